// Host side of latent attention's entry points (include/kda.h): argument validation before any HIP
// call, workspace sizing, dispatch.
#include <math.h>
#include <stdint.h>

#include "kda.h"
#include "latent_launch.h"

namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
bool bad_scale(float s) { return !isfinite(s) || !(s > 0.f); }

kda::LatentLaunch shape(bool packed, int N, int H, int T, int S, int dn, int dr, int io) {
    kda::LatentLaunch p{};
    p.N = N; p.B = packed ? 1 : N; p.H = H; p.T = T; p.S = S; p.dn = dn; p.dr = dr;
    p.fp32 = io == KDA_FP32;
    p.packed = packed;
    return p;
}

int check_shape(bool backward, bool packed, int N, int H, int T, int S, int dn, int dr, int io) {
    if (io != KDA_BF16 && io != KDA_FP32) return KDA_ERR_DTYPE;
    if (N < 1 || H < 1 || T < 0 || S < 0 || H > 65535) return KDA_ERR_SHAPE;
    if ((dn != 64 && dn != 128) || (dr != 32 && dr != 64)) return KDA_ERR_SHAPE;
    if (!packed && N > 65535) return KDA_ERR_SHAPE;
    if (T > 2147483647 - 256 || S > 2147483647 - 256) return KDA_ERR_SHAPE;
    return kda::latent_grids_fit(shape(packed, N, H, T, S, dn, dr, io), backward) ? KDA_OK : KDA_ERR_SHAPE;
}

// b, h, t strides of a tensor of B entries, H heads (0: none) and T rows of `inner` elements; a dimension
// of one has none
bool set_strides(long long (&s)[3], const kda_strides *given, int B, long long H, long long T, long long inner, int unit) {
    if (given == nullptr) {
        s[2] = inner;
        s[1] = H > 0 ? T * inner : 0;
        s[0] = (H > 0 ? H : 1) * T * inner;
        return true;
    }
    s[0] = B > 1 ? given->b : 0;
    s[1] = H > 1 ? given->h : 0;
    s[2] = T > 1 ? given->t : 0;
    return s[0] % unit == 0 && s[1] % unit == 0 && s[2] % unit == 0;
}

// the kernels step through 64 rows with 32-bit offsets, forwards
bool far_rows(const long long (&s)[3], long long rows, bool fp32) {
    return rows > 1 && (s[2] < 0 || s[2] > 2147483647LL / 64 / (fp32 ? 4 : 2));
}

int inputs(kda::LatentLaunch &p, const void *q, const kda_strides *qs, const void *k, const kda_strides *ks, const void *v,
           const kda_strides *vs, const void *kr, const kda_strides *krs, const int *cu_q, const int *cu_k, float scale) {
    const int unit = p.fp32 ? 4 : 8;
    if (bad_scale(scale)) return KDA_ERR_SCALE;
    if ((cu_q == nullptr) != (cu_k == nullptr)) return KDA_ERR_NULL;
    if ((p.T > 0 && !q) || (p.S > 0 && (!k || !v || !kr))) return KDA_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(kr, 16) || !aligned(cu_q, 4) || !aligned(cu_k, 4))
        return KDA_ERR_ALIGN;
    if (!set_strides(p.sq, qs, p.B, p.H, p.T, p.dn + p.dr, unit) || !set_strides(p.sk, ks, p.B, p.H, p.S, p.dn, unit) ||
        !set_strides(p.sv, vs, p.B, p.H, p.S, p.dn, unit) || !set_strides(p.skr, krs, p.B, 0, p.S, p.dr, unit))
        return KDA_ERR_ALIGN;
    if (far_rows(p.sq, p.T, p.fp32) || far_rows(p.sk, p.S, p.fp32) || far_rows(p.sv, p.S, p.fp32) || far_rows(p.skr, p.S, p.fp32))
        return KDA_ERR_SHAPE;
    p.q = q; p.k = k; p.v = v; p.kr = kr;
    p.cu_q = cu_q; p.cu_k = cu_k;
    p.scale = scale;
    return KDA_OK;
}

kda::LatentLaunch decode_shape(int B, int H, int page, int max_pages, int dc, int io) {
    kda::LatentLaunch p{};
    p.B = B; p.H = H; p.page = page; p.max_pages = max_pages; p.dc = dc;
    p.fp32 = io == KDA_FP32;
    return p;
}

int check_decode(int B, int H, int page, int max_pages, int dc, int dr, int io) {
    if (io != KDA_BF16 && io != KDA_FP32) return KDA_ERR_DTYPE;
    if (B < 1 || B > 65535 || H < 1 || H > 65535 || page < 1 || max_pages < 1) return KDA_ERR_SHAPE;
    if ((dc != 256 && dc != 512) || dr != 64) return KDA_ERR_SHAPE;
    if ((long long)max_pages * page > 2147483647LL - 128) return KDA_ERR_SHAPE;
    return kda::latent_decode_grid_fits(decode_shape(B, H, page, max_pages, dc, io)) ? KDA_OK : KDA_ERR_SHAPE;
}

kda::LatentTreeLaunch tree_shape(int B, int T, int H, int page, int max_pages, int dc, int io) {
    kda::LatentTreeLaunch p{};
    p.B = B; p.T = T; p.H = H; p.page = page; p.max_pages = max_pages; p.dc = dc;
    p.fp32 = io == KDA_FP32;
    return p;
}

int check_tree(int B, int T, int H, int page, int max_pages, int dc, int dr, int io) {
    if (io != KDA_BF16 && io != KDA_FP32) return KDA_ERR_DTYPE;
    if (B < 1 || B > 65535 || T < 1 || T > 64 || H < 1 || H > 65535 || page < 1 || max_pages < 1) return KDA_ERR_SHAPE;
    if ((dc != 256 && dc != 512) || dr != 64) return KDA_ERR_SHAPE;
    if ((long long)max_pages * page > 2147483647LL - 128) return KDA_ERR_SHAPE;
    return kda::latent_tree_grid_fits(tree_shape(B, T, H, page, max_pages, dc, io)) ? KDA_OK : KDA_ERR_SHAPE;
}

// strides of rows that start at multiples of 16 bytes; a dimension of one has none
bool append_stride(long long &s, long long given, long long n, int unit) {
    s = n > 1 ? given : 0;
    return s % unit == 0;
}

}  // namespace

extern "C" {

int kda_latent_attn_fwd(const void *q, const kda_strides *q_strides, const void *k, const kda_strides *k_strides,
                        const void *v, const kda_strides *v_strides, const void *k_rope,
                        const kda_strides *k_rope_strides, const int *cu_seqlens_q, const int *cu_seqlens_k, int N,
                        int H, int T, int S, int dn, int dr, int io_dtype, float scale, void *out, float *lse,
                        hipStream_t stream) {
    const bool packed = cu_seqlens_q != nullptr;
    int st = check_shape(false, packed, N, H, T, S, dn, dr, io_dtype);
    if (st != KDA_OK) return st;
    kda::LatentLaunch p = shape(packed, N, H, T, S, dn, dr, io_dtype);
    if (T > 0 && (!out || !lse)) return KDA_ERR_NULL;
    if (!aligned(out, 16) || !aligned(lse, 4)) return KDA_ERR_ALIGN;
    st = inputs(p, q, q_strides, k, k_strides, v, v_strides, k_rope, k_rope_strides, cu_seqlens_q, cu_seqlens_k, scale);
    if (st != KDA_OK || T == 0) return st;
    p.out = out;
    p.lse = lse;
    p.stream = stream;
    return kda::launch_latent_fwd(p) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t kda_latent_attn_bwd_workspace_bytes(int packed, int N, int H, int T, int S, int dn, int dr, int io_dtype) {
    if (check_shape(true, packed != 0, N, H, T, S, dn, dr, io_dtype) != KDA_OK) return 0;
    return kda::latent_bwd_bytes(shape(packed != 0, N, H, T, S, dn, dr, io_dtype));
}

int kda_latent_attn_bwd(const void *q, const kda_strides *q_strides, const void *k, const kda_strides *k_strides,
                        const void *v, const kda_strides *v_strides, const void *k_rope,
                        const kda_strides *k_rope_strides, const void *out, const float *lse, const void *dout,
                        const kda_strides *dout_strides, const int *cu_seqlens_q, const int *cu_seqlens_k, int N,
                        int H, int T, int S, int dn, int dr, int io_dtype, float scale, void *dq, void *dk_out,
                        void *dv_out, void *dk_rope, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    const bool packed = cu_seqlens_q != nullptr;
    int st = check_shape(true, packed, N, H, T, S, dn, dr, io_dtype);
    if (st != KDA_OK) return st;
    kda::LatentLaunch p = shape(packed, N, H, T, S, dn, dr, io_dtype);
    if ((T > 0 && (!out || !lse || !dout || !dq)) || (S > 0 && (!dk_out || !dv_out || !dk_rope))) return KDA_ERR_NULL;
    if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(dout, 16) || !aligned(dq, 16) || !aligned(dk_out, 16) ||
        !aligned(dv_out, 16) || !aligned(dk_rope, 16) || !set_strides(p.sdo, dout_strides, p.B, H, T, dn, p.fp32 ? 4 : 8))
        return KDA_ERR_ALIGN;
    st = inputs(p, q, q_strides, k, k_strides, v, v_strides, k_rope, k_rope_strides, cu_seqlens_q, cu_seqlens_k, scale);
    if (st != KDA_OK) return st;
    if (far_rows(p.sdo, T, p.fp32)) return KDA_ERR_SHAPE;
    const size_t need = kda::latent_bwd_bytes(p);
    if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return KDA_ERR_ALIGN;
    if (T == 0 && S == 0) return KDA_OK;
    p.fwd_out = out;
    p.fwd_lse = lse;
    p.dout = dout;
    p.dq = dq; p.dk = dk_out; p.dv = dv_out; p.dkr = dk_rope;
    p.workspace = static_cast<unsigned char *>(workspace);
    p.stream = stream;
    return kda::launch_latent_bwd(p) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t kda_latent_decode_workspace_bytes(int B, int H, int page, int max_pages, int dc, int dr, int io_dtype) {
    if (check_decode(B, H, page, max_pages, dc, dr, io_dtype) != KDA_OK) return 0;
    return kda::latent_decode_bytes(decode_shape(B, H, page, max_pages, dc, io_dtype));
}

int kda_latent_decode_step(const void *q, const void *cache, const int *block_table, const int *lengths, int B, int H,
                           int pages, int page, int max_pages, int dc, int dr, int io_dtype, float scale, void *out,
                           float *lse, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    const int st = check_decode(B, H, page, max_pages, dc, dr, io_dtype);
    if (st != KDA_OK) return st;
    if (pages < 1) return KDA_ERR_SHAPE;
    if (bad_scale(scale)) return KDA_ERR_SCALE;
    if (!q || !cache || !block_table || !lengths || !out || !lse) return KDA_ERR_NULL;
    if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(block_table, 4) || !aligned(lengths, 4) || !aligned(out, 16) ||
        !aligned(lse, 4) || !aligned(workspace, 16))
        return KDA_ERR_ALIGN;
    kda::LatentLaunch p = decode_shape(B, H, page, max_pages, dc, io_dtype);
    const size_t need = kda::latent_decode_bytes(p);
    if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    p.q = q; p.cache = cache; p.table = block_table; p.lengths = lengths;
    p.pages = pages;
    p.scale = scale;
    p.out = out;
    p.lse = lse;
    p.workspace = static_cast<unsigned char *>(workspace);
    p.stream = stream;
    return kda::launch_latent_decode(p) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

int kda_latent_append(const void *latent, const kda_strides *latent_strides, const void *k_rope,
                      const kda_strides *k_rope_strides, void *cache, const int *block_table, const int *lengths,
                      const float *freqs, const void *norm_weight, float eps, const int *positions, const int *counts,
                      const void *q_rope, const kda_strides *q_rope_strides, void *q, const int *cu_seqlens, int N, int T,
                      int H, int pages, int page, int max_pages, int dc, int dr, int io_dtype, int interleaved,
                      hipStream_t stream) {
    if (io_dtype != KDA_BF16 && io_dtype != KDA_FP32) return KDA_ERR_DTYPE;
    if (N < 1 || T < 0 || H < 0 || H > 65535 || pages < 1 || page < 1 || max_pages < 1) return KDA_ERR_SHAPE;
    if ((dc != 256 && dc != 512) || dr != 64) return KDA_ERR_SHAPE;
    if ((long long)max_pages * page > 2147483647LL - 128) return KDA_ERR_SHAPE;
    const bool packed = cu_seqlens != nullptr;
    kda::LatentAppendLaunch p{};
    p.N = N; p.B = packed ? 1 : N; p.T = T; p.H = H; p.pages = pages; p.page = page; p.max_pages = max_pages; p.dc = dc;
    p.fp32 = io_dtype == KDA_FP32;
    p.interleaved = interleaved != 0;
    if (!kda::latent_append_grid_fits(p)) return KDA_ERR_SHAPE;
    if (norm_weight && !(isfinite(eps) && eps >= 0.f)) return KDA_ERR_SCALE;
    if (packed && counts) return KDA_ERR_NULL;
    if (!cache || !block_table || !lengths || !freqs || (T > 0 && (!latent || !k_rope)) || (T > 0 && H > 0 && (!q_rope || !q)))
        return KDA_ERR_NULL;
    const int unit = p.fp32 ? 4 : 8;
    if (!aligned(latent, 16) || !aligned(k_rope, 16) || !aligned(cache, 16) || !aligned(norm_weight, 16) || !aligned(q_rope, 16) ||
        !aligned(q, 16) || !aligned(block_table, 4) || !aligned(lengths, 4) || !aligned(freqs, 4) || !aligned(positions, 4) ||
        !aligned(counts, 4) || !aligned(cu_seqlens, 4))
        return KDA_ERR_ALIGN;
    const kda_strides l = latent_strides ? *latent_strides : kda_strides{(long long)T * dc, 0, dc};
    const kda_strides k = k_rope_strides ? *k_rope_strides : kda_strides{(long long)T * dr, 0, dr};
    const kda_strides r = q_rope_strides ? *q_rope_strides : kda_strides{(long long)T * H * dr, dr, (long long)H * dr};
    if (!append_stride(p.sl[0], l.b, p.B, unit) || !append_stride(p.sl[1], l.t, T, unit) || !append_stride(p.sk[0], k.b, p.B, unit) ||
        !append_stride(p.sk[1], k.t, T, unit) || !append_stride(p.sq[0], r.b, p.B, unit) || !append_stride(p.sq[1], r.t, T, unit) ||
        !append_stride(p.sq[2], r.h, H, unit))
        return KDA_ERR_ALIGN;
    if (T == 0) return KDA_OK;
    p.latent = latent; p.kr = k_rope; p.qr = q_rope; p.weight = norm_weight;
    p.cache = cache; p.q = q;
    p.table = block_table; p.lengths = lengths; p.positions = positions; p.counts = counts; p.cu = cu_seqlens;
    p.freqs = freqs;
    p.eps = eps;
    p.stream = stream;
    return kda::launch_latent_append(p) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

size_t kda_latent_tree_workspace_bytes(int B, int T, int H, int page, int max_pages, int dc, int dr, int io_dtype) {
    if (check_tree(B, T, H, page, max_pages, dc, dr, io_dtype) != KDA_OK) return 0;
    return kda::latent_tree_bytes(tree_shape(B, T, H, page, max_pages, dc, io_dtype));
}

int kda_latent_tree_step(const void *q, const void *cache, const int *block_table, const int *lengths, const int *counts,
                         const unsigned long long *tree_mask, int B, int T, int H, int pages, int page, int max_pages, int dc,
                         int dr, int io_dtype, float scale, void *out, float *lse, void *workspace, size_t workspace_bytes,
                         hipStream_t stream) {
    const int st = check_tree(B, T, H, page, max_pages, dc, dr, io_dtype);
    if (st != KDA_OK) return st;
    if (pages < 1) return KDA_ERR_SHAPE;
    if (bad_scale(scale)) return KDA_ERR_SCALE;
    if (!q || !cache || !block_table || !lengths || !tree_mask || !out || !lse) return KDA_ERR_NULL;
    if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(block_table, 4) || !aligned(lengths, 4) || !aligned(counts, 4) ||
        !aligned(tree_mask, 8) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 16))
        return KDA_ERR_ALIGN;
    kda::LatentTreeLaunch p = tree_shape(B, T, H, page, max_pages, dc, io_dtype);
    const size_t need = kda::latent_tree_bytes(p);
    if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    p.q = q; p.cache = cache; p.table = block_table; p.lengths = lengths; p.counts = counts;
    p.mask = tree_mask;
    p.pages = pages;
    p.scale = scale;
    p.out = out;
    p.lse = lse;
    p.workspace = static_cast<unsigned char *>(workspace);
    p.stream = stream;
    return kda::launch_latent_tree(p) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
