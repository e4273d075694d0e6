// Host side of decayed linear attention's entry points (include/kda.h): argument validation before any
// HIP call, workspace sizing, dispatch.
#include <math.h>
#include <stdint.h>

#include "kda.h"
#include "lin_launch.h"

namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

kda::LinLaunch shape(bool packed, int N, int Hk, int H, int T, int dk, int dv, int io) {
    kda::LinLaunch p{};
    p.packed = packed;
    p.N = N; p.B = packed ? 1 : N; p.Hk = Hk; p.H = H; p.T = T; p.dk = dk; p.dv = dv;
    p.fp32 = io == KDA_FP32;
    return p;
}

int check_shape(bool backward, bool packed, int N, int Hk, int H, int T, int dk, int dv, int io) {
    if (io != KDA_BF16 && io != KDA_FP32) return KDA_ERR_DTYPE;
    if (N < 1 || Hk < 1 || H < 1 || T < 0 || H % Hk != 0 || H > 65535) return KDA_ERR_SHAPE;
    if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128)) return KDA_ERR_SHAPE;
    if (!packed && N > 65535) return KDA_ERR_SHAPE;
    if (T > 2147483647 - (1 << 19) || (long long)T / 64 + N > 2147483647LL) return KDA_ERR_SHAPE;  // a segment behind T still counts in 32 bits
    if ((packed ? 1.0 : (double)N) * H * (double)T * (dk > dv ? dk : dv) >= 1099511627776.0) return KDA_ERR_SHAPE;  // 2^40
    if (backward && (packed ? 1 : N) * (long long)H * (((long long)T + 15) / 16) >= 1 << 24) return KDA_ERR_SHAPE;
    return kda::lin_grids_fit(shape(packed, N, Hk, H, T, dk, dv, io), backward) ? KDA_OK : KDA_ERR_SHAPE;
}

// g in float32, or in the other tensors' type
int check_g(int io, int g) { return g == KDA_FP32 || (g == KDA_BF16 && io == KDA_BF16) ? KDA_OK : KDA_ERR_DTYPE; }

// strides of a tensor of B x H x T rows of `inner` elements; unit: elements that a row's start must be a
// multiple of (1: any).  A dimension of one has none.
bool set_strides(long long (&s)[3], const kda_strides *given, int B, long long H, long long T, long long inner, int unit) {
    if (given == nullptr) {
        s[2] = inner;
        s[1] = T * inner;
        s[0] = H * T * inner;
        return true;
    }
    s[0] = B > 1 ? given->b : 0;
    s[1] = H > 1 ? given->h : 0;
    s[2] = T > 1 ? given->t : 0;
    return s[0] % unit == 0 && s[1] % unit == 0 && s[2] % unit == 0;
}

// the kernels step through 64 rows with 32-bit offsets, forwards
bool far_rows(const kda::LinLaunch &p, const long long (&s)[3]) {
    return p.T > 1 && (s[2] < 0 || s[2] > 2147483647LL / 64 / (p.fp32 ? 4 : 2));
}

int inputs(kda::LinLaunch &p, const void *q, const kda_strides *qs, const void *k, const kda_strides *ks, const void *v,
           const kda_strides *vs, const void *g, const kda_strides *gs, int g_dtype, const int *cu, float scale, const float *init,
           void *workspace, size_t given, size_t need) {
    const int unit = p.fp32 ? 4 : 8;
    if (!isfinite(scale)) return KDA_ERR_SCALE;
    if (p.T > 0 && (!q || !k || !v || !g)) return KDA_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(g, g_dtype == KDA_FP32 ? 4 : 2) || !aligned(cu, 4) ||
        !aligned(init, 16))
        return KDA_ERR_ALIGN;
    if (!set_strides(p.sq, qs, p.B, p.Hk, p.T, p.dk, unit) || !set_strides(p.sk, ks, p.B, p.Hk, p.T, p.dk, unit) ||
        !set_strides(p.sv, vs, p.B, p.H, p.T, p.dv, unit) || !set_strides(p.sg, gs, p.B, p.H, p.T, 1, 1))
        return KDA_ERR_ALIGN;
    if (far_rows(p, p.sq) || far_rows(p, p.sk) || far_rows(p, p.sv)) return KDA_ERR_SHAPE;
    if (need > 0 && (!workspace || given < need)) return KDA_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return KDA_ERR_ALIGN;
    p.q = q; p.k = k; p.v = v; p.g = g;
    p.g32 = g_dtype == KDA_FP32;
    p.cu = cu;
    p.scale = scale;
    p.init_state = init;
    p.workspace = static_cast<unsigned char *>(workspace);
    return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_lin_workspace_bytes(int backward, int packed, int N, int Hk, int H, int T, int dk, int dv, int io_dtype) {
    if (check_shape(backward != 0, packed != 0, N, Hk, H, T, dk, dv, io_dtype) != KDA_OK) return 0;
    const kda::LinLaunch p = shape(packed != 0, N, Hk, H, T, dk, dv, io_dtype);
    return backward ? kda::lin_bwd_bytes(p, backward != 2) : kda::lin_fwd_bytes(p);
}

int kda_lin_chunk_fwd(const void *q, const kda_strides *q_strides, const void *k, const kda_strides *k_strides,
                      const void *v, const kda_strides *v_strides, const void *g, const kda_strides *g_strides,
                      const int *cu_seqlens, int N, int Hk, int H, int T, int dk, int dv, int io_dtype, int g_dtype,
                      float scale, const float *initial_state, void *out, float *final_state, void *workspace,
                      size_t workspace_bytes, hipStream_t stream) {
    int st = check_shape(false, cu_seqlens != nullptr, N, Hk, H, T, dk, dv, io_dtype);
    if (st == KDA_OK) st = check_g(io_dtype, g_dtype);
    if (st != KDA_OK) return st;
    kda::LinLaunch p = shape(cu_seqlens != nullptr, N, Hk, H, T, dk, dv, io_dtype);
    if (T > 0 && !out) return KDA_ERR_NULL;
    if (!aligned(out, 16) || !aligned(final_state, 16)) return KDA_ERR_ALIGN;
    st = inputs(p, q, q_strides, k, k_strides, v, v_strides, g, g_strides, g_dtype, cu_seqlens, scale, initial_state, workspace,
                workspace_bytes, kda::lin_fwd_bytes(p));
    if (st != KDA_OK || (T == 0 && !final_state)) return st;
    p.out = out;
    p.final_state = final_state;
    p.stream = stream;
    return kda::launch_lin_fwd(p) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

int kda_lin_chunk_bwd(const void *q, const kda_strides *q_strides, const void *k, const kda_strides *k_strides,
                      const void *v, const kda_strides *v_strides, const void *g, const kda_strides *g_strides,
                      const void *dout, const kda_strides *dout_strides, const int *cu_seqlens, int N, int Hk, int H,
                      int T, int dk, int dv, int io_dtype, int g_dtype, float scale, const float *initial_state,
                      const float *dfinal_state, void *dq, void *dk_out, void *dv_out, void *dg, float *dinitial_state,
                      void *workspace, size_t workspace_bytes, hipStream_t stream) {
    int st = check_shape(true, cu_seqlens != nullptr, N, Hk, H, T, dk, dv, io_dtype);
    if (st == KDA_OK) st = check_g(io_dtype, g_dtype);
    if (st != KDA_OK) return st;
    kda::LinLaunch p = shape(cu_seqlens != nullptr, N, Hk, H, T, dk, dv, io_dtype);
    if (T > 0 && (!dout || !dq || !dk_out || !dv_out)) return KDA_ERR_NULL;
    if (!aligned(dout, 16) || !aligned(dq, 16) || !aligned(dk_out, 16) || !aligned(dv_out, 16) ||
        !aligned(dg, g_dtype == KDA_FP32 ? 4 : 2) || !aligned(dfinal_state, 16) || !aligned(dinitial_state, 16) ||
        !set_strides(p.sdo, dout_strides, p.B, H, T, dv, p.fp32 ? 4 : 8))
        return KDA_ERR_ALIGN;
    st = inputs(p, q, q_strides, k, k_strides, v, v_strides, g, g_strides, g_dtype, cu_seqlens, scale, initial_state, workspace,
                workspace_bytes, kda::lin_bwd_bytes(p, dg && dfinal_state));
    if (st != KDA_OK) return st;
    if (far_rows(p, p.sdo)) return KDA_ERR_SHAPE;
    if (T == 0 && !dinitial_state) return KDA_OK;
    p.dout = dout;
    p.dfinal = dfinal_state;
    p.dq = dq; p.dk_ = dk_out; p.dv_ = dv_out; p.dg = dg;
    p.dinit = dinitial_state;
    p.stream = stream;
    return kda::launch_lin_bwd(p) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

int kda_lin_decode_step(const void *q, const void *k, const void *v, const void *g, int B, int Hk, int H, int dk, int dv,
                        int io_dtype, int g_dtype, float scale, float *state, void *out, hipStream_t stream) {
    if (io_dtype != KDA_BF16 && io_dtype != KDA_FP32) return KDA_ERR_DTYPE;
    if (check_g(io_dtype, g_dtype) != KDA_OK) return KDA_ERR_DTYPE;
    if (B < 1 || Hk < 1 || H < 1 || H % Hk != 0 || H > 65535 || (dk != 64 && dk != 128) || (dv != 64 && dv != 128)) return KDA_ERR_SHAPE;
    kda::LinLaunch p{};
    p.B = B; p.Hk = Hk; p.H = H; p.T = 1; p.dk = dk; p.dv = dv;
    if (!kda::lin_decode_grid_fits(p)) return KDA_ERR_SHAPE;
    if (!isfinite(scale)) return KDA_ERR_SCALE;
    if (!q || !k || !v || !g || !state || !out) return KDA_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(g, g_dtype == KDA_FP32 ? 4 : 2) || !aligned(state, 16) ||
        !aligned(out, 16))
        return KDA_ERR_ALIGN;
    p.q = q; p.k = k; p.v = v; p.g = g;
    p.fp32 = io_dtype == KDA_FP32;
    p.g32 = g_dtype == KDA_FP32;
    p.scale = scale;
    p.state = state;
    p.out = out;
    p.stream = stream;
    return kda::launch_lin_decode(p) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
