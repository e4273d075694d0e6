// Sequential stage of the gated delta rule (gdr_common.h): walks the chunks of one (sequence, value
// head) with the state P = S^T in registers.  A wave owns 16 value columns, for which it does every
// product of the chunk on its own: the accumulator layout of one product is the B operand of the
// next, so the chain K P -> Y -> X -> U = T X -> K^T U' exchanges nothing between waves; the chunk's
// K, Q, T and M are shared through LDS, filled one chunk ahead by direct global-to-LDS loads.
//
// A chunk costs a wave 104 MFMAs of 16x16x32 (dk = 128, bf16 inputs), about 1,700 cycles, and the
// conversions of P, X and U to fp16 pieces.  The chain of chunks bounds the stage while there are
// fewer waves (sequences x heads x dv / 16) than SIMDs, so a work-group takes as few waves as fill
// the chip (gdr_waves): fewer waves share a fill, but each then has its CU's LDS to itself.
//
// SAVE = 1 (backward): instead of outputs it stores every chunk's start state and U, as fp16 pieces.
#pragma once
#include "gdr_common.h"

namespace kda {

struct GdrStateArgs {
    const unsigned char *keys, *vals;
    const void *v;
    Strides3 sv;
    GdrSeqs seqs;
    int H, r, nslot, dv;       // value heads; value heads per key head; chunk slots
    float scale;
    float *final_state;        // nullable [N][H][dv][dk]
    const float *init_state;   // nullable
    void *out;                 // [B][H][T][dv], contiguous
    unsigned char *save;       // SAVE: records, GdrSave
};

// Saved by the SAVE pass, one record per (batch, head, chunk, 16-column slice): 64 ints (exponent of
// P, of U), then P's pieces ([dk / 32] fragments each) and U's pieces (2 fragments each), B operands.
struct GdrSave {
    int ni, dk;
    __host__ __device__ constexpr int p_off(int piece) const { return 256 + piece * (dk / 32) * 1024; }
    __host__ __device__ constexpr int u_off(int piece) const { return 256 + ni * (dk / 32) * 1024 + piece * 2048; }
    __host__ __device__ constexpr size_t bytes() const { return 256 + (size_t)ni * (dk / 32) * 1024 + ni * 2048; }
};

// LDS of one buffered chunk: the value record (header, T, M) and the key record's K (and Q)
template <int DK, int NI, int SAVE> struct GdrStateLds {
    static constexpr GdrLayout L{NI, DK, NI};
    static constexpr int VAL = GdrLayout::kHead + (SAVE ? 2 : 2 + NI) * GdrLayout::kTri;
    static constexpr int KEY = (SAVE ? 1 : 2) * NI * L.mat();
    static constexpr int BYTES = VAL + KEY;
    static constexpr int NBUF = 2 * BYTES <= 160 * 1024 ? 2 : 1;
    static constexpr int K = VAL, Q = VAL + NI * L.mat();
    static constexpr int T = GdrLayout::kHead, M = T + 2 * GdrLayout::kTri;
};

// mp: pieces of M in the records (2 for the backward's records, which keep it exact)
template <int DK, bool F32, int SAVE, int NW, int MP>
__global__ __launch_bounds__(64 * NW) void gdr_state_kernel(const GdrStateArgs p) {
    using E = typename std::conditional<F32, float, __bf16>::type;
    constexpr int NI = F32 ? 2 : 1, NKB = DK / 32, NT = DK / 16;
    using S = GdrStateLds<DK, NI, SAVE>;
    constexpr GdrLayout L{NI, DK, MP};
    constexpr GdrSave SV{NI, DK};
    __shared__ __attribute__((aligned(1024))) unsigned char smem[S::NBUF * S::BYTES];
    const int lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // the work-groups of one head share an XCD's L2: ids 8 apart
    const int gh = p.dv / 16 / NW, id = blockIdx.x;
    const int unit = id / (8 * gh) * 8 + (id & 7), slice = (id >> 3) % gh * NW + w;
    if (unit >= p.seqs.N * p.H) return;
    const int seq = unit / p.H, h = unit % p.H, b = p.seqs.batch(seq);
    const int len = p.seqs.length(seq), start = p.seqs.start(seq), nchunk = (len + 63) / 64;
    const int col = slice * 16 + n, nkey = p.H / p.r;
    const size_t slot0 = p.seqs.slot0(seq);
    const unsigned char *krec = p.keys + ((size_t)(b * nkey + h / p.r) * p.nslot + slot0) * L.key_bytes();
    const unsigned char *vrec = p.vals + ((size_t)(b * p.H + h) * p.nslot + slot0) * L.val_bytes();
    const E *vp = reinterpret_cast<const E *>(p.v) + b * p.sv.b + h * p.sv.h + (long long)start * p.sv.t + col;
    E *op = reinterpret_cast<E *>(p.out) + ((size_t)(b * p.H + h) * p.seqs.T + start) * p.dv + col;
    unsigned char *save = p.save + (((size_t)(b * p.H + h) * p.nslot + slot0) * (p.dv / 16) + slice) * SV.bytes();

    auto fill = [&](int c, int buf) {
        const unsigned char *vs = vrec + (size_t)c * L.val_bytes(), *ks = krec + (size_t)c * L.key_bytes() + 256;
        lds_u8 *dst = lds_base(smem) + buf * S::BYTES;
        for (int u = w; u < S::BYTES / 1024; u += NW) {
            const unsigned char *src = u < S::VAL / 1024 ? vs + u * 1024 : ks + (u * 1024 - S::VAL);
            load_lds16(src + lane * 16, dst + u * 1024);
        }
    };
    E vr[16], vn[16];
    auto load_v = [&](int c) {
#pragma unroll
        for (int x = 0; x < 16; ++x) {
            const int row = 64 * c + 32 * (x >> 3) + 8 * g + (x & 7), last = len - 1;
            vn[x] = vp[(long long)(row < last ? row : last) * p.sv.t];
        }
    };

    // the state: tile t row 4 g + i is key channel perm_row(t, 4 g + i), column n
    f32x4 P[NT];
    const size_t state0 = ((size_t)(seq * p.H + h) * p.dv + col) * DK;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if (p.init_state != nullptr)
            P[t] = *reinterpret_cast<const f32x4 *>(p.init_state + state0 + perm_row(t, 4 * g));
        else
            P[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    E o_prev[16];
    if (nchunk > 0) {
        fill(0, 0);
        load_v(0);
    }
    for (int c = 0; c < nchunk; ++c) {
        const int buf = S::NBUF == 2 ? (c & 1) : 0;
        // own loads done, then everybody's; with two buffers the other one is free after this
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
        barrier_lds();
#pragma unroll
        for (int x = 0; x < 16; ++x) vr[x] = vn[x];
        if constexpr (S::NBUF == 2)
            if (c + 1 < nchunk) fill(c + 1, buf ^ 1);
        if (c + 1 < nchunk) load_v(c + 1);
        if constexpr (!SAVE)
            if (c > 0) {  // the last chunk's outputs (whole chunks but the very last)
#pragma unroll
                for (int x = 0; x < 16; ++x)
                    op[(size_t)(64 * (c - 1) + 32 * (x >> 3) + 8 * g + (x & 7)) * p.dv] = o_prev[x];
            }
        const lds_u8 *sb = lds_base(smem) + buf * S::BYTES;
        const auto *hd = reinterpret_cast<const __attribute__((address_space(3))) float *>(sb);
        const auto *hi_ = reinterpret_cast<const __attribute__((address_space(3))) int *>(sb);
        const float last = hd[192];
        const int et = __builtin_amdgcn_readfirstlane(hi_[193]), em = __builtin_amdgcn_readfirstlane(hi_[194]);
        const int ek = __builtin_amdgcn_readfirstlane(hi_[195]), eq = __builtin_amdgcn_readfirstlane(hi_[196]);
        auto row4 = [&](int arr, int rt) {  // header array at this lane's four rows of tile rt
            return *reinterpret_cast<const __attribute__((address_space(3))) f32x4 *>(hd + 64 * arr + perm_row(rt, 4 * g));
        };

        // P as fp16 pieces
        f16x8 ph[NKB], pl[NKB];
        float mx = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t) mx = max_abs4(P[t], mx);
        const int ep = gdr_exp(wave_max(mx));
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) split_pair(P[2 * kb], P[2 * kb + 1], pow2f(ep), ph[kb], pl[kb]);
        if constexpr (SAVE) {
            unsigned char *sv = save + (size_t)c * (p.dv / 16) * SV.bytes();
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                f16x8 one = ph[kb];
                if constexpr (NI == 1) one = round_pair(P[2 * kb], P[2 * kb + 1], pow2f(ep));
                *reinterpret_cast<f16x8 *>(sv + SV.p_off(0) + kb * 1024 + frag_slot(g, n)) = one;
                if constexpr (NI == 2) *reinterpret_cast<f16x8 *>(sv + SV.p_off(1) + kb * 1024 + frag_slot(g, n)) = pl[kb];
            }
            if (lane == 0) reinterpret_cast<int *>(sv)[0] = ep;
        }
        // Z = K P; X = diag(b) (V - e^G Z); Q P alongside
        f32x4 X[4], O[4];
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        float xm = 0.f;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            f32x4 z = zero, z1 = zero;
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                const f16x8 f = ld_frag(sb + S::K + (rt * NKB + kb) * 1024, lane);
                z = mma16(f, ph[kb], z);
                z1 = mma16(f, pl[kb], z1);
                if constexpr (NI == 2)
                    z1 = mma16(ld_frag(sb + S::K + L.mat() + (rt * NKB + kb) * 1024, lane), ph[kb], z1);
            }
            const f32x4 eG = row4(0, rt), be = row4(2, rt);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                X[rt][i] = be[i] * (to_f(vr[4 * rt + i]) - eG[i] * scale_down(z[i] + z1[i], ek + ep));
            xm = max_abs4(X[rt], xm);
        }
        if constexpr (!SAVE) {
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                f32x4 z = zero;
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb) {
                    const f16x8 f = ld_frag(sb + S::Q + (rt * NKB + kb) * 1024, lane);
                    z = mma16(f, ph[kb], z);
                    if constexpr (NI == 2) {
                        z = mma16(f, pl[kb], z);
                        z = mma16(ld_frag(sb + S::Q + L.mat() + (rt * NKB + kb) * 1024, lane), ph[kb], z);
                    }
                }
                O[rt] = z;
            }
        }
        // U = T X
        const int ex = gdr_exp(wave_max(xm));
        f16x8 xh[2], xl[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) split_pair(X[2 * kb], X[2 * kb + 1], pow2f(ex), xh[kb], xl[kb]);
        f32x4 U[4], V2[4];
        float um = 0.f, vm = 0.f;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            f32x4 z = zero, z1 = zero;
#pragma unroll
            for (int kb = 0; kb < (rt < 2 ? 1 : 2); ++kb) {
                const f16x8 th = ld_frag(sb + S::T + tri_frag(rt, kb) * 1024, lane);
                const f16x8 tl = ld_frag(sb + S::T + GdrLayout::kTri + tri_frag(rt, kb) * 1024, lane);
                z = mma16(th, xh[kb], z);
                z1 = mma16(tl, xh[kb], mma16(th, xl[kb], z1));
            }
            const f32x4 eL = row4(1, rt);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                U[rt][i] = scale_down(z[i] + z1[i], et + ex);
                V2[rt][i] = U[rt][i] * eL[i];
            }
            um = max_abs4(U[rt], um);
            vm = max_abs4(V2[rt], vm);
        }
        // P' = e^{G_last} P + K^T (e^{G_last - G} U)
        const int ev = gdr_exp(wave_max(vm)), eu = gdr_exp(wave_max(um));
        {
            f16x8 vh[2], vl[2];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) split_pair(V2[2 * kb], V2[2 * kb + 1], pow2f(ev), vh[kb], vl[kb]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                f32x4 z = zero, z1 = zero;
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    const lds_u8 *f0 = sb + S::K + (2 * kb * NKB + (t >> 1)) * 1024, *f1 = f0 + NKB * 1024;
                    const f16x8 f = ld_frag_t(f0, f1, t, lane);
                    z = mma16(f, vh[kb], z);
                    z1 = mma16(f, vl[kb], z1);
                    if constexpr (NI == 2) z1 = mma16(ld_frag_t(f0 + L.mat(), f1 + L.mat(), t, lane), vh[kb], z1);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) P[t][i] = fmaf(P[t][i], last, scale_down(z[i] + z1[i], ek + ev));
            }
        }
        // O = scale e^G Q P + M U (M holds the scale)
        f16x8 uh[2], ul[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            if constexpr (NI == 2) split_pair(U[2 * kb], U[2 * kb + 1], pow2f(eu), uh[kb], ul[kb]);
            else uh[kb] = round_pair(U[2 * kb], U[2 * kb + 1], pow2f(eu));
        }
        if constexpr (SAVE) {
            unsigned char *sv = save + (size_t)c * (p.dv / 16) * SV.bytes();
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                *reinterpret_cast<f16x8 *>(sv + SV.u_off(0) + kb * 1024 + frag_slot(g, n)) = uh[kb];
                if constexpr (NI == 2) *reinterpret_cast<f16x8 *>(sv + SV.u_off(1) + kb * 1024 + frag_slot(g, n)) = ul[kb];
            }
            if (lane == 0) reinterpret_cast<int *>(sv)[1] = eu;
        } else {
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                f32x4 z = zero;
#pragma unroll
                for (int kb = 0; kb < (rt < 2 ? 1 : 2); ++kb) {
                    const f16x8 f = ld_frag(sb + S::M + tri_frag(rt, kb) * 1024, lane);
                    z = mma16(f, uh[kb], z);
                    if constexpr (NI == 2) {
                        z = mma16(f, ul[kb], z);
                        z = mma16(ld_frag(sb + S::M + GdrLayout::kTri + tri_frag(rt, kb) * 1024, lane), uh[kb], z);
                    }
                }
                const f32x4 eG = row4(0, rt);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o_prev[4 * rt + i] = from_f<E>(scale_down(z[i], em + eu) + p.scale * eG[i] * scale_down(O[rt][i], eq + ep));
            }
        }
        if constexpr (S::NBUF == 1) {
            barrier_lds();  // everybody has read the buffer
            if (c + 1 < nchunk) fill(c + 1, 0);
        }
    }
    if constexpr (!SAVE) {
#pragma unroll
        for (int x = 0; x < 16; ++x) {
            const int row = 64 * (nchunk - 1) + 32 * (x >> 3) + 8 * g + (x & 7);
            if (row >= 0 && row < len) op[(size_t)row * p.dv] = o_prev[x];
        }
    }
    if (p.final_state != nullptr)
#pragma unroll
        for (int t = 0; t < NT; ++t)
            *reinterpret_cast<f32x4 *>(p.final_state + state0 + perm_row(t, 4 * g)) = P[t];
}

}  // namespace kda
