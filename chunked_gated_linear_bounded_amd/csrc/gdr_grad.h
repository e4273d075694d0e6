// Gradient stage of the gated delta rule's backward (gdr_common.h): one 512-thread work-group per
// (chunk, key head, batch) loops over the value heads that share the key head and sums their dQ and
// dK in registers (no atomics).  From the two sequential passes it has, per value head, P and U, dP'
// and dX; with E1 = dO P^T, E2 = dX P^T, E3 = U dP'^T, D_ij = e^{G_i - G_j},
//   X1 = scale lower(dO U^T) o D,   X2 = -strict(dX U^T) o D,   R = X2 K,
//   dQ = scale e^G E1 + X1 K,
//   dK = X1^T Q + e^{G_last - G} E3 - b e^G E2 + b R + X2^T diag(b) K,
//   db_i = dX_i . V_i - e^G_i k_i . E2_i + k_i . R_i,
//   dG_i = q_i . dQ_i - k_i . (X1^T Q + e^{G_last - G} E3 + b e^G E2 - b R + X2^T diag(b) K)_i,
//   dG_last += sum_i e^{G_last - G_i} k_i . E3_i + e^{G_last} <P, dP'>,   dg_t = sum_{s >= t} dG_s:
// every sum over a row of dM o M or dA o A is a dot product of q or k with a row that is there anyway.
//
// Wave (rw, ch) owns token tile rw and one half of the key channels.  Operands are fp16 with one
// exponent per block (float32 inputs: two pieces); what the passes kept with an exponent per 16
// columns is brought to the smallest of them on its way into LDS.  diag(b) X2 takes b times the power of
// two that brings max |b| below 1: X2 itself sits at 2^13 .. 2^14, and a beta of 4 would reach fp16's end.
// The stage reads about 200 KiB a chunk and value head at d = 128 (bf16) and writes 32 KiB a key head;
// its 656 MFMAs a head are a tenth of that traffic's time (4096 tokens x 32 heads: 168 us, most of it
// the four phases' barriers with one work-group of eight waves a CU), so the four phases share one 64
// KiB buffer (P, then dP', then K and Q; dX, then X1 and X2).
#pragma once
#include "gdr_state.h"

namespace kda {

struct GdrGradArgs {
    const unsigned char *keys, *vals;
    const void *v, *g, *dout;
    Strides3 sv, sg, sdo;
    GdrSeqs seqs;
    int Hk, r, nslot;
    float scale;
    const unsigned char *fwd, *rev;  // GdrSave records: P, U and dP', dX
    void *dq, *dk, *dg, *dbeta;      // contiguous
};

// operand (rows = the 16 entries perm_row(tile, .) of a slice block's fragment columns, k = value
// channels 32 kbv + 8 g + j) from slice records in LDS: fragment (slice, block) at (slice nb + block) KiB
__device__ __forceinline__ f16x8 ld_slices(const lds_u8 *f, int nb, int kbv, int tile, int lane) {
    const int g = lane >> 4, s = lane & 15, m = 8 * (g & 1) + (s >> 2);
    const lds_u8 *q = f + ((2 * kbv + (g >> 1)) * nb + (tile >> 1)) * 1024 + 8 * (tile & 1);
    const f16x4 a = ld_tr16<f16x4>(q + frag_slot(s & 3, m)), b = ld_tr16<f16x4>(q + frag_slot(s & 3, m + 4));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
// rows 4 g + i of row tile (fragment f), column perm_row(tile, n): a matrix in accumulator layout
__device__ __forceinline__ f16x4 ld_acc(const lds_u8 *f, int tile, int lane) {
    const int g = lane >> 4, s = lane & 15;
    return ld_tr16<f16x4>(f + frag_slot(s & 3, 4 * g + (s >> 2)) + 8 * (tile & 1));
}
// sum over the 16 lanes of a row
__device__ __forceinline__ float row_sum(float x) {
    x += dpp_mov<0xB1>(x);
    x += dpp_mov<0x4E>(x);
    x += dpp_mov<0x141>(x);
    x += dpp_mov<0x140>(x);
    return x;
}

template <int DK, int DV, bool F32>
__global__ __launch_bounds__(512) void gdr_grad_kernel(const GdrGradArgs p) {
    using E = typename std::conditional<F32, float, __bf16>::type;
    constexpr int NI = F32 ? 2 : 1, NKB = DK / 32, NTH = DK / 32, NVB = DV / 32, NSL = DV / 16;  // NTH: dk tiles per wave
    constexpr GdrLayout L{NI, DK, 2};
    constexpr GdrSave SV{NI, DK};
    typedef __attribute__((address_space(3))) f16x8 lds_f16x8;
    // buffers: P / dP' / K and Q; U; dX / X1 and X2 (8 KiB a piece each)
    constexpr int PP = NSL * NKB * 1024, PU = NSL * 2048;
    constexpr int BA = NI * (PP > 2 * L.mat() ? PP : 2 * L.mat()), BU = NI * PU, BX = NI * (PU > 16384 ? PU : 16384);
    __shared__ __attribute__((aligned(1024))) unsigned char smem[BA + BU + BX];
    __shared__ double sG[64];
    __shared__ __attribute__((aligned(16))) _Float16 sBh[64];  // b 2^eb
    __shared__ float sGi[2][64], sBe[2][64], sRed[4][8];  // per half: dG, dbeta; per wave: max X1, X2, <P, dP'>, sum for dG_last
    lds_u8 *sa = lds_base(smem), *su = sa + BA, *sxx = su + BU;
    const int slot = blockIdx.x, kh = blockIdx.y, b = blockIdx.z, H = p.Hk * p.r;
    int t0, seq;
    const int nrow = p.seqs.find(b, slot, t0, seq);
    if (nrow <= 0) return;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), rw = w & 3, ch = w >> 2;
    __builtin_assume(w >= 0 && w < 8);
    const unsigned char *krec = p.keys + ((size_t)(b * p.Hk + kh) * p.nslot + slot) * L.key_bytes();
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    f32x4 dq[NTH], dk[NTH];
#pragma unroll
    for (int t = 0; t < NTH; ++t) dq[t] = dk[t] = zero;

    for (int x = 0; x < p.r; ++x) {
        // opaque in every round, or the LDS addresses of all phases stay in registers across rounds
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));
        const int g = lane >> 4, n = lane & 15, h = kh * p.r + x, row0 = perm_row(rw, 4 * g);
        const unsigned char *vrec = p.vals + ((size_t)(b * H + h) * p.nslot + slot) * L.val_bytes();
        const size_t sbase = ((size_t)(b * H + h) * p.nslot + slot) * NSL * SV.bytes();
        const unsigned char *fr = p.fwd + sbase, *rr = p.rev + sbase;
        const float *hd = reinterpret_cast<const float *>(vrec);
        const f32x4 eG = *reinterpret_cast<const f32x4 *>(hd + row0), eL = *reinterpret_cast<const f32x4 *>(hd + 64 + row0);
        const f32x4 be = *reinterpret_cast<const f32x4 *>(hd + 128 + row0);
        const float last = hd[192];
        const int ek = reinterpret_cast<const int *>(vrec)[195], eq = reinterpret_cast<const int *>(vrec)[196];
        const int eb = max(gdr_exp(hd[198]) - 14, -126);  // max |b| 2^eb in [0.5, 1)
        // the smallest exponents over the slices
        int ep = 1 << 20, eu = ep, epr = ep, ex = ep;
#pragma unroll
        for (int s = 0; s < NSL; ++s) {
            const int *a = reinterpret_cast<const int *>(fr + s * SV.bytes()), *c = reinterpret_cast<const int *>(rr + s * SV.bytes());
            ep = min(ep, a[0]);
            eu = min(eu, a[1]);
            epr = min(epr, c[0]);
            ex = min(ex, c[1]);
        }
        auto shift = [](int e, int es) {  // 2^(e - es), e <= es; far smaller blocks vanish beside the largest
            const int d = e - es;
            return (_Float16)pow2f(d < -24 ? -24 : d);
        };
        // slice records into LDS; dot: with what lies there now
        auto stage = [&](const unsigned char *rec, int nb, int off, int piece_off, int eidx, int e, lds_u8 *dst, int piece_dst,
                         auto &&dot) {
            for (int u = w; u < NSL * nb; u += 8) {
                const int s = u / nb, kb = u % nb;
                const unsigned char *r = rec + (size_t)s * SV.bytes();
                const _Float16 f = shift(e, reinterpret_cast<const int *>(r)[eidx]);
                f16x8 v[NI];
#pragma unroll
                for (int y = 0; y < NI; ++y) {
                    v[y] = *reinterpret_cast<const f16x8 *>(r + off + y * piece_off + kb * 1024 + lane * 16);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[y][j] *= f;
                }
                dot(v, dst + u * 1024 + lane * 16);
#pragma unroll
                for (int y = 0; y < NI; ++y) *reinterpret_cast<lds_f16x8 *>(dst + y * piece_dst + u * 1024 + lane * 16) = v[y];
            }
        };
        auto none = [](const f16x8 (&)[NI], const lds_u8 *) {};
        stage(fr, NKB, SV.p_off(0), SV.p_off(1) - SV.p_off(0), 0, ep, sa, PP, none);
        stage(fr, 2, SV.u_off(0), SV.u_off(1) - SV.u_off(0), 1, eu, su, PU, none);
        stage(rr, 2, SV.u_off(0), SV.u_off(1) - SV.u_off(0), 1, ex, sxx, PU, none);
        if (w == 0) {  // G as in the chunk stage
            float gv = 0.f;
            if (lane < nrow)
                gv = to_f(reinterpret_cast<const E *>(p.g)[b * p.sg.b + h * p.sg.h + (long long)(t0 + lane) * p.sg.t]);
            double G = (double)(gv < -1000.f ? -1000.f : gv) * 1.4426950408889634;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const double y = __shfl_up(G, d, 64);
                if (lane >= d) G += y;
            }
            sG[lane] = G;
            sBh[lane] = (_Float16)(hd[128 + lane] * pow2f(eb));
        }
        // dO and V rows of this wave's tile, lane (g, n): token perm_row(rw, n)
        const int tok = perm_row(rw, n), tokc = tok < nrow ? tok : nrow - 1;
        const E *dop = reinterpret_cast<const E *>(p.dout) + b * p.sdo.b + h * p.sdo.h + (long long)(t0 + tokc) * p.sdo.t + 8 * g;
        const E *vp = reinterpret_cast<const E *>(p.v) + b * p.sv.b + h * p.sv.h + (long long)(t0 + tokc) * p.sv.t + 8 * g;
        float xo[NVB][8], xv[(NVB + 1) / 2][8];
        Most mo;
#pragma unroll
        for (int kb = 0; kb < NVB; ++kb) {
            ld8(dop + 32 * kb, xo[kb]);
            if ((kb & 1) == ch) ld8(vp + 32 * kb, xv[kb >> 1]);
        }
#pragma unroll
        for (int kb = 0; kb < NVB; ++kb)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (tok >= nrow) xo[kb][j] = 0.f;
                mo.add(xo[kb][j]);
            }
        const int eo = gdr_exp(mo.wave());
        f16x8 of[NI][NVB];
#pragma unroll
        for (int kb = 0; kb < NVB; ++kb) {
            const f32x4 a = {xo[kb][0], xo[kb][1], xo[kb][2], xo[kb][3]}, c = {xo[kb][4], xo[kb][5], xo[kb][6], xo[kb][7]};
            if constexpr (NI == 2) split_pair(a, c, pow2f(eo), of[0][kb], of[1][kb]);
            else of[0][kb] = round_pair(a, c, pow2f(eo));
        }
        __syncthreads();

        // ---- E1, E2, dO U^T, dX U^T
        f32x4 E1[NTH], E2[NTH], dM[2], dA[2];
#pragma unroll
        for (int t = 0; t < NTH; ++t) E1[t] = E2[t] = zero;
        dM[0] = dM[1] = dA[0] = dA[1] = zero;
        const int nc = rw < 2 ? 1 : 2, c0 = rw < 2 ? ch : 2 * ch;  // token tiles c0 .. c0 + nc - 1
        float xdot = 0.f;
#pragma unroll
        for (int kb = 0; kb < NVB; ++kb) {
            f16x8 xf[NI];
#pragma unroll
            for (int y = 0; y < NI; ++y) xf[y] = ld_slices(sxx + y * PU, 2, kb, rw, lane);
            if ((kb & 1) == ch)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float d = (float)xf[0][j];
                    if constexpr (NI == 2) d += (float)xf[NI - 1][j];
                    xdot = fmaf(d, xv[kb >> 1][j], xdot);
                }
#pragma unroll
            for (int t = 0; t < NTH; ++t) {
                const f16x8 pf = ld_slices(sa, NKB, kb, NTH * ch + t, lane);
                E1[t] = mma16(of[0][kb], pf, E1[t]);
                E2[t] = mma16(xf[0], pf, E2[t]);
                if constexpr (NI == 2) {
                    const f16x8 p1 = ld_slices(sa + PP, NKB, kb, NTH * ch + t, lane);
                    E1[t] = mma16(of[NI - 1][kb], pf, mma16(of[0][kb], p1, E1[t]));
                    E2[t] = mma16(xf[NI - 1], pf, mma16(xf[0], p1, E2[t]));
                }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c)
                if (c < nc) {
                    const f16x8 uf = ld_slices(su, 2, kb, c0 + c, lane);
                    dM[c] = mma16(of[0][kb], uf, dM[c]);
                    dA[c] = mma16(xf[0], uf, dA[c]);
                    if constexpr (NI == 2) {
                        const f16x8 u1 = ld_slices(su + PU, 2, kb, c0 + c, lane);
                        dM[c] = mma16(of[NI - 1][kb], uf, mma16(of[0][kb], u1, dM[c]));
                        dA[c] = mma16(xf[NI - 1], uf, mma16(xf[0], u1, dA[c]));
                    }
                }
        }
        Most m1_, m2_;
#pragma unroll
        for (int c = 0; c < 2; ++c)
            if (c < nc) {
                const int j = perm_row(c0 + c, n);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = row0 + i;
                    const float dec = row >= j ? ex2((float)(sG[row] - sG[j])) : 0.f;
                    dM[c][i] = row >= j ? scale_down(dM[c][i], eo + eu) * dec * p.scale : 0.f;
                    dA[c][i] = row > j ? -scale_down(dA[c][i], ex + eu) * dec : 0.f;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // four rows
                    m1_.add(dM[c][i]);
                    m2_.add(dA[c][i]);
                }
            }
        const float m1 = m1_.wave(), m2 = m2_.wave();
        if (lane == 0) {
            sRed[0][w] = m1;
            sRed[1][w] = m2;
        }
        xdot += __shfl_xor(xdot, 16, 64);
        xdot += __shfl_xor(xdot, 32, 64);
        xdot = scale_down(xdot, ex);  // sum of dX V over this half's value channels, token perm_row(rw, n)
#pragma unroll
        for (int t = 0; t < NTH; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                E1[t][i] = p.scale * eG[i] * scale_down(E1[t][i], eo + ep);
                E2[t][i] = eG[i] * scale_down(E2[t][i], ex + ep);
            }
        __syncthreads();

        // ---- dP' over P, X1 and X2 over dX
        int e1, e2;
        {
            float a = 0.f, c = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                a = fmaxf(a, sRed[0][i]);
                c = fmaxf(c, sRed[1][i]);
            }
            e1 = gdr_exp(a);
            e2 = gdr_exp(c);
        }
        float pd = 0.f;
        stage(rr, NKB, SV.p_off(0), SV.p_off(1) - SV.p_off(0), 0, epr, sa, PP, [&](const f16x8(&v)[NI], const lds_u8 *at) {
            const f16x8 a = *reinterpret_cast<const lds_f16x8 *>(at);
            f16x8 a1 = a;
            if constexpr (NI == 2) a1 = *reinterpret_cast<const lds_f16x8 *>(at + PP);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (NI == 2) pd = fmaf((float)a[j] + (float)a1[j], (float)v[0][j] + (float)v[NI - 1][j], pd);
                else pd = fmaf((float)a[j], (float)v[0][j], pd);
            }
        });
        pd = scale_down(pd, ep + epr);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) pd += __shfl_xor(pd, d, 64);
        if (lane == 0) sRed[2][w] = pd;
        lds_u8 *s1 = sxx, *s2 = sxx + NI * 8192;  // [piece][column tile][kb]
#pragma unroll
        for (int c = 0; c < 2; ++c)
            if (c < nc) {
                f16x4 hi, lo;
                const int at = ((c0 + c) * 2 + (rw >> 1)) * 1024;
                if constexpr (NI == 2) {
                    split4(dM[c], pow2f(e1), hi, lo);
                    st_half_frag(s1 + 8192 + at, rw & 1, g, n, lo);
                } else {
                    hi = round4(dM[c], pow2f(e1));
                }
                st_half_frag(s1 + at, rw & 1, g, n, hi);
                if constexpr (NI == 2) {
                    split4(dA[c], pow2f(e2), hi, lo);
                    st_half_frag(s2 + 8192 + at, rw & 1, g, n, lo);
                } else {
                    hi = round4(dA[c], pow2f(e2));
                }
                st_half_frag(s2 + at, rw & 1, g, n, hi);
            }
        __syncthreads();

        // ---- E3 = U dP'^T
        f32x4 E3[NTH];
#pragma unroll
        for (int t = 0; t < NTH; ++t) E3[t] = zero;
#pragma unroll
        for (int kb = 0; kb < NVB; ++kb) {
            f16x8 uf[NI];
#pragma unroll
            for (int y = 0; y < NI; ++y) uf[y] = ld_slices(su + y * PU, 2, kb, rw, lane);
#pragma unroll
            for (int t = 0; t < NTH; ++t) {
                const f16x8 pf = ld_slices(sa, NKB, kb, NTH * ch + t, lane);
                E3[t] = mma16(uf[0], pf, E3[t]);
                if constexpr (NI == 2)
                    E3[t] = mma16(uf[NI - 1], pf, mma16(uf[0], ld_slices(sa + PP, NKB, kb, NTH * ch + t, lane), E3[t]));
            }
        }
#pragma unroll
        for (int t = 0; t < NTH; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) E3[t][i] = eL[i] * scale_down(E3[t][i], eu + epr);
        __syncthreads();

        // ---- K and Q over dP'
        for (int u = w; u < 2 * NI * L.mat() / 1024; u += 8)
            *reinterpret_cast<lds_f16x8 *>(sa + u * 1024 + lane * 16) =
                *reinterpret_cast<const f16x8 *>(krec + 256 + u * 1024 + lane * 16);
        __syncthreads();
        const lds_u8 *sk = sa, *sq = sa + NI * L.mat();
        float aG[4] = {0.f, 0.f, 0.f, 0.f}, aB[4] = {0.f, 0.f, 0.f, 0.f}, aL[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = 0; t < NTH; ++t) {
            const int tile = NTH * ch + t;
            auto tok_op = [&](const lds_u8 *base, int kb) {  // k = tokens of block kb, columns = dk tile
                const lds_u8 *f0 = base + (2 * kb * NKB + (tile >> 1)) * 1024;
                return ld_frag_t(f0, f0 + NKB * 1024, tile, lane);
            };
            f32x4 q1 = zero, k1 = zero, r = zero, s = zero;  // X1 K, X1^T Q, X2 K, X2^T diag(b) K
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                f16x8 kf[NI], qf[NI];
#pragma unroll
                for (int y = 0; y < NI; ++y) {
                    kf[y] = tok_op(sk + y * L.mat(), kb);
                    qf[y] = tok_op(sq + y * L.mat(), kb);
                }
                if (kb == 0 || rw >= 2) {  // rows of X: tokens of tile rw over columns of block kb
                    const int at = (4 * kb + (rw >> 1)) * 1024;
                    f16x8 a[NI], c[NI];
#pragma unroll
                    for (int y = 0; y < NI; ++y) {
                        a[y] = ld_frag_t(s1 + y * 8192 + at, s1 + y * 8192 + at + 2048, rw, lane);
                        c[y] = ld_frag_t(s2 + y * 8192 + at, s2 + y * 8192 + at + 2048, rw, lane);
                    }
                    q1 = mma16(a[0], kf[0], q1);
                    r = mma16(c[0], kf[0], r);
                    if constexpr (NI == 2) {
                        q1 = mma16(a[NI - 1], kf[0], mma16(a[0], kf[NI - 1], q1));
                        r = mma16(c[NI - 1], kf[0], mma16(c[0], kf[NI - 1], r));
                    }
                }
                if (kb == 1 || rw < 2) {  // columns of X: tokens of tile rw over rows of block kb
                    const int at = (2 * rw + kb) * 1024;
                    f16x8 a[NI], c[NI];
#pragma unroll
                    for (int y = 0; y < NI; ++y) {
                        a[y] = ld_frag(s1 + y * 8192 + at, lane);
                        c[y] = ld_frag(s2 + y * 8192 + at, lane);
                    }
                    if constexpr (NI == 2) {
                        f32x4 lo4, hi4;
                        const float *bb = hd + 128 + 32 * kb + 8 * g;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            lo4[j] = ((float)c[0][j] + (float)c[NI - 1][j]) * (bb[j] * pow2f(eb));
                            hi4[j] = ((float)c[0][4 + j] + (float)c[NI - 1][4 + j]) * (bb[4 + j] * pow2f(eb));
                        }
                        split_pair(lo4, hi4, 1.f, c[0], c[NI - 1]);
                    } else {
                        c[0] *= *reinterpret_cast<const f16x8 *>(sBh + 32 * kb + 8 * g);
                    }
                    k1 = mma16(a[0], qf[0], k1);
                    s = mma16(c[0], kf[0], s);
                    if constexpr (NI == 2) {
                        k1 = mma16(a[NI - 1], qf[0], mma16(a[0], qf[NI - 1], k1));
                        s = mma16(c[NI - 1], kf[0], mma16(c[0], kf[NI - 1], s));
                    }
                }
            }
            f16x4 kd = ld_acc(sk + (rw * NKB + (tile >> 1)) * 1024, tile, lane);
            f16x4 qd = ld_acc(sq + (rw * NKB + (tile >> 1)) * 1024, tile, lane);
            f16x4 kd1 = kd, qd1 = qd;
            if constexpr (NI == 2) {
                kd1 = ld_acc(sk + L.mat() + (rw * NKB + (tile >> 1)) * 1024, tile, lane);
                qd1 = ld_acc(sq + L.mat() + (rw * NKB + (tile >> 1)) * 1024, tile, lane);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float kv = (float)kd[i], qv = (float)qd[i];
                if constexpr (NI == 2) {
                    kv += (float)kd1[i];
                    qv += (float)qd1[i];
                }
                kv = scale_down(kv, ek);
                qv = scale_down(qv, eq);
                const float dqh = E1[t][i] + scale_down(q1[i], e1 + ek);
                const float x1 = scale_down(k1[i], e1 + eq), rr_ = scale_down(r[i], e2 + ek), ss = scale_down(s[i], e2 + ek + eb);
                dq[t][i] += dqh;
                dk[t][i] += x1 + E3[t][i] - be[i] * E2[t][i] + be[i] * rr_ + ss;
                aG[i] += qv * dqh - kv * (x1 + E3[t][i] + be[i] * E2[t][i] - be[i] * rr_ + ss);
                aB[i] += kv * (rr_ - E2[t][i]);
                aL[i] += kv * E3[t][i];
            }
        }
        float sl = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            aG[i] = row_sum(aG[i]);
            aB[i] = row_sum(aB[i]);
            sl += aL[i];
            if (n == 0) {
                sGi[ch][row0 + i] = aG[i];
                sBe[ch][row0 + i] = aB[i];
            }
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) sl += __shfl_xor(sl, d, 64);
        if (lane == 0) sRed[3][w] = sl;
        __syncthreads();
        if (g == 0) sBe[ch][tok] += xdot;  // one lane per (half, token)
        __syncthreads();
        if (w == 0) {
            float gl = 0.f, pl = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                gl += sRed[3][i];
                pl += sRed[2][i];
            }
            float dG = sGi[0][lane] + sGi[1][lane];
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const float y = __shfl_down(dG, d, 64);
                if (lane + d < 64) dG += y;
            }
            if (lane < nrow) {
                const size_t at = (size_t)(b * H + h) * p.seqs.T + t0 + lane;
                reinterpret_cast<E *>(p.dg)[at] = from_f<E>(dG + gl + last * pl);
                reinterpret_cast<E *>(p.dbeta)[at] = from_f<E>(sBe[0][lane] + sBe[1][lane]);
            }
        }
    }
    const int lane = threadIdx.x & 63, row0 = perm_row(rw, 4 * (lane >> 4));
    E *qo = reinterpret_cast<E *>(p.dq) + ((size_t)(b * p.Hk + kh) * p.seqs.T + t0 + row0) * DK;
    E *ko = reinterpret_cast<E *>(p.dk) + ((size_t)(b * p.Hk + kh) * p.seqs.T + t0 + row0) * DK;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (row0 + i < nrow)
#pragma unroll
            for (int t = 0; t < NTH; ++t) {
                const int c = perm_row(NTH * ch + t, lane & 15);
                qo[i * DK + c] = from_f<E>(dq[t][i]);
                ko[i * DK + c] = from_f<E>(dk[t][i]);
            }
}

// Gradients of the tokens of a packed stream that no document covers: zeros in front of the first
// boundary and behind the last.
template <typename E>
__global__ __launch_bounds__(256) void gdr_uncovered_kernel(GdrSeqs seqs, int Hk, int H, int dk, int dv, E *dq, E *dko, E *dvo,
                                                           E *dg, E *db) {
    const int y = blockIdx.y, a = seqs.clip(seqs.cu[0]), z = max(a, seqs.clip(seqs.cu[seqs.N]));
    const long long n = a + (seqs.T - z);
    auto fill = [&](E *to, long long w) {  // rows of w values
        for (long long i = blockIdx.x * 256 + threadIdx.x; i < n * w; i += 256 * gridDim.x) {
            const long long row = i / w;
            to[((size_t)y * seqs.T + (row < a ? row : z + row - a)) * w + i % w] = (E)0.f;
        }
    };
    if (y < Hk) {
        fill(dq, dk);
        fill(dko, dk);
    }
    fill(dvo, dv);
    fill(dg, 1);
    fill(db, 1);
}

}  // namespace kda
