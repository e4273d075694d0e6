// Reverse pass of the gated delta rule's backward (gdr_common.h): walks the chunks of one (sequence,
// value head) from the last to the first with 16 NCT columns of dP, the gradient of a chunk's end
// state P', in the registers of four waves laid out as in gdr_state.h:
//   1. dU = M^T dO + e^{G_last - G} K dP'                 pieces of dU to LDS, barrier
//   2. dX = T^T dU                                        pieces of F = b e^G dX to LDS, barrier
//   3. dP = e^{G_last} dP' + Q^T (scale e^G dO) - K^T F   pieces of dP to LDS, barrier
// Four more waves make the terms without the state a chunk ahead, M^T dO and Q^T (scale e^G dO), which
// reach the chain as float32 tiles, lane to lane; they load everything but K's plain fragments, write
// dV = diag(b) dX, and keep every chunk's dP' and dX, as fp16, for the gradient stage.
//
// M, T, Q and K are all needed transposed, so they go through LDS; each part is brought there two
// intervals before it is read, Q, M and dO two chunks ahead, K and T in the chunk itself.  The
// exponents of the pieces come from bounds as in gdr_state.h, |dU| <= max|M^T dO| + max(e^{G_last - G}
// |k|_1) max|dP'|, |dX| <= 64 max|T| max|dU|, |dP| <= e^{G_last} max|dP'| + max|Q^T H| + sum(max|k|)
// max|F|.  H and F have their own, of the decayed values, F_j = b_j sum_i (T_ij e^{G_j - G_i}) e^{G_i} dU_i
// with |e^G dU| <= max|e^G M^T dO| + e^{G_last} max|k|_1 max|dP'|: where the chunk's first tokens have no
// gradient, both are as small as the decay over them.  A state gradient that a caller asks for
// (dinitial_state, float32) is exact to the same 22 bits as the final state.
//
// 4096 tokens x 32 heads: 2.5 us a chunk, 159 us; with everything on the chain's four waves, and a
// fourth barrier for dP's maximum, 3.2 us, 204 us.
#pragma once
#include "gdr_state.h"

namespace kda {

struct GdrRevArgs {
    const unsigned char *keys, *vals;
    const void *dout;
    Strides3 sdo;
    GdrSeqs seqs;
    int H, r, nslot, dv;
    float scale;
    const float *dfinal;       // nullable [N][H][dv][dk]
    float *dinit;              // nullable
    void *dv_out;              // [B][H][T][dv], contiguous
    unsigned char *save;       // GdrSave records: dP' in the place of P, dX in the place of U
};

template <int DK, int NI, int NCT> struct GdrRevLds {
    static constexpr int NKB = DK / 32, KB = NI * 64 * DK * 2;
    // dP' [piece][kb][ct]; dU, F = b e^G dX, H = scale e^G dO [piece][kb 2][ct]; dO [piece < NI][kb 2][ct]
    static constexpr int XP = 0, XU = XP + 2 * NKB * NCT * 1024, XF = XU + 4 * NCT * 1024, XH = XF + 4 * NCT * 1024;
    static constexpr int XO = XH + 4 * NCT * 1024;
    // float32 tiles from lane to lane: M^T dO and dX [wave][ct], Q^T H [wave][tile][ct]
    static constexpr int D0 = XO + NI * 2 * NCT * 1024, DX = D0 + 4 * NCT * 1024, DQ = DX + 4 * NCT * 1024;
    static constexpr int K = DQ + (DK / 16) * NCT * 1024, T = K + KB, Q = T + 2 * GdrLayout::kTri, M = Q + KB;
    static constexpr int HEAD = M + 2 * GdrLayout::kTri, BYTES = HEAD + 2 * GdrLayout::kHead;
};

template <int DK, bool F32, int NCT>
__global__ __launch_bounds__(512) void gdr_rev_kernel(const GdrRevArgs p) {
    using E = typename std::conditional<F32, float, __bf16>::type;
    constexpr int NI = F32 ? 2 : 1, NKB = DK / 32, NTW = DK / 64;
    using S = GdrRevLds<DK, NI, NCT>;
    constexpr GdrLayout L{NI, DK, 2};
    constexpr GdrSave SV{NI, DK};
    typedef __attribute__((address_space(3))) f16x8 lds_f16x8;
    typedef __attribute__((address_space(3))) f32x4 lds_f4;
    typedef __attribute__((address_space(3))) float lds_f1;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[S::BYTES];
    // per wave: max |dP'|, |dU|, |F|, |dO|, |M^T dO|, |Q^T H|, |e^G M^T dO|, |e^G dO|
    __shared__ __attribute__((aligned(16))) float sMax[32];
    __shared__ int sExp[2];     // exponents of dP's and of dX's pieces
    const int lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wid & 3;
    __builtin_assume(w >= 0 && w < 4);
    const int gh = p.dv / (16 * NCT), id = blockIdx.x;
    const int unit = id / (8 * gh) * 8 + (id & 7), slice = (id >> 3) % gh * NCT;
    if (unit >= p.seqs.N * p.H) return;
    const int seq = unit / p.H, h = unit % p.H, b = p.seqs.batch(seq);
    const int len = p.seqs.length(seq), start = p.seqs.start(seq), nchunk = (len + 63) / 64;
    const int col = slice * 16 + n, nkey = p.H / p.r;
    const size_t slot0 = p.seqs.slot0(seq);
    const unsigned char *krec = p.keys + ((size_t)(b * nkey + h / p.r) * p.nslot + slot0) * L.key_bytes();
    const unsigned char *vrec = p.vals + ((size_t)(b * p.H + h) * p.nslot + slot0) * L.val_bytes();
    const int row0 = perm_row(w, 4 * g), fo = frag_slot(g, n);
    lds_u8 *sx = lds_base(smem);
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    // rows of the transpose of a 64x64 lower triangle: column tile w, contraction block kb (>= w's own)
    auto tri_t = [&](const lds_u8 *f, int kb) {
        const lds_u8 *f0 = f + tri_frag(2 * kb, w >> 1) * 1024, *f1 = f + tri_frag(2 * kb + 1, w >> 1) * 1024;
        return ld_frag_t(f0, f1, w, lane);
    };

    if (wid >= 4) {  // ------------------------- loads, the terms without the state, outputs
        const E *dop = reinterpret_cast<const E *>(p.dout) + b * p.sdo.b + h * p.sdo.h + (long long)start * p.sdo.t + col;
        E *dvp = reinterpret_cast<E *>(p.dv_out) + ((size_t)(b * p.H + h) * p.seqs.T + start + row0) * p.dv + col;
        unsigned char *save = p.save + (((size_t)(b * p.H + h) * p.nslot + slot0) * (p.dv / 16) + slice) * SV.bytes();
        // a quarter of each; chunks before the first are loaded as the first and not used
        f16x8 kf[NI][NKB], tf[3], qf[NI][NKB], mf[3];
        E vn[NCT][4];
        f32x4 eG;
        float head;
        int em, eq, at = 0;  // at: the chunk of qf, mf, vn
        auto load_kt = [&](int c) {
            c = max(c, 0);
            const unsigned char *r = krec + (size_t)c * L.key_bytes() + w * NKB * 1024 + fo;
            const unsigned char *t = vrec + (size_t)c * L.val_bytes() + 3 * w * 1024 + fo;
#pragma unroll
            for (int x = 0; x < NI; ++x)
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb) kf[x][kb] = *reinterpret_cast<const f16x8 *>(r + L.k_off(x) + kb * 1024);
#pragma unroll
            for (int i = 0; i < 3; ++i) tf[i] = *reinterpret_cast<const f16x8 *>(t + L.t_off(0) + i * 1024);
        };
        auto load_head = [&](int c) {
            head = *reinterpret_cast<const float *>(vrec + (size_t)max(c, 0) * L.val_bytes() + 4 * (64 * w + lane));
        };
        auto load_qm = [&](int c) {
            at = c = max(c, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = min(64 * c + row0 + i, len - 1);
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) vn[ct][i] = dop[(long long)row * p.sdo.t + 16 * ct];
            }
            const unsigned char *r = krec + (size_t)c * L.key_bytes() + w * NKB * 1024 + fo;
            const unsigned char *v = vrec + (size_t)c * L.val_bytes();
            eG = *reinterpret_cast<const f32x4 *>(v + 4 * row0);
#pragma unroll
            for (int x = 0; x < NI; ++x)
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb) qf[x][kb] = *reinterpret_cast<const f16x8 *>(r + L.q_off(x) + kb * 1024);
#pragma unroll
            for (int i = 0; i < 3; ++i) mf[i] = *reinterpret_cast<const f16x8 *>(v + L.m_off(0) + (3 * w + i) * 1024 + fo);
            em = reinterpret_cast<const int *>(v)[194];
            eq = reinterpret_cast<const int *>(v)[196];
        };
        auto grad_of = [&](int ct, int i) { return 64 * at + row0 + i < len ? to_f(vn[ct][i]) : 0.f; };  // none past the last row
        auto publish_max = [&]() {
            __builtin_amdgcn_sched_barrier(0);  // mixed in with what stands before, 2 % slower
            Most mo, mg;
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                const f32x4 d = {grad_of(ct, 0), grad_of(ct, 1), grad_of(ct, 2), grad_of(ct, 3)};
                mo.add4(d);
                mg.add4(eG * d);
            }
            const float m = mo.wave(), mh = mg.wave();
            if (lane == 0) {
                sMax[12 + w] = m;
                sMax[28 + w] = mh;
            }
        };
        auto put_kt = [&]() {
#pragma unroll
            for (int x = 0; x < NI; ++x)
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb)
                    *reinterpret_cast<lds_f16x8 *>(sx + S::K + x * L.mat() + (w * NKB + kb) * 1024 + fo) = kf[x][kb];
#pragma unroll
            for (int i = 0; i < 3; ++i) *reinterpret_cast<lds_f16x8 *>(sx + S::T + (3 * w + i) * 1024 + fo) = tf[i];
        };
        auto put_head = [&](int c) { *reinterpret_cast<lds_f1 *>(sx + S::HEAD + (c & 1) * L.kHead + 4 * (64 * w + lane)) = head; };
        int eo = 0, eh = 0, em_ = 0, eq_ = 0;  // of what is in LDS
        f32x4 eG_ = zero;
        auto put_qm = [&]() {
            eo = gdr_exp(max4(sMax + 12));
            eh = gdr_exp(fabsf(p.scale) * max4(sMax + 28));
            em_ = em;
            eq_ = eq;
            eG_ = eG;
#pragma unroll
            for (int x = 0; x < NI; ++x)
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb)
                    *reinterpret_cast<lds_f16x8 *>(sx + S::Q + x * L.mat() + (w * NKB + kb) * 1024 + fo) = qf[x][kb];
#pragma unroll
            for (int i = 0; i < 3; ++i) *reinterpret_cast<lds_f16x8 *>(sx + S::M + (3 * w + i) * 1024 + fo) = mf[i];
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                const f32x4 d = {grad_of(ct, 0), grad_of(ct, 1), grad_of(ct, 2), grad_of(ct, 3)};
                f32x4 hd;
#pragma unroll
                for (int i = 0; i < 4; ++i) hd[i] = p.scale * eG[i] * d[i];
                f16x4 hi, lo;
                const int to = ((w >> 1) * NCT + ct) * 1024;
                if constexpr (NI == 2) {
                    split4(d, pow2f(eo), hi, lo);
                    st_half_frag(sx + S::XO + 2 * NCT * 1024 + to, w & 1, g, n, lo);
                } else {
                    hi = round4(d, pow2f(eo));  // exact
                }
                st_half_frag(sx + S::XO + to, w & 1, g, n, hi);
                split4(hd, pow2f(eh), hi, lo);
                st_half_frag(sx + S::XH + to, w & 1, g, n, hi);
                st_half_frag(sx + S::XH + 2 * NCT * 1024 + to, w & 1, g, n, lo);
            }
        };
        f32x4 d0[NCT];
        auto mul_m = [&]() {  // M^T dO
            f32x4 y[NCT], y1[NCT];
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) y[ct] = y1[ct] = zero;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
                if (kb == 1 || w < 2) {
                    const f16x8 mh = tri_t(sx + S::M, kb), ml = tri_t(sx + S::M + L.kTri, kb);
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct) {
                        const f16x8 oh = ld_frag(sx + S::XO + (kb * NCT + ct) * 1024, lane);
                        y[ct] = mma16(mh, oh, y[ct]);
                        y1[ct] = mma16(ml, oh, y1[ct]);
                        if constexpr (NI == 2) y1[ct] = mma16(mh, ld_frag(sx + S::XO + ((2 + kb) * NCT + ct) * 1024, lane), y1[ct]);
                    }
                }
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                for (int i = 0; i < 4; ++i) d0[ct][i] = scale_down(y[ct][i] + y1[ct][i], em_ + eo);
        };
        auto put_terms = [&]() {  // M^T dO, and Q^T (scale e^G dO)
            Most m0_, mg_, mq_;
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                *reinterpret_cast<lds_f4 *>(sx + S::D0 + (w * NCT + ct) * 1024 + 16 * lane) = d0[ct];
                m0_.add4(d0[ct]);
                mg_.add4(eG_ * d0[ct]);
            }
#pragma unroll
            for (int t = 0; t < NTW; ++t) {
                const int tile = NTW * w + t;
                f32x4 a[NCT], a1[NCT];
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) a[ct] = a1[ct] = zero;
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    const lds_u8 *f0 = sx + S::Q + (2 * kb * NKB + (tile >> 1)) * 1024, *f1 = f0 + NKB * 1024;
                    const f16x8 q = ld_frag_t(f0, f1, tile, lane);
                    f16x8 q1 = q;
                    if constexpr (NI == 2) q1 = ld_frag_t(f0 + L.mat(), f1 + L.mat(), tile, lane);
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct) {
                        const f16x8 hh = ld_frag(sx + S::XH + (kb * NCT + ct) * 1024, lane);
                        const f16x8 hl = ld_frag(sx + S::XH + ((2 + kb) * NCT + ct) * 1024, lane);
                        a[ct] = mma16(q, hh, a[ct]);
                        a1[ct] = mma16(q, hl, a1[ct]);
                        if constexpr (NI == 2) a1[ct] = mma16(q1, hh, a1[ct]);
                    }
                }
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[ct][i] = scale_down(a[ct][i] + a1[ct][i], eq_ + eh);
                    *reinterpret_cast<lds_f4 *>(sx + S::DQ + (tile * NCT + ct) * 1024 + 16 * lane) = a[ct];
                    mq_.add4(a[ct]);
                }
            }
            const float m0 = m0_.wave(), mg = mg_.wave(), mq = mq_.wave();
            if (lane == 0) {
                sMax[16 + w] = m0;
                sMax[24 + w] = mg;
                sMax[20 + w] = mq;
            }
        };
        if (nchunk > 0) {
            load_qm(nchunk - 1);
            load_head(nchunk - 1);
            publish_max();
            barrier_lds();  // (a)
            put_qm();
            load_qm(nchunk - 2);
            barrier_lds();  // (b)
            mul_m();
            put_terms();
            put_head(nchunk - 1);
            load_head(nchunk - 2);
            publish_max();
            barrier_lds();  // (c)
            put_qm();
            load_qm(nchunk - 3);
            load_kt(nchunk - 1);
        }
        // chunk c's K and T, c - 1's terms and header, c - 2's Q, M and dO go to LDS
        for (int c = nchunk - 1; c >= 0; --c) {
            barrier_lds();  // (1)
            const int ep = sExp[0];
            put_kt();
            mul_m();
            if (w < NKB)
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) {
                    const f16x8 ph = ld_frag(sx + S::XP + (w * NCT + ct) * 1024, lane);
                    const f16x8 pl = ld_frag(sx + S::XP + ((NKB + w) * NCT + ct) * 1024, lane);
                    unsigned char *sv = save + ((size_t)c * (p.dv / 16) + ct) * SV.bytes() + w * 1024 + fo;
                    if constexpr (NI == 2) {
                        *reinterpret_cast<f16x8 *>(sv + SV.p_off(0)) = ph;
                        *reinterpret_cast<f16x8 *>(sv + SV.p_off(1)) = pl;
                    } else {
                        *reinterpret_cast<f16x8 *>(sv + SV.p_off(0)) = ph + pl;  // both pieces together round to one
                    }
                }
            barrier_lds();  // (2)
            load_kt(c - 1);
            put_terms();
            put_head(c - 1);
            load_head(c - 2);
            publish_max();
            barrier_lds();  // (3)
            const int ex = sExp[1];
            f32x4 dX[NCT];
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) dX[ct] = *reinterpret_cast<const lds_f4 *>(sx + S::DX + (w * NCT + ct) * 1024 + 16 * lane);
            const f32x4 be = *reinterpret_cast<const lds_f4 *>(sx + S::HEAD + (c & 1) * L.kHead + 512 + 4 * row0);
            put_qm();
            load_qm(c - 3);
            unsigned char *sv = save + (size_t)c * (p.dv / 16) * SV.bytes();
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                f16x4 hi, lo;
                if constexpr (NI == 2) split4(dX[ct], pow2f(ex), hi, lo);
                else hi = round4(dX[ct], pow2f(ex));
                unsigned char *to = sv + ct * SV.bytes() + (w >> 1) * 1024 + fo + 8 * (w & 1);
                *reinterpret_cast<f16x4 *>(to + SV.u_off(0)) = hi;
                if constexpr (NI == 2) *reinterpret_cast<f16x4 *>(to + SV.u_off(1)) = lo;
                if (w == 0 && lane == 0) {
                    reinterpret_cast<int *>(sv + ct * SV.bytes())[0] = ep;
                    reinterpret_cast<int *>(sv + ct * SV.bytes())[1] = ex;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (64 * c + row0 + i < len) dvp[(size_t)(64 * c + i) * p.dv + 16 * ct] = from_f<E>(be[i] * dX[ct][i]);
            }
        }
        return;
    }

    // ------------------------------------------ the chain
    __builtin_amdgcn_s_setprio(3);
    f32x4 P[NTW][NCT];  // dP
    const size_t state0 = ((size_t)(seq * p.H + h) * p.dv + col) * DK;
#pragma unroll
    for (int t = 0; t < NTW; ++t)
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
            P[t][ct] = p.dfinal == nullptr ? zero
                           : *reinterpret_cast<const f32x4 *>(p.dfinal + state0 + (size_t)16 * ct * DK + perm_row(NTW * w + t, 4 * g));
    auto max_p = [&]() {
        Most m;
#pragma unroll
        for (int t = 0; t < NTW; ++t)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) m.add4(P[t][ct]);
        return m.wave();
    };
    auto put_p = [&](int e) {
        const float s = pow2f(e);
#pragma unroll
        for (int t = 0; t < NTW; ++t)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                f16x4 hi, lo;
                split4(P[t][ct], s, hi, lo);
                const int tile = NTW * w + t;
                lds_u8 *f = sx + S::XP + ((tile >> 1) * NCT + ct) * 1024;
                st_half_frag(f, tile & 1, g, n, hi);
                st_half_frag(f + NKB * NCT * 1024, tile & 1, g, n, lo);
            }
    };
    f16x8 kf[NI][NKB];
    f32x4 eG, eL, be, h0, h1, h2, D0[NCT], DQ[NTW][NCT];
    f32x4 md, mdg, mq;
    auto load_k = [&](int c) {
        const unsigned char *r = krec + (size_t)max(c, 0) * L.key_bytes() + w * NKB * 1024 + fo;
#pragma unroll
        for (int x = 0; x < NI; ++x)
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) kf[x][kb] = *reinterpret_cast<const f16x8 *>(r + L.k_off(x) + kb * 1024);
    };
    // what the other waves have laid out for chunk c
    auto get = [&](int c) {
        const lds_u8 *hd = sx + S::HEAD + (c & 1) * L.kHead;
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
            D0[ct] = *reinterpret_cast<const lds_f4 *>(sx + S::D0 + (w * NCT + ct) * 1024 + 16 * lane);
#pragma unroll
            for (int t = 0; t < NTW; ++t)
                DQ[t][ct] = *reinterpret_cast<const lds_f4 *>(sx + S::DQ + ((NTW * w + t) * NCT + ct) * 1024 + 16 * lane);
        }
        eG = *reinterpret_cast<const lds_f4 *>(hd + 4 * row0);
        eL = *reinterpret_cast<const lds_f4 *>(hd + 256 + 4 * row0);
        be = *reinterpret_cast<const lds_f4 *>(hd + 512 + 4 * row0);
        h0 = *reinterpret_cast<const lds_f4 *>(hd + 768);
        h1 = *reinterpret_cast<const lds_f4 *>(hd + 784);
        h2 = *reinterpret_cast<const lds_f4 *>(hd + 800);
        md = *reinterpret_cast<const f32x4 *>(sMax + 16);  // their maxima where they are used
        mdg = *reinterpret_cast<const f32x4 *>(sMax + 24);
        mq = *reinterpret_cast<const f32x4 *>(sMax + 20);
    };
    int ep = 0;
    if (nchunk > 0) {
        load_k(nchunk - 1);
        const float mp = max_p();
        if (lane == 0) sMax[w] = mp;
        barrier_lds();  // (a)
        ep = gdr_exp(max4(sMax));
        put_p(ep);
        if (threadIdx.x == 0) sExp[0] = ep;
        barrier_lds();  // (b)
        barrier_lds();  // (c)
        get(nchunk - 1);
    }
    for (int c = nchunk - 1; c >= 0; --c) {
        barrier_lds();  // (1)
        const float et_ = h0[1], ek_ = h0[3];
        const int et = __builtin_bit_cast(int, et_), ek = __builtin_bit_cast(int, ek_);
        const float pmax = max4(sMax), last = h0[0], bm = h1[2], ksum = h2[0], cl = h2[1], ubound = h2[2], k1 = h2[3];

        // ---- 1. dU = M^T dO + e^{G_last - G} K dP'
        f32x4 Z[NCT], Z1[NCT];
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) Z[ct] = Z1[ct] = zero;
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                const f16x8 ph = ld_frag(sx + S::XP + (kb * NCT + ct) * 1024, lane);
                const f16x8 pl = ld_frag(sx + S::XP + ((NKB + kb) * NCT + ct) * 1024, lane);
                Z[ct] = mma16(kf[0][kb], ph, Z[ct]);
                Z1[ct] = mma16(kf[0][kb], pl, Z1[ct]);
                if constexpr (NI == 2) Z1[ct] = mma16(kf[1][kb], ph, Z1[ct]);
            }
        const int eu = gdr_exp(max4(md) + cl * pmax);
        Most mu;
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
            f32x4 dU;
#pragma unroll
            for (int i = 0; i < 4; ++i) dU[i] = D0[ct][i] + eL[i] * scale_down(Z[ct][i] + Z1[ct][i], ek + ep);
            mu.add4(dU);
            f16x4 hi, lo;
            split4(dU, pow2f(eu), hi, lo);
            lds_u8 *f = sx + S::XU + ((w >> 1) * NCT + ct) * 1024;
            st_half_frag(f, w & 1, g, n, hi);
            st_half_frag(f + 2 * NCT * 1024, w & 1, g, n, lo);
        }
        const float um = mu.wave();
        if (lane == 0) sMax[4 + w] = um;
        const float gbound = 64.f * ubound * (max4(mdg) + last * pmax * k1);  // of e^G dX
        load_k(c - 1);
        barrier_lds();  // (2)

        // ---- 2. dX = T^T dU, F = b e^G dX
        const float xbound = 64.f * ldexp2(1.f, 14 - et) * max4(sMax + 4);
        const int ex = gdr_exp(xbound), ef = gdr_exp(bm * fminf(xbound, gbound));
        Most mf;
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
            f32x4 z = zero, z1 = zero;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
                if (kb == 1 || w < 2) {
                    const f16x8 th = tri_t(sx + S::T, kb), tl = tri_t(sx + S::T + L.kTri, kb);
                    const f16x8 uh = ld_frag(sx + S::XU + (kb * NCT + ct) * 1024, lane);
                    const f16x8 ul = ld_frag(sx + S::XU + ((2 + kb) * NCT + ct) * 1024, lane);
                    z = mma16(th, uh, z);
                    z1 = mma16(tl, uh, mma16(th, ul, z1));
                }
            f32x4 dX, F;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dX[i] = scale_down(z[i] + z1[i], et + eu);
                F[i] = be[i] * eG[i] * dX[i];
            }
            mf.add4(F);
            f16x4 hi, lo;
            split4(F, pow2f(ef), hi, lo);
            lds_u8 *f = sx + S::XF + ((w >> 1) * NCT + ct) * 1024;
            st_half_frag(f, w & 1, g, n, hi);
            st_half_frag(f + 2 * NCT * 1024, w & 1, g, n, lo);
            *reinterpret_cast<lds_f4 *>(sx + S::DX + (w * NCT + ct) * 1024 + 16 * lane) = dX;
        }
        const float fm = mf.wave();
        if (lane == 0) sMax[8 + w] = fm;
        if (threadIdx.x == 0) sExp[1] = ex;
        barrier_lds();  // (3)

        // ---- 3. dP = e^{G_last} dP' + Q^T H - K^T F
        f16x8 fh[2][NCT], fl[2][NCT], kt[NI][NTW][2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                fh[kb][ct] = ld_frag(sx + S::XF + (kb * NCT + ct) * 1024, lane);
                fl[kb][ct] = ld_frag(sx + S::XF + ((2 + kb) * NCT + ct) * 1024, lane);
            }
#pragma unroll
            for (int t = 0; t < NTW; ++t) {
                const int tile = NTW * w + t;
                const lds_u8 *f0 = sx + S::K + (2 * kb * NKB + (tile >> 1)) * 1024, *f1 = f0 + NKB * 1024;
#pragma unroll
                for (int x = 0; x < NI; ++x) kt[x][t][kb] = ld_frag_t(f0 + x * L.mat(), f1 + x * L.mat(), tile, lane);
            }
        }
        const float fmax = max4(sMax + 8);
        f32x4 base[NTW][NCT];
#pragma unroll
        for (int t = 0; t < NTW; ++t)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                for (int i = 0; i < 4; ++i) base[t][ct][i] = fmaf(P[t][ct][i], last, DQ[t][ct][i]);
        const float qmax = max4(mq);
        __builtin_amdgcn_sched_barrier(0);
        get(c - 1);  // behind the reads that are waited for
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < NTW; ++t) {
            f32x4 d[NCT], d1[NCT];
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) d[ct] = d1[ct] = zero;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) {
                    d[ct] = mma16(kt[0][t][kb], fh[kb][ct], d[ct]);
                    d1[ct] = mma16(kt[0][t][kb], fl[kb][ct], d1[ct]);
                    if constexpr (NI == 2) d1[ct] = mma16(kt[1][t][kb], fh[kb][ct], d1[ct]);
                }
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                for (int i = 0; i < 4; ++i) P[t][ct][i] = base[t][ct][i] - scale_down(d[ct][i] + d1[ct][i], ek + ef);
        }
        ep = gdr_exp(last * pmax + qmax + ksum * fmax);
        put_p(ep);
        const float mp = max_p();
        if (lane == 0) sMax[w] = mp;
        if (threadIdx.x == 0) sExp[0] = ep;
    }
    if (p.dinit != nullptr)
#pragma unroll
        for (int t = 0; t < NTW; ++t)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
                *reinterpret_cast<f32x4 *>(p.dinit + state0 + (size_t)16 * ct * DK + perm_row(NTW * w + t, 4 * g)) = P[t][ct];
}

}  // namespace kda
