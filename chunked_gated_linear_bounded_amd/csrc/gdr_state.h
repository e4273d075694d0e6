// Sequential stage of the gated delta rule (gdr_common.h): walks the chunks of one (sequence, value
// head) with 16 NCT columns of the state P = S^T in the registers of a four-wave work-group.  Wave w
// owns tokens perm_row(w, .) of a chunk's Z, X, U and O, and key channels 32 w .. (dk = 128) of P:
//   1. Z = K P, X = diag(b) (V - e^G Z)             X's pieces to LDS, barrier
//   2. U = T X                                      pieces of U and e^{G_last - G} U to LDS, barrier
//   3. P' = e^{G_last} P + K^T (e^{G_last - G} U)   pieces of P' to LDS
//   4. O = scale e^G Q P + M U                      barrier, next chunk
// A product's accumulator tiles are the next one's B operands in the layout they have, so LDS holds
// them as the MFMA reads them.  Of a chunk's records every wave needs its own row tile only (Q, T, M,
// the decays: registers), but for K^T, which goes through LDS.  Each record is loaded for the next
// chunk as soon as its registers are free, so the loads spread over the chunk: issued together they
// held every wave up for 1,700 of 6,500 cycles, the vector memory unit taking 16 cycles for each.
//
// The exponents of the fp16 pieces have to be the same in all four waves.  They come from a bound,
// one norm away from a maximum that was published with the operand before: |X| <= max b max|V| +
// max(b e^G |k|_1) max|P|, |U| <= |T|_inf max|X|, |P'| <= e^{G_last} max|P| + sum(e^{G_last - G}
// max|k|) max|U|.  A bound that is 2^10 too large still leaves two pieces their 22 bits.
//
// The chain of chunks is what bounds the stage: one wave on its own (16 columns, everything in its
// registers, no barriers) took 6.3 us a chunk, 1,400 instructions one behind the other with nothing
// to hide the LDS latency; four waves on the same columns take 1.8 us.
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

// LDS: K's fragments, and the operands the waves exchange: P [piece][kb][ct], X [piece][kb 2][ct],
// E = e^{G_last - G} U likewise, U [piece < NI][kb 2][ct]
template <int DK, int NI, int NCT, int SAVE> struct GdrStateLds {
    static constexpr int NKB = DK / 32;
    static constexpr int XP = 0, XX = XP + 2 * NKB * NCT * 1024, XE = XX + 4 * NCT * 1024, XU = XE + 4 * NCT * 1024;
    static constexpr int K = XU + (SAVE ? 0 : NI * 2 * NCT * 1024), BYTES = K + NI * 64 * DK * 2;
};

// half of a fragment (tile `half` of a pair, this lane's four rows) as fp16
typedef __attribute__((address_space(3))) f16x4 lds_f16x4;
__device__ __forceinline__ void st_half_frag(lds_u8 *f, int half, int g, int m, const f16x4 &x) {
    *reinterpret_cast<lds_f16x4 *>(f + frag_slot(g, m) + 8 * half) = x;
}
__device__ __forceinline__ void split4(const f32x4 &x, float s, f16x4 &hi, f16x4 &lo) {
    f16x2 h[2], l[2];
    split2(x[0] * s, x[1] * s, h[0], l[0]);
    split2(x[2] * s, x[3] * s, h[1], l[1]);
    hi = f16x4{h[0][0], h[0][1], h[1][0], h[1][1]};
    lo = f16x4{l[0][0], l[0][1], l[1][0], l[1][1]};
}
__device__ __forceinline__ f16x4 round4(const f32x4 &x, float s) {
    f16x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (_Float16)(x[i] * s);
    return r;
}
__device__ __forceinline__ float max4(const float *p) { return fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])); }

template <int DK, bool F32, int NCT, int SAVE, int MP>
__global__ __launch_bounds__(256) void gdr_state_kernel(const GdrStateArgs p) {
    using E = typename std::conditional<F32, float, __bf16>::type;
    constexpr int NI = F32 ? 2 : 1, NKB = DK / 32, NTW = DK / 64;  // tiles of P per wave and column tile
    using S = GdrStateLds<DK, NI, NCT, SAVE>;
    constexpr GdrLayout L{NI, DK, MP};
    constexpr GdrSave SV{NI, DK};
    __shared__ __attribute__((aligned(1024))) unsigned char smem[S::BYTES];
    __shared__ float sMax[16];  // per wave: max |P|, |X|, |e^{G_last-G} U|, |V| of the next chunk
    const int lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    __builtin_assume(w >= 0 && w < 4);
    // the work-groups of one head share an XCD's L2: ids 8 apart
    const int gh = p.dv / (16 * NCT), id = blockIdx.x;
    const int unit = id / (8 * gh) * 8 + (id & 7), slice = (id >> 3) % gh * NCT;
    if (unit >= p.seqs.N * p.H) return;
    const int seq = unit / p.H, h = unit % p.H, b = p.seqs.batch(seq);
    const int len = p.seqs.length(seq), start = p.seqs.start(seq), nchunk = (len + 63) / 64;
    const int col = slice * 16 + n, nkey = p.H / p.r;
    const size_t slot0 = p.seqs.slot0(seq);
    const unsigned char *krec = p.keys + ((size_t)(b * nkey + h / p.r) * p.nslot + slot0) * L.key_bytes();
    const unsigned char *vrec = p.vals + ((size_t)(b * p.H + h) * p.nslot + slot0) * L.val_bytes();
    const int row0 = perm_row(w, 4 * g);  // this lane's first row of the wave's token tile
    const E *vp = reinterpret_cast<const E *>(p.v) + b * p.sv.b + h * p.sv.h + (long long)start * p.sv.t + col;
    E *op = reinterpret_cast<E *>(p.out) + ((size_t)(b * p.H + h) * p.seqs.T + start + row0) * p.dv + col;
    unsigned char *save = p.save + (((size_t)(b * p.H + h) * p.nslot + slot0) * (p.dv / 16) + slice) * SV.bytes();
    lds_u8 *sx = lds_base(smem);

    E vr[NCT][4], vn[NCT][4], o_prev[NCT][4];
    auto load_v = [&](int c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 64 * c + row0 + i, rc = row < len ? row : len - 1;  // rows past the last repeat it
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) vn[ct][i] = vp[(long long)rc * p.sv.t + 16 * ct];
        }
    };
    auto max_v = [&]() {
        float m = 0.f;
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
            for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(to_f(vn[ct][i])));
        return wave_max(m);
    };

    // tile t of this wave, row 4 g + i: key channel perm_row(NTW w + t, 4 g + i), column n
    f32x4 P[NTW][NCT];
    const size_t state0 = ((size_t)(seq * p.H + h) * p.dv + col) * DK;
#pragma unroll
    for (int t = 0; t < NTW; ++t)
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
            P[t][ct] = p.init_state == nullptr ? f32x4{0.f, 0.f, 0.f, 0.f}
                           : *reinterpret_cast<const f32x4 *>(p.init_state + state0 + (size_t)16 * ct * DK + perm_row(NTW * w + t, 4 * g));
    auto max_p = [&]() {
        float m = 0.f;
#pragma unroll
        for (int t = 0; t < NTW; ++t)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) m = max_abs4(P[t][ct], m);
        return wave_max(m);
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
    // this wave's part of a chunk's records, each loaded for the next chunk once it has been used
    f16x8 kf[NI][NKB], qf[SAVE ? 1 : NI][NKB], tf[2][2], mf[SAVE ? 1 : NI][2];
    f32x4 eG, eL, be;
    float last_, ck_, cb_, ct_, cc_;  // e^{G_last} and the four norms of the value record's header
    int et_, em_, ek_, eq_;
    const int fo = frag_slot(g, n);
    auto load_kq = [&](int c) {
        const unsigned char *r = krec + (size_t)c * L.key_bytes() + w * NKB * 1024 + fo;
#pragma unroll
        for (int x = 0; x < NI; ++x)
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                kf[x][kb] = *reinterpret_cast<const f16x8 *>(r + L.k_off(x) + kb * 1024);
                if constexpr (!SAVE) qf[x][kb] = *reinterpret_cast<const f16x8 *>(r + L.q_off(x) + kb * 1024);
            }
    };
    const int tri = (w < 2 ? w : 2 * w - 2) * 1024 + fo, tri1 = w < 2 ? 0 : 1024;  // waves 0, 1: one fragment
    auto load_t = [&](int c) {
        const unsigned char *r = vrec + (size_t)c * L.val_bytes() + tri;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            tf[x][0] = *reinterpret_cast<const f16x8 *>(r + L.t_off(x));
            tf[x][1] = *reinterpret_cast<const f16x8 *>(r + L.t_off(x) + tri1);
        }
    };
    auto load_m = [&](int c) {
        const unsigned char *r = vrec + (size_t)c * L.val_bytes() + tri;
#pragma unroll
        for (int x = 0; x < NI; ++x) {
            mf[x][0] = *reinterpret_cast<const f16x8 *>(r + L.m_off(x));
            mf[x][1] = *reinterpret_cast<const f16x8 *>(r + L.m_off(x) + tri1);
        }
    };
    auto load_head = [&](int c) {
        const float *r = reinterpret_cast<const float *>(vrec + (size_t)c * L.val_bytes());
        eG = *reinterpret_cast<const f32x4 *>(r + row0);
        eL = *reinterpret_cast<const f32x4 *>(r + 64 + row0);
        be = *reinterpret_cast<const f32x4 *>(r + 128 + row0);
        const int *e = reinterpret_cast<const int *>(r);
        last_ = r[192];
        et_ = e[193];
        em_ = e[194];
        ek_ = e[195];
        eq_ = e[196];
        ck_ = r[197];
        cb_ = r[198];
        ct_ = r[199];
        cc_ = r[200];
    };
    int ep = 0;
    if (nchunk > 0) {
        load_kq(0);
        load_t(0);
        load_head(0);
        if constexpr (!SAVE) load_m(0);
        load_v(0);
        const float mp = max_p(), mv = max_v();
        if (lane == 0) {
            sMax[w] = mp;
            sMax[12 + w] = mv;
        }
        barrier_lds();
        ep = gdr_exp(max4(sMax));
        put_p(ep);
    }
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < nchunk; ++c) {
        const int next = c + 1 < nchunk ? c + 1 : c;  // the last chunk's loads are not used: no branches
        barrier_lds();
        // K for step 3: its readers of the last chunk are past this barrier, those of this one past the next
#pragma unroll
        for (int x = 0; x < NI; ++x)
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb)
                *reinterpret_cast<__attribute__((address_space(3))) f16x8 *>(sx + S::K + x * L.mat() + (w * NKB + kb) * 1024 + fo) =
                    kf[x][kb];
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
            for (int i = 0; i < 4; ++i) vr[ct][i] = vn[ct][i];
        load_v(next);
        if constexpr (!SAVE)
            if (c > 0) {  // the last chunk's outputs, a whole chunk
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct) op[(size_t)(64 * (c - 1) + i) * p.dv + 16 * ct] = o_prev[ct][i];
            }
        const float pmax = max4(sMax), last = last_, kbound = ck_, bbound = cb_, tbound = ct_, kcol = cc_;
        const int et = et_, em = em_, ek = ek_, eq = eq_;
        const f32x4 eG0 = eG;

        // ---- 1. Z = K P, X = diag(b) (V - e^G Z); Q P alongside
        f32x4 Z[NCT], Z1[NCT], O[NCT];
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) Z[ct] = Z1[ct] = O[ct] = zero;
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                const f16x8 ph = ld_frag(sx + S::XP + (kb * NCT + ct) * 1024, lane);
                const f16x8 pl = ld_frag(sx + S::XP + ((NKB + kb) * NCT + ct) * 1024, lane);
                Z[ct] = mma16(kf[0][kb], ph, Z[ct]);
                Z1[ct] = mma16(kf[0][kb], pl, Z1[ct]);
                if constexpr (NI == 2) Z1[ct] = mma16(kf[1][kb], ph, Z1[ct]);
                if constexpr (!SAVE) {
                    O[ct] = mma16(qf[0][kb], ph, O[ct]);
                    if constexpr (NI == 2) O[ct] = mma16(qf[1][kb], ph, mma16(qf[0][kb], pl, O[ct]));
                }
                if constexpr (SAVE) {
                    if (kb == w && NKB == 4 || kb == w >> 1 && NKB == 2 && (w & 1) == 0) {
                        // one wave per fragment keeps it; both pieces together round to one
                        unsigned char *sv = save + ((size_t)c * (p.dv / 16) + ct) * SV.bytes() + kb * 1024 + frag_slot(g, n);
                        if constexpr (NI == 2) {
                            *reinterpret_cast<f16x8 *>(sv + SV.p_off(0)) = ph;
                            *reinterpret_cast<f16x8 *>(sv + SV.p_off(1)) = pl;
                        } else {
                            *reinterpret_cast<f16x8 *>(sv + SV.p_off(0)) = ph + pl;
                        }
                    }
                }
            }
        }
        f32x4 X[NCT];
        float xm = 0.f;
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                X[ct][i] = be[i] * (to_f(vr[ct][i]) - eG[i] * scale_down(Z[ct][i] + Z1[ct][i], ek + ep));
            xm = max_abs4(X[ct], xm);
        }
        const int ex = gdr_exp(bbound * max4(sMax + 12) + kbound * pmax);
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
            f16x4 hi, lo;
            split4(X[ct], pow2f(ex), hi, lo);
            lds_u8 *f = sx + S::XX + ((w >> 1) * NCT + ct) * 1024;
            st_half_frag(f, w & 1, g, n, hi);
            st_half_frag(f + 2 * NCT * 1024, w & 1, g, n, lo);
        }
        xm = wave_max(xm);
        if (lane == 0) sMax[4 + w] = xm;
        load_kq(next);
        barrier_lds();

        // ---- 2. U = T X
        const int eu = gdr_exp(tbound * max4(sMax + 4));
        float um = 0.f;
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
            f32x4 z = zero, z1 = zero;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
                if (kb == 0 || w >= 2) {
                    const f16x8 xh = ld_frag(sx + S::XX + (kb * NCT + ct) * 1024, lane);
                    const f16x8 xl = ld_frag(sx + S::XX + ((2 + kb) * NCT + ct) * 1024, lane);
                    z = mma16(tf[0][kb], xh, z);
                    z1 = mma16(tf[1][kb], xh, mma16(tf[0][kb], xl, z1));
                }
            f32x4 U, EU;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                U[i] = scale_down(z[i] + z1[i], et + ex);
                EU[i] = U[i] * eL[i];
            }
            um = max_abs4(EU, um);
            f16x4 hi, lo;
            split4(EU, pow2f(eu), hi, lo);
            lds_u8 *f = sx + S::XE + ((w >> 1) * NCT + ct) * 1024;
            st_half_frag(f, w & 1, g, n, hi);
            st_half_frag(f + 2 * NCT * 1024, w & 1, g, n, lo);
            if constexpr (NI == 2) split4(U, pow2f(eu), hi, lo);
            else hi = round4(U, pow2f(eu));
            if constexpr (SAVE) {
                unsigned char *sv = save + ((size_t)c * (p.dv / 16) + ct) * SV.bytes() + (w >> 1) * 1024 + frag_slot(g, n) + 8 * (w & 1);
                *reinterpret_cast<f16x4 *>(sv + SV.u_off(0)) = hi;
                if constexpr (NI == 2) *reinterpret_cast<f16x4 *>(sv + SV.u_off(1)) = lo;
                if (threadIdx.x == 0) {
                    int *e = reinterpret_cast<int *>(save + ((size_t)c * (p.dv / 16) + ct) * SV.bytes());
                    e[0] = ep;
                    e[1] = eu;
                }
            } else {
                f = sx + S::XU + ((w >> 1) * NCT + ct) * 1024;
                st_half_frag(f, w & 1, g, n, hi);
                if constexpr (NI == 2) st_half_frag(f + 2 * NCT * 1024, w & 1, g, n, lo);
            }
        }
        um = wave_max(um);
        if (lane == 0) sMax[8 + w] = um;
        load_t(next);
        load_head(next);
        barrier_lds();

        // ---- 3. P' = e^{G_last} P + K^T (e^{G_last - G} U)
        f16x8 eh[2][NCT], el[2][NCT];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                eh[kb][ct] = ld_frag(sx + S::XE + (kb * NCT + ct) * 1024, lane);
                el[kb][ct] = ld_frag(sx + S::XE + ((2 + kb) * NCT + ct) * 1024, lane);
            }
#pragma unroll
        for (int t = 0; t < NTW; ++t) {
            f32x4 z[NCT], z1[NCT];
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) z[ct] = z1[ct] = zero;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const int tile = NTW * w + t;
                const lds_u8 *f0 = sx + S::K + (2 * kb * NKB + (tile >> 1)) * 1024, *f1 = f0 + NKB * 1024;
                const f16x8 f = ld_frag_t(f0, f1, tile, lane);
                f16x8 fl = f;
                if constexpr (NI == 2) fl = ld_frag_t(f0 + L.mat(), f1 + L.mat(), tile, lane);
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) {
                    z[ct] = mma16(f, eh[kb][ct], z[ct]);
                    z1[ct] = mma16(f, el[kb][ct], z1[ct]);
                    if constexpr (NI == 2) z1[ct] = mma16(fl, eh[kb][ct], z1[ct]);
                }
            }
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    P[t][ct][i] = fmaf(P[t][ct][i], last, scale_down(z[ct][i] + z1[ct][i], ek + eu));
        }
        const int ep_old = ep;
        ep = gdr_exp(last * pmax + kcol * max4(sMax + 8));
        put_p(ep);
        const float mp = max_p();
        const float mv = max_v();  // of the next chunk
        if (lane == 0) {
            sMax[w] = mp;
            sMax[12 + w] = mv;
        }

        // ---- 4. O = scale e^G Q P + M U (M holds the scale)
        if constexpr (!SAVE) {
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                f32x4 z = zero;
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
                    if (kb == 0 || w >= 2) {
                        const f16x8 uh = ld_frag(sx + S::XU + (kb * NCT + ct) * 1024, lane);
                        z = mma16(mf[0][kb], uh, z);
                        if constexpr (NI == 2) {
                            z = mma16(mf[0][kb], ld_frag(sx + S::XU + ((2 + kb) * NCT + ct) * 1024, lane), z);
                            z = mma16(mf[1][kb], uh, z);
                        }
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o_prev[ct][i] = from_f<E>(scale_down(z[i], em + eu) + p.scale * eG0[i] * scale_down(O[ct][i], eq + ep_old));
            }
        }
        if constexpr (!SAVE) load_m(next);
    }
    if constexpr (!SAVE)
        if (nchunk > 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (64 * (nchunk - 1) + row0 + i < len)
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct) op[(size_t)(64 * (nchunk - 1) + i) * p.dv + 16 * ct] = o_prev[ct][i];
        }
    if (p.final_state != nullptr)
#pragma unroll
        for (int t = 0; t < NTW; ++t)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
                *reinterpret_cast<f32x4 *>(p.final_state + state0 + (size_t)16 * ct * DK + perm_row(NTW * w + t, 4 * g)) = P[t][ct];
}

}  // namespace kda
