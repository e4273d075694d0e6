// Sequential stage of the gated delta rule (gdr_common.h): walks the chunks of one (sequence, value
// head) with 16 NCT columns of the state P = S^T in the registers of four waves, the chain.  Wave w
// of them owns tokens perm_row(w, .) of a chunk's Z, X and U, and key channels 32 w .. (dk = 128) of P:
//   1. Z = K P, X = diag(b) (V - e^G Z)             X's pieces to LDS, barrier
//   2. U = T X                                      pieces of U and e^{G_last - G} U to LDS, barrier
//   3. P' = e^{G_last} P + K^T (e^{G_last - G} U)   pieces of P' to LDS, barrier
// A product's accumulator tiles are the next one's B operands in the layout they have, so LDS holds
// them as the MFMA reads them.  Four more waves of the same work-group do what the next chunk's state
// does not need, O = scale e^G Q P + M U, and load: the next chunk's K, T, V and decays from global
// memory to LDS, each a whole chunk ahead (a load waited for in the chunk that issued it held all
// eight waves up by 800 of 4,000 cycles).
//
// The exponents of the fp16 pieces have to be the same in all four waves.  They come from a bound,
// one norm away from a maximum that was published with the operand before: |X| <= max b max|V| +
// max(b e^G |k|_1) max|P|, |U| <= |T|_inf max|X|, |P'| <= e^{G_last} max|P| + sum(max|k|) max|e^{G_last - G}
// U|: the maximum is that of the decayed U, so the sum is not decayed again (keys that end before the
// chunk does would leave it far below P').  The decayed U has a bound of its own, e^{G_last - G_i} U_i =
// sum_j (T_ij e^{G_j - G_i}) e^{G_last - G_j} X_j with |e^{G_last - G} X| <= max(b e^{G_last - G} |V|) +
// e^{G_last} max b max|k|_1 max|P|: where the chunk's last tokens write nothing, all of it is as small as
// the decay over them, and U's exponent would leave its pieces no bits.  A bound that is 2^10 too large
// still leaves two pieces their 22 bits.
//
// The chain of chunks is what bounds the stage, three exchanges through LDS one behind the other.
// 65,536 tokens x 32 heads (16 columns a work-group, one work-group a CU): 1.48 us a chunk; the chain's
// waves with the loads and outputs on them 1.78 us, 215 of their vector instructions and the LDS reads
// of 100 KiB a chunk being left; one wave on its own columns, no barriers, 6.3 us.
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

// LDS: K's and T's fragments, the value record's header and V's tile of two chunks, and the operands the waves exchange: P [piece][kb][ct],
// X [piece][kb 2][ct], E = e^{G_last - G} U likewise, U [piece < NI][kb 2][ct]
template <int DK, int NI, int NCT> struct GdrStateLds {
    static constexpr int NKB = DK / 32, VB = NI * 2048 * NCT;
    static constexpr int XP = 0, XX = XP + 2 * NKB * NCT * 1024, XE = XX + 4 * NCT * 1024, XU = XE + 4 * NCT * 1024;
    static constexpr int IN = XU + NI * 2 * NCT * 1024;  // two of: K, T, V, header
    static constexpr int T = NI * 64 * DK * 2, V = T + 2 * GdrLayout::kTri, HEAD = V + VB, INB = HEAD + GdrLayout::kHead;
    static constexpr int BYTES = IN + 2 * INB;
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
__global__ __launch_bounds__(512) void gdr_state_kernel(const GdrStateArgs p) {
    using E = typename std::conditional<F32, float, __bf16>::type;
    typedef __attribute__((ext_vector_type(4))) E E4;
    typedef __attribute__((address_space(3))) E4 lds_e4;
    typedef __attribute__((address_space(3))) f16x8 lds_f16x8;
    typedef __attribute__((address_space(3))) f32x4 lds_f4;
    typedef __attribute__((address_space(3))) int lds_i32;
    constexpr int NI = F32 ? 2 : 1, NKB = DK / 32, NTW = DK / 64;  // tiles of P per wave and column tile
    using S = GdrStateLds<DK, NI, NCT>;
    constexpr GdrLayout L{NI, DK, MP};
    constexpr GdrSave SV{NI, DK};
    __shared__ __attribute__((aligned(1024))) unsigned char smem[S::BYTES];
    // per wave: max |P|, |X|, |e^{G_last-G} U|; |V| of two chunks, b e^{G_last-G} |V| of two
    __shared__ __attribute__((aligned(16))) float sMax[28];
    __shared__ int sExp[2];     // exponents of P and of U's pieces
    const int lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wid & 3;
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
    const int fo = frag_slot(g, n);
    const int tri = (w < 2 ? w : 2 * w - 2) * 1024 + fo, tri1 = w < 2 ? 0 : 1024;  // waves 0, 1: one fragment
    lds_u8 *sx = lds_base(smem);
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

    if (wid >= 4) {  // ---------------------------------------------- loads, outputs
        const E *vp = reinterpret_cast<const E *>(p.v) + b * p.sv.b + h * p.sv.h + (long long)start * p.sv.t + col;
        E *op = reinterpret_cast<E *>(p.out) + ((size_t)(b * p.H + h) * p.seqs.T + start + row0) * p.dv + col;
        unsigned char *save = p.save + (((size_t)(b * p.H + h) * p.nslot + slot0) * (p.dv / 16) + slice) * SV.bytes();
        E vn[NCT][4];  // a vector would be put together, and waited for, where it is loaded
        f16x8 kf[NI][NKB], tf[3], qf[SAVE ? 1 : NI][NKB], mf[SAVE ? 1 : NI][2];
        f32x4 eG, el, bl;
        float head;
        int em, eq;
        // a quarter of K's and T's fragments, of the header and of V
        auto load_kt = [&](int c) {
            c = min(c, nchunk - 1);  // behind the last chunk: loaded and not used
            const unsigned char *r = krec + (size_t)c * L.key_bytes() + w * NKB * 1024 + fo;
            const unsigned char *t = vrec + (size_t)c * L.val_bytes();
#pragma unroll
            for (int x = 0; x < NI; ++x)
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb) kf[x][kb] = *reinterpret_cast<const f16x8 *>(r + L.k_off(x) + kb * 1024);
#pragma unroll
            for (int i = 0; i < 3; ++i) tf[i] = *reinterpret_cast<const f16x8 *>(t + L.t_off(0) + (3 * w + i) * 1024 + fo);
            head = *reinterpret_cast<const float *>(t + 4 * (64 * w + lane));
            el = *reinterpret_cast<const f32x4 *>(t + 256 + 4 * row0);
            bl = *reinterpret_cast<const f32x4 *>(t + 512 + 4 * row0);
        };
        auto load_v = [&](int c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = min(64 * c + row0 + i, len - 1);  // rows past the last repeat it
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) vn[ct][i] = vp[(long long)row * p.sv.t + 16 * ct];
            }
        };
        auto put = [&](int c) {
            lds_u8 *to = sx + S::IN + (c & 1) * S::INB;
#pragma unroll
            for (int x = 0; x < NI; ++x)
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb)
                    *reinterpret_cast<lds_f16x8 *>(to + x * L.mat() + (w * NKB + kb) * 1024 + fo) = kf[x][kb];
#pragma unroll
            for (int i = 0; i < 3; ++i) *reinterpret_cast<lds_f16x8 *>(to + S::T + (3 * w + i) * 1024 + fo) = tf[i];
            *reinterpret_cast<__attribute__((address_space(3))) float *>(to + S::HEAD + 4 * (64 * w + lane)) = head;
            __builtin_amdgcn_sched_barrier(0);  // mixed in with what stands before, 2 % slower
            Most mv, mbl;
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                *reinterpret_cast<lds_e4 *>(to + S::V + ct * NI * 2048 + (w * 64 + lane) * 4 * (int)sizeof(E)) = E4{vn[ct][0], vn[ct][1], vn[ct][2], vn[ct][3]};
                const f32x4 x = {(float)vn[ct][0], (float)vn[ct][1], (float)vn[ct][2], (float)vn[ct][3]};
                mv.add4(x);
                mbl.add4(bl * el * x);
            }
            const float m = mv.wave(), ml = mbl.wave();
            if (lane == 0) {
                sMax[12 + 4 * (c & 1) + w] = m;
                sMax[20 + 4 * (c & 1) + w] = ml;
            }
        };
        auto load_q = [&](int c) {
            const unsigned char *r = krec + (size_t)min(c, nchunk - 1) * L.key_bytes() + w * NKB * 1024 + fo;
#pragma unroll
            for (int x = 0; x < NI; ++x)
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb) qf[x][kb] = *reinterpret_cast<const f16x8 *>(r + L.q_off(x) + kb * 1024);
        };
        auto load_m = [&](int c) {
            const unsigned char *m = vrec + (size_t)min(c, nchunk - 1) * L.val_bytes() + tri;
#pragma unroll
            for (int x = 0; x < NI; ++x) {
                mf[x][0] = *reinterpret_cast<const f16x8 *>(m + L.m_off(x));
                mf[x][1] = *reinterpret_cast<const f16x8 *>(m + L.m_off(x) + tri1);
            }
        };
        if (nchunk > 0) {
            load_kt(0);
            load_v(0);
            put(0);
            load_kt(1);
            load_v(1);
            if constexpr (!SAVE) {
                load_q(0);
                load_m(0);
            }
            barrier_lds();  // (A)
        }
        for (int c = 0; c < nchunk; ++c) {
            barrier_lds();  // (1)
            const int ep = sExp[0];
            const lds_u8 *hd = sx + S::IN + (c & 1) * S::INB + S::HEAD;
            if constexpr (!SAVE) {
                eG = *reinterpret_cast<const lds_f4 *>(hd + 4 * row0);
                em = reinterpret_cast<const lds_i32 *>(hd)[194];
                eq = reinterpret_cast<const lds_i32 *>(hd)[196];
            }
            f32x4 O[NCT];
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) O[ct] = zero;
            if constexpr (!SAVE) {
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct) {
                        const f16x8 ph = ld_frag(sx + S::XP + (kb * NCT + ct) * 1024, lane);
                        O[ct] = mma16(qf[0][kb], ph, O[ct]);
                        if constexpr (NI == 2) {
                            const f16x8 pl = ld_frag(sx + S::XP + ((NKB + kb) * NCT + ct) * 1024, lane);
                            O[ct] = mma16(qf[1][kb], ph, mma16(qf[0][kb], pl, O[ct]));
                        }
                    }
                load_q(c + 1);
            } else {
                // both pieces together round to one
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
                            *reinterpret_cast<f16x8 *>(sv + SV.p_off(0)) = ph + pl;
                        }
                    }
            }
            barrier_lds();  // (2)
            put(c + 1);     // read from behind (3) on
            barrier_lds();  // (3)
            load_kt(c + 2);
            load_v(c + 2);
            const int eu = sExp[1];
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
                        if (64 * c + row0 + i < len)
                            op[(size_t)(64 * c + i) * p.dv + 16 * ct] =
                                from_f<E>(scale_down(z[i], em + eu) + p.scale * eG[i] * scale_down(O[ct][i], eq + ep));
                }
                load_m(c + 1);
            } else {
                // fragment w & 1 of U's piece w / 2
                if (w < 2 * NI)
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct)
                        *reinterpret_cast<f16x8 *>(save + ((size_t)c * (p.dv / 16) + ct) * SV.bytes() + SV.u_off(w >> 1) + (w & 1) * 1024 + fo) =
                            ld_frag(sx + S::XU + (w * NCT + ct) * 1024, lane);
                if (w == 3 && lane == 0)
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct) {
                        int *e = reinterpret_cast<int *>(save + ((size_t)c * (p.dv / 16) + ct) * SV.bytes());
                        e[0] = ep;
                        e[1] = eu;
                    }
            }
        }
        return;
    }

    // -------------------------------------------------------------- the chain
    __builtin_amdgcn_s_setprio(3);
    // tile t of this wave, row 4 g + i: key channel perm_row(NTW w + t, 4 g + i), column n
    f32x4 P[NTW][NCT];
    const size_t state0 = ((size_t)(seq * p.H + h) * p.dv + col) * DK;
#pragma unroll
    for (int t = 0; t < NTW; ++t)
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
            P[t][ct] = p.init_state == nullptr ? zero
                           : *reinterpret_cast<const f32x4 *>(p.init_state + state0 + (size_t)16 * ct * DK + perm_row(NTW * w + t, 4 * g));
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
    f16x8 kf[NI][NKB], tf[2][2];
    E4 v[NCT];
    f32x4 eG, eL, be, h0, h1, h2, mv, ml;
    // what the other waves have laid out for chunk c
    auto get = [&](int c) {
        const lds_u8 *in = sx + S::IN + (c & 1) * S::INB;
#pragma unroll
        for (int x = 0; x < NI; ++x)
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) kf[x][kb] = ld_frag(in + x * L.mat() + (w * NKB + kb) * 1024, lane);
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) v[ct] = *reinterpret_cast<const lds_e4 *>(in + S::V + ct * NI * 2048 + (w * 64 + lane) * 4 * (int)sizeof(E));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            tf[x][0] = *reinterpret_cast<const lds_f16x8 *>(in + S::T + x * L.kTri + tri);
            tf[x][1] = *reinterpret_cast<const lds_f16x8 *>(in + S::T + x * L.kTri + tri + tri1);
        }
        const lds_u8 *hd = in + S::HEAD;
        eG = *reinterpret_cast<const lds_f4 *>(hd + 4 * row0);
        eL = *reinterpret_cast<const lds_f4 *>(hd + 256 + 4 * row0);
        be = *reinterpret_cast<const lds_f4 *>(hd + 512 + 4 * row0);
        h0 = *reinterpret_cast<const lds_f4 *>(hd + 768);
        h1 = *reinterpret_cast<const lds_f4 *>(hd + 784);
        h2 = *reinterpret_cast<const lds_f4 *>(hd + 800);
        mv = *reinterpret_cast<const f32x4 *>(sMax + 12 + 4 * (c & 1));  // their maxima where they are used
        ml = *reinterpret_cast<const f32x4 *>(sMax + 20 + 4 * (c & 1));
    };
    int ep = 0;
    if (nchunk > 0) {
        const float mp = max_p();
        if (lane == 0) sMax[w] = mp;
        barrier_lds();  // (A)
        get(0);
        ep = gdr_exp(max4(sMax));
        put_p(ep);
        if (threadIdx.x == 0) sExp[0] = ep;
    }
    for (int c = 0; c < nchunk; ++c) {
        barrier_lds();  // (1)
        const float pmax = max4(sMax), last = h0[0], kbound = h1[1], bbound = h1[2], tbound = h1[3];
        const float ksum = h2[0], ubound = h2[2], k1 = h2[3];
        const float et_ = h0[1], ek_ = h0[3];
        const int et = __builtin_bit_cast(int, et_), ek = __builtin_bit_cast(int, ek_);

        // ---- 1. Z = K P, X = diag(b) (V - e^G Z)
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
        const int ex = gdr_exp(bbound * max4(mv) + kbound * pmax);
        f32x4 X[NCT];
        Most mx;
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                X[ct][i] = be[i] * ((float)v[ct][i] - eG[i] * scale_down(Z[ct][i] + Z1[ct][i], ek + ep));
            mx.add4(X[ct]);
        }
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
            f16x4 hi, lo;
            split4(X[ct], pow2f(ex), hi, lo);
            lds_u8 *f = sx + S::XX + ((w >> 1) * NCT + ct) * 1024;
            st_half_frag(f, w & 1, g, n, hi);
            st_half_frag(f + 2 * NCT * 1024, w & 1, g, n, lo);
        }
        const float xm = mx.wave();
        if (lane == 0) sMax[4 + w] = xm;
        const float lbound = ubound * (max4(ml) + last * pmax * (bbound * k1));  // of e^{G_last - G} U
        barrier_lds();  // (2)

        // ---- 2. U = T X
        const float umost = tbound * max4(sMax + 4);
        const int eu = gdr_exp(umost), ee = gdr_exp(fminf(umost, lbound));
        Most mu;
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
            mu.add4(EU);
            f16x4 hi, lo;
            split4(EU, pow2f(ee), hi, lo);
            lds_u8 *f = sx + S::XE + ((w >> 1) * NCT + ct) * 1024;
            st_half_frag(f, w & 1, g, n, hi);
            st_half_frag(f + 2 * NCT * 1024, w & 1, g, n, lo);
            if constexpr (NI == 2) split4(U, pow2f(eu), hi, lo);
            else hi = round4(U, pow2f(eu));
            f = sx + S::XU + ((w >> 1) * NCT + ct) * 1024;
            st_half_frag(f, w & 1, g, n, hi);
            if constexpr (NI == 2) st_half_frag(f + 2 * NCT * 1024, w & 1, g, n, lo);
        }
        const float um = mu.wave();
        if (lane == 0) sMax[8 + w] = um;
        if (threadIdx.x == 0) sExp[1] = eu;
        barrier_lds();  // (3)

        // ---- 3. P' = e^{G_last} P + K^T (e^{G_last - G} U)
        f16x8 eh[2][NCT], el[2][NCT];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                eh[kb][ct] = ld_frag(sx + S::XE + (kb * NCT + ct) * 1024, lane);
                el[kb][ct] = ld_frag(sx + S::XE + ((2 + kb) * NCT + ct) * 1024, lane);
            }
        f16x8 kt[NI][NTW][2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int t = 0; t < NTW; ++t) {
                const int tile = NTW * w + t;
                const lds_u8 *f0 = sx + S::IN + (c & 1) * S::INB + (2 * kb * NKB + (tile >> 1)) * 1024, *f1 = f0 + NKB * 1024;
#pragma unroll
                for (int x = 0; x < NI; ++x) kt[x][t][kb] = ld_frag_t(f0 + x * L.mat(), f1 + x * L.mat(), tile, lane);
            }
        const float emax = max4(sMax + 8);
        __builtin_amdgcn_sched_barrier(0);
        get(c + 1);  // behind the reads that are waited for
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < NTW; ++t) {
            f32x4 z[NCT], z1[NCT];
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) z[ct] = z1[ct] = zero;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) {
                    z[ct] = mma16(kt[0][t][kb], eh[kb][ct], z[ct]);
                    z1[ct] = mma16(kt[0][t][kb], el[kb][ct], z1[ct]);
                    if constexpr (NI == 2) z1[ct] = mma16(kt[1][t][kb], eh[kb][ct], z1[ct]);
                }
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    P[t][ct][i] = fmaf(P[t][ct][i], last, scale_down(z[ct][i] + z1[ct][i], ek + ee));
        }
        ep = gdr_exp(last * pmax + ksum * emax);
        put_p(ep);
        const float mp = max_p();
        if (lane == 0) sMax[w] = mp;
        if (threadIdx.x == 0) sExp[0] = ep;
    }
    if (p.final_state != nullptr)
#pragma unroll
        for (int t = 0; t < NTW; ++t)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
                *reinterpret_cast<f32x4 *>(p.final_state + state0 + (size_t)16 * ct * DK + perm_row(NTW * w + t, 4 * g)) = P[t][ct];
}

}  // namespace kda
