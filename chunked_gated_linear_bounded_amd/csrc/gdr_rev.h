// Reverse pass of the gated delta rule's backward (gdr_common.h): walks the chunks of one (sequence,
// value head) from the last to the first with 16 NCT columns of dP, the gradient of a chunk's end
// state P', in the registers of a four-wave work-group laid out as in gdr_state.h:
//   1. dU = M^T dO + diag(e^{G_last - G}) K dP'                 pieces of dU to LDS, barrier
//   2. dX = T^T dU, dV = diag(b) dX                             pieces of b e^G dX to LDS, barrier
//   3. dP = e^{G_last} dP' + Q^T (scale e^G dO) - K^T (b e^G dX)   pieces of dP to LDS, barrier
// Every chunk's dP' and dX are kept, as fp16, for the gradient stage; dV is final here.
//
// M, T, Q and K are all needed transposed, so they go through LDS (56 KiB at dk = 128, bf16), each
// wave bringing its row tile.  The exponents of the pieces come from bounds as in gdr_state.h; the
// column sums of |M| and |T| are bounded by 64 times their largest entry.  A state gradient that a
// caller asks for (dinitial_state, float32) is exact to the same 22 bits as the final state.
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
    static constexpr int NKB = DK / 32;
    // dP' [piece][kb][ct]; dO [piece < NI][kb 2][ct]; dU, H = scale e^G dO, F = b e^G dX [piece][kb 2][ct]
    static constexpr int XP = 0, XO = XP + 2 * NKB * NCT * 1024, XU = XO + NI * 2 * NCT * 1024, XH = XU + 4 * NCT * 1024;
    static constexpr int XF = XH + 4 * NCT * 1024, K = XF + 4 * NCT * 1024, Q = K + NI * 64 * DK * 2;
    static constexpr int T = Q + NI * 64 * DK * 2, M = T + 2 * GdrLayout::kTri, BYTES = M + 2 * GdrLayout::kTri;
};

template <int DK, bool F32, int NCT>
__global__ __launch_bounds__(256) void gdr_rev_kernel(const GdrRevArgs p) {
    using E = typename std::conditional<F32, float, __bf16>::type;
    constexpr int NI = F32 ? 2 : 1, NKB = DK / 32, NTW = DK / 64;
    using S = GdrRevLds<DK, NI, NCT>;
    constexpr GdrLayout L{NI, DK, 2};
    constexpr GdrSave SV{NI, DK};
    typedef __attribute__((address_space(3))) f16x8 lds_f16x8;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[S::BYTES];
    __shared__ float sMax[16];  // per wave: max |dP'|, |dU|, |dO| of the next chunk
    const int lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
    const E *dop = reinterpret_cast<const E *>(p.dout) + b * p.sdo.b + h * p.sdo.h + (long long)start * p.sdo.t + col;
    E *dvp = reinterpret_cast<E *>(p.dv_out) + ((size_t)(b * p.H + h) * p.seqs.T + start + row0) * p.dv + col;
    unsigned char *save = p.save + (((size_t)(b * p.H + h) * p.nslot + slot0) * (p.dv / 16) + slice) * SV.bytes();
    lds_u8 *sx = lds_base(smem);

    E vn[NCT][4];
    auto load_do = [&](int c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 64 * c + row0 + i, rc = row < len ? row : len - 1;
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                const E x = dop[(long long)rc * p.sdo.t + 16 * ct];
                vn[ct][i] = row < len ? x : (E)0.f;  // rows past the last have no gradient
            }
        }
    };
    auto max_do = [&]() {
        float m = 0.f;
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
            for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(to_f(vn[ct][i])));
        return wave_max(m);
    };
    f32x4 P[NTW][NCT];  // dP
    const size_t state0 = ((size_t)(seq * p.H + h) * p.dv + col) * DK;
#pragma unroll
    for (int t = 0; t < NTW; ++t)
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
            P[t][ct] = p.dfinal == nullptr ? f32x4{0.f, 0.f, 0.f, 0.f}
                           : *reinterpret_cast<const f32x4 *>(p.dfinal + state0 + (size_t)16 * ct * DK + perm_row(NTW * w + t, 4 * g));
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
    f16x8 kf[NI][NKB], qf[NI][NKB], tf[2][2], mf[2][2];
    f32x4 eG, eL, be;
    float last_, bm_, cl_;
    int et_, em_, ek_, eq_;
    const int tri0 = w < 2 ? w : 2 * w - 2, tri1 = w < 2 ? 0 : 1024;  // waves 0, 1: one causal fragment
    auto load_rec = [&](int c) {
        const unsigned char *r = krec + (size_t)c * L.key_bytes() + w * NKB * 1024 + fo;
        const unsigned char *v = vrec + (size_t)c * L.val_bytes(), *t = v + tri0 * 1024 + fo;
#pragma unroll
        for (int x = 0; x < NI; ++x)
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                kf[x][kb] = *reinterpret_cast<const f16x8 *>(r + L.k_off(x) + kb * 1024);
                qf[x][kb] = *reinterpret_cast<const f16x8 *>(r + L.q_off(x) + kb * 1024);
            }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                tf[x][o] = *reinterpret_cast<const f16x8 *>(t + L.t_off(x) + o * tri1);
                mf[x][o] = *reinterpret_cast<const f16x8 *>(t + L.m_off(x) + o * tri1);
            }
        const float *f = reinterpret_cast<const float *>(v);
        const int *e = reinterpret_cast<const int *>(v);
        eG = *reinterpret_cast<const f32x4 *>(f + row0);
        eL = *reinterpret_cast<const f32x4 *>(f + 64 + row0);
        be = *reinterpret_cast<const f32x4 *>(f + 128 + row0);
        last_ = f[192];
        et_ = e[193];
        em_ = e[194];
        ek_ = e[195];
        eq_ = e[196];
        bm_ = f[198];
        cl_ = f[201];
    };
    // rows of the transpose of a 64x64 lower triangle: column tile w, contraction block kb (>= w's own)
    auto tri_t = [&](const lds_u8 *f, int kb) {
        const lds_u8 *f0 = f + tri_frag(2 * kb, w >> 1) * 1024, *f1 = f + tri_frag(2 * kb + 1, w >> 1) * 1024;
        return ld_frag_t(f0, f1, w, lane);
    };
    int ep = 0;
    if (nchunk > 0) {
        load_rec(nchunk - 1);
        load_do(nchunk - 1);
        const float mp = max_p(), mo = max_do();
        if (lane == 0) {
            sMax[w] = mp;
            sMax[8 + w] = mo;
        }
        barrier_lds();
        ep = gdr_exp(max4(sMax));
        put_p(ep);
    }
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    for (int c = nchunk - 1; c >= 0; --c) {
        const int next = c > 0 ? c - 1 : 0;
        barrier_lds();  // dP' is there; the last chunk's LDS has been read
        const float pmax = max4(sMax), omax = max4(sMax + 8), last = last_, bm = bm_, cl = cl_;
        const int et = et_, em = em_, ek = ek_, eq = eq_;
        const f32x4 eL0 = eL, eG0 = eG, be0 = be;
        const int eo = gdr_exp(omax), eh = gdr_exp(fabsf(p.scale) * omax);
#pragma unroll
        for (int x = 0; x < NI; ++x)
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                *reinterpret_cast<lds_f16x8 *>(sx + S::K + x * L.mat() + (w * NKB + kb) * 1024 + fo) = kf[x][kb];
                *reinterpret_cast<lds_f16x8 *>(sx + S::Q + x * L.mat() + (w * NKB + kb) * 1024 + fo) = qf[x][kb];
            }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int o = 0; o < 2; ++o)
                if (o == 0 || w >= 2) {
                    *reinterpret_cast<lds_f16x8 *>(sx + S::T + x * GdrLayout::kTri + (tri0 + o) * 1024 + fo) = tf[x][o];
                    *reinterpret_cast<lds_f16x8 *>(sx + S::M + x * GdrLayout::kTri + (tri0 + o) * 1024 + fo) = mf[x][o];
                }
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
            const f32x4 d = {to_f(vn[ct][0]), to_f(vn[ct][1]), to_f(vn[ct][2]), to_f(vn[ct][3])};
            f32x4 hd;
#pragma unroll
            for (int i = 0; i < 4; ++i) hd[i] = p.scale * eG0[i] * d[i];
            f16x4 hi, lo;
            const int at = ((w >> 1) * NCT + ct) * 1024;
            if constexpr (NI == 2) {
                split4(d, pow2f(eo), hi, lo);
                st_half_frag(sx + S::XO + 2 * NCT * 1024 + at, w & 1, g, n, lo);
            } else {
                hi = round4(d, pow2f(eo));  // exact
            }
            st_half_frag(sx + S::XO + at, w & 1, g, n, hi);
            split4(hd, pow2f(eh), hi, lo);
            st_half_frag(sx + S::XH + at, w & 1, g, n, hi);
            st_half_frag(sx + S::XH + 2 * NCT * 1024 + at, w & 1, g, n, lo);
        }
        barrier_lds();

        // ---- 1. dU = M^T dO + e^{G_last - G} K dP'
        f32x4 Z[NCT], Z1[NCT], Y[NCT], Y1[NCT];
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) Z[ct] = Z1[ct] = Y[ct] = Y1[ct] = zero;
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                const f16x8 ph = ld_frag(sx + S::XP + (kb * NCT + ct) * 1024, lane);
                const f16x8 pl = ld_frag(sx + S::XP + ((NKB + kb) * NCT + ct) * 1024, lane);
                Z[ct] = mma16(kf[0][kb], ph, Z[ct]);
                Z1[ct] = mma16(kf[0][kb], pl, Z1[ct]);
                if constexpr (NI == 2) Z1[ct] = mma16(kf[1][kb], ph, Z1[ct]);
                if (kb == w && NKB == 4 || kb == w >> 1 && NKB == 2 && (w & 1) == 0) {
                    unsigned char *sv = save + ((size_t)c * (p.dv / 16) + ct) * SV.bytes() + kb * 1024 + fo;
                    if constexpr (NI == 2) {
                        *reinterpret_cast<f16x8 *>(sv + SV.p_off(0)) = ph;
                        *reinterpret_cast<f16x8 *>(sv + SV.p_off(1)) = pl;
                    } else {
                        *reinterpret_cast<f16x8 *>(sv + SV.p_off(0)) = ph + pl;
                    }
                }
            }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
            if (kb == 1 || w < 2) {
                const f16x8 mh = tri_t(sx + S::M, kb), ml = tri_t(sx + S::M + GdrLayout::kTri, kb);
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) {
                    const f16x8 oh = ld_frag(sx + S::XO + (kb * NCT + ct) * 1024, lane);
                    Y[ct] = mma16(mh, oh, Y[ct]);
                    Y1[ct] = mma16(ml, oh, Y1[ct]);
                    if constexpr (NI == 2) Y1[ct] = mma16(mh, ld_frag(sx + S::XO + ((2 + kb) * NCT + ct) * 1024, lane), Y1[ct]);
                }
            }
        const int eu = gdr_exp(64.f * ldexp2(1.f, 14 - em) * omax + cl * pmax);
        float um = 0.f;
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
            f32x4 dU;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                dU[i] = scale_down(Y[ct][i] + Y1[ct][i], em + eo) + eL0[i] * scale_down(Z[ct][i] + Z1[ct][i], ek + ep);
            um = max_abs4(dU, um);
            f16x4 hi, lo;
            split4(dU, pow2f(eu), hi, lo);
            lds_u8 *f = sx + S::XU + ((w >> 1) * NCT + ct) * 1024;
            st_half_frag(f, w & 1, g, n, hi);
            st_half_frag(f + 2 * NCT * 1024, w & 1, g, n, lo);
        }
        um = wave_max(um);
        if (lane == 0) sMax[4 + w] = um;
        load_rec(next);
        load_do(next);
        barrier_lds();

        // ---- 2. dX = T^T dU, dV = b dX, F = b e^G dX
        const float xbound = 64.f * ldexp2(1.f, 14 - et) * max4(sMax + 4);
        const int ex = gdr_exp(xbound), ef = gdr_exp(bm * xbound);
        f32x4 dX[NCT];
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
            f32x4 z = zero, z1 = zero;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
                if (kb == 1 || w < 2) {
                    const f16x8 th = tri_t(sx + S::T, kb), tl = tri_t(sx + S::T + GdrLayout::kTri, kb);
                    const f16x8 uh = ld_frag(sx + S::XU + (kb * NCT + ct) * 1024, lane);
                    const f16x8 ul = ld_frag(sx + S::XU + ((2 + kb) * NCT + ct) * 1024, lane);
                    z = mma16(th, uh, z);
                    z1 = mma16(tl, uh, mma16(th, ul, z1));
                }
            f32x4 F;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dX[ct][i] = scale_down(z[i] + z1[i], et + eu);
                F[i] = be0[i] * eG0[i] * dX[ct][i];
            }
            f16x4 hi, lo;
            split4(F, pow2f(ef), hi, lo);
            lds_u8 *f = sx + S::XF + ((w >> 1) * NCT + ct) * 1024;
            st_half_frag(f, w & 1, g, n, hi);
            st_half_frag(f + 2 * NCT * 1024, w & 1, g, n, lo);
        }
        barrier_lds();

        // ---- 3. dP = e^{G_last} dP' + Q^T (scale e^G dO) - K^T F
#pragma unroll
        for (int t = 0; t < NTW; ++t) {
            const int tile = NTW * w + t;
            f32x4 a[NCT], a1[NCT], d[NCT], d1[NCT];
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) a[ct] = a1[ct] = d[ct] = d1[ct] = zero;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const int at = (2 * kb * NKB + (tile >> 1)) * 1024;
                const f16x8 q = ld_frag_t(sx + S::Q + at, sx + S::Q + at + NKB * 1024, tile, lane);
                const f16x8 k = ld_frag_t(sx + S::K + at, sx + S::K + at + NKB * 1024, tile, lane);
                f16x8 q1 = q, k1 = k;
                if constexpr (NI == 2) {
                    q1 = ld_frag_t(sx + S::Q + L.mat() + at, sx + S::Q + L.mat() + at + NKB * 1024, tile, lane);
                    k1 = ld_frag_t(sx + S::K + L.mat() + at, sx + S::K + L.mat() + at + NKB * 1024, tile, lane);
                }
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) {
                    const f16x8 hh = ld_frag(sx + S::XH + (kb * NCT + ct) * 1024, lane);
                    const f16x8 hl = ld_frag(sx + S::XH + ((2 + kb) * NCT + ct) * 1024, lane);
                    const f16x8 fh = ld_frag(sx + S::XF + (kb * NCT + ct) * 1024, lane);
                    const f16x8 fl = ld_frag(sx + S::XF + ((2 + kb) * NCT + ct) * 1024, lane);
                    a[ct] = mma16(q, hh, a[ct]);
                    a1[ct] = mma16(q, hl, a1[ct]);
                    d[ct] = mma16(k, fh, d[ct]);
                    d1[ct] = mma16(k, fl, d1[ct]);
                    if constexpr (NI == 2) {
                        a1[ct] = mma16(q1, hh, a1[ct]);
                        d1[ct] = mma16(k1, fh, d1[ct]);
                    }
                }
            }
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    P[t][ct][i] = fmaf(P[t][ct][i], last, scale_down(a[ct][i] + a1[ct][i], eq + eh)) -
                                  scale_down(d[ct][i] + d1[ct][i], ek + ef);
        }
        // the state's bound needs the next maximum, so it is taken, not bounded: one more barrier
        const float mp = max_p(), mo = max_do();
        if (lane == 0) {
            sMax[12 + w] = mp;
            sMax[8 + w] = mo;
        }
        // outputs of this chunk meanwhile
        unsigned char *sv = save + (size_t)c * (p.dv / 16) * SV.bytes();
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
            f16x4 hi, lo;
            if constexpr (NI == 2) split4(dX[ct], pow2f(ex), hi, lo);
            else hi = round4(dX[ct], pow2f(ex));
            unsigned char *to = sv + ct * SV.bytes() + (w >> 1) * 1024 + fo + 8 * (w & 1);
            *reinterpret_cast<f16x4 *>(to + SV.u_off(0)) = hi;
            if constexpr (NI == 2) *reinterpret_cast<f16x4 *>(to + SV.u_off(1)) = lo;
            if (threadIdx.x == 0) {
                reinterpret_cast<int *>(sv + ct * SV.bytes())[0] = ep;
                reinterpret_cast<int *>(sv + ct * SV.bytes())[1] = ex;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (64 * c + row0 + i < len) dvp[(size_t)(64 * c + i) * p.dv + 16 * ct] = from_f<E>(be0[i] * dX[ct][i]);
        }
        barrier_lds();
        const float newmax = max4(sMax + 12);
        if (threadIdx.x < 4) sMax[threadIdx.x] = sMax[12 + threadIdx.x];
        ep = gdr_exp(newmax);
        put_p(ep);
    }
    if (p.dinit != nullptr)
#pragma unroll
        for (int t = 0; t < NTW; ++t)
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
                *reinterpret_cast<f32x4 *>(p.dinit + state0 + (size_t)16 * ct * DK + perm_row(NTW * w + t, 4 * g)) = P[t][ct];
}

}  // namespace kda
