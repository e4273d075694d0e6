// Chunk-parallel stage of the gated delta rule (gdr_common.h): one 256-thread work-group per
// (chunk, value head, batch) writes the value record (T, M and the decays); the first value head of
// a key head also writes the key record (Q and K as fp16 fragments).  K K^T and Q K^T are formed
// again for every value head: they are 1 % of the work-group's time, and a loop over the heads that
// kept them cost more in registers (one wave per SIMD) than it saved.
//
//  1. Q and K are read once (16-byte pieces, the fragment layout), scaled to fp16 and written out;
//     K's fragments also go to LDS.  Wave w owns row tile w and forms its rows of K K^T and Q K^T
//     with MFMAs.
//  2. The prefix sum of g in double precision, so that a difference G_i - G_j late in
//     the chunk is not hurt by a large decay early in it; A to LDS in float32.
//  3. T = (I + A)^-1: each wave inverts one 16x16 diagonal block by forward substitution (lane =
//     column), then two levels of blocks, T21 = -T22 (A21 T11), on float32 MFMAs.
//  4. T as two fp16 pieces, M as one (or two), in fragment order.
//
// Per chunk and value head the stage reads 128 dk values (once from HBM for a key head) and writes 19
// KiB, and 32 KiB a key head; the LDS is kept at 35 KiB (dk = 128, bf16) to have four work-groups on a
// CU, which hide the latency of step 3.  65,536 tokens, 16 key heads, 32 value heads: 422 us for 1.7
// GB, 4.0 TB/s, 86 % of a copy's rate.
#pragma once
#include "gdr_common.h"

namespace kda {

struct GdrChunkArgs {
    const void *q, *k, *g, *beta;
    Strides3 sq, sk, sg, sb;
    GdrSeqs seqs;
    int Hk, r, nslot;  // key heads, value heads per key head, chunk slots per batch entry
    float scale;
    unsigned char *keys, *vals;
};

// eight consecutive values as floats
__device__ __forceinline__ void ld8(const __bf16 *p, float (&x)[8]) {
    const bf16x8 v = *reinterpret_cast<const bf16x8 *>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)v[i];
}
__device__ __forceinline__ void ld8(const float *p, float (&x)[8]) {
    const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) { x[i] = a[i]; x[4 + i] = b[i]; }
}

// maximum over the work-group (256 threads); red: 4 floats, free again after the next barrier
__device__ __forceinline__ float block_most(const Most &m, float *red) {
    const float x = m.wave();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}

template <int DK, bool F32, int MP>
__global__ __launch_bounds__(256, 4) void gdr_chunk_kernel(const GdrChunkArgs p) {
    using E = typename std::conditional<F32, float, __bf16>::type;
    constexpr int NI = F32 ? 2 : 1, NKB = DK / 32, LD = 68;
    constexpr GdrLayout L{NI, DK, MP};
    constexpr int kMat = 64 * LD * 4, kFrag = NI * L.mat();
    // K's fragments die before A and T come to life
    constexpr int kBuf = 2 * kMat > kFrag ? 2 * kMat : kFrag;
    __shared__ __attribute__((aligned(16))) unsigned char smem[kBuf];
    __shared__ double sG[64];
    __shared__ float sBeta[64], sK1[64], sKm[64];  // beta; sum and maximum of |k| per token
    __shared__ __attribute__((aligned(16))) float sGf[64];  // G in float32, for a bound
    __shared__ float red[24];
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, m = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slot = blockIdx.x, h = blockIdx.y, b = blockIdx.z, H = p.Hk * p.r, kh = h / p.r;
    const bool first = h % p.r == 0;  // writes the key record
    int t0, n;
    const int nrow = p.seqs.find(b, slot, t0, n);
    if (nrow <= 0) return;
    float *sA = reinterpret_cast<float *>(smem), *sT = sA + 64 * LD;

    // ---- 1. Q, K
    const int tr = perm_row(w, m), trc = tr < nrow ? tr : nrow - 1;  // rows past the last repeat it
    const E *qp = reinterpret_cast<const E *>(p.q) + b * p.sq.b + kh * p.sq.h + (long long)(t0 + trc) * p.sq.t + 8 * g;
    const E *kp = reinterpret_cast<const E *>(p.k) + b * p.sk.b + kh * p.sk.h + (long long)(t0 + trc) * p.sk.t + 8 * g;
    float xk[NKB][8], xq[NKB][8];
    Most mk_, mq;
#pragma unroll
    for (int kb = 0; kb < NKB; ++kb) {
        ld8(kp + 32 * kb, xk[kb]);
        ld8(qp + 32 * kb, xq[kb]);
    }
#pragma unroll
    for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
            mk_.add4(f32x4{xk[kb][j], xk[kb][j + 1], xk[kb][j + 2], xk[kb][j + 3]});
            mq.add4(f32x4{xq[kb][j], xq[kb][j + 1], xq[kb][j + 2], xq[kb][j + 3]});
        }
    const int ek = gdr_exp(block_most(mk_, red)), eq = gdr_exp(block_most(mq, red + 4));
    {
        float k1 = 0.f, mk = mk_.lane();
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
            for (int j = 0; j < 8; ++j) k1 += fabsf(xk[kb][j]);
        k1 += __shfl_xor(k1, 16, 64);
        k1 += __shfl_xor(k1, 32, 64);
        mk = fmaxf(mk, __shfl_xor(mk, 16, 64));
        mk = fmaxf(mk, __shfl_xor(mk, 32, 64));
        if (g == 0) {
            sK1[tr] = k1;
            sKm[tr] = mk;
        }
    }
    unsigned char *krec = p.keys + ((size_t)(b * p.Hk + kh) * p.nslot + slot) * L.key_bytes();
    lds_u8 *sK = lds_base(smem);
    f16x8 fk[NI][NKB], fq[NI][NKB];
    {
        const float s = pow2f(ek), t = pow2f(eq);
        const int fo = frag_slot(g, m);
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
            const f32x4 k0 = {xk[kb][0], xk[kb][1], xk[kb][2], xk[kb][3]}, k1 = {xk[kb][4], xk[kb][5], xk[kb][6], xk[kb][7]};
            const f32x4 q0 = {xq[kb][0], xq[kb][1], xq[kb][2], xq[kb][3]}, q1 = {xq[kb][4], xq[kb][5], xq[kb][6], xq[kb][7]};
            if constexpr (NI == 2) {
                split_pair(k0, k1, s, fk[0][kb], fk[1][kb]);
                split_pair(q0, q1, t, fq[0][kb], fq[1][kb]);
            } else {
                fk[0][kb] = round_pair(k0, k1, s);  // exact: bf16 values at most 2^14
                fq[0][kb] = round_pair(q0, q1, t);
            }
#pragma unroll
            for (int x = 0; x < NI; ++x) {
                const int at = (w * NKB + kb) * 1024 + fo;
                if (first) {
                    *reinterpret_cast<f16x8 *>(krec + L.k_off(x) + at) = fk[x][kb];
                    *reinterpret_cast<f16x8 *>(krec + L.q_off(x) + at) = fq[x][kb];
                }
                *reinterpret_cast<__attribute__((address_space(3))) f16x8 *>(sK + x * L.mat() + at) = fk[x][kb];
            }
        }
    }
    __syncthreads();
    // rows perm_row(w, 4 g + i), columns perm_row(c, m), c up to the end of w's 32-token block
    const int nc = w < 2 ? 2 : 4;
    f32x4 kk[4], qk[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        kk[c] = f32x4{0.f, 0.f, 0.f, 0.f};
        qk[c] = kk[c];
        if (c < nc) {
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                const f16x8 f0 = ld_frag(sK + (c * NKB + kb) * 1024, lane);
                kk[c] = mma16(fk[0][kb], f0, kk[c]);
                qk[c] = mma16(fq[0][kb], f0, qk[c]);
                if constexpr (NI == 2) {
                    const f16x8 f1 = ld_frag(sK + L.mat() + (c * NKB + kb) * 1024, lane);
                    kk[c] = mma16(fk[1][kb], f0, mma16(fk[0][kb], f1, kk[c]));
                    qk[c] = mma16(fq[1][kb], f0, mma16(fq[0][kb], f1, qk[c]));
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                kk[c][i] = scale_down(kk[c][i], 2 * ek);
                qk[c][i] = scale_down(qk[c][i], ek + eq) * p.scale;
            }
        }
    }

    unsigned char *vrec = p.vals + ((size_t)(b * H + h) * p.nslot + slot) * L.val_bytes();
    __syncthreads();  // K's fragments have been read
    // ---- 2. decays
    if (w == 0) {
        const bool in = lane < nrow;
        float gv = 0.f, bv = 0.f;
        if (in) {
            gv = to_f(reinterpret_cast<const E *>(p.g)[b * p.sg.b + h * p.sg.h + (long long)(t0 + lane) * p.sg.t]);
            bv = to_f(reinterpret_cast<const E *>(p.beta)[b * p.sb.b + h * p.sb.h + (long long)(t0 + lane) * p.sb.t]);
        }
        // a decay below e^-1000 is zero, -inf among them; NaN stays
        double G = (double)(gv < -1000.f ? -1000.f : gv) * 1.4426950408889634;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const double y = __shfl_up(G, d, 64);
            if (lane >= d) G += y;
        }
        const double last = __shfl(G, 63, 64);
        sG[lane] = G;
        sGf[lane] = (float)G;
        sBeta[lane] = bv;
        float *hd = reinterpret_cast<float *>(vrec);
        hd[lane] = ex2((float)G);
        hd[64 + lane] = ex2((float)(last - G));
        hd[128 + lane] = bv;
        // what the state stage bounds its operands with (GdrLayout)
        auto norm = [](float x) { return wave_max(finite_mag(x)); };
        const float ck = norm(bv * sK1[lane] * ex2((float)G)), bm = norm(bv);
        const float cl = norm(ex2((float)(last - G)) * sK1[lane]), k1 = norm(sK1[lane]);
        float ks = in ? sKm[lane] : 0.f;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) ks += __shfl_xor(ks, d, 64);
        if (lane == 0) {
            hd[192] = ex2((float)last);
            reinterpret_cast<int *>(vrec)[195] = ek;
            reinterpret_cast<int *>(vrec)[196] = eq;
            hd[197] = ck;
            hd[198] = bm;
            hd[200] = ks;
            hd[201] = cl;
            hd[203] = k1;
        }
    }
    __syncthreads();
    f32x4 dec[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        dec[c] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (c < nc) {
            const int j = perm_row(c, m);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = perm_row(w, 4 * g + i);
                dec[c][i] = row >= j ? ex2((float)(sG[row] - sG[j])) : 0.f;
                sA[row * LD + j] = row > j ? kk[c][i] * dec[c][i] * sBeta[row] : 0.f;
            }
        }
    }
    __syncthreads();
    // ---- 3. T = (I + A)^-1
    {
        // row i + 1 is read while row i is summed; no further ahead, which would only spill
        float t[16];
        f32x4 a[4], an[4];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                a[j] = an[j];
                if (4 * j < i + 1 && i < 15)
                    an[j] = *reinterpret_cast<const f32x4 *>(sA + (16 * w + i + 1) * LD + 16 * w + 4 * j);
            }
            __builtin_amdgcn_sched_barrier(0);
            float acc = i == m ? 1.f : 0.f;
#pragma unroll
            for (int j = 0; j < i; ++j) acc = fmaf(-a[j >> 2][j & 3], t[j], acc);
            asm volatile("" : "+v"(acc));  // summed here, not where T is stored
            t[i] = acc;
        }
        float mine[4];  // rows 4 g .. 4 g + 3
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[i] = g < 2 ? (g == 0 ? t[i] : t[4 + i]) : (g == 2 ? t[8 + i] : t[12 + i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float *to = sT + (16 * w + 4 * g + i) * LD + 16 * w + m;
            to[0] = mine[i];
            if (w & 1) to[-16 * LD] = 0.f;
        }
    }
    __syncthreads();
    // one 16x16x16 product with float32 operands: A row-major at a, B from LDS or registers
    auto a4 = [&](const float *a) { return *reinterpret_cast<const f32x4 *>(a + m * LD + 4 * g); };
    auto b4 = [&](const float *bm) {
        return f32x4{bm[(4 * g) * LD + m], bm[(4 * g + 1) * LD + m], bm[(4 * g + 2) * LD + m], bm[(4 * g + 3) * LD + m]};
    };
    auto prod = [&](const f32x4 &a, const f32x4 &bb, f32x4 c) {
#pragma unroll
        for (int s = 0; s < 4; ++s) c = mma4(a[s], bb[s], c);
        return c;
    };
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    if (w < 2) {
        const int br = 2 * w + 1, bc = 2 * w;
        const f32x4 z = prod(a4(sA + 16 * br * LD + 16 * bc), b4(sT + 16 * bc * LD + 16 * bc), zero);
        const f32x4 t = prod(a4(sT + 16 * br * LD + 16 * br), z, zero);
#pragma unroll
        for (int i = 0; i < 4; ++i) sT[(16 * br + 4 * g + i) * LD + 16 * bc + m] = -t[i];
    }
    __syncthreads();
    if (w < 2) {
        f32x4 z[2];
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
            z[rt] = prod(a4(sA + 16 * (2 + rt) * LD + 16), b4(sT + 16 * LD + 16 * w), zero);
            if (w == 0) z[rt] = prod(a4(sA + 16 * (2 + rt) * LD), b4(sT), z[rt]);
        }
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
            f32x4 t = prod(a4(sT + 16 * (2 + rt) * LD + 32), z[0], zero);
            if (rt == 1) t = prod(a4(sT + 48 * LD + 48), z[1], t);
#pragma unroll
            for (int i = 0; i < 4; ++i) sT[(32 + 16 * rt + 4 * g + i) * LD + 16 * w + m] = -t[i];
        }
    }
    __syncthreads();
    // ---- 4. T and M as fragments; M takes A's place
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (c < nc) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sA[perm_row(w, 4 * g + i) * LD + perm_row(c, m)] = qk[c][i] * dec[c][i];
        }
    __syncthreads();
    f32x4 ft[2][2], fm[2][2];
    Most mt, mm, mrs, mrt;
    float rs = 0.f, rt = 0.f;
    const float gi = sGf[perm_row(w, m)];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
        if (kb == 0 || w >= 2) {
            const int at = perm_row(w, m) * LD + 32 * kb + 8 * g;
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                ft[kb][o] = *reinterpret_cast<const f32x4 *>(sT + at + 4 * o);
                fm[kb][o] = *reinterpret_cast<const f32x4 *>(sA + at + 4 * o);
                mt.add4(ft[kb][o]);
                mm.add4(fm[kb][o]);
#pragma unroll
                for (int i = 0; i < 4; ++i) rs += fabsf(ft[kb][o][i]);
                const f32x4 gj = *reinterpret_cast<const f32x4 *>(sGf + 32 * kb + 8 * g + 4 * o);
#pragma unroll
                for (int i = 0; i < 4; ++i) rt = fmaf(fabsf(ft[kb][o][i]), ex2(fminf(gj[i] - gi, 126.f)), rt);
            }
        }
    rt += __shfl_xor(rt, 16, 64);
    rt += __shfl_xor(rt, 32, 64);
    mrt.add(rt);
    rt = block_most(mrt, red + 20);
    rs += __shfl_xor(rs, 16, 64);
    rs += __shfl_xor(rs, 32, 64);
    mrs.add(rs);
    rs = block_most(mrs, red + 16);
    const int et = gdr_exp(block_most(mt, red + 8)), em = gdr_exp(block_most(mm, red + 12));
    if (tid == 0) {
        reinterpret_cast<int *>(vrec)[193] = et;
        reinterpret_cast<int *>(vrec)[194] = em;
        reinterpret_cast<float *>(vrec)[199] = rs;
        reinterpret_cast<float *>(vrec)[202] = rt;
    }
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
        if (kb == 0 || w >= 2) {
            const int at = tri_frag(w, kb) * 1024 + frag_slot(g, m);
            f16x8 hi, lo;
            split_pair(ft[kb][0], ft[kb][1], pow2f(et), hi, lo);
            *reinterpret_cast<f16x8 *>(vrec + L.t_off(0) + at) = hi;
            *reinterpret_cast<f16x8 *>(vrec + L.t_off(1) + at) = lo;
            if constexpr (MP == 2) {
                split_pair(fm[kb][0], fm[kb][1], pow2f(em), hi, lo);
                *reinterpret_cast<f16x8 *>(vrec + L.m_off(0) + at) = hi;
                *reinterpret_cast<f16x8 *>(vrec + L.m_off(1) + at) = lo;
            } else {
                *reinterpret_cast<f16x8 *>(vrec + L.m_off(0) + at) = round_pair(fm[kb][0], fm[kb][1], pow2f(em));
            }
        }
}

}  // namespace kda
