// Expanded latent attention, forward: one work-group per 128 queries of one head, keys in tiles of 64
// through LDS, 32 queries a wave (two column tiles).  Per tile a wave does 2 x 4 x (dn + dr) / 32 + 2 x
// 2 x dn / 16 MFMAs (80 at 128 + 64, 1,280 cycles) on 40 KiB of LDS reads.  The next tile is loaded
// into registers between the score products and stored into the other of two 40 KiB buffers between
// the value products, one barrier a tile.  One pass over the keys with the running maximum and sum of
// the softmax.  Work-groups of a head share an XCD's L2; the last queries, which see most keys, start
// first.
//
// NG = 1: four waves, two work-groups on a CU, one's softmax beside the other's MFMAs.  NG = 2: two
// groups of four waves take every other key tile for the same queries and join their accumulators at
// the end.  While no more work-groups come after the first two on a CU, a long row of a causal triangle
// soon runs alone with one wave a SIMD (4,600 cycles a tile), and two groups keep both waves at work:
// 16 heads x 4096 tokens (512 work-groups) 118 us with two groups, 140 with one; 1,184 work-groups of
// ragged packed prompts 148 with two, 124 with one.  So two groups up to two work-groups a CU.
// (float32: one group, one buffer.)
#pragma once
#include "latent_common.h"

namespace kda {

struct LatentFwdArgs {
    const void *q, *k, *kr, *v;
    Strides3 sq, sk, skr, sv;  // kr: b, (unused), t
    AttnSeqs seqs;
    int H, NB, ntile;          // heads; batch entries (1: packed); query tiles per batch entry
    float scale;
    void *out;                 // [B][H][T][dn], contiguous
    float *lse;                // [B][H][T]
};

template <int DN, int DR, bool F32, int NG>
__global__ __launch_bounds__(256 * NG, F32 ? 1 : 2) void latent_fwd_kernel(const LatentFwdArgs p) {
    using Op = AttnOp<F32>;
    using E = typename Op::E;
    using V8 = typename Op::V8;
    constexpr int NKB = (DN + DR) / 32, NDB = DN / 32, NT = DN / 16, NQ = 2;
    constexpr int TILE = (4 * NKB + 4 * NDB) * Op::FB, NBUF = F32 ? 1 : 2;
    static_assert(NG == 1 || 256 * (NT * NQ + 1) * 16 <= NG * NBUF * TILE, "the second group's accumulators fit");
    __shared__ __attribute__((aligned(1024))) unsigned char smem[NG * NBUF * TILE];
    const int tid = threadIdx.x & 255, lane = tid & 63, g = lane >> 4, n = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6), grp = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
    const int unit = (blockIdx.x >> 3) / p.ntile * 8 + (blockIdx.x & 7);
    const int slot = p.ntile - 1 - (blockIdx.x >> 3) % p.ntile;
    if (unit >= p.NB * p.H) return;
    const int b = unit / p.H, h = unit % p.H;
    int seq, tile, q0, nq, k0, nk;
    if (!p.seqs.template find<128>(p.seqs.cu_q, p.seqs.T, b, slot, seq, tile)) return;
    AttnSeqs::range(p.seqs.cu_q, seq, p.seqs.T, q0, nq);
    AttnSeqs::range(p.seqs.cu_k, seq, p.seqs.S, k0, nk);
    if (tile * 128 >= nq) return;
    const int qw = tile * 128 + 32 * w, shift = nk - nq;  // query i sees keys 0 .. i + shift
    const E *kp = reinterpret_cast<const E *>(p.k) + b * p.sk.b + h * p.sk.h + (long long)k0 * p.sk.t;
    const E *rp = reinterpret_cast<const E *>(p.kr) + b * p.skr.b + (long long)k0 * p.skr.t;
    const E *vp = reinterpret_cast<const E *>(p.v) + b * p.sv.b + h * p.sv.h + (long long)k0 * p.sv.t;
    const E *qp = reinterpret_cast<const E *>(p.q) + b * p.sq.b + h * p.sq.h + (long long)q0 * p.sq.t + 8 * g;
    const int lastq = min(tile * 128 + 127, nq - 1);
    const int nkey = max(0, min(nk, lastq + shift + 1)), ntk = (nkey + 63) / 64;
    const float c = p.scale * kLog2e;

    V8 qf[NQ][NKB];
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        const int r = min(qw + 16 * x + n, nq - 1);
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) qf[x][kb] = Op::load(qp + (long long)r * p.sq.t + 32 * kb);
    }
    f32x4 O[NT][NQ];
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int x = 0; x < NQ; ++x) O[t][x] = zero;
    float m[NQ], l[NQ];  // running maximum (of the scaled scores, log2 units) and sum of a lane's column
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        m[x] = -INFINITY;
        l[x] = 0.f;
    }
    TileStage<F32, DN / 8> stk, stv;
    TileStage<F32, DR / 8> str;
    auto load_tile = [&](int kt, int part) {
        if (part == 0) stk.load(kp, p.sk.t, 64 * kt, nk, tid);
        if (part == 1) str.load(rp, p.skr.t, 64 * kt, nk, tid);
        if (part == 2) stv.load(vp, p.sv.t, 64 * kt, nk, tid);
    };
    auto store_tile = [&](lds_u8 *to, int part) {
        if (part == 0) stk.store(to, NKB, 0, tid);
        if (part == 1) str.store(to, NKB, NDB, tid);
        if (part == 2) stv.store(to + 4 * NKB * Op::FB, NDB, 0, tid);
    };
    lds_u8 *mine = lds_base(smem) + grp * NBUF * TILE;
    if (ntk > 0) {
#pragma unroll
        for (int part = 0; part < 3; ++part) load_tile(grp, part);
#pragma unroll
        for (int part = 0; part < 3; ++part) store_tile(mine, part);
        barrier_lds();
    }
    int buf = 0;
    for (int k2 = 0; k2 < ntk; k2 += NG) {  // as many rounds for either group: a tile past the last is all masked
        const int kt = k2 + grp;
        const lds_u8 *sk = mine + (NBUF == 2 ? buf * TILE : 0), *sv = sk + 4 * NKB * Op::FB;
        const int first = 64 * kt;
        f32x4 s[4][NQ];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            V8 kf[NKB];
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) kf[kb] = Op::get(sk + (t * NKB + kb) * Op::FB, kb, lane);
            if (t < 3) load_tile(kt + NG, t);  // behind the last tile it loads nothing
#pragma unroll
            for (int x = 0; x < NQ; ++x) s[t][x] = zero;
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
                for (int x = 0; x < NQ; ++x) s[t][x] = Op::mma(kf[kb], qf[x][kb], s[t][x]);
            __builtin_amdgcn_sched_barrier(0);  // no fragments of later tiles in registers yet
        }
        float mx[NQ];
        bool grown = false;
        if (first + 64 > nk || first + 63 > qw + shift) {
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                const int see = min(nk - 1, qw + 16 * x + n + shift) - first - 8 * g;  // last visible key
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (perm_row(t, i) > see) s[t][x][i] = -INFINITY;
            }
        }
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            float a = fmaxf(fmaxf(s[0][x][0], s[0][x][1]), fmaxf(s[0][x][2], s[0][x][3]));
#pragma unroll
            for (int t = 1; t < 4; ++t) a = fmaxf(a, fmaxf(fmaxf(s[t][x][0], s[t][x][1]), fmaxf(s[t][x][2], s[t][x][3])));
            mx[x] = col_max(a) * c;
            grown |= mx[x] > m[x] + 8.f;  // any finite score at first: m is -inf
        }
        // the exponentials are taken against a maximum that may be 2^8 too small: bf16 and float32 keep
        // their relative precision there, and the accumulator is scaled a few times a row, not every tile
        if (__builtin_amdgcn_ballot_w64(grown) != 0) {
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                const float now = fmaxf(m[x], mx[x]), alpha = now == -INFINITY ? 1.f : ex2(m[x] - now);
                m[x] = now;
                l[x] *= alpha;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) O[t][x][i] *= alpha;
            }
        }
        V8 pf[2][NQ];
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            const float mm = m[x] == -INFINITY ? 0.f : m[x];  // a column that has seen nothing yet
            f32x4 sum = zero;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[t][x][i] = ex2(fmaf(s[t][x][i], c, -mm));
                    sum[i] += s[t][x][i];
                }
            l[x] += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            pf[0][x] = Op::pair(s[0][x], s[1][x]);
            pf[1][x] = Op::pair(s[2][x], s[3][x]);
        }
        buf ^= 1;
        lds_u8 *to = mine + (NBUF == 2 ? buf * TILE : 0);
        V8 vf[2][2];
        auto load_v = [&](int t) {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const lds_u8 *f0 = sv + (2 * kb * NDB + (t >> 1)) * Op::FB;
                vf[t & 1][kb] = Op::get_t(f0, f0 + NDB * Op::FB, t, lane);
            }
        };
        load_v(0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t + 1 < NT) load_v(t + 1);
            if (NBUF == 2 && t < 3) store_tile(to, t);  // the next tile into the other buffer
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int x = 0; x < NQ; ++x) O[t][x] = Op::mma(vf[t & 1][kb], pf[kb][x], O[t][x]);
            __builtin_amdgcn_sched_barrier(0);
        }
        barrier_lds();  // this tile has been read, and (two buffers) the next one is there
        if constexpr (NBUF == 1) {
#pragma unroll
            for (int part = 0; part < 3; ++part) store_tile(to, part);
            barrier_lds();
        }
    }
    if constexpr (NG == 2) {  // the second group hands its accumulators over; both are past the last barrier
        typedef __attribute__((address_space(3))) f32x4 lds_f4;
        lds_f4 *ex = reinterpret_cast<lds_f4 *>(lds_base(smem)) + tid;
        if (grp == 1) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int x = 0; x < NQ; ++x) ex[256 * (t * NQ + x)] = O[t][x];
            ex[256 * NT * NQ] = f32x4{m[0], l[0], m[1], l[1]};
        }
        barrier_lds();
        if (grp == 1) return;
        const f32x4 ml = ex[256 * NT * NQ];
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            const float now = fmaxf(m[x], ml[2 * x]);
            const float a = now == -INFINITY ? 0.f : ex2(m[x] - now), d = now == -INFINITY ? 0.f : ex2(ml[2 * x] - now);
            m[x] = now;
            l[x] = l[x] * a + ml[2 * x + 1] * d;
#pragma unroll
            for (int t = 0; t < NT; ++t) O[t][x] = O[t][x] * a + ex[256 * (t * NQ + x)] * d;
        }
    }
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        const int r = qw + 16 * x + n;
        l[x] = col_sum(l[x]);
        if (r >= nq) continue;
        const size_t row = ((size_t)(b * p.H + h)) * p.seqs.T + q0 + r;
        const float inv = l[x] == 0.f ? 0.f : 1.f / l[x];  // a query that sees nothing: zeros, -inf; NaN stays
#pragma unroll
        for (int t = 0; t < NT; t += 2) {
            f32x4 a = O[t][x], d = O[t + 1][x];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] *= inv;
                d[i] *= inv;
            }
            Op::store8(reinterpret_cast<E *>(p.out) + row * DN + 16 * t + 8 * g, a, d);
        }
        if (g == 0) p.lse[row] = l[x] == 0.f ? -INFINITY : (m[x] + lg2(l[x])) * kLn2;
    }
}

}  // namespace kda
