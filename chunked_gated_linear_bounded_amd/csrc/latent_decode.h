// Absorbed latent attention, one token per sequence against a paged cache of latent rows
// c = [latent (dc), rotary part (dr)]: s_j = scale q . c_j, o = sum p_j c_j[:dc].
//
// A row serves every head as key and as value, so the cache is read once for up to 64 heads: a
// work-group of NW waves takes one sequence, one part of its keys and 16 NW / WS heads, with WS waves
// on each 16 heads.  32 keys at a time go through registers into LDS (36 KiB at 512 + 64, bf16); S^T is
// C Q^T, and O^T = C^T P^T reads the same tile transposed.  The waves on the same heads split S by key
// tile (WS = 4: also by half of the contraction), hand it round through LDS, and split the dc rows of
// O^T: one wave alone would need 128 registers for O^T and 72 for its queries, and spilled.
//
// Up to 16 heads the 2 * 16 * (576 + 512) flops a 1,152-byte row costs are far below what HBM lets
// pass; at 128 heads (two work-groups on the same keys, side by side on one XCD) the 272 KiB of LDS
// reads per tile and work-group take about the time HBM needs for the tile.  The keys are split
// over work-groups until there are 512, two a CU (on 64 heads at dc = 512 one behind the other: 221
// registers leave a CU one work-group of eight waves), but a sequence into at most 64 parts; the parts
// are joined by their log-sum-exps in a second kernel, which walks them one behind the other.  48
// sequences of 6,000 to 12,000 rows, 128 heads: 309 us and 14 for the join (768 work-groups: 345 and
// 24).  One sequence of 20,000 rows, 16 heads, whole calls: 47 us with 64 parts, 105 with 256, 151
// with 313.
#pragma once
#include "latent_common.h"

namespace kda {

struct LatentDecodeArgs {
    const void *q;             // [B][H][dc + dr]
    const void *cache;         // [pages][page][dc + dr]
    const int *table;          // [B][max_pages]
    const int *lengths;        // [B]
    int B, H, pages, page, max_pages, nsplit, hgroups;
    float scale;
    void *out;                 // [B][H][dc]
    float *lse;                // [B][H]
    float *part;               // nsplit > 1: [B][nsplit][H][dc], then [B][nsplit][H] log-sum-exps (log2)
    float *part_lse;
    // 32-key tiles of sequence b, and of each of its parts
    __device__ __forceinline__ int tiles(int b, int &len, int &per) const {
        const long long most = (long long)max_pages * page;
        const int given = lengths[b];
        len = given < 0 ? 0 : (given > most ? (int)most : given);
        const int n = (len + 31) / 32;
        per = (n + nsplit - 1) / nsplit;
        return n;
    }
};

template <int DC, int DR, bool F32, int WS, int NW>
__global__ __launch_bounds__(64 * NW, F32 ? 1 : 2) void latent_decode_kernel(const LatentDecodeArgs p) {
    using Op = AttnOp<F32>;
    using E = typename Op::E;
    using V8 = typename Op::V8;
    constexpr int D = DC + DR, NKB = D / 32, NC = D / 8, HT = NW / WS;  // head tiles of the work-group
    constexpr int NT = DC / 16 / WS;                                   // rows tiles of O^T per wave
    constexpr int KP = WS == 4 ? 2 : 1, NB = (NKB + KP - 1) / KP;      // parts of the contraction
    constexpr int TPR = 2 * NW, NST = (NC + TPR - 1) / TPR;            // threads on a row, pieces a thread
    static_assert(WS > 1 && TPR % 4 == 0, "S goes through LDS; a thread's pieces keep their place in a block");
    typedef __attribute__((address_space(3))) f32x4 lds_f4;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[2 * NKB * Op::FB];
    __shared__ __attribute__((aligned(16))) unsigned char sx[HT * KP * 2 * 1024];
    __shared__ long long soff[2][32];
    lds_u8 *sc = lds_base(smem), *ss = lds_base(sx);
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, n = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6), ws = w % WS, ht = w / WS;
    const int unit = blockIdx.x / (8 * p.hgroups) * 8 + (blockIdx.x & 7), hg = (blockIdx.x >> 3) % p.hgroups;
    if (unit >= p.B * p.nsplit) return;
    const int b = unit / p.nsplit, split = unit % p.nsplit;
    const int head = (hg * HT + ht) * 16 + n, hc = head < p.H ? head : p.H - 1;
    int len, per;
    const int ntile = p.tiles(b, len, per);
    const int first = split * per, last = min(first + per, ntile);
    const E *cache = reinterpret_cast<const E *>(p.cache);
    const float c = p.scale * kLog2e;

    const int kpart = WS == 4 ? ws >> 1 : 0, kb0 = kpart * NB;
    V8 qf[NB];
#pragma unroll
    for (int kb = 0; kb < NB; ++kb)
        qf[kb] = kb0 + kb < NKB ? Op::load(reinterpret_cast<const E *>(p.q) + ((size_t)b * p.H + hc) * D + 32 * (kb0 + kb) + 8 * g)
                                : Op::zero();
    // Row r of a tile: key 32 tile + r (past the last: the last), on a page of the table; pages outside the
    // cache are clipped.  The table is read two tiles before the rows, in front of the rows' loads: a
    // wait for it is then no wait for them.
    const int *table = p.table + (size_t)b * p.max_pages;
    auto key_of = [&](int tile) { return min(32 * min(tile, last - 1) + (tid & 31), len - 1); };
    auto put_row = [&](int tile, int pg) {
        pg = pg < 0 ? 0 : (pg >= p.pages ? p.pages - 1 : pg);
        if (tid < 32) soff[tile & 1][tid] = ((long long)pg * p.page + key_of(tile) % p.page) * D;
    };
    V8 st[NST];
    auto load = [&](int tile) {
        const E *row = cache + soff[tile & 1][tid / TPR];
#pragma unroll
        for (int i = 0; i < NST; ++i) {
            const int piece = tid % TPR + TPR * i;
            st[i] = Op::load(row + 8 * (NC % TPR == 0 || piece < NC ? piece : NC - 1));
        }
    };
    f32x4 O[NT];
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < NT; ++t) O[t] = zero;
    float m = -INFINITY, l = 0.f;
    int pg = 0;  // this thread's page of the tile after next
    if (first < last) {
        put_row(first, table[key_of(first) / p.page]);
        put_row(first + 1, table[key_of(first + 1) / p.page]);
        pg = table[key_of(first + 2) / p.page];
        __syncthreads();
        load(first);
    }
    for (int tile = first; tile < last; ++tile) {
        barrier_lds();  // the last tile has been read
        const int r = tid / TPR, c0 = tid % TPR;
        lds_u8 *to = sc + (perm_tile(r) * NKB + (c0 >> 2)) * Op::FB;
#pragma unroll
        for (int i = 0; i < NST; ++i)
            if (NC % TPR == 0 || TPR * i + TPR <= NC || c0 + TPR * i < NC)
                Op::put(to + TPR / 4 * i * Op::FB, TPR / 4 * i + (c0 >> 2), c0 & 3, perm_m(r), st[i]);
        barrier_lds();
        put_row(tile + 2, pg);
        pg = table[key_of(tile + 3) / p.page];
        load(tile + 1);  // behind the last tile: its last rows again, not used
        f32x4 s[2];
        f32x4 x = zero;
        const int t = ws & 1;
#pragma unroll
        for (int kb = 0; kb < NB; ++kb)
            if (kb0 + kb < NKB) x = Op::mma(Op::get(sc + (t * NKB + kb0 + kb) * Op::FB, kb0 + kb, lane), qf[kb], x);
        lds_f4 *sp = reinterpret_cast<lds_f4 *>(ss + (ht * KP * 2) * 1024);
        sp[(kpart * 2 + t) * 64 + lane] = x;
        barrier_lds();
        s[0] = sp[lane];
        s[1] = sp[64 + lane];
        if constexpr (KP == 2) {
            s[0] += sp[128 + lane];
            s[1] += sp[192 + lane];
        }
        if (32 * tile + 32 > len) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (32 * tile + perm_row(t, 4 * g + i) >= len) s[t][i] = -INFINITY;
        }
        float a = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3]));
        a = fmaxf(a, fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
        const float mx = fmaxf(m, col_max(a) * c);
        if (__builtin_amdgcn_ballot_w64(mx > m) != 0) {
            const float alpha = mx == -INFINITY ? 1.f : ex2(m - mx);
            m = mx;
            l *= alpha;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) O[t][i] *= alpha;
        }
        const float mm = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[t][i] = ex2(fmaf(s[t][i], c, -mm));
                l += s[t][i];
            }
        const V8 pf = Op::pair(s[0], s[1]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int tt = ws * NT + t;
            const lds_u8 *f0 = sc + (tt >> 1) * Op::FB;
            O[t] = Op::mma(Op::get_t(f0, f0 + NKB * Op::FB, tt, lane), pf, O[t]);
            if (t % 8 == 7) __builtin_amdgcn_sched_barrier(0);  // eight fragments in flight, not all
        }
    }
    l = col_sum(l);
    // no keys: zeros, -inf; a sum that is NaN stays one
    const float inv = l == 0.f ? 0.f : 1.f / l, lse2 = l == 0.f ? -INFINITY : m + lg2(l);
    if (head >= p.H) return;
    if (p.nsplit == 1) {
        E *o = reinterpret_cast<E *>(p.out) + ((size_t)b * p.H + head) * DC;
#pragma unroll
        for (int t = 0; t < NT; t += 2) {
            const f32x4 x = O[t] * inv, y = O[t + 1] * inv;
            Op::store8(o + 16 * (ws * NT + t) + 8 * g, x, y);
            __builtin_amdgcn_sched_barrier(0);  // not all scaled copies at once: they would push Q into scratch
        }
        if (g == 0 && ws == 0) p.lse[(size_t)b * p.H + head] = lse2 * kLn2;
        return;
    }
    const size_t row = ((size_t)b * p.nsplit + split) * p.H + head;
    if (g == 0 && ws == 0) p.part_lse[row] = lse2;
    if (first >= last) return;  // nothing here, and the join reads the parts that have keys
#pragma unroll
    for (int t = 0; t < NT; t += 2) {
        float *o = p.part + row * DC + 16 * (ws * NT + t) + 8 * g;
        *reinterpret_cast<f32x4 *>(o) = O[t] * inv;
        *reinterpret_cast<f32x4 *>(o + 4) = O[t + 1] * inv;
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Joins the parts of one (sequence, head): weights 2^(lse_i - max), 4 values a thread.  Every part that
// has keys counts, so that one whose result is not finite shows.
template <int DC, typename E>
__global__ __launch_bounds__(DC / 4) void latent_join_kernel(const LatentDecodeArgs p) {
    const int b = blockIdx.y, h = blockIdx.x;
    const float *e = p.part_lse + (size_t)b * p.nsplit * p.H + h;
    int len, per;
    const int ntile = p.tiles(b, len, per), parts = per > 0 ? (ntile + per - 1) / per : 0;
    float m = -INFINITY, sum = 0.f;
    for (int i = 0; i < parts; ++i) m = fmaxf(m, e[(size_t)i * p.H]);
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < parts; ++i) {
        const float x = e[(size_t)i * p.H], wgt = x == -INFINITY ? 0.f : ex2(x - m);
        sum += wgt;
        o += wgt * *reinterpret_cast<const f32x4 *>(p.part + (((size_t)b * p.nsplit + i) * p.H + h) * DC + 4 * threadIdx.x);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    E *to = reinterpret_cast<E *>(p.out) + ((size_t)b * p.H + h) * DC + 4 * threadIdx.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] = from_f<E>(o[i] * inv);
    if (threadIdx.x == 0) p.lse[(size_t)b * p.H + h] = sum == 0.f ? -INFINITY : (m + lg2(sum)) * kLn2;
}

}  // namespace kda
