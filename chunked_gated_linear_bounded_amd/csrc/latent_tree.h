// Absorbed latent attention of several drafted tokens a sequence against the paged cache:
//   s_j = scale q . c_j over the committed rows and the drafted rows that the token's bits name,
//   o = sum softmax_j(s_j) c_j[:dc].
// Every head of every drafted token is a row of one problem: R = T H rows against the same keys, 2 (2 dc +
// dr) flops a row and key.  From a few hundred rows on the matrix units bound it, and what feeds them is
// LDS: a wave that takes 16 rows reads a fragment of keys for every MFMA, 64 lanes x 16 bytes in the 8
// cycles of LDS for 16 cycles of matrix unit, on four units.  So a work-group of four waves, one a SIMD
// with all 512 registers, takes up to 64 rows (NQ = 4 column tiles), and
//  - scores: wave w holds the 64 rows' queries whole (NQ D / 32 fragments) and takes the 16 keys of row tile
//    w: S^T = C Q^T, a fragment feeds NQ MFMAs, no sums are exchanged;
//  - values: wave w takes a quarter of the latent's channels: O^T = C^T P^T, a transposed fragment feeds NQ
//    MFMAs; P is handed round through LDS.
// 64 keys are a tile, loaded straight into LDS, the next one into a second buffer meanwhile: 136 MFMAs a
// wave (2,176 cycles) on 45 KiB of LDS reads.
//
// The exponentials are taken against a maximum that may be 2^8 too small, so that the accumulator is
// scaled a few times a row and not every tile: a wave makes P with the maximum it has, says whether a row
// has outgrown it, and only where one has all four waves agree on new maxima and make P again.
//
// A fragment (16 rows x 32 channels) is rows of 64 bytes, because a direct load fills LDS in lane order and
// is fast where four neighbouring lanes read one row: with a row a lane it made 64 accesses to the cache in
// place of 16 and took most of the time.  Row m's four 16-byte pieces are exchanged by m / 4, which puts the
// 16 lanes of a plain read on all banks.  The transposed read of 16 channels takes 8-byte halves; with the
// same half of every piece it would meet its neighbour's banks.  So channel tile o of a column block takes
// half o of the even pieces and half 1 - o of the odd ones, and a lane's pair of channel tiles changes
// places where g is odd.
#pragma once
#include "latent_common.h"

namespace kda {

struct LatentTreeArgs {
    const void *q;             // [B][T][H][dc + dr]
    const void *cache;         // [pages][page][dc + dr]
    const int *table;          // [B][max_pages]
    const int *lengths;        // [B]
    const int *counts;         // [B] (NULL: T)
    const unsigned long long *mask;  // [B][T]
    int B, T, H, pages, page, max_pages, nsplit, rgroups;
    float scale;
    void *out;                 // [B][T][H][dc]
    float *lse;                // [B][T][H]
    float *part, *part_lse;    // nsplit > 1: [B][nsplit][T H][dc]; [B][nsplit][T H] log-sum-exps (log2)
    // 64-key tiles of sequence b, and of each of its parts
    __device__ __forceinline__ int tiles(int b, int &len, int &per) const {
        const long long most = (long long)max_pages * page;
        const int given = lengths[b];
        len = given < 0 ? 0 : (given > most ? (int)most : given);
        const int n = (len + 63) / 64;
        per = (n + nsplit - 1) / nsplit;
        return n;
    }
};

template <bool F32> struct TreeOp;
template <> struct TreeOp<false> : AttnOp<false> {
    static constexpr int NL = 1;  // direct loads a fragment
    // row of the fragment that lane `lane` of load i fills, and the element of the row it starts at
    __device__ __forceinline__ static int load_row(int lane, int) { return lane >> 2; }
    __device__ __forceinline__ static int load_col(int lane, int) { return 8 * ((lane & 3) ^ (lane >> 4)); }
    __device__ __forceinline__ static int slot(int piece, int m) { return 64 * m + 16 * (piece ^ (m >> 2)); }
    __device__ __forceinline__ static V8 get(const lds_u8 *f, int lane) {
        return *reinterpret_cast<const lds_b8 *>(f + slot(lane >> 4, lane & 15));
    }
    __device__ __forceinline__ static void put(lds_u8 *f, int lane, const V8 &x) {
        *reinterpret_cast<lds_b8 *>(f + slot(lane >> 4, lane & 15)) = x;
    }
    __device__ __forceinline__ static V8 get_t(const lds_u8 *f0, const lds_u8 *f1, int o, int lane) {
        const int g = lane >> 4, s = lane & 15, cg = s & 3;
        const int off = slot(cg, 4 * g + (s >> 2)) + 8 * (o ^ (cg & 1));
        const bf16x4 a = ld_tr16<bf16x4>(f0 + off), b = ld_tr16<bf16x4>(f1 + off);
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    static constexpr bool kSwap = true;
    // half `h` of a lane's eight values of P
    __device__ __forceinline__ static void put_half(lds_u8 *f, int lane, int h, const f32x4 &x) {
        bf16x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = (__bf16)x[i];
        *reinterpret_cast<lds_b4 *>(f + 16 * lane + 8 * h) = r;
    }
    // zero in the place of what is not finite; whether anything was not
    __device__ __forceinline__ static bool mend(V8 &x) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool here = !(fabsf((float)x[i]) <= 3.4e38f);
            bad |= here;
            if (here) x[i] = (__bf16)0.f;
        }
        return bad;
    }
};
template <> struct TreeOp<true> : AttnOp<true> {
    static constexpr int NL = 2;
    __device__ __forceinline__ static int load_row(int lane, int i) { return 8 * i + (lane >> 3); }
    __device__ __forceinline__ static int load_col(int lane, int i) { return 4 * ((lane & 7) ^ (load_row(lane, i) >> 1)); }
    __device__ __forceinline__ static int slot(int piece, int m) { return 128 * m + 16 * (piece ^ (m >> 1)); }
    __device__ __forceinline__ static V8 get(const lds_u8 *f, int lane) {
        const int g = lane >> 4, m = lane & 15;
        return V8{*reinterpret_cast<const lds_f4 *>(f + slot(2 * g, m)), *reinterpret_cast<const lds_f4 *>(f + slot(2 * g + 1, m))};
    }
    __device__ __forceinline__ static void put(lds_u8 *f, int lane, const V8 &x) {
        const int g = lane >> 4, m = lane & 15;
        *reinterpret_cast<lds_f4 *>(f + slot(2 * g, m)) = x.a;
        *reinterpret_cast<lds_f4 *>(f + slot(2 * g + 1, m)) = x.b;
    }
    __device__ __forceinline__ static V8 get_t(const lds_u8 *f0, const lds_u8 *f1, int o, int lane) {
        const int g = lane >> 4, m = lane & 15;
        V8 r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int off = slot(2 * (m >> 2) + o, 4 * g + j) + 4 * (m & 3);
            r.a[j] = *reinterpret_cast<const __attribute__((address_space(3))) float *>(f0 + off);
            r.b[j] = *reinterpret_cast<const __attribute__((address_space(3))) float *>(f1 + off);
        }
        return r;
    }
    static constexpr bool kSwap = false;
    __device__ __forceinline__ static void put_half(lds_u8 *f, int lane, int h, const f32x4 &x) {
        *reinterpret_cast<lds_f4 *>(f + 16 * lane + 1024 * h) = x;
    }
    __device__ __forceinline__ static bool mend(V8 &x) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool a = !(fabsf(x.a[i]) <= 3.4028235e38f), b = !(fabsf(x.b[i]) <= 3.4028235e38f);
            bad |= a | b;
            if (a) x.a[i] = 0.f;
            if (b) x.b[i] = 0.f;
        }
        return bad;
    }
};

// Lane l's 16 bytes at `src` + STEP kb to dst + 16 l, past the registers.  In assembly, because behind the
// builtin every LDS read waits for all direct loads, those of the other buffer too; the caller waits with
// wait_vmcnt.  The instruction adds its offset to both addresses.
template <int STEP>
__device__ __forceinline__ void direct_load(const void *src, lds_u8 *dst, int kb) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off offset:%2" ::"v"(src),
                 "s"(__builtin_amdgcn_readfirstlane((int)(unsigned)(size_t)dst - STEP * kb)), "n"(STEP * kb)
                 : "memory", "m0");
}

template <int DC, int DR, bool F32, int NQ>
__global__ __launch_bounds__(256, 1) void latent_tree_kernel(const LatentTreeArgs p) {
    using Op = TreeOp<F32>;
    using E = typename Op::E;
    using V8 = typename Op::V8;
    constexpr int D = DC + DR, NKB = D / 32, NT = DC / 64, FB = Op::FB, NBUF = F32 ? 1 : 2, TILE = 4 * NKB * FB, NL = Op::NL;
    constexpr int ES = (int)sizeof(E), AHEAD = F32 ? 1 : 3;
    typedef __attribute__((address_space(3))) float lds_f;
    typedef __attribute__((address_space(3))) int lds_i;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[NBUF * TILE];
    __shared__ __attribute__((aligned(1024))) unsigned char sp_[2 * NQ * FB];
    __shared__ float smax_[2 * 4 * 16 * NQ];  // by tile parity: waves' maxima of their keys
    __shared__ int sgrown_[2 * 4];
    lds_u8 *sk = lds_base(smem), *sp = lds_base(sp_);
    lds_f *smax = (lds_f *)lds_base(smax_);
    lds_i *sgrown = (lds_i *)lds_base(sgrown_);
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, n = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    // work-groups in eight runs, one an XCD: those on the same keys are neighbours there
    const unsigned all = (unsigned)p.B * p.nsplit * p.rgroups, run = (all + 7) / 8, at_ = (blockIdx.x & 7) * run + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= run || at_ >= all) return;
    const int unit = at_ / p.rgroups, rg = at_ % p.rgroups;
    const int b = unit / p.nsplit, split = unit % p.nsplit, R = p.T * p.H, row0 = rg * 16 * NQ;
    int len, per;
    const int ntile = p.tiles(b, len, per), count = p.counts ? AttnSeqs::clip(p.counts[b], p.T) : p.T;
    const int base = len - count;  // the first drafted row; below 0 where fewer rows than drafted tokens are there
    // rows of tokens past the count see nothing
    const int first = split * per, last = row0 / p.H >= count ? first : min(first + per, ntile);
    const E *cache = reinterpret_cast<const E *>(p.cache);
    const float c = p.scale * kLog2e;

    V8 qf[NQ][NKB];
    unsigned long long bits[NQ];  // the drafted rows that a lane's row sees
    bool dead[NQ];
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        const int row = min(row0 + 16 * x + n, R - 1), node = row / p.H;
        bits[x] = p.mask[(size_t)b * p.T + node];
        dead[x] = node >= count;
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb)
            qf[x][kb] = Op::load(reinterpret_cast<const E *>(p.q) + ((size_t)b * R + row) * D + 32 * kb + 8 * g);
    }
    // as many as fit stay in accumulation registers, where MFMAs take operands from as well
    if constexpr (!F32 && NQ * NKB * 4 > 128) {
#pragma unroll
        for (int x = 0; x < NQ; ++x)
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb)
                if ((x * NKB + kb) * 4 < 256) asm volatile("" : "+a"(qf[x][kb]));
    }
    // rows of a tile: a lane's key(s), past the last the last; pages outside the cache are clipped
    const int *table = p.table + (size_t)b * p.max_pages;
    auto key_of = [&](int tile, int i) { return min(64 * min(tile, last - 1) + perm_row(w, Op::load_row(lane, i)), len - 1); };
    int pg[NL];
    auto fetch = [&](int tile) {
#pragma unroll
        for (int i = 0; i < NL; ++i) pg[i] = table[key_of(tile, i) / p.page];
    };
    const E *from[NL];
    auto find = [&](int tile) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int at = pg[i] < 0 ? 0 : (pg[i] >= p.pages ? p.pages - 1 : pg[i]);
            from[i] = cache + ((long long)at * p.page + key_of(tile, i) % p.page) * D + Op::load_col(lane, i);
        }
    };
    auto load = [&](lds_u8 *to, int kb) {
#pragma unroll
        for (int i = 0; i < NL; ++i) direct_load<32 * ES>(from[i], to + (w * NKB + kb) * FB + 1024 * i, kb);
    };
    auto load_all = [&](lds_u8 *to) {
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) load(to, kb);
    };
    f32x4 O[NT][NQ];
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int x = 0; x < NQ; ++x) O[t][x] = zero;
    float m[NQ], l[NQ];  // the rows' maximum (log2 units); the wave's keys' part of their sum
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        m[x] = -INFINITY;
        l[x] = 0.f;
    }
    if (first < last) {
        fetch(first);
        find(first);
        load_all(sk);
        fetch(first + 1);
    }
    for (int tile = first; tile < last; ++tile) {
        const int par = (tile - first) & 1;
        lds_u8 *here = sk + (NBUF == 2 ? par * TILE : 0);
        wait_vmcnt<0>();
        barrier_lds();  // the tile is there, and the other buffer has been read
        find(tile + 1);  // behind the last tile its last row again
        fetch(tile + 2);
        f32x4 s[NQ];
#pragma unroll
        for (int x = 0; x < NQ; ++x) s[x] = zero;
        lds_u8 *mine = here + w * NKB * FB;
        const bool edge = 64 * tile + 64 > base;  // drafted rows, or rows past the last
        unsigned badrows = 0;
        if (edge) {
            // a drafted row that is not finite reaches the tokens that see it, as NaN, and no others: the
            // products take it as zeros
            bool bad = false;
#pragma unroll 1
            for (int kb = 0; kb < NKB; ++kb) {
                V8 x = Op::get(mine + kb * FB, lane);
                if (Op::mend(x)) {
                    Op::put(mine + kb * FB, lane, x);
                    bad = true;
                }
            }
            const unsigned long long k = __builtin_amdgcn_ballot_w64(bad);
            badrows = (unsigned)(k | k >> 16 | k >> 32 | k >> 48) & 0xffff;
        }
        // fragments AHEAD steps before their MFMAs, in this order: left alone, the scheduler reads each one
        // right before its use, and the wave waits; a piece of the next tile is asked for in each step
        V8 ring[AHEAD + 1];
#pragma unroll
        for (int kb = 0; kb < AHEAD; ++kb) ring[kb] = Op::get(mine + kb * FB, lane);
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
            if (kb + AHEAD < NKB) ring[(kb + AHEAD) % (AHEAD + 1)] = Op::get(mine + (kb + AHEAD) * FB, lane);
            if constexpr (NBUF == 2) load(sk + (par ^ 1) * TILE, kb);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int x = 0; x < NQ; ++x) s[x] = Op::mma(ring[kb % (AHEAD + 1)], qf[x][kb], s[x]);
        }
        if (edge) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = 64 * tile + perm_row(w, 4 * g + i), j = key - base;
                const bool bad = badrows >> (4 * g + i) & 1;
#pragma unroll
                for (int x = 0; x < NQ; ++x) {
                    const bool see = key < len && (j < 0 || (bits[x] >> (j & 63) & 1) != 0);
                    s[x][i] = !see ? -INFINITY : bad ? NAN : s[x][i];
                }
            }
        }
        float mx[NQ];
        bool grown = false;
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            mx[x] = col_max(max4(s[x])) * c;
            grown |= mx[x] > m[x] + 8.f;  // any finite score at first: m is -inf
        }
        f32x4 P[NQ];
        auto make = [&]() {
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                const float mm = m[x] == -INFINITY ? 0.f : m[x];
#pragma unroll
                for (int i = 0; i < 4; ++i) P[x][i] = ex2(fmaf(s[x][i], c, -mm));
                Op::put_half(sp + ((w >> 1) * NQ + x) * FB, lane, w & 1, P[x]);
            }
        };
        make();
        const bool any = __builtin_amdgcn_ballot_w64(grown) != 0;
        if (lane == 0) sgrown[4 * par + w] = any;
        if (g == 0) {
#pragma unroll
            for (int x = 0; x < NQ; ++x) smax[((4 * par + w) * NQ + x) * 16 + n] = mx[x];
        }
        barrier_lds();  // P is there
        if (sgrown[4 * par] | sgrown[4 * par + 1] | sgrown[4 * par + 2] | sgrown[4 * par + 3]) {
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                float now = m[x];
#pragma unroll
                for (int k = 0; k < 4; ++k) now = fmaxf(now, smax[((4 * par + k) * NQ + x) * 16 + n]);
                const float alpha = now == -INFINITY ? 1.f : ex2(m[x] - now);
                m[x] = now;
                l[x] *= alpha;
#pragma unroll
                for (int t = 0; t < NT; ++t) O[t][x] *= alpha;
            }
            make();
            barrier_lds();
        }
#pragma unroll
        for (int x = 0; x < NQ; ++x) l[x] += (P[x][0] + P[x][1]) + (P[x][2] + P[x][3]);
        auto value = [&](int k) {  // step k: keys 32 (k / NT) .., channel tile k % NT
            const int tt = w * NT + k % NT;
            const lds_u8 *f = here + (k / NT * 2 * NKB + (tt >> 1)) * FB;
            return Op::get_t(f, f + NKB * FB, tt & 1, lane);
        };
        V8 pf[NQ];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) ring[k] = value(k);
#pragma unroll
        for (int k = 0; k < 2 * NT; ++k) {
            if (k % NT == 0) {
#pragma unroll
                for (int x = 0; x < NQ; ++x) pf[x] = Op::get_lane(sp + (k / NT * NQ + x) * FB, lane);
            }
            if (k + AHEAD < 2 * NT) ring[(k + AHEAD) % (AHEAD + 1)] = value(k + AHEAD);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int x = 0; x < NQ; ++x) O[k % NT][x] = Op::mma(ring[k % (AHEAD + 1)], pf[x], O[k % NT][x]);
        }
        if constexpr (NBUF == 1) {
            barrier_lds();  // the tile has been read
            if (tile + 1 < last) load_all(sk);
        }
    }
    // the sum over the waves' keys; the loads behind the last tile end before the wave does
    wait_vmcnt<0>();
    barrier_lds();
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        const float sum = col_sum(l[x]);
        if (g == 0) smax[(w * NQ + x) * 16 + n] = sum;
    }
    barrier_lds();
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) sum += smax[(k * NQ + x) * 16 + n];
        const int row = row0 + 16 * x + n;
        if (row >= R) continue;
        // nothing seen: zeros, -inf; a sum that is NaN stays one
        const bool none = dead[x] || sum == 0.f;
        const float inv = 1.f / sum, lse2 = none ? -INFINITY : m[x] + lg2(sum);
        if (p.nsplit == 1) {
            E *o = reinterpret_cast<E *>(p.out) + ((size_t)b * R + row) * DC + w * (DC / 4) + 8 * g;
#pragma unroll
            for (int t = 0; t < NT; t += 2) {
                const bool swap = Op::kSwap && (g & 1);
                f32x4 u = swap ? O[t + 1][x] : O[t][x], v = swap ? O[t][x] : O[t + 1][x];
                u = none ? zero : u * inv;
                v = none ? zero : v * inv;
                Op::store8(o + 16 * t, u, v);
            }
            if (g == 0 && w == 0) p.lse[(size_t)b * R + row] = lse2 * kLn2;
        } else {
            const size_t at = ((size_t)b * p.nsplit + split) * R + row;
            if (g == 0 && w == 0) p.part_lse[at] = lse2;
            if (first >= last && !dead[x]) continue;  // nothing here, and the join reads the parts that have keys
            float *o = p.part + at * DC + w * (DC / 4) + 8 * g;
#pragma unroll
            for (int t = 0; t < NT; t += 2) {
                const bool swap = Op::kSwap && (g & 1);
                f32x4 u = swap ? O[t + 1][x] : O[t][x], v = swap ? O[t][x] : O[t + 1][x];
                u = none ? zero : u * inv;
                v = none ? zero : v * inv;
                *reinterpret_cast<f32x4 *>(o + 16 * t) = u;
                *reinterpret_cast<f32x4 *>(o + 16 * t + 4) = v;
            }
        }
    }
}

// Joins the parts of a row: weights 2^(lse_i - max), 4 values a thread.  Every part that has keys counts, so
// that one whose result is not finite shows.
template <int DC, typename E>
__global__ __launch_bounds__(256) void latent_tree_join_kernel(const LatentTreeArgs p) {
    constexpr int TPR = DC / 4;  // threads a row
    const int R = p.T * p.H;
    const long long at = (long long)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
    if (at >= (long long)p.B * R) return;
    const int b = (int)(at / R), row = (int)(at % R), d = 4 * (threadIdx.x % TPR);
    const float *e = p.part_lse + (size_t)b * p.nsplit * R + row;
    const float *o_ = p.part + ((size_t)b * p.nsplit * R + row) * DC + d;
    int len, per;
    const int ntile = p.tiles(b, len, per), parts = per > 0 ? (ntile + per - 1) / per : 0;
    float m = -INFINITY, sum = 0.f;
    for (int i = 0; i < parts; ++i) m = fmaxf(m, e[(size_t)i * R]);
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < parts; ++i) {
        const float x = e[(size_t)i * R], wgt = x == -INFINITY ? 0.f : ex2(x - m);
        sum += wgt;
        o += wgt * *reinterpret_cast<const f32x4 *>(o_ + (size_t)i * R * DC);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    st_tile(reinterpret_cast<E *>(p.out) + at * DC + d, 0, o * inv);
    if (d == 0) p.lse[at] = sum == 0.f ? -INFINITY : (m + lg2(sum)) * kLn2;
}

}  // namespace kda
