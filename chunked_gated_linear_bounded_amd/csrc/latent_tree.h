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
// 24 sequences x 8 tokens x 128 heads on up to 9000 rows: 409 to 444 us, 0.8 to 0.9 PFLOP/s, matrix units 43 % busy,
// vector unit 25 %, LDS 41 % and 7 in bank conflicts.  With one wave a SIMD nothing covers a tile's softmax, its
// barrier and the first reads behind it; a third buffer, for the next scores to run beside them, does not fit the
// LDS.
//
// The exponentials are taken against a maximum that may be 2^8 too small, so that the accumulator is
// scaled a few times a row and not every tile: a wave makes P with the maximum it has, says whether a row
// has outgrown it, and only where one has all four waves agree on new maxima and make P again.
//
// With bf16 inputs P is rounded to bf16 as the products' operand, as in the one-token step: half the matrix work and
// half of what is handed round in LDS, against out's error of 1.8e-3 (histories of thousands of rows) to 2.1e-3 (of
// hundreds) of its norm, where its own rounding to bf16 alone is 1.7e-3.  Sums of P, maxima and the accumulator are
// float32, and the sum is that of the exponentials before they are rounded.
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
    int B, T, H, pages, page, max_pages, rgroups;
    float scale;
    void *out;                 // [B][T][H][dc]
    float *lse;                // [B][T][H]
    // groups > 0: that many work-groups share the tiles of all units evenly, and what each has of its first
    // and last unit goes to part, [2 groups][rows of a unit][dc], and part_lse (log2); from: [B + 1], the
    // first tile of sequence b's units, and [B + 1 ..] the tiles of a work-group.  0: a work-group a unit.
    int groups;
    float *part, *part_lse;
    int *from;
    __device__ __forceinline__ int length(int b) const {
        const long long most = (long long)max_pages * page;
        const int given = lengths[b];
        return given < 0 ? 0 : (given > most ? (int)most : given);
    }
    // 64-key tiles of one of sequence b's units; one at least, so that somebody writes its rows
    __device__ __forceinline__ int tiles(int b) const { return max(1, (length(b) + 63) / 64); }
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

// Lane l's 16 bytes at `src` + STEP kb to the LDS address `to` (the same in all lanes) + FB kb + off + 16 l,
// past the registers.  In assembly, because behind the builtin every LDS read waits for all direct loads,
// those of the other buffer too; the caller waits with wait_vmcnt.  The instruction adds its offset to both
// addresses.
template <int STEP, int FB>
__device__ __forceinline__ void direct_load(const void *src, int to, int kb, int off) {
    asm volatile("s_add_u32 m0, %1, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off offset:%2" ::"v"(src), "s"(to), "n"(STEP * kb),
                 "n"(FB * kb + off - STEP * kb)
                 : "memory", "m0", "scc");
}
// A barrier and nothing else: LDS reads in flight stay in flight.
__device__ __forceinline__ void barrier_only() {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

template <int DC, int DR, bool F32, int NQ>
__global__ __launch_bounds__(256, 1) void latent_tree_kernel(const LatentTreeArgs p) {
    using Op = TreeOp<F32>;
    using E = typename Op::E;
    using V8 = typename Op::V8;
    constexpr int D = DC + DR, NKB = D / 32, NT = DC / 64, FB = Op::FB, NBUF = F32 ? 1 : 2, TILE = 4 * NKB * FB, NL = Op::NL;
    constexpr int ES = (int)sizeof(E), AHEAD = F32 ? 1 : 3, RING = AHEAD + 1, NV = 2 * NT;  // NV: steps of the value products
    static_assert(NBUF == 1 || NV % RING == 0, "the ring's places carry on from the values into the next scores");
    typedef __attribute__((address_space(3))) float lds_f;
    typedef __attribute__((address_space(3))) int lds_i;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[NBUF * TILE];
    __shared__ __attribute__((aligned(1024))) unsigned char sp_[2 * NQ * FB];
    __shared__ float smax_[4 * 16 * NQ];
    __shared__ int sgrown_[2 * 4];  // by tile parity
    lds_u8 *sk = lds_base(smem), *sp = lds_base(sp_);
    lds_f *smax = (lds_f *)lds_base(smax_);
    lds_i *sgrown = (lds_i *)lds_base(sgrown_);
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int R = p.T * p.H;
    const E *cache = reinterpret_cast<const E *>(p.cache);
    const float c = p.scale * kLog2e;

    // what this work-group does: `left` tiles from tile t0 of unit (b, rg) on.  Work-groups in eight runs, one
    // an XCD: those on the same keys are neighbours there.
    const unsigned all = p.groups > 0 ? p.groups : (unsigned)p.B * p.rgroups, run = (all + 7) / 8;
    const unsigned me = (blockIdx.x & 7) * run + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= run || me >= all) return;
    int b, rg, t0 = 0, left;
    if (p.groups > 0) {
        // tiles in front of each sequence (fewer than 1024 where work is shared): 256 sequences a step
        lds_i *si = (lds_i *)lds_base(smem);
        int total = 0;
        for (int b0 = 0; b0 < p.B; b0 += 256) {
            int x = b0 + tid < p.B ? p.tiles(b0 + tid) * p.rgroups : 0;
            const int mine = x;
#pragma unroll
            for (int k = 1; k < 64; k <<= 1) {
                const int y = __shfl_up(x, k);
                x += lane >= k ? y : 0;
            }
            if (lane == 63) si[2048 + w] = x;
            __syncthreads();
            int before = total;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k < w) before += si[2048 + k];
                total += si[2048 + k];
            }
            if (b0 + tid < p.B) si[b0 + tid] = before + x - mine;
            __syncthreads();
        }
        const int each = (total + p.groups - 1) / p.groups;
        const long long at = (long long)me * each;
        if (me == 0) {
            for (int i = tid; i < p.B; i += 256) p.from[i] = si[i];
            if (tid == 0) {
                p.from[p.B] = total;
                p.from[p.B + 1] = each;
            }
        }
        if (at >= total) return;
        left = min(each, total - (int)at);
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (si[mid] <= (int)at) lo = mid;
            else hi = mid - 1;
        }
        b = lo;
        const int nt = p.tiles(b), in = (int)at - si[b];
        rg = in / nt;
        t0 = in % nt;
    } else {
        b = me / p.rgroups;
        rg = me % p.rgroups;
        left = p.tiles(b);
    }

    while (left > 0) {
        const int nt = p.tiles(b), t1 = min(nt, t0 + left), row0 = rg * 16 * NQ;
        const int len = p.length(b), count = p.counts ? AttnSeqs::clip(p.counts[b], p.T) : p.T;
        const int base = len - count;  // the first drafted row; below 0 where fewer rows than drafted tokens are there
        // rows of tokens past the count see nothing
        const int last = len == 0 || row0 / p.H >= count ? t0 : t1;
        // rows of a tile: a lane's key(s), past the last the last; pages outside the cache are clipped
        const int *table = p.table + (size_t)b * p.max_pages;
        int pg[NL], in[NL];  // page and row in it of the tile after next
        auto fetch = [&](int tile) {
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int key = min(64 * min(tile, last - 1) + perm_row(w, Op::load_row(lane, i)), len - 1);
                pg[i] = table[key / p.page];
                in[i] = key % p.page;
            }
        };
        const E *from[NL];
        auto find = [&]() {
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int at = pg[i] < 0 ? 0 : (pg[i] >= p.pages ? p.pages - 1 : pg[i]);
                from[i] = cache + ((long long)at * p.page + in[i]) * D + Op::load_col(lane, i);
            }
        };
        auto load = [&](int to, int kb) {  // to: the wave's fragments in LDS
#pragma unroll
            for (int i = 0; i < NL; ++i) direct_load<32 * ES, FB>(from[i], to, kb, 1024 * i);
        };
        const int mine0 = __builtin_amdgcn_readfirstlane((int)(unsigned)(size_t)(sk + w * NKB * FB));
        f32x4 O[NT][NQ];
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int x = 0; x < NQ; ++x) O[t][x] = zero;
        // of a row: minus the maximum that its exponentials are taken against (0 while there is none), the score
        // that outgrows it, and the wave's keys' part of the sum.  The maximum is taken off before the scale: scaled
        // first, its own rounding would be an exponent beyond 2^127 from scores of some 10^9 on.
        float nm[NQ], most[NQ], l[NQ];
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            nm[x] = 0.f;
            most[x] = -INFINITY;
            l[x] = 0.f;
        }
        V8 ring[RING];
        barrier_lds();  // what was in LDS has been read
        if (t0 < last) {
            fetch(t0);
            find();
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) load(mine0, kb);
            fetch(t0 + 1);
        }
        V8 qf[NQ][NKB];
        {
            const int ln = lane_here(lane);
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                const int row = min(row0 + 16 * x + (ln & 15), R - 1);
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb)
                    qf[x][kb] = Op::load(reinterpret_cast<const E *>(p.q) + ((size_t)b * R + row) * D + 32 * kb + 8 * (ln >> 4));
            }
        }
        // as many as fit stay in accumulation registers, where MFMAs take operands from as well; and all are
        // there before the loop, in which a wait for them would be one for the direct loads
        if constexpr (!F32) {
#pragma unroll
            for (int x = 0; x < NQ; ++x)
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb) {
                    if (NQ * NKB * 4 > 128 && (x * NKB + kb) * 4 < 256) asm volatile("" : "+a"(qf[x][kb]));
                    else asm volatile("" : "+v"(qf[x][kb]));
                }
        }
        if (NBUF == 2 && t0 < last) {
            wait_vmcnt<0>();
#pragma unroll
            for (int kb = 0; kb < AHEAD; ++kb) ring[kb] = Op::get(sk + (w * NKB + kb) * FB, lane);
        }
        for (int tile = t0; tile < last; ++tile) {
            const int par = (tile - t0) & 1;
            lds_u8 *here = sk + (NBUF == 2 ? par * TILE : 0), *mine = here + w * NKB * FB;
            // a wave's row tile is its own load; the others' are there behind the barrier in front of the values
            if constexpr (NBUF == 1) wait_vmcnt<0>();
            find();  // behind the last tile its last row again
            fetch(tile + 2);
            f32x4 s[NQ];
#pragma unroll
            for (int x = 0; x < NQ; ++x) s[x] = zero;
            const bool edge = 64 * tile + 64 > base;  // drafted rows, or rows past the last
            unsigned badrows = 0;
            if (edge) {
                // a drafted row that is not finite reaches the tokens that see it, as NaN, and no others: the
                // products take it as zeros
                bool bad = false;
                const int ln = lane_here(lane);
#pragma unroll 1
                for (int kb = 0; kb < NKB; ++kb) {
                    V8 x = Op::get(mine + kb * FB, ln);
                    if (Op::mend(x)) {
                        Op::put(mine + kb * FB, ln, x);
                        bad = true;
                    }
                }
                const unsigned long long k = __builtin_amdgcn_ballot_w64(bad);
                badrows = (unsigned)(k | k >> 16 | k >> 32 | k >> 48) & 0xffff;
            }
            if (NBUF == 1 || edge) {
#pragma unroll
                for (int kb = 0; kb < AHEAD; ++kb) ring[kb] = Op::get(mine + kb * FB, lane);
            }
            // fragments AHEAD steps before their MFMAs, in this order: left alone, the scheduler reads each one
            // right before its use, and the wave waits; a piece of the next tile is asked for in each step, once
            // all waves have read the buffer it goes to
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
                if (kb + AHEAD < NKB) ring[(kb + AHEAD) % RING] = Op::get(mine + (kb + AHEAD) * FB, lane);
                if constexpr (NBUF == 2) {
                    if (kb == 1) barrier_only();
                    if (kb > 0) load(mine0 + (par ^ 1) * TILE, kb - 1);
                    if (kb == NKB - 1) load(mine0 + (par ^ 1) * TILE, kb);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int x = 0; x < NQ; ++x) s[x] = Op::mma(ring[kb % RING], qf[x][kb], s[x]);
            }
            if (edge) {
                const int ln = lane_here(lane);
#pragma unroll
                for (int x = 0; x < NQ; ++x) {
                    const int node = min(row0 + 16 * x + (ln & 15), R - 1) / p.H;
                    const unsigned long long bits = p.mask[(size_t)b * p.T + node];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 4 * (ln >> 4) + i, key = 64 * tile + perm_row(w, r), j = key - base;
                        const bool see = key < len && (j < 0 || (bits >> (j & 63) & 1) != 0), bad = badrows >> r & 1;
                        s[x][i] = !see ? -INFINITY : bad ? NAN : s[x][i];
                    }
                }
            }
            // P against the maxima there are, and whether a row has outgrown its own by 2^8 (at first: has any)
            auto value = [&](int k) {  // step k: keys 32 (k / NT) .., channel tile k % NT
                const int tt = w * NT + k % NT;
                const lds_u8 *f = here + (k / NT * 2 * NKB + (tt >> 1)) * FB;
                return Op::get_t(f, f + NKB * FB, tt & 1, lane);
            };
            auto make = [&](float (&sum)[NQ]) {
#pragma unroll
                for (int x = 0; x < NQ; ++x) {
                    f32x4 P;
#pragma unroll
                    for (int i = 0; i < 4; ++i) P[i] = ex2((s[x][i] + nm[x]) * c);
                    Op::put_half(sp + ((w >> 1) * NQ + x) * FB, lane, w & 1, P);
                    sum[x] += (P[0] + P[1]) + (P[2] + P[3]);
                }
            };
            bool grown = false;
#pragma unroll
            for (int x = 0; x < NQ; ++x) grown |= max4(s[x]) > most[x];
            float sum[NQ];
#pragma unroll
            for (int x = 0; x < NQ; ++x) sum[x] = l[x];
            make(sum);
            const bool any = __builtin_amdgcn_ballot_w64(grown) != 0;
            if (lane == 0) sgrown[4 * par + w] = any;
            barrier_lds();  // P and the whole tile are there
            if (__builtin_amdgcn_readfirstlane(sgrown[4 * par] | sgrown[4 * par + 1] | sgrown[4 * par + 2] | sgrown[4 * par + 3])) {
                // new maxima, of all four waves' keys, and P again
                const int ln = lane_here(lane);
#pragma unroll
                for (int x = 0; x < NQ; ++x) {
                    const float a = col_max(max4(s[x]));
                    if (ln < 16) smax[(w * NQ + x) * 16 + ln] = a;
                }
                barrier_lds();
#pragma unroll
                for (int x = 0; x < NQ; ++x) {
                    const float was = most[x] == -INFINITY ? -INFINITY : -nm[x];
                    float now = was;
#pragma unroll
                    for (int k = 0; k < 4; ++k) now = fmaxf(now, smax[(k * NQ + x) * 16 + (ln & 15)]);
                    const float alpha = now == -INFINITY ? 1.f : ex2((was - now) * c);
                    nm[x] = now == -INFINITY ? 0.f : -now;
                    most[x] = now == -INFINITY ? now : now + 8.f / c;
                    sum[x] = l[x] * alpha;
#pragma unroll
                    for (int t = 0; t < NT; ++t) O[t][x] *= alpha;
                }
                make(sum);
                barrier_lds();
            }
            V8 pf[NQ];
#pragma unroll
            for (int x = 0; x < NQ; ++x) pf[x] = Op::get_lane(sp + x * FB, lane);
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) ring[k] = value(k);
#pragma unroll
            for (int x = 0; x < NQ; ++x) l[x] = sum[x];
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (k == NT) {
#pragma unroll
                    for (int x = 0; x < NQ; ++x) pf[x] = Op::get_lane(sp + (NQ + x) * FB, lane);
                }
                if (k + AHEAD < NV) {
                    ring[(k + AHEAD) % RING] = value(k + AHEAD);
                } else if constexpr (NBUF == 2) {  // into the next tile's scores
                    if (k + AHEAD == NV) wait_vmcnt<0>();
                    ring[(k + AHEAD) % RING] = Op::get(sk + (par ^ 1) * TILE + (w * NKB + k + AHEAD - NV) * FB, lane);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int x = 0; x < NQ; ++x) O[k % NT][x] = Op::mma(ring[k % RING], pf[x], O[k % NT][x]);
            }
            if constexpr (NBUF == 1) {
                barrier_lds();  // the tile has been read
                if (tile + 1 < last) {
#pragma unroll
                    for (int kb = 0; kb < NKB; ++kb) load(mine0, kb);
                }
            }
        }
        // the sum over the waves' keys; the loads behind the last tile end before the wave does
        wait_vmcnt<0>();
        barrier_lds();
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            const float sum = col_sum(l[x]);
            if (lane < 16) smax[(w * NQ + x) * 16 + lane] = sum;
        }
        barrier_lds();
        const bool whole = t0 == 0 && t1 == nt;
        const int ln = lane_here(lane), n2 = ln & 15, g2 = ln >> 4;
        const size_t slot = 2 * (size_t)me + (t0 == 0 ? 1 : 0);
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) sum += smax[(k * NQ + x) * 16 + n2];
            const int row = row0 + 16 * x + n2;
            if (row >= R) continue;
            // nothing seen: zeros, -inf; a sum that is NaN stays one
            const bool none = row / p.H >= count || sum == 0.f;
            const float inv = 1.f / sum, lse2 = none ? -INFINITY : fmaf(-nm[x], c, lg2(sum));
            const size_t at = (size_t)b * R + row, in_part = slot * (16 * NQ) + 16 * x + n2;
            if (g2 == 0 && w == 0) {
                if (whole) p.lse[at] = lse2 * kLn2;
                else p.part_lse[in_part] = lse2;
            }
            const int d = w * (DC / 4) + 8 * g2;
#pragma unroll
            for (int t = 0; t < NT; t += 2) {
                const bool swap = Op::kSwap && (g2 & 1);
                f32x4 u = swap ? O[t + 1][x] : O[t][x], v = swap ? O[t][x] : O[t + 1][x];
                u = none ? zero : u * inv;
                v = none ? zero : v * inv;
                if (whole) {
                    Op::store8(reinterpret_cast<E *>(p.out) + at * DC + d + 16 * t, u, v);
                } else {
                    float *o = p.part + in_part * DC + d + 16 * t;
                    *reinterpret_cast<f32x4 *>(o) = u;
                    *reinterpret_cast<f32x4 *>(o + 4) = v;
                }
            }
        }
        left -= t1 - t0;
        t0 = 0;
        if (++rg == p.rgroups) {
            rg = 0;
            ++b;
        }
    }
}

// Joins the pieces of the units that more than one work-group had: weights 2^(lse_i - max).  Work-group x of
// the first grid dimension takes the unit that work-group x of the kernel above began and did not end; a
// wave takes 256 channels of one row, lane i the weight of piece i, and four pieces' values are on their way
// at a time.  It moves bytes: 24 x 8 x 128 heads 23 us, 67 MB read and 17 written.
template <int DC, int NQ, typename E>
__global__ __launch_bounds__(256) void latent_tree_join_kernel(const LatentTreeArgs p) {
    constexpr int WPR = DC / 256, ROWS = 4 / WPR;  // waves a row; rows a work-group
    const int total = p.from[p.B], each = p.from[p.B + 1], me = blockIdx.x, R = p.T * p.H;
    const long long end = (long long)(me + 1) * each;
    if (end >= total) return;
    int lo = 0, hi = p.B - 1;  // the sequence that has tile end - 1
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.from[mid] < end) lo = mid;
        else hi = mid - 1;
    }
    const int b = lo, nt = p.tiles(b), rg = ((int)end - 1 - p.from[b]) / nt, begin = p.from[b] + rg * nt;
    // it ended there, or this work-group did not begin it
    if (begin + nt == end || begin < (long long)me * each) return;
    const int parts = (begin + nt - 1) / each - me + 1;
    auto slot = [&](int i) { return (size_t)(i == 0 ? 2 * me + 1 : 2 * (me + i)) * (16 * NQ); };
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = ROWS * blockIdx.y + w / WPR, row = rg * 16 * NQ + r, d = 256 * (w % WPR) + 4 * lane;
    if (row >= R) return;
    float m = -INFINITY, sum = 0.f;
    for (int i = lane; i < parts; i += 64) m = fmaxf(m, p.part_lse[slot(i) + r]);
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor(m, k));
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    for (int i0 = 0; i0 < parts; i0 += 64) {
        const float x = i0 + lane < parts ? p.part_lse[slot(i0 + lane) + r] : -INFINITY;
        const float mine = x == -INFINITY ? 0.f : ex2(x - m);  // one that is NaN stays one
        const int here = min(64, parts - i0);
        sum += mine;
        for (int i = 0; i < here; i += 4) {
            f32x4 y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = *reinterpret_cast<const f32x4 *>(p.part + (slot(i0 + min(i + k, here - 1)) + r) * DC + d);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k < here) o += __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, mine), i + k)) * y[k];
        }
    }
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) sum += __shfl_xor(sum, k);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const size_t at = (size_t)b * R + row;
    st_tile(reinterpret_cast<E *>(p.out) + at * DC + d, 0, o * inv);
    if (d == 0) p.lse[at] = sum == 0.f ? -INFINITY : (m + lg2(sum)) * kLn2;
}

}  // namespace kda
