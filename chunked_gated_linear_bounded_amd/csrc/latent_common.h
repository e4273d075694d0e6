// Building blocks of latent attention: attention whose keys and values come from one latent vector a
// token.  Expanded form: per head a key part k and a value v made from the latent, and a rotary key
// part k_rope that all heads share,
//   s_ij = scale (q_i[:dn] . k_j + q_i[dn:] . k_rope_j),  p = softmax over the visible j,  o_i = sum p_ij v_j;
// absorbed form: the query multiplied into the latent's space, one row c_j of the cache a token,
//   s_j = scale q . c_j,  o = sum p_j c_j[:dc].
//
// Everything is computed transposed: S^T = K Q^T puts keys on the accumulator's rows and queries on
// its columns, so a lane's column is one query, the softmax reduces over a lane's own rows and two
// lane exchanges, and the rows' scaling factors are lane scalars; and two key tiles of P^T are, as
// they lie, the B operand of O^T = V^T P^T.  The permuted row index and the transposed LDS read are
// those of gdr_common.h.
//
// A fragment in LDS (16 rows x 32 columns of 16 bits, 1 KiB) is two planes of 64 8-byte slots: the
// first and the last four columns of each lane's eight.  The transposed read takes 8 bytes from each
// of 64 rows and column groups; from a plane they are 512 bytes one after the other, where out of
// 16-byte slots they would use every second pair of banks (60 % of the LDS cycles were conflicts).
// Lane (g, m) of column block kb has slot 16 g + (m ^ 8 (g / 2) ^ 2 (kb % 4)): all 32 lanes of a half
// wave fall on different banks in the plain read, in the transposed one, and when rows are stored.
//
// bf16 inputs use 16x16x32 bf16 MFMAs, P and dS rounded to bf16 (dS of few keys to two pieces);
// float32 inputs use float32 MFMAs (eight 16x16x4 steps).  Softmax statistics and all sums are float32.
#pragma once
#include "gdr_common.h"

namespace kda {

struct f32x8s {
    f32x4 a, b;
};

template <bool F32> struct AttnOp;
template <> struct AttnOp<false> {
    using E = __bf16;
    using V8 = bf16x8;
    static constexpr int FB = 1024;  // bytes of a fragment
    __device__ __forceinline__ static f32x4 mma(const V8 &a, const V8 &b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    __device__ __forceinline__ static V8 load(const E *p) { return *reinterpret_cast<const V8 *>(p); }
    __device__ __forceinline__ static V8 zero() { return V8{}; }
    __device__ __forceinline__ static V8 pair(const f32x4 &x, const f32x4 &y) {
        V8 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) { r[i] = (__bf16)x[i]; r[4 + i] = (__bf16)y[i]; }
        return r;
    }
    // what pair(x, y) = r left of x and y
    __device__ __forceinline__ static V8 rest(const f32x4 &x, const f32x4 &y, const V8 &r) {
        V8 l;
#pragma unroll
        for (int i = 0; i < 4; ++i) { l[i] = (__bf16)(x[i] - (float)r[i]); l[4 + i] = (__bf16)(y[i] - (float)r[4 + i]); }
        return l;
    }
    typedef __attribute__((address_space(3))) bf16x4 lds_b4;
    typedef __attribute__((address_space(3))) bf16x8 lds_b8;
    __device__ __forceinline__ static int slot(int kb, int g, int m) { return 8 * (16 * g + (m ^ (8 * (g >> 1)) ^ (2 * (kb & 3)))); }
    // f: the fragment; kb: its column block
    __device__ __forceinline__ static void put(lds_u8 *f, int kb, int g, int m, const V8 &x) {
        lds_u8 *p = f + slot(kb, g, m);
        *reinterpret_cast<lds_b4 *>(p) = __builtin_shufflevector(x, x, 0, 1, 2, 3);
        *reinterpret_cast<lds_b4 *>(p + 512) = __builtin_shufflevector(x, x, 4, 5, 6, 7);
    }
    __device__ __forceinline__ static V8 get(const lds_u8 *f, int kb, int lane) {
        const lds_u8 *p = f + slot(kb, lane >> 4, lane & 15);
        const bf16x4 a = *reinterpret_cast<const lds_b4 *>(p), b = *reinterpret_cast<const lds_b4 *>(p + 512);
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    // an operand handed to the same lane of another wave
    __device__ __forceinline__ static void put_lane(lds_u8 *f, int lane, const V8 &x) { *reinterpret_cast<lds_b8 *>(f + 16 * lane) = x; }
    __device__ __forceinline__ static V8 get_lane(const lds_u8 *f, int lane) { return *reinterpret_cast<const lds_b8 *>(f + 16 * lane); }
    // transposed: rows = columns perm_row(tile, .), k = rows of the fragments f0 (row tile 2 kb), f1 (2 kb
    // + 1) of column block tile / 2
    __device__ __forceinline__ static V8 get_t(const lds_u8 *f0, const lds_u8 *f1, int tile, int lane) {
        const int g = lane >> 4, s = lane & 15;
        const int off = slot(tile >> 1, s & 3, 4 * g + (s >> 2)) + 512 * (tile & 1);
        const bf16x4 a = ld_tr16<bf16x4>(f0 + off), b = ld_tr16<bf16x4>(f1 + off);
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    __device__ __forceinline__ static void store8(E *p, const f32x4 &x, const f32x4 &y) {
        *reinterpret_cast<V8 *>(p) = pair(x, y);
    }
};
template <> struct AttnOp<true> {
    using E = float;
    using V8 = f32x8s;
    typedef __attribute__((address_space(3))) f32x4 lds_f4;
    static constexpr int FB = 2048;
    __device__ __forceinline__ static f32x4 mma(const V8 &a, const V8 &b, f32x4 c) {
#pragma unroll
        for (int j = 0; j < 4; ++j) c = mma4(a.a[j], b.a[j], c);
#pragma unroll
        for (int j = 0; j < 4; ++j) c = mma4(a.b[j], b.b[j], c);
        return c;
    }
    __device__ __forceinline__ static V8 load(const E *p) {
        return V8{*reinterpret_cast<const f32x4 *>(p), *reinterpret_cast<const f32x4 *>(p + 4)};
    }
    __device__ __forceinline__ static V8 zero() { return V8{f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}}; }
    __device__ __forceinline__ static V8 pair(const f32x4 &x, const f32x4 &y) { return V8{x, y}; }
    __device__ __forceinline__ static void put(lds_u8 *f, int, int g, int m, const V8 &x) {
        lds_f4 *p = reinterpret_cast<lds_f4 *>(f + 2 * frag_slot(g, m));
        p[0] = x.a;
        p[1] = x.b;
    }
    __device__ __forceinline__ static V8 get(const lds_u8 *f, int, int lane) {
        const lds_f4 *p = reinterpret_cast<const lds_f4 *>(f + 2 * frag_slot(lane >> 4, lane & 15));
        return V8{p[0], p[1]};
    }
    __device__ __forceinline__ static void put_lane(lds_u8 *f, int lane, const V8 &x) {
        *reinterpret_cast<lds_f4 *>(f + 16 * lane) = x.a;
        *reinterpret_cast<lds_f4 *>(f + 1024 + 16 * lane) = x.b;
    }
    __device__ __forceinline__ static V8 get_lane(const lds_u8 *f, int lane) {
        return V8{*reinterpret_cast<const lds_f4 *>(f + 16 * lane), *reinterpret_cast<const lds_f4 *>(f + 1024 + 16 * lane)};
    }
    __device__ __forceinline__ static V8 get_t(const lds_u8 *f0, const lds_u8 *f1, int tile, int lane) {
        const int g = lane >> 4, m = lane & 15, e = 4 * (4 * (tile & 1) + (m & 3));
        V8 r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int off = 2 * frag_slot(m >> 2, 4 * g + j) + e;
            r.a[j] = *reinterpret_cast<const __attribute__((address_space(3))) float *>(f0 + off);
            r.b[j] = *reinterpret_cast<const __attribute__((address_space(3))) float *>(f1 + off);
        }
        return r;
    }
    __device__ __forceinline__ static void store8(E *p, const f32x4 &x, const f32x4 &y) {
        *reinterpret_cast<f32x4 *>(p) = x;
        *reinterpret_cast<f32x4 *>(p + 4) = y;
    }
};

// row tile and row of index r inside a 64-row block (the inverse of perm_row)
__device__ __forceinline__ int perm_tile(int r) { return 2 * (r >> 5) + ((r >> 2) & 1); }
__device__ __forceinline__ int perm_m(int r) { return 4 * ((r >> 3) & 3) + (r & 3); }

// maximum / sum over the four lanes that hold one column: lanes l and l ^ 32, then l and l ^ 16,
// exchanged in the vector unit (a shuffle through LDS takes some hundred cycles)
template <typename F>
__device__ __forceinline__ float col_reduce(float x, F f) {
    const unsigned u = __builtin_bit_cast(unsigned, x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const unsigned r0 = r[0], r1 = r[1];  // whole values: a bit cast of a vector's element takes element 0
    const float y = f(__builtin_bit_cast(float, r0), __builtin_bit_cast(float, r1));
    const unsigned v = __builtin_bit_cast(unsigned, y);
    const auto q = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    const unsigned q0 = q[0], q1 = q[1];
    return f(__builtin_bit_cast(float, q0), __builtin_bit_cast(float, q1));
}
__device__ __forceinline__ float col_max(float x) {
    return col_reduce(x, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float col_sum(float x) {
    return col_reduce(x, [](float a, float b) { return a + b; });
}

// Sequences of queries and keys.  cu_q, cu_k NULL: N sequences of T queries and S keys.  Otherwise
// packed streams of T queries and S keys with N + 1 boundaries each, clipped to the streams.  The last
// query of a sequence stands at its last key: query i sees keys 0 .. i + (keys - queries).
struct AttnSeqs {
    const int *cu_q, *cu_k;
    int N, T, S;
    __device__ __forceinline__ static int clip(int x, int hi) { return x < 0 ? 0 : (x > hi ? hi : x); }
    __device__ __forceinline__ static void range(const int *cu, int n, int total, int &start, int &len) {
        start = 0;
        len = total;
        if (cu) {
            start = clip(cu[n], total);
            const int e = clip(cu[n + 1], total);
            len = e > start ? e - start : 0;
        }
    }
    // tile j of BT rows of batch entry b on the query side (cu = cu_q) or key side: as in GdrSeqs
    template <int BT>
    __device__ __forceinline__ bool find(const int *cu, int total, int b, int j, int &n, int &tile) const {
        n = b;
        tile = j;
        if (cu) {
            int lo = 0, hi = N - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (clip(cu[mid], total) / BT + mid <= j) lo = mid;
                else hi = mid - 1;
            }
            n = lo;
            tile = j - (clip(cu[n], total) / BT + n);
        }
        return tile >= 0;
    }
    static int tiles(bool packed, int N, int total, int bt) { return packed ? total / bt + N : (total + bt - 1) / bt; }
};

// One operand tile of ROWS rows and 8 NC columns into LDS: 16-byte pieces through registers, in
// fragment order; NTH threads, piece p = i NTH + tid: row p / NC.  Loads go through a buffer
// resource that starts at the tile's first row and ends behind the sequence's last: one 32-bit
// offset a thread in place of an address a piece, and rows past the last arrive as zeros.
template <bool F32, int NC, int ROWS = 64, int NTH = 256> struct TileStage {
    using Op = AttnOp<F32>;
    using E = typename Op::E;
    static constexpr int N = (ROWS * NC + NTH - 1) / NTH, STEP = NTH / NC;  // STEP: rows from piece to piece
    static constexpr bool ALL = ROWS * NC >= NTH;  // every thread has a piece
    static_assert(ROWS * NC % NTH == 0 || !ALL, "whole pieces per thread");
    static_assert(STEP % 16 == 0, "whole row tiles from piece to piece");
    typename Op::V8 x[N];
    // rows row0 .. of the nrow rows at base; `stride` in elements, a tile of it below 2^31 bytes
    __device__ __forceinline__ void load(const E *base, long long stride, int row0, int nrow, int tid) {
        const int st = (int)stride * (int)sizeof(E), left = min(max(nrow - row0, 0), ROWS);
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<E *>(base + (long long)row0 * stride), 0, left > 0 ? (left - 1) * st + 8 * NC * (int)sizeof(E) : 0, 0x00027000);
        const int step = STEP * st;
        int off = (tid / NC) * st + (tid % NC) * 8 * (int)sizeof(E);
        asm volatile("" : "+v"(off));  // or all N offsets would be kept in registers across the tiles
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = piece(r, off);
            off += step;
        }
    }
    static __device__ __forceinline__ typename Op::V8 piece(__amdgpu_buffer_rsrc_t r, int off) {
        typedef __attribute__((ext_vector_type(4))) unsigned u32x4;
        if constexpr (F32) {
            return f32x8s{__builtin_bit_cast(f32x4, (u32x4)__builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0)),
                          __builtin_bit_cast(f32x4, (u32x4)__builtin_amdgcn_raw_buffer_load_b128(r, off + 16, 0, 0))};
        } else {
            return __builtin_bit_cast(bf16x8, (u32x4)__builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
        }
    }
    // fragments [row tile][nb blocks], this tile's columns from block b0 on.  Rows of later pieces are
    // 16 or a multiple of 32 behind, which moves the fragment by a constant and flips at most one
    // address bit: a few addresses and immediate offsets.
    __device__ __forceinline__ void store(lds_u8 *f, int nb, int b0, int tid) const {
        static_assert(NC == 4 || NC == 8 || NC == 16, "32, 64 or 128 columns");
        const int r = tid / NC, c = tid % NC, kb = b0 + (c >> 2);
        lds_u8 *to = f + (perm_tile(r) * nb + kb) * Op::FB;
        if (!ALL && tid >= ROWS * NC) return;
#pragma unroll
        for (int i = 0; i < N; ++i)
            Op::put(to + i * STEP / 32 * 2 * nb * Op::FB, kb, c & 3, perm_m(r) ^ (STEP % 32 ? 8 * (i & 1) : 0), x[i]);
    }
};

}  // namespace kda
