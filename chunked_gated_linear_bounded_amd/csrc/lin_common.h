// Building blocks of linear attention with one log-decay per token and value head:
//   S_t = e^{g_t} S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t,   g_t <= 0,   S dv x dk.
// In chunks of 64 tokens, with P = S^T at a chunk's start, G the inclusive prefix sum of g inside the
// chunk and D_ij = e^{G_i - G_j} (i >= j):
//   O = scale ((Q K^T o D) V + e^G Q P),   P' = e^{G_last} P + K^T diag(e^{G_last - G}) V.
// The gradients are three operators of the same form.  With R the gradient by the state behind a token,
// transposed as P is,
//   dQ = scale ((dO V^T o D) K + e^G dO P^T)                   forwards, the state P^T;
//   dK = scale (dO V^T o D)^T Q + e^{G_last - G} V R^T         backwards in time;
//   dV = scale (Q K^T o D)^T dO + e^{G_last - G} K R           backwards in time;
//   R at the chunk's start = e^{G_last} R + scale Q^T diag(e^G) dO.
// So one walk over chunks does all four: out = a-rows against b-rows, times c-rows, plus a-rows against
// a state that gathers b c^T (lin_walk.h), forwards or backwards.
//
// The state has no delta rule in it: what a piece of a sequence adds to it does not depend on what came
// before.  So a sequence is cut into segments, walked side by side: first each segment's own
// contribution (b and c are read), then a scan over the segments (lin_scan.h), then the outputs.
//
// log-decays are summed in float64 and kept as two floats, so that a difference of two prefix sums is
// as exact where strong decays came before as where none did.
#pragma once
#include "latent_common.h"

namespace kda {

struct LinSeqs {
    const int *cu;    // NULL: fixed-length
    int N, T, seg;    // sequences; tokens of one sequence (fixed) or of the stream; tokens of a segment
    bool sparse;      // where states lie (state_slot)
    __device__ __forceinline__ int clip(int x) const { return x < 0 ? 0 : (x > T ? T : x); }
    __device__ __forceinline__ int start(int n) const { return cu ? clip(cu[n]) : 0; }
    __device__ __forceinline__ int length(int n) const {
        if (!cu) return T;
        const int s = clip(cu[n]), e = clip(cu[n + 1]);
        return e > s ? e - s : 0;
    }
    // first work slot of sequence n inside its batch entry; as in GdrSeqs, floor(start / seg) + n
    // leaves every sequence room for its segments (and at least one slot)
    __device__ __forceinline__ int slot0(int n) const { return cu ? clip(cu[n]) / seg + n : 0; }
    // state slot of segment c of sequence n, which is longer than a segment (no other has states in the
    // workspace).  sparse: 2 floor(start / seg) + c, whatever the number of sequences: one of m segments and a
    // piece, m >= 1, has m + 1 slots, and the next one starts m segments behind it or later, 2 m slots.  Else
    // the segment's work slot.
    __device__ __forceinline__ int state_slot(int n, int c, int slot) const { return sparse ? 2 * (clip(cu[n]) / seg) + c : slot; }
    __device__ __forceinline__ int segments(int n) const { return (length(n) + seg - 1) / seg; }
    // the segment at slot j of batch entry b: its sequence n, its number in it; false: none there
    __device__ __forceinline__ bool find(int b, int j, int &n, int &c) const {
        n = b;
        c = j;
        if (cu) {
            int lo = 0, hi = N - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (slot0(mid) <= j) lo = mid;
                else hi = mid - 1;
            }
            n = lo;
            c = j - slot0(n);
        }
        const int have = segments(n);
        return c >= 0 && (c < have || c == 0);
    }
};

// ---------------------------------------------------------------- log-decays
template <int CTRL, int ROWMASK>
__device__ __forceinline__ double dpp_add64(double x) {
    const unsigned long long u = __builtin_bit_cast(unsigned long long, x);
    const unsigned lo = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)u, CTRL, ROWMASK, 0xF, false);
    const unsigned hi = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)(u >> 32), CTRL, ROWMASK, 0xF, false);
    return x + __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
// inclusive prefix sum over the 64 lanes
__device__ __forceinline__ double wave_scan64(double x) {
    x = dpp_add64<0x111, 0xF>(x);  // row_shr 1, 2, 4, 8
    x = dpp_add64<0x112, 0xF>(x);
    x = dpp_add64<0x114, 0xF>(x);
    x = dpp_add64<0x118, 0xF>(x);
    x = dpp_add64<0x142, 0xA>(x);  // row_bcast:15 into rows 1 and 3
    x = dpp_add64<0x143, 0xC>(x);  // row_bcast:31 into rows 2 and 3
    return x;
}
__device__ __forceinline__ double lane64(double x, int lane) {
    const unsigned long long u = __builtin_bit_cast(unsigned long long, x);
    const unsigned lo = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)u, lane);
    const unsigned hi = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)(u >> 32), lane);
    return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
// a log-decay in log2 units; below -1000 (-inf too) it is a decay to zero, and sums stay finite
__device__ __forceinline__ double decay_log2(float g) { return (double)(g < -1000.f ? -1000.f : g) * 1.4426950408889634; }

// a log-decay as it lies in memory, and its value: apart, so that nothing waits for the load before its use
__device__ __forceinline__ unsigned load_g_bits(const void *g, long long at, bool g32) {
    return g32 ? reinterpret_cast<const unsigned *>(g)[at] : reinterpret_cast<const unsigned short *>(g)[at];
}
__device__ __forceinline__ float g_value(unsigned bits, bool g32) { return __builtin_bit_cast(float, g32 ? bits : bits << 16); }
__device__ __forceinline__ float load_g(const void *g, long long at, bool g32) { return g_value(load_g_bits(g, at, g32), g32);
}

// ---------------------------------------------------------------- operands
// What is computed in float32 and enters a product again is carried in pieces where operands are bf16:
// x = hi + lo keeps 16 bits (M and P, whose products are rounded to bf16 outputs: these are off by 1.7e-3 of their
// norm, as float32's rounded once), a third piece all 24 (what a float32 state that can be handed on gathers).  bf16 has float's exponents, so pieces need no
// scaling.  float32 inputs use float32 MFMAs and need no pieces.
template <bool F32> struct LinOp;
template <> struct LinOp<true> : AttnOp<true> {};
template <> struct LinOp<false> : AttnOp<false> {
    typedef __attribute__((ext_vector_type(4))) unsigned u32x4;
    // x[i], x[i + 1] as a bf16 pair, taken off them.  The pair is a whole number from here on: as two bf16
    // values the compiler converts each a second time to subtract it (64k x 32 heads: 855 us instead of 811).
    __device__ __forceinline__ static unsigned take(f32x4 &x, int i) {
        typedef __attribute__((ext_vector_type(2))) __bf16 b2;
        unsigned u = __builtin_bit_cast(unsigned, b2{(__bf16)x[i], (__bf16)x[i + 1]});
        asm("" : "+v"(u));
        x[i] -= __builtin_bit_cast(float, u << 16);
        x[i + 1] -= __builtin_bit_cast(float, u & 0xffff0000u);
        return u;
    }
    template <int NP>
    __device__ __forceinline__ static void pieces(f32x4 x, f32x4 y, bf16x8 (&r)[NP]) {
#pragma unroll
        for (int p = 0; p < NP; ++p) r[p] = __builtin_bit_cast(bf16x8, u32x4{take(x, 0), take(x, 2), take(y, 0), take(y, 2)});
    }
    __device__ __forceinline__ static void split(const bf16x8 &v, f32x4 &x, f32x4 &y) {
        const u32x4 u = __builtin_bit_cast(u32x4, v);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[2 * i] = __builtin_bit_cast(float, u[i] << 16);
            x[2 * i + 1] = __builtin_bit_cast(float, u[i] & 0xffff0000u);
            y[2 * i] = __builtin_bit_cast(float, u[2 + i] << 16);
            y[2 * i + 1] = __builtin_bit_cast(float, u[2 + i] & 0xffff0000u);
        }
    }
};

}  // namespace kda
