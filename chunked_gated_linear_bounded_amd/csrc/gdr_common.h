// Building blocks of the gated delta rule with one log-decay per token and value head:
//   S_t = e^{g_t} S_{t-1} (I - b_t k_t k_t^T) + b_t v_t k_t^T,   o_t = scale S_t q_t,   g_t <= 0,
// S dv x dk.  A sequence is cut into chunks of 64 tokens.  With P = S^T at a chunk's start, G the
// inclusive prefix sum of g inside the chunk and D_ij = e^{G_i - G_j} (i >= j):
//   A = strict_lower(b_i (k_i . k_j) D_ij),  T = (I + A)^-1,  M = scale lower((q_i . k_j) D_ij),
//   Y = V - e^G K P,   X = diag(b) Y,   U = T X,
//   O = scale e^G Q P + M U,   P' = e^{G_last} P + K^T diag(e^{G_last - G}) U.
// A decay per token commutes with the products over the head dimension, so it multiplies float32
// results and never an operand: Q, K (and V) enter the matrix products as they were given, and no
// bound on g is needed.
//
// Operands are fp16 with a power-of-two exponent per block (a bf16 value is exact in fp16 once its
// block's largest magnitude sits at 2^13 .. 2^14).  A float32 value that feeds the state (T, P, X,
// U) is carried as two pieces, x = hi + lo, which keep 22 bits: three fp16 MFMAs then cost 48
// cycles per 16x16x32 block where eight float32 ones cost 256, and the float32 final state stays
// exact to a few 1e-7.  float32 inputs are split the same way (NI = 2 pieces; bf16: NI = 1).
//
// Fragment order.  A wave keeps [64 tokens or dk rows] x [16 value columns] blocks as 16x16
// accumulator tiles; two tiles 2 kb, 2 kb + 1 form the B operand of one 16x16x32 MFMA with no data
// movement if the accumulator row 4 g + i of tile 2 kb + o stands for index 32 kb + 8 g + 4 o + i:
// lane group g then holds indexes 32 kb + 8 g .. + 7, eight consecutive ones, and the matching A
// operand of a row-major matrix is one 16-byte piece per lane.  perm_row() is that index; tokens
// and key channels both use it.  A fragment is 64 lanes x 8 values (1 KiB), lane (g, m) at
// 16-byte slot 16 g + (m ^ 4 g): the exclusive-or spreads the transposed 8-byte reads of the same
// block (ld_tr16) over all LDS banks.
#pragma once
#include "kda_device.h"

namespace kda {

constexpr int kGdrChunk = 64;

// element strides of a [B][H][T][*] tensor (the last dimension is contiguous)
struct Strides3 {
    long long b, h, t;
};

__host__ __device__ constexpr int perm_row(int tile, int m) {
    return 32 * (tile >> 1) + 8 * (m >> 2) + 4 * (tile & 1) + (m & 3);
}

// byte offsets of the records; sizes for NI input pieces
struct GdrLayout {
    int ni, dk, mp;  // input pieces, key channels, pieces of M
    // key record, one per (batch, key head, chunk): int exponent of K, Q; K pieces; Q pieces
    __host__ __device__ constexpr int mat() const { return 64 * dk * 2; }
    __host__ __device__ constexpr int k_off(int piece) const { return 256 + piece * mat(); }
    __host__ __device__ constexpr int q_off(int piece) const { return 256 + (ni + piece) * mat(); }
    __host__ __device__ constexpr size_t key_bytes() const { return 256 + 2 * (size_t)ni * mat(); }
    // value record, one per (batch, value head, chunk): header, T hi, T lo, M hi (, M lo)
    // header: float eG[64], eL[64] (e^{G_last - G}), beta[64]; then at float 192: e^{G_last}; int
    // exponents of T, M, K, Q; and seven norms, max b e^G |k|_1, max b, max row sum of |T|, sum over
    // the tokens of max |k|, max e^{G_last - G} |k|_1, max row sum of |T_ij| e^{G_j - G_i}, max |k|_1
    static constexpr int kTri = 6 * 1024;  // six causal 16x32 fragments of a 64x64 lower triangle
    static constexpr int kHead = 1024;
    __host__ __device__ constexpr int t_off(int piece) const { return kHead + piece * kTri; }
    __host__ __device__ constexpr int m_off(int piece) const { return kHead + (2 + piece) * kTri; }
    __host__ __device__ constexpr size_t val_bytes() const { return kHead + (2 + (size_t)mp) * kTri; }
};

// index of the causal fragment (row tile rt, 32-column block kb): rt 0, 1 have kb 0 only
__host__ __device__ constexpr int tri_frag(int rt, int kb) { return rt < 2 ? rt : 2 + 2 * (rt - 2) + kb; }

// Where a chunk lies.  Fixed-length batches: sequence n = batch entry, chunk c of it.  Packed
// documents (cu not NULL): document n covers tokens cu[n] .. cu[n+1] of one stream, its chunk c has
// slot cu[n] / 64 + n + c, which needs no table: floor(cu[n] / 64) + n + ceil(len / 64) is at most
// floor(cu[n+1] / 64) + n + 1.  Boundaries are clipped to [0, T] and an end to at least its start,
// so no content of cu makes an index leave the arrays.
struct GdrSeqs {
    const int *cu;  // NULL: fixed-length
    int N, T;       // sequences; tokens of one sequence (fixed) or of the stream
    __device__ __forceinline__ int clip(int x) const { return x < 0 ? 0 : (x > T ? T : x); }
    __device__ __forceinline__ int start(int n) const { return cu ? clip(cu[n]) : 0; }
    __device__ __forceinline__ int length(int n) const {
        if (!cu) return T;
        const int s = clip(cu[n]), e = clip(cu[n + 1]);
        return e > s ? e - s : 0;
    }
    // first chunk slot of sequence n inside its batch entry
    __device__ __forceinline__ int slot0(int n) const { return cu ? clip(cu[n]) / kGdrChunk + n : 0; }
    // batch entry that sequence n's tensors and records belong to
    __device__ __forceinline__ int batch(int n) const { return cu ? 0 : n; }
    // the chunk at slot j of batch entry b: first token and its rows (0: no chunk there)
    __device__ __forceinline__ int find(int b, int j, int &t0, int &n) const {
        int c = j;
        n = b;
        if (cu) {
            int lo = 0, hi = N;  // the last n with slot0(n) <= j (slot0 grows with n)
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (slot0(mid) <= j && mid < N) lo = mid;
                else hi = mid - 1;
            }
            n = lo;
            c = j - slot0(n);
        }
        const int len = length(n), left = c < 0 ? 0 : len - c * kGdrChunk;
        t0 = start(n) + c * kGdrChunk;
        return left < 0 ? 0 : (left > kGdrChunk ? kGdrChunk : left);
    }
};

// ---------------------------------------------------------------- fp16 pieces
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;

// x = hi + lo to 22 bits: hi is x cut off (not rounded) to fp16, so what is left is exact in
// float32 and lo takes its upper 11 bits.
__device__ __forceinline__ void split2(float x0, float x1, f16x2 &hi, f16x2 &lo) {
    hi = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_pkrtz(x0, x1));
    lo = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_pkrtz(x0 - (float)hi[0], x1 - (float)hi[1]));
}
// B operand pieces from an accumulator tile pair, times 2^e
__device__ __forceinline__ void split_pair(const f32x4 &t0, const f32x4 &t1, float s, f16x8 &hi, f16x8 &lo) {
    f16x2 h[4], l[4];
    split2(t0[0] * s, t0[1] * s, h[0], l[0]);
    split2(t0[2] * s, t0[3] * s, h[1], l[1]);
    split2(t1[0] * s, t1[1] * s, h[2], l[2]);
    split2(t1[2] * s, t1[3] * s, h[3], l[3]);
    hi = f16x8{h[0][0], h[0][1], h[1][0], h[1][1], h[2][0], h[2][1], h[3][0], h[3][1]};
    lo = f16x8{l[0][0], l[0][1], l[1][0], l[1][1], l[2][0], l[2][1], l[3][0], l[3][1]};
}
// one piece, rounded to nearest
__device__ __forceinline__ f16x8 round_pair(const f32x4 &t0, const f32x4 &t1, float s) {
    f16x8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) { r[i] = (_Float16)(t0[i] * s); r[4 + i] = (_Float16)(t1[i] * s); }
    return r;
}
__device__ __forceinline__ f32x4 mma16(const f16x8 &a, const f16x8 &b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// The largest finite magnitude.  Exponents and bounds come from a block's finite values; an infinity or a
// NaN stays one in its pieces and reaches the rows or columns of the products that its element takes part
// in, and the others keep their digits.  Whole numbers order as the magnitudes whose bits they are:
// shifted past the sign and moved up by 2^24, a zero is 2^24, and infinities and NaN have gone round the
// end to below that.  add4 takes four values of one row or column that the products spoil as a whole: an
// infinity among them leaves all four out, for one instruction more than a maximum of floats.
struct Most {
    unsigned t = 1u << 24;
    __device__ __forceinline__ void add(float x) {
        const unsigned y = (__builtin_bit_cast(unsigned, x) << 1) + (1u << 24);
        t = y > t ? y : t;
    }
    __device__ __forceinline__ void add4(const f32x4 &x) {
        add(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
    }
    __device__ __forceinline__ static float value(unsigned t) { return __builtin_bit_cast(float, (t - (1u << 24)) >> 1); }
    __device__ __forceinline__ float lane() const { return value(t); }
    __device__ __forceinline__ float wave() const {
        return value(__builtin_bit_cast(unsigned, wave_max(__builtin_bit_cast(float, t))));
    }
};
__device__ __forceinline__ float finite_mag(float x) {
    Most m;
    m.add(x);
    return m.lane();
}

// exponent that puts magnitudes up to m at 2^13 .. 2^14, kept where 2^e and 2^-e are normal floats (m may
// be a bound that has left float's range).  A block of zeros has the largest, so that it does not count
// where several blocks are brought to the smallest of their exponents.
__device__ __forceinline__ int gdr_exp(float m) {
    if (!(m > 0.f)) return 120;
    const int e = pow2_scale(fminf(m, 3.402823466e38f));
    return e > 120 ? 120 : (e < -120 ? -120 : e);
}
__device__ __forceinline__ float pow2f(int e) { return __builtin_bit_cast(float, (127 + e) << 23); }
// 2^-(a+b), also where the sum leaves the range of one float's exponent
__device__ __forceinline__ float scale_down(float x, int e) { return ldexp2(x, -e); }

__device__ __forceinline__ float max4(const f32x4 &x) { return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])); }

// ---------------------------------------------------------------- fragments in LDS
// byte offset of lane (g, m) inside a fragment
__device__ __forceinline__ int frag_slot(int g, int m) { return (16 * g + (m ^ (4 * g))) * 16; }

__device__ __forceinline__ f16x8 ld_frag(const lds_u8 *f, int lane) {
    return *reinterpret_cast<const __attribute__((address_space(3))) f16x8 *>(f + frag_slot(lane >> 4, lane & 15));
}
// A operand of the transpose: rows = the 16 columns perm_row(tile, .) of a block whose row-major
// fragments start at `base` ((row tile, column block) at (row tile * ncb + column block) KiB),
// k = its rows 32 kb .. 32 kb + 31.  Lane (g, m): slots j = rows 32 kb + 8 g + j.
__device__ __forceinline__ f16x8 ld_frag_t(const lds_u8 *f0, const lds_u8 *f1, int tile, int lane) {
    // f0, f1: the fragments (row tiles 2 kb, 2 kb + 1) x (column block tile >> 1)
    const int g = lane >> 4, s = lane & 15, m = 4 * g + (s >> 2), cg = s & 3;
    const int off = frag_slot(cg, m) + 8 * (tile & 1);
    const f16x4 a = ld_tr16<f16x4>(f0 + off), b = ld_tr16<f16x4>(f1 + off);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

}  // namespace kda
