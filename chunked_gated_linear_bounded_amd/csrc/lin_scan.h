// Decayed linear attention between segments: the scan that turns segments' own contributions into
// start states, and what the backward pass still does behind its walks (the log-decays' gradient, sums
// over value heads, rows that no document covers).  All of it moves bytes and nothing else.  Training step of
// 2 x 4096 x 8/16 heads of 128 x 128 (288 us): scans 2 x 8 us, 34 MB each read and written; the gradient of the
// log-decays 11, of which the <R, S> are 34 MB; the sums over heads 32, 134 MB read and 34 written (5.2 TB/s).
#pragma once
#include "lin_common.h"

namespace kda {

struct LinScanArgs {
    LinSeqs seqs;
    int B, H, nslot, n4;         // n4: dk dv / 4
    struct Side {
        const float *init;       // [N][H] (NULL: zero)
        float *seg, *last;       // [B][H][nslot] in place; [N][H] end states (NULL: not wanted)
        const float *decay;      // [B][H][nslot]
        bool all;                // segments that are alone in their sequence take part as others do
    } side[2];                   // forwards; backwards in time
};

// seg[s] <- state before segment s (in the walk's direction): four floats a thread, eight segments'
// loads in flight.
static __global__ __launch_bounds__(256) void lin_scan_kernel(const LinScanArgs p) {
    const bool rev = blockIdx.y != 0;
    const LinScanArgs::Side &a = p.side[blockIdx.y];
    const unsigned parts = p.n4 / 256, unit = blockIdx.x / parts;
    const int seq = unit / p.H, h = unit % p.H, e = (blockIdx.x % parts) * 256 + threadIdx.x;
    if (a.seg == nullptr) return;
    const int len = p.seqs.length(seq);
    if (!a.all && len <= p.seqs.seg) return;
    const int ns = max(1, p.seqs.segments(seq)), b = p.seqs.cu ? 0 : seq;
    const size_t s0 = ((size_t)b * p.H + h) * p.nslot + p.seqs.slot0(seq);
    f32x4 *st = reinterpret_cast<f32x4 *>(a.seg) + s0 * p.n4 + e;
    const size_t at = ((size_t)seq * p.H + h) * p.n4 + e;
    f32x4 carry = {0.f, 0.f, 0.f, 0.f};
    if (a.init) carry = reinterpret_cast<const f32x4 *>(a.init)[at];
    for (int s = 0; s < ns; s += 8) {
        f32x4 x[8];
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = min(s + i, ns - 1), k = rev ? ns - 1 - c : c;
            x[i] = st[(size_t)k * p.n4];
            d[i] = a.decay[s0 + k];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (s + i >= ns) break;
            const int k = rev ? ns - 1 - s - i : s + i;
            st[(size_t)k * p.n4] = carry;
            carry = carry * d[i] + x[i];
        }
    }
    if (a.last) reinterpret_cast<f32x4 *>(a.last)[at] = carry;
}

struct LinDecayGradArgs {
    LinSeqs seqs;
    int B, H, nslot, n4;
    bool g32;
    const float *fwd, *rev;      // start states of the segments, of either walk
    const float *last, *dfinal;  // [N][H]: end states, and the gradient by them (NULL: zero)
    const float *row, *col;      // [B][H][T]: q . dq and k . dk, the pairs of a token with itself left out
    void *dg;                    // [B][H][T]
};

// dg_t = sum over the pairs (i, j) of tokens with i >= t > j of their part of the loss.  Inside a segment
// that is the sum over u >= t of row_u - col_u, plus the pairs that reach over the segment's end, <R, S>
// there.
static __global__ __launch_bounds__(256) void lin_decay_grad_kernel(const LinDecayGradArgs p) {
    __shared__ double part[4];
    __shared__ double tail[4];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int slot = blockIdx.x % p.nslot, h = blockIdx.x / p.nslot % p.H, b = blockIdx.x / p.nslot / p.H;
    int seq, piece;
    if (!p.seqs.find(b, slot, seq, piece)) return;
    const int len = p.seqs.length(seq), rows = min(p.seqs.seg, len - piece * p.seqs.seg);
    if (rows <= 0) return;
    const size_t sunit = ((size_t)b * p.H + h) * p.nslot + slot, row0 = ((size_t)b * p.H + h) * p.seqs.T + p.seqs.start(seq) + piece * p.seqs.seg;
    const bool end = (piece + 1) * (long long)p.seqs.seg >= len;
    const size_t at = ((size_t)seq * p.H + h) * p.n4;
    const f32x4 *R = end ? reinterpret_cast<const f32x4 *>(p.dfinal) + at : reinterpret_cast<const f32x4 *>(p.rev) + sunit * p.n4;
    const f32x4 *S = end ? reinterpret_cast<const f32x4 *>(p.last) + at : reinterpret_cast<const f32x4 *>(p.fwd) + (sunit + 1) * p.n4;
    double over = 0.0;
    if (!end || p.dfinal) {
        for (int e = tid; e < p.n4; e += 256) {
            const f32x4 x = R[e], y = S[e];
            over += (double)((x[0] * y[0] + x[1] * y[1]) + (x[2] * y[2] + x[3] * y[3]));
        }
        over = lane64(wave_scan64(over), 63);
    }
    if (lane == 0) tail[w] = over;
    __syncthreads();
    double carry = (tail[0] + tail[1]) + (tail[2] + tail[3]);
    for (int top = rows - 1; top >= 0; top -= 256) {
        const int t = top - tid;  // later tokens on lower lanes
        const double x = t >= 0 ? (double)p.row[row0 + t] - (double)p.col[row0 + t] : 0.0;
        double s = wave_scan64(x);
        __syncthreads();  // part has been read
        if (lane == 63) part[w] = s;
        __syncthreads();
        double before = carry;
        for (int i = 0; i < 4; ++i) {
            if (i < w) before += part[i];
            carry += part[i];
        }
        if (t >= 0) {
            const float d = (float)(before + s);
            if (p.g32) reinterpret_cast<float *>(p.dg)[row0 + t] = d;
            else reinterpret_cast<__bf16 *>(p.dg)[row0 + t] = (__bf16)d;
        }
    }
}

// Sums over the r value heads of a key head of their float32 partials, of dq (y = 0) and dk: four
// elements a thread, n4 = T dk / 4 of a head, `all` of them.
template <typename E>
__global__ __launch_bounds__(256) void lin_head_sum_kernel(const float *part0, const float *part1, E *out0, E *out1, int r, long long n4,
                                                           long long all) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= all) return;
    const f32x4 *x = reinterpret_cast<const f32x4 *>(blockIdx.y ? part1 : part0) + (i / n4 * r) * n4 + i % n4;
    f32x4 s = x[0];
    for (int k = 1; k < r; ++k) s += x[k * n4];
    st_tile((blockIdx.y ? out1 : out0) + 4 * i, 0, s);
}

// Gradients of the rows of a packed stream that no document covers, [0, cu[0]) and [cu[N], T): zeros.
template <typename E> struct LinUncovered {
    E *dq, *dk, *dv;
    void *dg;
    LinSeqs seqs;
    int Hk, H, DK, DV;
    bool g32;
};
template <typename E>
__global__ __launch_bounds__(256) void lin_uncovered_kernel(const LinUncovered<E> p) {
    const int from = p.seqs.clip(p.seqs.cu[0]), to = max(from, p.seqs.clip(p.seqs.cu[p.seqs.N])), h = blockIdx.y;
    const int t0 = blockIdx.x * 64, t1 = min(t0 + 64, p.seqs.T);
    if (t0 >= from && t1 <= to) return;
    auto clear = [&](E *x, int d) {
        for (int i = threadIdx.x; i < (t1 - t0) * d; i += 256) {
            const int t = t0 + i / d;
            if (t < from || t >= to) x[((size_t)h * p.seqs.T + t0) * d + i] = (E)0.f;
        }
    };
    if (h < p.Hk) {
        clear(p.dq, p.DK);
        clear(p.dk, p.DK);
    }
    clear(p.dv, p.DV);
    const int t = t0 + threadIdx.x;
    if (p.dg && t < t1 && (t < from || t >= to)) {
        if (p.g32) static_cast<float *>(p.dg)[(size_t)h * p.seqs.T + t] = 0.f;
        else static_cast<__bf16 *>(p.dg)[(size_t)h * p.seqs.T + t] = (__bf16)0.f;
    }
}

}  // namespace kda
