// Decayed linear attention between segments: the scan that turns segments' own contributions into
// start states, and what the backward pass still does behind its walks (the log-decays' gradient, sums
// over value heads, rows that no document covers).  All of it moves bytes and nothing else.  Training step of
// 2 x 4096 x 8/16 heads of 128 x 128 (286 us): scans 2 x 8 us, 34 MB each read and written; all that is behind the
// walks 33 to 35, 134 MB of partials and 34 of states read, 34 written (5.8 TB/s; as launches of their own the
// sums over heads took 32 and the log-decays 11).
#pragma once
#include "lin_common.h"

namespace kda {

struct LinScanArgs {
    LinSeqs seqs;
    int B, H, nslot, nstate, n4; // n4: dk dv / 4
    struct Side {
        const float *init;       // [N][H] (NULL: zero)
        float *seg, *last;       // [B][H][nstate] in place; [N][H] end states (NULL: not wanted)
        const float *decay;      // [B][H][nslot]
        bool all;                // last holds what segments that are alone in their sequence add to its state
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
    const int ns = p.seqs.segments(seq), b = p.seqs.cu ? 0 : seq, slot = p.seqs.slot0(seq);
    const size_t s0 = ((size_t)b * p.H + h) * p.nslot + slot;
    const size_t at = ((size_t)seq * p.H + h) * p.n4 + e;
    f32x4 carry = {0.f, 0.f, 0.f, 0.f};
    if (a.init) carry = reinterpret_cast<const f32x4 *>(a.init)[at];
    if (len <= p.seqs.seg) {
        f32x4 *last = reinterpret_cast<f32x4 *>(a.last) + at;
        *last = carry * a.decay[s0] + *last;
        return;
    }
    f32x4 *st = reinterpret_cast<f32x4 *>(a.seg) + (((size_t)b * p.H + h) * p.nstate + p.seqs.state_slot(seq, 0, slot)) * p.n4 + e;
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
    int B, H, nslot, nstate, n4;
    bool g32;
    const float *fwd, *rev;      // start states of the segments, of either walk
    const float *last, *dfinal;  // [N][H]: end states, and the gradient by them (NULL: zero)
    const float *row, *col;      // [B][H][T]: q . dq and k . dk, the pairs of a token with itself left out
    void *dg;                    // [B][H][T]
};

// dg_t = sum over the pairs (i, j) of tokens with i >= t > j of their part of the loss.  Inside a segment
// that is the sum over u >= t of row_u - col_u, plus the pairs that reach over the segment's end, <R, S>
// there.
static __device__ __forceinline__ void lin_decay_grad(const LinDecayGradArgs &p, unsigned block) {
    __shared__ double part[4];
    __shared__ double tail[4];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int slot = block % p.nslot, h = block / p.nslot % p.H, b = block / p.nslot / p.H;
    int seq, piece;
    if (!p.seqs.find(b, slot, seq, piece)) return;
    const int len = p.seqs.length(seq), rows = min(p.seqs.seg, len - piece * p.seqs.seg);
    if (rows <= 0) return;
    const size_t state = ((size_t)b * p.H + h) * p.nstate + p.seqs.state_slot(seq, piece, slot), row0 = ((size_t)b * p.H + h) * p.seqs.T + p.seqs.start(seq) + piece * p.seqs.seg;
    const bool end = (piece + 1) * (long long)p.seqs.seg >= len;
    const size_t at = ((size_t)seq * p.H + h) * p.n4;
    const f32x4 *R = end ? reinterpret_cast<const f32x4 *>(p.dfinal) + at : reinterpret_cast<const f32x4 *>(p.rev) + state * p.n4;
    const f32x4 *S = end ? reinterpret_cast<const f32x4 *>(p.last) + at : reinterpret_cast<const f32x4 *>(p.fwd) + (state + 1) * p.n4;
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

// What the backward pass does behind its walks, in one launch of `grads` work-groups for the log-decays'
// gradient, `sums` for the sums over the r value heads of a key head of their float32 partials of dq and dk
// (four elements of both a thread, n4 = T dk / 4 of a head, `all` of them; r = 1: none), and the rest for the rows
// of a packed stream that no document covers, [0, cu[0]) and [cu[N], T): zeros.
template <typename E> struct LinFinish {
    LinDecayGradArgs d;
    unsigned grads, sums;
    const float *part[2];
    E *dq, *dk, *dv;
    int r, Hk, H, DK, DV;
    long long n4, all;
};
template <typename E>
__global__ __launch_bounds__(256) void lin_finish_kernel(const LinFinish<E> p) {
    unsigned block = blockIdx.x;
    if (block < p.grads) {
        lin_decay_grad(p.d, block);
        return;
    }
    block -= p.grads;
    const LinSeqs &seqs = p.d.seqs;
    int from = 0, to = seqs.T;  // the rows that documents cover
    if (seqs.cu) {
        from = seqs.clip(seqs.cu[0]);
        to = max(from, seqs.clip(seqs.cu[seqs.N]));
    }
    if (block < p.sums) {
        const long long i = (long long)block * 256 + threadIdx.x;
        if (i >= p.all) return;
        const int t = (int)(i % p.n4 / (p.DK / 4));
        const long long at = (i / p.n4 * p.r) * p.n4 + i % p.n4;
        const f32x4 *x = reinterpret_cast<const f32x4 *>(p.part[0]) + at, *y = reinterpret_cast<const f32x4 *>(p.part[1]) + at;
        f32x4 u = x[0], v = y[0];
        for (int k = 1; k < p.r; ++k) {
            u += x[k * p.n4];
            v += y[k * p.n4];
        }
        const bool none = t < from || t >= to;
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        st_tile(p.dq + 4 * i, 0, none ? zero : u);
        st_tile(p.dk + 4 * i, 0, none ? zero : v);
        return;
    }
    block -= p.sums;
    const int nx = (seqs.T + 63) / 64, h = block / nx, t0 = block % nx * 64, t1 = min(t0 + 64, seqs.T);
    if (t0 >= from && t1 <= to) return;
    auto clear = [&](E *x, int d) {
        for (int i = threadIdx.x; i < (t1 - t0) * d; i += 256) {
            const int t = t0 + i / d;
            if (t < from || t >= to) x[((size_t)h * seqs.T + t0) * d + i] = (E)0.f;
        }
    };
    if (p.sums == 0) {  // (else with the sums)
        clear(p.dq, p.DK);
        clear(p.dk, p.DK);
    }
    clear(p.dv, p.DV);
    const int t = t0 + threadIdx.x;
    if (p.d.dg && t < t1 && (t < from || t >= to)) {
        if (p.d.g32) static_cast<float *>(p.d.dg)[(size_t)h * seqs.T + t] = 0.f;
        else static_cast<__bf16 *>(p.d.dg)[(size_t)h * seqs.T + t] = (__bf16)0.f;
    }
}

}  // namespace kda
