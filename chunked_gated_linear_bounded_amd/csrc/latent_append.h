// New tokens into a paged cache of latent rows [latent (dc), rotary key part (dr)], and the rotary part of
// their queries behind the absorbed part:
//   c' = c / sqrt(mean c^2 + eps) w (or c as it is),   (x, y)' = (x cos a - y sin a, x sin a + y cos a),
//   a = position freq_i for the pair i of a rotary part.
// Every byte is read once and written once: HBM bounds a prompt, the launch a single token.
//
// A wave takes one token and up to 32 heads: the wave of the first heads also the token's row of the cache.
// An item is 8 pairs of one head's rotary part, 16 elements, two loads and two stores of 16 bytes (bf16);
// items of a lane have the same pairs, so a lane keeps the 8 cosines and sines that it needs.  All loads
// are issued before the angles are computed.  The angle's turns are reduced in float64, so a position may
// be any int32: position times freq is off by 2^-53 of itself there, and by half a turn's 2^-24 after it, as it
// becomes the float32 that cosine and sine are taken of.
// The row's sum of squares is held in float32 (dc squares of one sign: off by dc 2^-24 at most).
//
// 16,411 tokens of 64 heads, 0.31 GB: 60 us, 5.1 TB/s.  Five tokens of 128 heads: 4.5 us, a launch and one
// round trip to memory behind another (lengths, the page, the row).
#pragma once
#include "latent_common.h"

namespace kda {

struct LatentAppendArgs {
    const void *latent, *kr, *qr, *weight;
    long long sl[2], sk[2], sq[3];  // element strides: b, t; b, t; b, t, head
    void *cache, *q;                // [pages][page][dc + dr]; [B][T][H][dc + dr]
    const int *table, *lengths, *positions, *counts, *cu;
    const float *freqs;             // [dr / 2]
    int N, B, T, H, parts, pages, page, max_pages;
    float eps;
};

constexpr int kAppendHeads = 32;  // heads of a wave

// two pieces of 8 elements: the pairs 8 p .. + 7 of a rotary part, as they lie
template <typename E> struct Piece8 {
    float x[8];
    __device__ __forceinline__ void load(const E *p) {
        if constexpr (sizeof(E) == 4) {
            const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = a[i];
                x[4 + i] = b[i];
            }
        } else {
            const bf16x8 a = *reinterpret_cast<const bf16x8 *>(p);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = (float)a[i];
        }
    }
    __device__ __forceinline__ void store(E *p) const {
        if constexpr (sizeof(E) == 4) {
            *reinterpret_cast<f32x4 *>(p) = f32x4{x[0], x[1], x[2], x[3]};
            *reinterpret_cast<f32x4 *>(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
        } else {
            bf16x8 a;
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = (__bf16)x[i];
            *reinterpret_cast<bf16x8 *>(p) = a;
        }
    }
};

template <int DC, int DR, bool F32, bool INTERLEAVED>
__global__ __launch_bounds__(256) void latent_append_kernel(const LatentAppendArgs p) {
    using E = typename std::conditional<F32, float, __bf16>::type;
    constexpr int D = DC + DR, IPH = DR / 16, NI = kAppendHeads * IPH / 64, HALF = DR / 2;  // items of a head; items a lane
    static_assert(DR == 64, "8 pairs an item, 4 items a head");
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const long long unit = (long long)blockIdx.x * 4 + w, token = unit / p.parts;
    const int part = (int)(unit % p.parts);
    if (token >= (long long)p.B * p.T) return;
    int b = (int)(token / p.T), t = (int)(token % p.T), n = b, i = t, count = p.T;
    if (p.cu) {
        int lo = 0, hi = p.N - 1;  // the last sequence that begins at t or before
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (AttnSeqs::clip(p.cu[mid], p.T) <= t) lo = mid;
            else hi = mid - 1;
        }
        n = lo;
        int start;
        AttnSeqs::range(p.cu, n, p.T, start, count);
        i = t - start;
    } else if (p.counts) {
        count = AttnSeqs::clip(p.counts[b], p.T);
    }
    if (i < 0 || i >= count) return;  // no token: nothing is written
    const long long row = (long long)p.lengths[n] - count + i;
    const long long pos = p.positions ? (long long)p.positions[token] : row;

    const int c = lane & (IPH - 1);  // the lane's pairs are 8 c .. + 7
    const int o0 = INTERLEAVED ? 16 * c : 8 * c, o1 = INTERLEAVED ? o0 + 8 : o0 + HALF;
    const int heads = min(kAppendHeads, p.H - part * kAppendHeads);
    Piece8<E> x[NI], y[NI], lat, kx, ky;
    const E *qr = reinterpret_cast<const E *>(p.qr) + b * p.sq[0] + t * p.sq[1] + (long long)part * kAppendHeads * p.sq[2];
    auto head = [&](int j) { return lane / IPH + 64 / IPH * j; };
#pragma unroll
    for (int j = 0; j < NI; ++j)
        if (head(j) < heads) {
            x[j].load(qr + head(j) * p.sq[2] + o0);
            y[j].load(qr + head(j) * p.sq[2] + o1);
        }
    bool to_cache = part == 0 && row >= 0 && row < (long long)p.max_pages * p.page;
    int pg = 0;
    if (to_cache) pg = p.table[(long long)n * p.max_pages + row / p.page];
    to_cache = to_cache && pg >= 0 && pg < p.pages;
    if (to_cache) {
        const E *l = reinterpret_cast<const E *>(p.latent) + b * p.sl[0] + t * p.sl[1], *k = reinterpret_cast<const E *>(p.kr) + b * p.sk[0] + t * p.sk[1];
        if (lane < DC / 8) lat.load(l + 8 * lane);
        if (lane < IPH) {
            kx.load(k + o0);
            ky.load(k + o1);
        }
    }
    // the angle of pair lane % HALF, in turns from -1/2 to 1/2
    const double turns = (double)pos * (double)p.freqs[lane % HALF] * 0.15915494309189535;
    float s, co;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &co);
    float sn[8], cs[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        sn[k] = __shfl(s, 8 * c + k);
        cs[k] = __shfl(co, 8 * c + k);
    }
    auto turn = [&](Piece8<E> &u, Piece8<E> &v) {
        if constexpr (INTERLEAVED) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float a = u.x[2 * k], d = u.x[2 * k + 1], e = v.x[2 * k], f = v.x[2 * k + 1];
                u.x[2 * k] = a * cs[k] - d * sn[k];
                u.x[2 * k + 1] = a * sn[k] + d * cs[k];
                v.x[2 * k] = e * cs[4 + k] - f * sn[4 + k];
                v.x[2 * k + 1] = e * sn[4 + k] + f * cs[4 + k];
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float a = u.x[k], d = v.x[k];
                u.x[k] = a * cs[k] - d * sn[k];
                v.x[k] = a * sn[k] + d * cs[k];
            }
        }
    };
    E *q = reinterpret_cast<E *>(p.q) + (token * p.H + (long long)part * kAppendHeads) * D + DC;
#pragma unroll
    for (int j = 0; j < NI; ++j)
        if (head(j) < heads) {
            turn(x[j], y[j]);
            x[j].store(q + (long long)head(j) * D + o0);
            y[j].store(q + (long long)head(j) * D + o1);
        }
    if (!to_cache) return;
    E *to = reinterpret_cast<E *>(p.cache) + ((long long)pg * p.page + row % p.page) * D;
    if (p.weight) {
        float sum = 0.f;
        if (lane < DC / 8) {
#pragma unroll
            for (int k = 0; k < 8; ++k) sum = fmaf(lat.x[k], lat.x[k], sum);
        }
#pragma unroll
        for (int k = 32; k > 0; k >>= 1) sum += __shfl_xor(sum, k);
        const float r = 1.f / sqrtf(sum * (1.f / DC) + p.eps);
        if (lane < DC / 8) {
            Piece8<E> wt;
            wt.load(reinterpret_cast<const E *>(p.weight) + 8 * lane);
#pragma unroll
            for (int k = 0; k < 8; ++k) lat.x[k] *= r * wt.x[k];
        }
    }
    if (lane < DC / 8) lat.store(to + 8 * lane);
    if (lane < IPH) {
        turn(kx, ky);
        kx.store(to + DC + o0);
        ky.store(to + DC + o1);
    }
}

}  // namespace kda
