// One token of decayed linear attention per (batch, value head), the float32 state in place:
//   S <- e^g S + v k^T,   o = scale S q.
// The state is read and written once (8 dk dv bytes a head), so HBM bounds a full batch and the launch a
// single user.  As in the gated delta rule's step a wave takes 4 value rows, 16 bytes of a row a lane,
// every load issued before the first use.  256 users x 32 heads of 128 x 128: 1.07 GB in 187 us, 5.7 TB/s.
#pragma once
#include "kda_decode.h"
#include "lin_common.h"

namespace kda {

struct LinDecodeArgs {
    const void *q, *k, *v, *g;  // [B][Hk][dk], [B][Hk][dk], [B][H][dv], [B][H]
    int H, r, dv;
    bool g32;
    float scale;
    float *state;
    void *out;
};

template <int DK, bool F32>
__global__ __launch_bounds__(256) void lin_decode_kernel(const LinDecodeArgs p) {
    using E = typename std::conditional<F32, float, __bf16>::type;
    constexpr int LPR = DK / 4, RPI = 64 / LPR, NI = kDecodeRowsPerWave / RPI;  // lanes a row, rows an access, accesses
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nb = p.dv / kDecodeRowsPerBlock;
    const size_t head = blockIdx.x / nb, key = (head / p.H) * (p.H / p.r) + (head % p.H) / p.r;
    const int c0 = 4 * (lane % LPR);
    const int row = (blockIdx.x % nb) * kDecodeRowsPerBlock + kDecodeRowsPerWave * wave + lane / LPR;
    float *st0 = p.state + (head * p.dv + row) * DK + c0;
    const E *vp = reinterpret_cast<const E *>(p.v) + head * p.dv + row;
    f32x4 st[NI];
    float vr[NI], kc[4], qc[4];
#pragma unroll
    for (int x = 0; x < NI; ++x) {
        st[x] = *reinterpret_cast<const f32x4 *>(st0 + x * RPI * DK);
        vr[x] = to_f(vp[RPI * x]);
    }
    load4(reinterpret_cast<const E *>(p.k) + key * DK + c0, kc);
    load4(reinterpret_cast<const E *>(p.q) + key * DK + c0, qc);
    const float dec = ex2(load_g(p.g, head, p.g32) * kLog2e);
#pragma unroll
    for (int x = 0; x < NI; ++x) {
        f32x4 s;
        float y = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[j] = fmaf(vr[x], kc[j], st[x][j] * dec);
            y += s[j] * qc[j];
        }
        y = group_sum<LPR>(y);
        *reinterpret_cast<f32x4 *>(st0 + x * RPI * DK) = s;
        if (lane % LPR == 0) reinterpret_cast<E *>(p.out)[head * p.dv + row + RPI * x] = from_f<E>(p.scale * y);
    }
}

}  // namespace kda
