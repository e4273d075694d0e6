// One token of the gated delta rule per (batch, value head), the float32 state in place:
//   S~ = e^g S,  S <- S~ + b (v - S~ k) k^T,  o = scale (S~ q + b (v - S~ k) (k . q)).
// The state is read and written once (8 dk dv bytes a head) and nothing else counts, so HBM bounds a
// full batch and the launch bounds a single user.  A wave takes 4 value rows, 16 bytes of a row per
// lane, with every load issued before the first use; a work-group takes 16 rows, so one user's 32
// heads already make 256 work-groups.  256 users x 32 heads: 190 us for 1.08 GB, 5.7 TB/s; one user
// 3 us, less than the call's way through the host.
#pragma once
#include "gdr_common.h"
#include "kda_decode.h"

namespace kda {

struct GdrDecodeArgs {
    const void *q, *k, *v, *g, *beta;  // [B][Hk][dk], [B][Hk][dk], [B][H][dv], [B][H], [B][H]
    int H, r, dv;
    float scale;
    float *state;
    void *out;
};

template <int DK, bool F32>
__global__ __launch_bounds__(256) void gdr_decode_kernel(const GdrDecodeArgs p) {
    using E = typename std::conditional<F32, float, __bf16>::type;
    constexpr int LPR = DK / 4;                          // lanes per state row
    constexpr int RPI = 64 / LPR;                        // rows per wave-wide access
    constexpr int NI = kDecodeRowsPerWave / RPI;         // accesses per wave
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
    const float dec = ex2(to_f(reinterpret_cast<const E *>(p.g)[head]) * kLog2e);
    const float b = to_f(reinterpret_cast<const E *>(p.beta)[head]);
    float kq = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) kq += kc[j] * qc[j];
    kq = group_sum<LPR>(kq);
#pragma unroll
    for (int x = 0; x < NI; ++x) {
        float s[4], yk = 0.f, yq = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[j] = st[x][j] * dec;
            yk += s[j] * kc[j];
            yq += s[j] * qc[j];
        }
        yk = group_sum<LPR>(yk);
        yq = group_sum<LPR>(yq);
        const float d = b * (vr[x] - yk);
        f32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = fmaf(d, kc[j], s[j]);
        *reinterpret_cast<f32x4 *>(st0 + x * RPI * DK) = o;
        if (lane % LPR == 0)
            reinterpret_cast<E *>(p.out)[head * p.dv + row + RPI * x] = from_f<E>(p.scale * fmaf(d, kq, yq));
    }
}

}  // namespace kda
