// Internal interface between the host side of decayed linear attention's entry points
// (kda_abi_lin.cpp) and its kernels.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stddef.h>

namespace kda {

struct LinLaunch {
    const void *q, *k, *v, *g;
    long long sq[3], sk[3], sv[3], sg[3];  // element strides b, h, t
    const int *cu;                         // NULL: fixed-length batch
    int N, B, Hk, H, T, dk, dv;            // sequences; batch entries (1 when packed)
    bool fp32, g32, packed;                // g32: g (and dg) in float32
    float scale;
    void *out;
    float *final_state;
    const float *init_state;
    float *state;                          // one-token step
    unsigned char *workspace;
    hipStream_t stream;
    // backward
    const void *dout;
    long long sdo[3];
    const float *dfinal;
    void *dq, *dk_, *dv_, *dg;             // dg NULL: not wanted
    float *dinit;
};

// Tokens of a segment, the piece of a sequence that one work-group walks through, and the segments of
// one batch entry.
inline int lin_segment(const LinLaunch &p) {
    const long long chunks = (((long long)p.T + 63) / 64) * p.B * p.H, most = p.fp32 ? 512 : 256;
    long long per = (chunks + most - 1) / most;
    per = per < 4 ? 4 : (per > 4096 ? 4096 : per);
    return (int)per * 64;
}
inline long long lin_slots(const LinLaunch &p) {
    const long long seg = lin_segment(p), n = p.packed ? p.T / seg + p.N : (p.T + seg - 1) / seg;
    return n < 1 ? 1 : n;
}
size_t lin_fwd_bytes(const LinLaunch &p);
size_t lin_bwd_bytes(const LinLaunch &p);

hipError_t launch_lin_fwd(const LinLaunch &p);
hipError_t launch_lin_bwd(const LinLaunch &p);
hipError_t launch_lin_decode(const LinLaunch &p);

// Whether the launches of a call stay below 2^32 work-items in x, which is as far as a launch goes, and
// their unit counts in 32 bits.
inline bool lin_grids_fit(const LinLaunch &p) {
    const long long most = 4294967295LL, units = (long long)p.B * p.H * lin_slots(p);
    const long long states = (long long)p.N * p.H * (p.dk * p.dv / 1024);
    const long long rows = (long long)p.B * p.H * (((long long)p.T + 15) / 16);
    return (units + 7) / 8 * 8 <= most / 256 && states <= most / 256 && rows <= most / 256;
}
inline bool lin_decode_grid_fits(const LinLaunch &p) { return (long long)p.B * p.H * (p.dv / 16) * 256 <= 4294967295LL; }

}  // namespace kda
