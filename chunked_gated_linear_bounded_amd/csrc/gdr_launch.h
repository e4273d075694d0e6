// Internal interface between the host side of the gated delta rule's entry points (kda_abi_gdr.cpp)
// and its kernels.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stddef.h>

namespace kda {

struct GdrLaunch {
    const void *q, *k, *v, *g, *beta;
    long long sq[3], sk[3], sv[3], sg[3], sb[3];  // element strides b, h, t
    const int *cu;                                // NULL: fixed-length batch
    int N, B, Hk, H, T, dk, dv;                   // sequences; batch entries (1 when packed)
    bool fp32;
    float scale;
    void *out;
    float *final_state;
    const float *init_state;
    float *state;                                 // one-token step
    unsigned char *workspace;
    hipStream_t stream;
    // backward
    const void *dout;
    long long sdo[3];
    const float *dfinal;
    void *dq, *dk_, *dv_, *dg, *dbeta;
    float *dinit;
};

// chunk slots of one batch entry, and the bytes of the forward's and the backward's workspace
int gdr_slots(const GdrLaunch &p);
size_t gdr_fwd_bytes(const GdrLaunch &p);
size_t gdr_bwd_bytes(const GdrLaunch &p);

hipError_t launch_gdr_fwd(const GdrLaunch &p);
hipError_t launch_gdr_bwd(const GdrLaunch &p);
hipError_t launch_gdr_decode(const GdrLaunch &p);

// The sequential stages take 32 columns a work-group in place of 16 once those of 16 outnumber the
// places for them: one a CU, or two where two fit (dk = 64, bf16).  Packed documents are ragged, a short
// one's place is soon free, and two a CU still run faster than fewer, longer steps.  Microseconds of the
// state stage and the reverse pass, 16 columns / 32: 5 sequences of 1024 x 12 heads (480 work-groups of
// 16), dk = 128: 51 and 80 / 42 and 60, dk = 64: 36 and 53 / 36 and 50; 11 documents of 5000 tokens x 4
// heads (352), dk = 128: 37 and 60 / 59 and 82, dk = 64: 23 and 36 / 33 and 47; 32 documents of 12,000
// tokens x 8 heads (2048), dk = 128: 99 and 161 / 79 and 119.  Lengths are on the device, so documents of
// one length get the ragged ones' choice: at 257 to 512 work-groups and dk = 128 the first line's loss.
inline bool gdr_two_tiles(const GdrLaunch &p) {
    const long long places = p.cu != nullptr || (p.dk == 64 && !p.fp32) ? 512 : 256;
    return (long long)p.N * p.H * (p.dv / 16) > places;
}

// Whether the launches of a call stay below 2^32 work-items in x, which is as far as a launch goes.
inline bool gdr_grids_fit(const GdrLaunch &p, bool backward) {
    const long long most = 4294967295LL, packed = p.cu != nullptr, units = ((long long)p.N * p.H + 7) / 8 * 8;
    const long long slots = packed ? (long long)p.T / 64 + p.N : ((long long)p.T + 63) / 64;
    const int columns = !gdr_two_tiles(p) || (backward && p.fp32 && p.dk == 128) ? 16 : 32;
    return slots * (backward ? 512 : 256) <= most && units * (p.dv / columns) * 512 <= most;
}
inline bool gdr_decode_grid_fits(const GdrLaunch &p) { return (long long)p.B * p.H * (p.dv / 16) * 256 <= 4294967295LL; }

}  // namespace kda
