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

}  // namespace kda
