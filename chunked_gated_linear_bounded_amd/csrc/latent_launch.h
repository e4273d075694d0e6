// Internal interface between the host side of latent attention's entry points (kda_abi_latent.cpp)
// and its kernels.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stddef.h>

namespace kda {

struct LatentLaunch {
    const void *q, *k, *kr, *v;
    long long sq[3], sk[3], skr[3], sv[3];  // element strides b, h, t (kr: h unused)
    const int *cu_q, *cu_k;                 // NULL: fixed-length batch
    int N, B, H, T, S, dn, dr;
    bool fp32, packed;
    float scale;
    void *out;
    float *lse;
    unsigned char *workspace;
    hipStream_t stream;
    // backward
    const void *fwd_out, *dout;
    const float *fwd_lse;
    long long sdo[3];
    void *dq, *dk, *dkr, *dv;
    // absorbed one-token step: q [B][H][dc + dr] against the paged cache
    const void *cache;
    const int *table, *lengths;
    int pages, page, max_pages, dc;
};

// Whether a call's launches stay below 2^32 work-items in x, which is as far as a launch goes.
inline bool latent_grids_fit(const LatentLaunch &p, bool backward) {
    const long long most = 4294967295LL, units = ((long long)p.B * p.H + 7) / 8 * 8, rows = backward && p.fp32 ? 64 : 128;
    auto fits = [&](long long total) {
        const long long tiles = p.packed ? total / rows + p.N : (total + rows - 1) / rows;
        return units * tiles <= most / (backward ? 512 : 256);
    };
    return fits(p.T) && (!backward || fits(p.S));
}
size_t latent_bwd_bytes(const LatentLaunch &p);
hipError_t launch_latent_fwd(const LatentLaunch &p);
hipError_t launch_latent_bwd(const LatentLaunch &p);

bool latent_decode_grid_fits(const LatentLaunch &p);
size_t latent_decode_bytes(const LatentLaunch &p);
hipError_t launch_latent_decode(const LatentLaunch &p);

// new tokens into the paged cache, and their queries' rotary part
struct LatentAppendLaunch {
    const void *latent, *kr, *qr, *weight;
    long long sl[2], sk[2], sq[3];  // element strides b, t (qr: and head)
    void *cache, *q;
    const int *table, *lengths, *positions, *counts, *cu;
    const float *freqs;
    int N, B, T, H, pages, page, max_pages, dc;  // H 0: no queries
    bool fp32, interleaved;
    float eps;
    hipStream_t stream;
};
bool latent_append_grid_fits(const LatentAppendLaunch &p);
hipError_t launch_latent_append(const LatentAppendLaunch &p);

// drafted tokens against the paged cache: q, out [B][T][H][..], lse [B][T][H]
struct LatentTreeLaunch {
    const void *q, *cache;
    const int *table, *lengths, *counts;
    const unsigned long long *mask;  // [B][T]
    int B, T, H, pages, page, max_pages, dc;
    bool fp32;
    float scale;
    void *out;
    float *lse;
    unsigned char *workspace;
    hipStream_t stream;
};
bool latent_tree_grid_fits(const LatentTreeLaunch &p);
size_t latent_tree_bytes(const LatentTreeLaunch &p);
hipError_t launch_latent_tree(const LatentTreeLaunch &p);

}  // namespace kda
