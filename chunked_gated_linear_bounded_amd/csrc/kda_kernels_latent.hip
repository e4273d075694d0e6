// Instantiations and launcher of expanded latent attention, forward.
#include <hip/hip_runtime.h>

#include "latent_fwd.h"
#include "latent_launch.h"

namespace kda {

static Strides3 st3(const long long (&s)[3]) { return Strides3{s[0], s[1], s[2]}; }
static unsigned grid_of(int units, int tiles) { return (unsigned)((units + 7) / 8 * 8) * (unsigned)tiles; }

template <int DN, int DR, bool F32>
static hipError_t fwd_t(const LatentLaunch &p) {
    const int nt = AttnSeqs::tiles(p.cu_q != nullptr, p.N, p.T, 128);
    const LatentFwdArgs a{p.q, p.k, p.kr, p.v, st3(p.sq), st3(p.sk), st3(p.skr), st3(p.sv),
                          AttnSeqs{p.cu_q, p.cu_k, p.N, p.T, p.S}, p.H, p.B, nt, p.scale, p.out, p.lse};
    const dim3 grid(grid_of(p.B * p.H, nt));
    if (!F32 && grid.x <= 512)  // two on each CU: see latent_fwd.h
        hipLaunchKernelGGL((latent_fwd_kernel<DN, DR, F32, F32 ? 1 : 2>), grid, dim3(F32 ? 256 : 512), 0, p.stream, a);
    else
        hipLaunchKernelGGL((latent_fwd_kernel<DN, DR, F32, 1>), grid, dim3(256), 0, p.stream, a);
    return hipGetLastError();
}

template <bool F32>
static hipError_t dispatch(const LatentLaunch &p) {
    if (p.dn == 64) return p.dr == 32 ? fwd_t<64, 32, F32>(p) : fwd_t<64, 64, F32>(p);
    return p.dr == 32 ? fwd_t<128, 32, F32>(p) : fwd_t<128, 64, F32>(p);
}
hipError_t launch_latent_fwd(const LatentLaunch &p) { return p.fp32 ? dispatch<true>(p) : dispatch<false>(p); }

}  // namespace kda
