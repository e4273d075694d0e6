// Instantiations and launcher of the writer of the paged latent cache.
#include <hip/hip_runtime.h>

#include "latent_append.h"
#include "latent_launch.h"

namespace kda {

static long long units(const LatentAppendLaunch &p) {
    const long long parts = p.H > 0 ? (p.H + kAppendHeads - 1) / kAppendHeads : 1;
    return (long long)p.B * p.T * parts;
}
bool latent_append_grid_fits(const LatentAppendLaunch &p) { return (units(p) + 3) / 4 <= 4294967295LL / 256; }

template <int DC, bool F32>
static hipError_t run(const LatentAppendLaunch &p) {
    LatentAppendArgs a{p.latent, p.kr, p.qr, p.weight, {p.sl[0], p.sl[1]}, {p.sk[0], p.sk[1]}, {p.sq[0], p.sq[1], p.sq[2]}, p.cache, p.q,
                       p.table, p.lengths, p.positions, p.counts, p.cu, p.freqs, p.N, p.B, p.T, p.H,
                       p.H > 0 ? (p.H + kAppendHeads - 1) / kAppendHeads : 1, p.pages, p.page, p.max_pages, p.eps};
    const dim3 grid((unsigned)((units(p) + 3) / 4));
    if (p.interleaved) hipLaunchKernelGGL((latent_append_kernel<DC, 64, F32, true>), grid, dim3(256), 0, p.stream, a);
    else hipLaunchKernelGGL((latent_append_kernel<DC, 64, F32, false>), grid, dim3(256), 0, p.stream, a);
    return hipGetLastError();
}
hipError_t launch_latent_append(const LatentAppendLaunch &p) {
    if (p.dc == 256) return p.fp32 ? run<256, true>(p) : run<256, false>(p);
    return p.fp32 ? run<512, true>(p) : run<512, false>(p);
}

}  // namespace kda
