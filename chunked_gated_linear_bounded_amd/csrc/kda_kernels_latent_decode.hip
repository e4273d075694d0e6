// Instantiations and launcher of absorbed latent attention.
#include <hip/hip_runtime.h>

#include "latent_decode.h"
#include "latent_launch.h"

namespace kda {

// Four waves on 16 heads or on 32, eight on 64 (float32, whose registers do not allow eight: 32).
static int heads_per_group(const LatentLaunch &p) { return p.H <= 16 ? 16 : p.H <= 32 || p.fp32 ? 32 : 64; }
static int head_groups(const LatentLaunch &p) { return (p.H + heads_per_group(p) - 1) / heads_per_group(p); }
// Parts the keys are cut into: up to 512 work-groups, each with at least 64 keys of the longest sequence
// that the table can hold (the lengths are on the device), and 64 of one sequence, whom the join takes
// one after the other (latent_decode.h has the times): one user's 20,000 rows keep 64 CUs busy, no more.
static int splits(const LatentLaunch &p) {
    const long long want = 512 / ((long long)p.B * head_groups(p)), most = ((long long)p.max_pages * p.page + 63) / 64;
    const long long n = want < most ? want : most;
    return n < 1 ? 1 : (n > 64 ? 64 : (int)n);
}
size_t latent_decode_bytes(const LatentLaunch &p) {
    const int n = splits(p);
    return n == 1 ? 0 : (size_t)p.B * n * p.H * (p.dc + 1) * 4;
}

// a group of 64 heads is eight waves
bool latent_decode_grid_fits(const LatentLaunch &p) {
    const long long groups = ((long long)p.B * splits(p) + 7) / 8 * 8 * head_groups(p);
    return groups <= 4294967295LL / (heads_per_group(p) == 64 ? 512 : 256);
}

template <int DC, bool F32, int WS, int NW>
static hipError_t run(const LatentLaunch &p) {
    LatentDecodeArgs a{p.q, p.cache, p.table, p.lengths, p.B, p.H, p.pages, p.page, p.max_pages, splits(p), head_groups(p),
                       p.scale, p.out, p.lse, reinterpret_cast<float *>(p.workspace), nullptr};
    a.part_lse = a.part + (size_t)p.B * a.nsplit * p.H * DC;
    const unsigned grid = (unsigned)((p.B * a.nsplit + 7) / 8 * 8) * (unsigned)a.hgroups;
    hipLaunchKernelGGL((latent_decode_kernel<DC, 64, F32, WS, NW>), dim3(grid), dim3(64 * NW), 0, p.stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.nsplit == 1) return e;
    hipLaunchKernelGGL((latent_join_kernel<DC, typename AttnOp<F32>::E>), dim3(p.H, p.B), dim3(DC / 4), 0, p.stream, a);
    return hipGetLastError();
}
template <int DC, bool F32>
static hipError_t by_heads(const LatentLaunch &p) {
    const int heads = heads_per_group(p);
    if (heads == 16) return run<DC, F32, 4, 4>(p);
    if constexpr (!F32)
        if (heads == 64) return run<DC, F32, 2, 8>(p);
    return run<DC, F32, 2, 4>(p);
}
hipError_t launch_latent_decode(const LatentLaunch &p) {
    if (p.dc == 256) return p.fp32 ? by_heads<256, true>(p) : by_heads<256, false>(p);
    return p.fp32 ? by_heads<512, true>(p) : by_heads<512, false>(p);
}

}  // namespace kda
