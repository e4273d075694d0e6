// Instantiations and launcher of absorbed latent attention of drafted tokens.
#include <hip/hip_runtime.h>

#include "latent_launch.h"
#include "latent_tree.h"

namespace kda {

static long long rows(const LatentTreeLaunch &p) { return (long long)p.T * p.H; }
// column tiles of 16 rows a work-group takes (float32: the queries of 32 rows fill the registers)
static int tiles(const LatentTreeLaunch &p) { return rows(p) <= 16 ? 1 : rows(p) <= 32 || p.fp32 ? 2 : 4; }
static int groups(const LatentTreeLaunch &p) { return (int)((rows(p) + 16 * tiles(p) - 1) / (16 * tiles(p))); }
// parts the keys are cut into: up to 512 work-groups, each with at least 64 keys of the longest sequence
// that the table can hold (the lengths are on the device)
static int splits(const LatentTreeLaunch &p) {
    const long long want = 512 / ((long long)p.B * groups(p)), most = ((long long)p.max_pages * p.page + 63) / 64;
    const long long n = want < most ? want : most;
    return n < 1 ? 1 : (n > 64 ? 64 : (int)n);
}
size_t latent_tree_bytes(const LatentTreeLaunch &p) {
    const int n = splits(p);
    return n == 1 ? 0 : (size_t)p.B * n * rows(p) * (p.dc + 1) * 4;
}
bool latent_tree_grid_fits(const LatentTreeLaunch &p) {
    return ((long long)p.B * splits(p) * groups(p) + 7) / 8 * 8 <= 4294967295LL / 256 && p.B * rows(p) <= 4294967295LL / 128;
}

template <int DC, bool F32, int NQ>
static hipError_t run(const LatentTreeLaunch &p) {
    LatentTreeArgs a{p.q, p.cache, p.table, p.lengths, p.counts, p.mask, p.B, p.T, p.H, p.pages, p.page, p.max_pages, splits(p), groups(p),
                     p.scale, p.out, p.lse, reinterpret_cast<float *>(p.workspace), nullptr};
    a.part_lse = a.part + (size_t)p.B * a.nsplit * rows(p) * DC;
    const unsigned grid = (unsigned)((p.B * (long long)a.nsplit * a.rgroups + 7) / 8 * 8);
    hipLaunchKernelGGL((latent_tree_kernel<DC, 64, F32, NQ>), dim3(grid), dim3(256), 0, p.stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.nsplit == 1) return e;
    const long long joins = (p.B * rows(p) + 1024 / DC - 1) / (1024 / DC);
    hipLaunchKernelGGL((latent_tree_join_kernel<DC, typename AttnOp<F32>::E>), dim3((unsigned)joins), dim3(256), 0, p.stream, a);
    return hipGetLastError();
}
template <int DC, bool F32>
static hipError_t by_rows(const LatentTreeLaunch &p) {
    const int n = tiles(p);
    if (n == 1) return run<DC, F32, 1>(p);
    if constexpr (!F32)
        if (n == 4) return run<DC, F32, 4>(p);
    return run<DC, F32, 2>(p);
}
hipError_t launch_latent_tree(const LatentTreeLaunch &p) {
    if (p.dc == 256) return p.fp32 ? by_rows<256, true>(p) : by_rows<256, false>(p);
    return p.fp32 ? by_rows<512, true>(p) : by_rows<512, false>(p);
}

}  // namespace kda
