// Instantiations and launcher of absorbed latent attention of drafted tokens.
#include <hip/hip_runtime.h>

#include "latent_launch.h"
#include "latent_tree.h"

namespace kda {

static long long rows(const LatentTreeLaunch &p) { return (long long)p.T * p.H; }
// column tiles of 16 rows a work-group takes (float32: the queries of 32 rows fill the registers)
static int tiles(const LatentTreeLaunch &p) {
    const int most = rows(p) <= 16 ? 1 : rows(p) <= 32 || p.fp32 ? 2 : 4;
    const long long keys = ((long long)p.max_pages * p.page + 63) / 64;
    for (int n = most; n > 1; n /= 2)
        if (p.B * ((rows(p) + 16 * n - 1) / (16 * n)) * keys >= 512) return n;
    return 1;
}
static int groups(const LatentTreeLaunch &p) { return (int)((rows(p) + 16 * tiles(p) - 1) / (16 * tiles(p))); }
// Work-groups that share all tiles evenly (latent_tree.h), one a CU, as long as the units alone do not fill
// the card four times over, and no more than there can be tiles; 0: one a unit.
static int shared(const LatentTreeLaunch &p) {
    const long long units = (long long)p.B * groups(p), most = units * (((long long)p.max_pages * p.page + 63) / 64);
    return units >= 1024 ? 0 : most < 256 ? (int)most : 256;
}
static size_t part_rows(const LatentTreeLaunch &p) { return 2 * (size_t)shared(p) * 16 * tiles(p); }
size_t latent_tree_bytes(const LatentTreeLaunch &p) {
    return shared(p) <= 1 ? 0 : part_rows(p) * (p.dc + 1) * 4 + ((size_t)p.B + 2) * 4;
}
bool latent_tree_grid_fits(const LatentTreeLaunch &p) {
    const long long units = (long long)p.B * groups(p), tiles = ((long long)p.max_pages * p.page + 63) / 64;
    return (units + 7) / 8 * 8 <= 4294967295LL / 256 && (units >= 1024 || units * tiles <= 2147483647LL);
}

template <int DC, bool F32, int NQ>
static hipError_t run(const LatentTreeLaunch &p) {
    LatentTreeArgs a{p.q, p.cache, p.table, p.lengths, p.counts, p.mask, p.B, p.T, p.H, p.pages, p.page, p.max_pages, groups(p),
                     p.scale, p.out, p.lse, shared(p), reinterpret_cast<float *>(p.workspace), nullptr, nullptr};
    if (a.groups == 1) a.groups = 0;  // one unit of one tile
    a.part_lse = a.part + part_rows(p) * DC;
    a.from = reinterpret_cast<int *>(a.part_lse + part_rows(p));
    const long long all = a.groups > 0 ? a.groups : (long long)p.B * a.rgroups;
    hipLaunchKernelGGL((latent_tree_kernel<DC, 64, F32, NQ>), dim3((unsigned)((all + 7) / 8 * 8)), dim3(256), 0, p.stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.groups == 0) return e;
    hipLaunchKernelGGL((latent_tree_join_kernel<DC, NQ, typename AttnOp<F32>::E>), dim3(a.groups, 16 * NQ * DC / 1024),
                       dim3(256), 0, p.stream, a);
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
