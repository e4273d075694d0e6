// Instantiations and launcher of absorbed latent attention of drafted tokens.
#include <hip/hip_runtime.h>

#include "latent_launch.h"
#include "latent_tree.h"

namespace kda {

static long long rows(const LatentTreeLaunch &p) { return (long long)p.T * p.H; }
static long long key_tiles(const LatentTreeLaunch &p) { return ((long long)p.max_pages * p.page + 63) / 64; }
// Column tiles of 16 rows a work-group takes: as many as there are rows for (float32: the queries of 32 rows fill
// the registers), because a fragment of keys is read once for all of them (24 sequences x 8 tokens x 128
// heads on 4500 to 9000 rows: 424 us with four, 593 with two); fewer where there would not be two tiles of keys for
// every CU (a call on 3 x 5 x 16 on up to 700: 20 us with one, 26 with two, 37 with four; 8 x 4 x 16 on up to 1500: 29
// with one, 37 with two).
static int tiles(const LatentTreeLaunch &p) {
    const int most = rows(p) <= 16 ? 1 : rows(p) <= 32 || p.fp32 ? 2 : 4;
    for (int n = most; n > 1; n /= 2)
        if (p.B * ((rows(p) + 16 * n - 1) / (16 * n)) * key_tiles(p) >= 512) return n;
    return 1;
}
static int groups(const LatentTreeLaunch &p) { return (int)((rows(p) + 16 * tiles(p) - 1) / (16 * tiles(p))); }
// Work-groups that share all tiles evenly (latent_tree.h), one a CU and no more than there can be tiles; 0: one a
// unit.  Pieces cost their float32 values written and read again and a launch, as much as some 24 tiles of 64
// rows; units of their own leave CUs idle in the last round.  Histories of half to all of the longest, shared
// against a unit each: 384 units on 9000 rows 394 to 430 us against 461 to 478, 24 x 8 x 128 all on 9000 511 against 605;
// 256 units on 3000 148 and 108, 512 units 242 and 194; 1 x 1 x 16 on 40,000 97 and 980.  Four rounds even out by
// themselves (1,008 units on up to 1000 keys 416 and 181).  Tiles of fewer rows are as much shorter.
// What a unit costs to begin and end is not counted, and the lengths are not known here: with histories from next to
// nothing on, where a work-group's share can be many short units, sharing is the worse (384 units on 8 to 9000 rows:
// 603 us against 375).  float32 tiles are eight times as long, and uneven lengths cost more than pieces: 256 units of 32
// rows on up to 2000 keys 258 us shared, 279 a unit each.
static int shared(const LatentTreeLaunch &p) {
    const long long units = (long long)p.B * groups(p), idle = ((units + 255) / 256 * 256 - units) * key_tiles(p) / 256;
    const long long most = units * key_tiles(p);
    if (units >= 1024 || most == 1 || (!p.fp32 && idle < 6 * tiles(p))) return 0;
    return most < 256 ? (int)most : 256;
}
static size_t part_rows(const LatentTreeLaunch &p) { return 2 * (size_t)shared(p) * 16 * tiles(p); }
size_t latent_tree_bytes(const LatentTreeLaunch &p) {
    return shared(p) == 0 ? 0 : part_rows(p) * (p.dc + 1) * 4 + ((size_t)p.B + 2) * 4;
}
bool latent_tree_grid_fits(const LatentTreeLaunch &p) {
    const long long units = (long long)p.B * groups(p);
    return (units + 7) / 8 * 8 <= 4294967295LL / 256 && (shared(p) == 0 || units * key_tiles(p) <= 2147483647LL);
}

template <int DC, bool F32, int NQ>
static hipError_t run(const LatentTreeLaunch &p) {
    LatentTreeArgs a{p.q, p.cache, p.table, p.lengths, p.counts, p.mask, p.B, p.T, p.H, p.pages, p.page, p.max_pages, groups(p),
                     p.scale, p.out, p.lse, shared(p), reinterpret_cast<float *>(p.workspace), nullptr, nullptr};
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
