// What the launchers of decayed linear attention's forward and backward share.
#pragma once
#include "lin_launch.h"
#include "lin_scan.h"
#include "lin_walk.h"

namespace kda {

inline Strides3 lin_st3(const long long (&s)[3]) { return Strides3{s[0], s[1], s[2]}; }

inline LinWalkArgs lin_walk_args(const LinLaunch &p) {
    LinWalkArgs a{};
    a.g = p.g;
    a.sg = lin_st3(p.sg);
    a.g32 = p.g32;
    a.ra = a.rb = a.rc = a.ry = 1;
    a.seqs = LinSeqs{p.cu, p.N, p.T, lin_segment(p), lin_sparse(p)};
    a.B = p.B;
    a.H = p.H;
    a.nslot = (int)lin_slots(p);
    a.nstate = (int)lin_states(p);
    a.scale = p.scale;
    a.inter = a.into = 1.f;
    a.parts = 1;
    return a;
}
inline unsigned lin_walk_grid(const LinLaunch &p, int parts = 1) {
    return (unsigned)(((long long)p.B * p.H * lin_slots(p) * parts + 7) / 8 * 8);
}

template <typename... W, typename... A>
inline hipError_t lin_walks(unsigned grid, hipStream_t stream, const A &...a) {
    static_assert(sizeof...(W) == sizeof...(A), "a walk's arguments each");
    hipLaunchKernelGGL((lin_pair_kernel<W...>), dim3(grid, sizeof...(W)), dim3(512), 0, stream, LinWalkList<sizeof...(W)>{{a...}});
    return hipGetLastError();
}
// float32's walks, one a launch
template <int DA, int DC, bool REV, bool TR, bool OUT, bool DOT>
inline hipError_t lin_walk32(const LinWalkArgs &a, unsigned grid, hipStream_t stream) {
    hipLaunchKernelGGL((lin_walk32_kernel<DA, DC, REV, TR, OUT, DOT>), dim3(grid), dim3(256), 0, stream, a);
    return hipGetLastError();
}

// Pass 1, the segments' own states.  In bf16 work-groups of 64 of c's channels: they read b twice, from the
// second's neighbour's L2, but two of them share a CU (64k x 32 heads 797 us a call against 808, the training step
// of 2 x 4096 x 16 heads 314 against 319).
template <int DA, bool REV> using LinOwnStates = LinWalk<DA, 64, REV, false, false, false, false>;
template <int DC>
inline LinWalkArgs lin_in_parts(LinWalkArgs a) {
    a.parts = DC / 64;
    return a;
}
template <int DA, int DC, bool F32, bool REV>
inline hipError_t lin_own_states(const LinLaunch &p, const LinWalkArgs &a) {
    if constexpr (F32) return lin_walk32<DA, DC, REV, false, false, false>(a, lin_walk_grid(p), p.stream);
    else return lin_walks<LinOwnStates<DA, REV>>(lin_walk_grid(p, DC / 64), p.stream, lin_in_parts<DC>(a));
}

}  // namespace kda
