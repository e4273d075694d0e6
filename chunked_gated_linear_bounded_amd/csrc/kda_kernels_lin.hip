// Instantiations and launchers of decayed linear attention's forward and one-token step.
#include <hip/hip_runtime.h>

#include "lin_decode.h"
#include "lin_launch.h"
#include "lin_run.h"

namespace kda {

size_t lin_fwd_bytes(const LinLaunch &p) {
    if (p.T <= lin_segment(p)) return 0;  // every sequence is one segment
    const size_t units = (size_t)p.B * p.H * lin_slots(p);
    return lin_all_states(p) * p.dk * p.dv * 4 + (units * 4 + 15) / 16 * 16;
}

template <int DK, int DV, bool F32>
static hipError_t fwd_t(const LinLaunch &p) {
    LinWalkArgs a = lin_walk_args(p);
    a.a = p.q; a.sa = lin_st3(p.sq); a.ra = p.H / p.Hk;
    a.b = p.k; a.sb = lin_st3(p.sk); a.rb = p.H / p.Hk;
    a.c = p.v; a.sc = lin_st3(p.sv); a.rc = 1;
    a.inter = p.scale;
    a.into = 1.f;
    a.init = p.init_state;
    a.final_state = p.final_state;
    a.out = p.out;
    const unsigned grid = lin_walk_grid(p);
    if (p.T > a.seqs.seg) {
        a.seg = reinterpret_cast<float *>(p.workspace);
        a.seg_decay = a.seg + lin_all_states(p) * DK * DV;
        hipError_t e = lin_own_states<DK, DV, F32, false>(p, a);
        if (e != hipSuccess) return e;
        LinScanArgs s{a.seqs, p.B, p.H, a.nslot, a.nstate, DK * DV / 4, {{p.init_state, a.seg, p.final_state, a.seg_decay, false}, {}}};
        hipLaunchKernelGGL(lin_scan_kernel, dim3((unsigned)p.N * p.H * (DK * DV / 1024)), dim3(256), 0, p.stream, s);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if constexpr (F32) return lin_walk32<DK, DV, false, false, true, false>(a, grid, p.stream);
    else return lin_walks<LinWalk<DK, DV, false, false, true, false, false>>(grid, p.stream, a);
}

template <bool F32>
static hipError_t fwd_io(const LinLaunch &p) {
    if (p.dk == 64) return p.dv == 64 ? fwd_t<64, 64, F32>(p) : fwd_t<64, 128, F32>(p);
    return p.dv == 64 ? fwd_t<128, 64, F32>(p) : fwd_t<128, 128, F32>(p);
}
hipError_t launch_lin_fwd(const LinLaunch &p) { return p.fp32 ? fwd_io<true>(p) : fwd_io<false>(p); }

hipError_t launch_lin_decode(const LinLaunch &p) {
    const LinDecodeArgs a{p.q, p.k, p.v, p.g, p.H, p.H / p.Hk, p.dv, p.g32, p.scale, p.state, p.out};
    const dim3 grid((unsigned)p.B * p.H * (p.dv / kDecodeRowsPerBlock));
    if (p.dk == 64) {
        if (p.fp32) hipLaunchKernelGGL((lin_decode_kernel<64, true>), grid, dim3(256), 0, p.stream, a);
        else hipLaunchKernelGGL((lin_decode_kernel<64, false>), grid, dim3(256), 0, p.stream, a);
    } else {
        if (p.fp32) hipLaunchKernelGGL((lin_decode_kernel<128, true>), grid, dim3(256), 0, p.stream, a);
        else hipLaunchKernelGGL((lin_decode_kernel<128, false>), grid, dim3(256), 0, p.stream, a);
    }
    return hipGetLastError();
}

}  // namespace kda
