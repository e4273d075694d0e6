// Instantiations and launchers of decayed linear attention's backward.
#include <hip/hip_runtime.h>

#include "lin_run.h"

namespace kda {

// Workspace: start states of the segments, forwards and backwards, and their decays; the two dot products a
// token that the decays' gradient is made of; where key heads are shared, the value heads' float32 partials
// of dq and dk; and, where the decays' gradient needs them, the sequences' end states.
struct LinBwdPlan {
    size_t units, state, states, tokens, part;
    size_t seg[2], decay[2], last, dots[2], parts[2], bytes;
    LinBwdPlan(const LinLaunch &p, bool end_states) {
        units = (size_t)p.B * p.H * lin_slots(p);
        state = (size_t)p.dk * p.dv;
        states = lin_all_states(p);
        tokens = (size_t)p.B * p.H * p.T;
        part = p.H == p.Hk ? 0 : tokens * p.dk;
        size_t at = 0;
        auto take = [&](size_t floats) {
            const size_t here = at;
            at += (floats * 4 + 255) / 256 * 256;
            return here;
        };
        for (int i = 0; i < 2; ++i) {
            seg[i] = take(states * state);
            decay[i] = take(units);
            dots[i] = take(tokens);
            parts[i] = take(part);
        }
        last = take(end_states ? (size_t)p.N * p.H * state : 0);
        bytes = at;
    }
};
size_t lin_bwd_bytes(const LinLaunch &p, bool end_states) { return LinBwdPlan(p, end_states).bytes; }

#define KDA_LAUNCH(...)                             \
    do {                                            \
        hipLaunchKernelGGL(__VA_ARGS__);            \
        const hipError_t e_ = hipGetLastError();    \
        if (e_ != hipSuccess) return e_;            \
    } while (0)

#define KDA_WALK(call)                  \
    do {                                \
        const hipError_t e_ = call;     \
        if (e_ != hipSuccess) return e_; \
    } while (0)

template <int DK, int DV, bool F32, bool DOT, bool SUM>
static hipError_t bwd_t(const LinLaunch &p) {
    using E = typename std::conditional<F32, float, __bf16>::type;
    const bool want_last = DOT && p.dfinal != nullptr, many = p.T > lin_segment(p);
    const LinBwdPlan m(p, want_last);
    auto f = [&](size_t at) { return reinterpret_cast<float *>(p.workspace + at); };
    const int r = p.H / p.Hk;
    const Strides3 sq = lin_st3(p.sq), sk = lin_st3(p.sk), sv = lin_st3(p.sv), sdo = lin_st3(p.sdo);
    const unsigned grid = lin_walk_grid(p);
    LinWalkArgs a = lin_walk_args(p);
    const dim3 block(256);
    // each segment's own part of the state, and of the gradient by it
    LinWalkArgs s0 = a, s1 = a;
    s0.b = p.k; s0.sb = sk; s0.rb = r; s0.c = p.v; s0.sc = sv;
    s0.seg = f(m.seg[0]);
    s0.seg_decay = f(m.decay[0]);
    s0.all = want_last;
    s0.final_state = f(m.last);
    s1.b = p.q; s1.sb = sq; s1.rb = r; s1.c = p.dout; s1.sc = sdo;
    s1.into = p.scale;
    s1.seg = f(m.seg[1]);
    s1.seg_decay = f(m.decay[1]);
    if (many && !F32) {
        if constexpr (!F32)
            KDA_WALK((lin_walks<LinOwnStates<DK, false>, LinOwnStates<DK, true>>(lin_walk_grid(p, DV / 64), p.stream, lin_in_parts<DV>(s0),
                                                                               lin_in_parts<DV>(s1))));
    } else {
        if (many || want_last) KDA_WALK((lin_own_states<DK, DV, F32, false>(p, s0)));
        if (many) KDA_WALK((lin_own_states<DK, DV, F32, true>(p, s1)));
    }
    if (many || want_last) {
        LinScanArgs s{a.seqs, p.B, p.H, a.nslot, a.nstate, DK * DV / 4, {}};
        s.side[0] = {p.init_state, f(m.seg[0]), want_last ? f(m.last) : nullptr, f(m.decay[0]), want_last};
        s.side[1] = {p.dfinal, many ? f(m.seg[1]) : nullptr, p.dinit, f(m.decay[1]), false};
        KDA_LAUNCH(lin_scan_kernel, dim3((unsigned)p.N * p.H * (DK * DV / 1024), 2), block, 0, p.stream, s);
    }
    // dq: forwards, with the transposed state
    LinWalkArgs wq = a, wk = a, wv = a;
    wq.a = p.dout; wq.sa = sdo;
    wq.b = p.v; wq.sb = sv;
    wq.c = p.k; wq.sc = sk; wq.rc = r;
    wq.y = p.q; wq.sy = sq; wq.ry = r;
    wq.inter = p.scale;
    wq.init = p.init_state;
    wq.seg = f(m.seg[0]);
    wq.dots = f(m.dots[0]);
    wq.out = SUM ? f(m.parts[0]) : p.dq;
    // dk and dv: backwards in time
    wk.a = p.v; wk.sa = sv;
    wk.b = p.dout; wk.sb = sdo;
    wk.c = p.q; wk.sc = sq; wk.rc = r;
    wk.y = p.k; wk.sy = sk; wk.ry = r;
    wk.into = p.scale;
    wk.init = p.dfinal;
    wk.seg = f(m.seg[1]);
    wk.dots = f(m.dots[1]);
    wk.out = SUM ? f(m.parts[1]) : p.dk_;
    wv.a = p.k; wv.sa = sk; wv.ra = r;
    wv.b = p.q; wv.sb = sq; wv.rb = r;
    wv.c = p.dout; wv.sc = sdo;
    wv.into = p.scale;
    wv.init = p.dfinal;
    wv.final_state = p.dinit;
    wv.seg = f(m.seg[1]);
    wv.out = p.dv_;
    if constexpr (F32) {
        KDA_WALK((lin_walk32<DV, DK, false, true, true, DOT>(wq, grid, p.stream)));
        KDA_WALK((lin_walk32<DV, DK, true, true, true, DOT>(wk, grid, p.stream)));
        KDA_WALK((lin_walk32<DK, DV, true, false, true, false>(wv, grid, p.stream)));
    } else {
        using Q = LinWalk<DV, DK, false, true, true, DOT, SUM>;
        using K = LinWalk<DV, DK, true, true, true, DOT, SUM>;
        using V = LinWalk<DK, DV, true, false, true, false, false>;
        KDA_WALK((lin_walks<Q, K, V>(grid, p.stream, wq, wk, wv)));
    }
    if (p.T == 0) return hipSuccess;
    LinFinish<E> z{};
    z.d = LinDecayGradArgs{a.seqs, p.B, p.H, a.nslot, a.nstate, DK * DV / 4, p.g32, f(m.seg[0]), f(m.seg[1]), f(m.last), p.dfinal,
                           f(m.dots[0]), f(m.dots[1]), p.dg};
    z.part[0] = f(m.parts[0]);
    z.part[1] = f(m.parts[1]);
    z.dq = static_cast<E *>(p.dq); z.dk = static_cast<E *>(p.dk_); z.dv = static_cast<E *>(p.dv_);
    z.r = r; z.Hk = p.Hk; z.H = p.H; z.DK = DK; z.DV = DV;
    z.n4 = (long long)p.T * DK / 4;
    z.all = z.n4 * p.B * p.Hk;
    z.grads = DOT ? (unsigned)m.units : 0;
    z.sums = SUM ? (unsigned)((z.all + 255) / 256) : 0;
    const unsigned blocks = (unsigned)lin_finish_grid(p, DOT);
    if (blocks > 0) KDA_LAUNCH((lin_finish_kernel<E>), dim3(blocks), block, 0, p.stream, z);
    return hipSuccess;
}
template <int DK, int DV, bool F32>
static hipError_t bwd_d(const LinLaunch &p) {
    if (p.dg) return p.H == p.Hk ? bwd_t<DK, DV, F32, true, false>(p) : bwd_t<DK, DV, F32, true, true>(p);
    return p.H == p.Hk ? bwd_t<DK, DV, F32, false, false>(p) : bwd_t<DK, DV, F32, false, true>(p);
}
template <bool F32>
static hipError_t bwd_io(const LinLaunch &p) {
    if (p.dk == 64) return p.dv == 64 ? bwd_d<64, 64, F32>(p) : bwd_d<64, 128, F32>(p);
    return p.dv == 64 ? bwd_d<128, 64, F32>(p) : bwd_d<128, 128, F32>(p);
}
hipError_t launch_lin_bwd(const LinLaunch &p) { return p.fp32 ? bwd_io<true>(p) : bwd_io<false>(p); }

}  // namespace kda
