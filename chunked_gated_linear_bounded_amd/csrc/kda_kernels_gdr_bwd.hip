// Instantiations and launcher of the gated delta rule's backward: the chunk stage and the state
// stage again (keeping every chunk's start state and U), the reverse pass, the gradient stage.
#include <hip/hip_runtime.h>

#include "gdr_chunk.h"
#include "gdr_grad.h"
#include "gdr_launch.h"
#include "gdr_rev.h"
#include "gdr_state.h"

namespace kda {

static Strides3 st3(const long long (&s)[3]) { return Strides3{s[0], s[1], s[2]}; }

// workspace: key records, value records, what the forward pass keeps, what the reverse pass keeps
struct BwdPlan {
    size_t keys, vals, save, total;
};
static BwdPlan plan(const GdrLaunch &p) {
    const int ni = p.fp32 ? 2 : 1;
    const GdrLayout L{ni, p.dk, 2};
    const GdrSave S{ni, p.dk};
    const size_t slots = (size_t)p.B * gdr_slots(p);
    BwdPlan r;
    r.keys = slots * p.Hk * L.key_bytes();
    r.vals = slots * p.H * L.val_bytes();
    r.save = slots * p.H * (p.dv / 16) * S.bytes();
    r.total = r.keys + r.vals + 2 * r.save;
    return r;
}
size_t gdr_bwd_bytes(const GdrLaunch &p) { return plan(p).total; }

template <int DK, bool F32, int NCT>
static hipError_t passes(const GdrLaunch &p, const GdrStateArgs &a, const GdrRevArgs &c) {
    constexpr int NR = F32 && DK == 128 ? 1 : NCT;  // two float32 tiles would need 170 KiB of LDS
    const int units = (p.N * p.H + 7) / 8 * 8;
    hipLaunchKernelGGL((gdr_state_kernel<DK, F32, NCT, 1, 2>), dim3(units * (p.dv / 16 / NCT)), dim3(512), 0, p.stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((gdr_rev_kernel<DK, F32, NR>), dim3(units * (p.dv / 16 / NR)), dim3(512), 0, p.stream, c);
    return hipGetLastError();
}

template <int DK, bool F32>
static hipError_t bwd_t(const GdrLaunch &p) {
    using E = typename std::conditional<F32, float, __bf16>::type;
    const int r = p.H / p.Hk, nslot = gdr_slots(p);
    const GdrSeqs seqs{p.cu, p.N, p.T};
    const BwdPlan w = plan(p);
    unsigned char *keys = p.workspace, *vals = keys + w.keys, *fwd = vals + w.vals, *rev = fwd + w.save;
    hipError_t e;
    if (p.T > 0) {
        const GdrChunkArgs a{p.q, p.k, p.g, p.beta, st3(p.sq), st3(p.sk), st3(p.sg), st3(p.sb), seqs,
                             p.Hk, r, nslot, p.scale, keys, vals};
        hipLaunchKernelGGL((gdr_chunk_kernel<DK, F32, 2>), dim3(nslot, p.H, p.B), dim3(256), 0, p.stream, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const GdrStateArgs a{keys, vals, p.v, st3(p.sv), seqs, p.H, r, nslot, p.dv, p.scale, nullptr, p.init_state, nullptr, fwd};
    const GdrRevArgs c{keys, vals, p.dout, st3(p.sdo), seqs, p.H, r, nslot, p.dv, p.scale, p.dfinal, p.dinit, p.dv_, rev};
    e = gdr_two_tiles(p) ? passes<DK, F32, 2>(p, a, c) : passes<DK, F32, 1>(p, a, c);
    if (e != hipSuccess || p.T == 0) return e;
    const GdrGradArgs d{keys, vals, p.v, p.g, p.dout, st3(p.sv), st3(p.sg), st3(p.sdo), seqs, p.Hk, r, nslot, p.scale,
                        fwd, rev, p.dq, p.dk_, p.dg, p.dbeta};
    if (p.dv == 64) hipLaunchKernelGGL((gdr_grad_kernel<DK, 64, F32>), dim3(nslot, p.Hk, p.B), dim3(512), 0, p.stream, d);
    else hipLaunchKernelGGL((gdr_grad_kernel<DK, 128, F32>), dim3(nslot, p.Hk, p.B), dim3(512), 0, p.stream, d);
    if ((e = hipGetLastError()) != hipSuccess || p.cu == nullptr) return e;
    hipLaunchKernelGGL((gdr_uncovered_kernel<E>), dim3(16, p.H), dim3(256), 0, p.stream, seqs, p.Hk, p.H, p.dk, p.dv,
                       (E *)p.dq, (E *)p.dk_, (E *)p.dv_, (E *)p.dg, (E *)p.dbeta);
    return hipGetLastError();
}

hipError_t launch_gdr_bwd(const GdrLaunch &p) {
    if (p.dk == 64) return p.fp32 ? bwd_t<64, true>(p) : bwd_t<64, false>(p);
    return p.fp32 ? bwd_t<128, true>(p) : bwd_t<128, false>(p);
}

}  // namespace kda
