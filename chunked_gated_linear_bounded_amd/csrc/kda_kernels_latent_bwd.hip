// Instantiations and launchers of expanded latent attention, backward.
#include <hip/hip_runtime.h>

#include "gdr_chunk.h"
#include "latent_bwd.h"
#include "latent_launch.h"

namespace kda {

static Strides3 st3(const long long (&s)[3]) { return Strides3{s[0], s[1], s[2]}; }
static unsigned grid_of(int units, int tiles) { return (unsigned)((units + 7) / 8 * 8) * (unsigned)tiles; }

// workspace: delta [B][H][T], then the partials of dk_rope [B][H][S][dr], float32
static size_t delta_bytes(const LatentLaunch &p) { return ((size_t)p.B * p.H * p.T * 4 + 255) / 256 * 256; }
size_t latent_bwd_bytes(const LatentLaunch &p) { return delta_bytes(p) + (size_t)p.B * p.H * p.S * p.dr * 4; }

template <int DN, int DR, bool F32>
static hipError_t bwd_t(const LatentLaunch &p) {
    using E = typename AttnOp<F32>::E;
    constexpr int BT = F32 ? 64 : 128;
    const bool packed = p.cu_q != nullptr;
    const AttnSeqs seqs{p.cu_q, p.cu_k, p.N, p.T, p.S};
    float *delta = reinterpret_cast<float *>(p.workspace), *part = reinterpret_cast<float *>(p.workspace + delta_bytes(p));
    LatentBwdArgs a{p.q, p.k, p.kr, p.v, p.fwd_out, p.dout, st3(p.sq), st3(p.sk), st3(p.skr), st3(p.sv), st3(p.sdo),
                    seqs, p.H, p.B, 0, p.scale, p.fwd_lse, delta, p.dq, p.dk, p.dv, part};
    hipError_t e = hipSuccess;
    if (p.T > 0) {
        a.ntile = AttnSeqs::tiles(packed, p.N, p.T, BT);
        hipLaunchKernelGGL((latent_dq_kernel<DN, DR, F32>), dim3(grid_of(p.B * p.H, a.ntile)), dim3(512), 0, p.stream, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (p.S > 0) {
        a.ntile = AttnSeqs::tiles(packed, p.N, p.S, BT);
        hipLaunchKernelGGL((latent_dkv_kernel<DN, DR, F32>), dim3(grid_of(p.B * p.H, a.ntile)), dim3(512), 0, p.stream, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        hipLaunchKernelGGL((latent_dkr_kernel<E>), dim3((unsigned)(((long long)p.S * DR / 4 + 255) / 256), p.B), dim3(256), 0,
                           p.stream, part, seqs, p.H, DR, (E *)p.dkr);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (packed) {
        const dim3 grid(16, p.H);
        if (p.T > 0)
            hipLaunchKernelGGL((latent_uncovered_kernel<E>), grid, dim3(256), 0, p.stream, p.cu_q, p.N, p.T, DN + DR, (E *)p.dq);
        if (p.S > 0) {
            hipLaunchKernelGGL((latent_uncovered_kernel<E>), grid, dim3(256), 0, p.stream, p.cu_k, p.N, p.S, DN, (E *)p.dk);
            hipLaunchKernelGGL((latent_uncovered_kernel<E>), grid, dim3(256), 0, p.stream, p.cu_k, p.N, p.S, DN, (E *)p.dv);
        }
        e = hipGetLastError();
    }
    return e;
}

template <bool F32>
static hipError_t dispatch(const LatentLaunch &p) {
    if (p.dn == 64) return p.dr == 32 ? bwd_t<64, 32, F32>(p) : bwd_t<64, 64, F32>(p);
    return p.dr == 32 ? bwd_t<128, 32, F32>(p) : bwd_t<128, 64, F32>(p);
}
hipError_t launch_latent_bwd(const LatentLaunch &p) {
    return p.fp32 ? dispatch<true>(p) : dispatch<false>(p);
}

}  // namespace kda
