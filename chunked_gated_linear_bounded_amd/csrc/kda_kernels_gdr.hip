// Instantiations and launchers of the gated delta rule's forward and one-token step.
#include <hip/hip_runtime.h>

#include "gdr_chunk.h"
#include "gdr_decode.h"
#include "gdr_launch.h"
#include "gdr_state.h"

namespace kda {

static Strides3 st3(const long long (&s)[3]) { return Strides3{s[0], s[1], s[2]}; }

int gdr_slots(const GdrLaunch &p) {
    return p.cu != nullptr ? p.T / kGdrChunk + p.N : (p.T + kGdrChunk - 1) / kGdrChunk;
}

static size_t key_part(const GdrLaunch &p, const GdrLayout &L) { return (size_t)p.B * p.Hk * gdr_slots(p) * L.key_bytes(); }

size_t gdr_fwd_bytes(const GdrLaunch &p) {
    const GdrLayout L{p.fp32 ? 2 : 1, p.dk, p.fp32 ? 2 : 1};
    return key_part(p, L) + (size_t)p.B * p.H * gdr_slots(p) * L.val_bytes();
}

template <int DK, bool F32, int NCT>
static hipError_t run_state(const GdrStateArgs &a, hipStream_t stream) {
    const int units = (a.seqs.N * a.H + 7) / 8 * 8;
    hipLaunchKernelGGL((gdr_state_kernel<DK, F32, NCT, 0, F32 ? 2 : 1>), dim3(units * (a.dv / 16 / NCT)), dim3(512), 0, stream, a);
    return hipGetLastError();
}

template <int DK, bool F32>
static hipError_t fwd_t(const GdrLaunch &p) {
    constexpr int MP = F32 ? 2 : 1;
    constexpr GdrLayout L{MP, DK, MP};
    const int r = p.H / p.Hk, nslot = gdr_slots(p);
    const GdrSeqs seqs{p.cu, p.N, p.T};
    unsigned char *vals = p.workspace + key_part(p, L);
    if (nslot > 0 && p.T > 0) {
        const GdrChunkArgs a{p.q, p.k, p.g, p.beta, st3(p.sq), st3(p.sk), st3(p.sg), st3(p.sb), seqs,
                             p.Hk, r, nslot, p.scale, p.workspace, vals};
        hipLaunchKernelGGL((gdr_chunk_kernel<DK, F32, MP>), dim3(nslot, p.H, p.B), dim3(256), 0, p.stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const GdrStateArgs a{p.workspace, vals, p.v, st3(p.sv), seqs, p.H, r, nslot, p.dv, p.scale,
                         p.final_state, p.init_state, p.out, nullptr};
    if (gdr_two_tiles(p)) return run_state<DK, F32, 2>(a, p.stream);
    return run_state<DK, F32, 1>(a, p.stream);
}

hipError_t launch_gdr_fwd(const GdrLaunch &p) {
    if (p.dk == 64) return p.fp32 ? fwd_t<64, true>(p) : fwd_t<64, false>(p);
    return p.fp32 ? fwd_t<128, true>(p) : fwd_t<128, false>(p);
}

hipError_t launch_gdr_decode(const GdrLaunch &p) {
    const GdrDecodeArgs a{p.q, p.k, p.v, p.g, p.beta, p.H, p.H / p.Hk, p.dv, p.scale, p.state, p.out};
    const dim3 grid((unsigned)p.B * p.H * (p.dv / kDecodeRowsPerBlock));
    if (p.dk == 64) {
        if (p.fp32) hipLaunchKernelGGL((gdr_decode_kernel<64, true>), grid, dim3(256), 0, p.stream, a);
        else hipLaunchKernelGGL((gdr_decode_kernel<64, false>), grid, dim3(256), 0, p.stream, a);
    } else {
        if (p.fp32) hipLaunchKernelGGL((gdr_decode_kernel<128, true>), grid, dim3(256), 0, p.stream, a);
        else hipLaunchKernelGGL((gdr_decode_kernel<128, false>), grid, dim3(256), 0, p.stream, a);
    }
    return hipGetLastError();
}

}  // namespace kda
