// Internal interface between the host side of decayed linear attention's entry points
// (kda_abi_lin.cpp) and its kernels.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stddef.h>

namespace kda {

struct LinLaunch {
    const void *q, *k, *v, *g;
    long long sq[3], sk[3], sv[3], sg[3];  // element strides b, h, t
    const int *cu;                         // NULL: fixed-length batch
    int N, B, Hk, H, T, dk, dv;            // sequences; batch entries (1 when packed)
    bool fp32, g32, packed;                // g32: g (and dg) in float32
    float scale;
    void *out;
    float *final_state;
    const float *init_state;
    float *state;                          // one-token step
    unsigned char *workspace;
    hipStream_t stream;
    // backward
    const void *dout;
    long long sdo[3];
    const float *dfinal;
    void *dq, *dk_, *dv_, *dg;             // dg NULL: not wanted
    float *dinit;
};

// Tokens of a segment, the piece of a sequence that one work-group walks through, and the segments of one
// batch entry.  A segment costs its state written, scanned and read again and its inputs read twice, so
// there are as many as keep the card busy and no more, counted over the chunks of all heads.
// bf16: one work-group a CU, whose eight waves have 130 KiB of LDS at 128 x 128 (256 against 512 segments in all:
// 4 x 8192 x 16 heads 210 us against 228, 1 x 65536 x 32 heads 729 against 738, the training step of 2 x 4096 x 8/16
// heads 280 against 341).  Where batch x heads does not divide 256 a head's last segment is short and there are up
// to a quarter more work-groups than CUs, so a second round: 8192 tokens of 24 heads take 126 us, of 32 heads 108.
// float32: 512 segments.  At 64 x 64 two work-groups fit a CU (67 KiB; 2 x 4096 x 16 heads 96 us against 116 with 256,
// backward 267 against 337); at 128 x 128 one does (115 KiB), and two rounds of shorter segments are as good as one (4
// x 8192 x 16 heads 920 against 978, backward 2,727 against 2,823; 2 x 4096 x 16 heads 259 against 262).
// A chunk of 64 tokens is the least, for short sequences wait for one chunk after the other (1 x 1024 x 4
// heads, forward and backward: 27 and 43 us with segments of 64 tokens, 31 and 46 with 256; float32 43 and
// 117, 118 and 332); only up to 256 tokens of bf16 is one launch over a single segment better (256 tokens:
// 18 us against 27 forward, 37 against 44 backward).
inline int lin_segment(const LinLaunch &p) {
    const long long chunks = (((long long)p.T + 63) / 64) * p.B * p.H, most = p.fp32 ? 512 : 256;
    long long per = (chunks + most - 1) / most;
    if (per < 1) per = 1;
    if (per < 4 && p.T <= 256 && !p.fp32) per = 4;
    if (per > 4096) per = 4096;
    return (int)per * 64;
}
inline long long lin_slots(const LinLaunch &p) {
    const long long seg = lin_segment(p), n = p.packed ? p.T / seg + p.N : (p.T + seg - 1) / seg;
    return n < 1 ? 1 : n;
}
// Segment states of one batch entry and head.  Only sequences longer than a segment have any, so that a packed
// stream needs no more of them the more short documents are in it; of the two ways to place them
// (LinSeqs::state_slot) the one that takes less.
inline bool lin_sparse(const LinLaunch &p) { return p.packed && p.N > p.T / lin_segment(p) + 1; }
inline long long lin_states(const LinLaunch &p) { return lin_sparse(p) ? 2 * (long long)(p.T / lin_segment(p)) + 1 : lin_slots(p); }
// all of them (one at least)
inline size_t lin_all_states(const LinLaunch &p) { return p.T <= lin_segment(p) ? 1 : (size_t)p.B * p.H * lin_states(p); }
size_t lin_fwd_bytes(const LinLaunch &p);
// end_states: of a call with dfinal and dg
size_t lin_bwd_bytes(const LinLaunch &p, bool end_states);

hipError_t launch_lin_fwd(const LinLaunch &p);
hipError_t launch_lin_bwd(const LinLaunch &p);
hipError_t launch_lin_decode(const LinLaunch &p);

// Work-groups of the backward's last launch (lin_scan.h).
inline long long lin_finish_grid(const LinLaunch &p, bool grads) {
    const long long sums = p.H == p.Hk ? 0 : ((long long)p.B * p.Hk * p.T * p.dk / 4 + 255) / 256;
    return (grads ? (long long)p.B * p.H * lin_slots(p) : 0) + sums + (p.packed ? ((long long)p.T + 63) / 64 * p.H : 0);
}

// Whether the launches of a call stay below 2^32 work-items in x, which is as far as a launch goes, and
// their unit counts in 32 bits.
inline bool lin_grids_fit(const LinLaunch &p, bool backward) {
    const long long most = 4294967295LL, units = (long long)p.B * p.H * lin_slots(p) * (p.dv / 64);
    const long long states = (long long)p.N * p.H * (p.dk * p.dv / 1024);
    return (units + 7) / 8 * 8 <= most / 512 && states <= most / 256 && (!backward || lin_finish_grid(p, true) <= most / 256);
}
inline bool lin_decode_grid_fits(const LinLaunch &p) { return (long long)p.B * p.H * (p.dv / 16) * 256 <= 4294967295LL; }

}  // namespace kda
