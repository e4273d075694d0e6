// The walk of decayed linear attention over the chunks of one segment (formulas: lin_common.h):
//   out_i = scale sum_j D_ij (a_i . b_j) c_j + inter wd_i a_i P,   P <- e^{G_last} P + into sum_j ws_j b_j c_j^T
// forwards (j <= i, D_ij = e^{G_i - G_j}, wd_i = e^{G_i}, ws_j = e^{G_last - G_j}) or, REV, backwards in
// time (j >= i, D_ij = e^{G_j - G_i}, wd and ws change places).
//
// A work-group of four waves takes one segment of one head, a wave a quarter of c's channels.  Everything but the scores is computed
// transposed: O^T = C^T M^T + P^T A^T has the channels on the accumulator's rows, so that a lane stores
// eight consecutive ones; the scores S^T = B A^T are, as they lie, the B operand of M^T; and the state P
// (rows b's channels, columns c's, 16 DC / 64 columns a wave, in registers throughout) is, as it lies,
// the A operand of P^T A^T.  C's transposed fragments serve O^T unscaled and, times ws in pieces, the
// state.  A wave makes the scores of 16 rows and hands them round through LDS.
#pragma once
#include "lin_common.h"

namespace kda {

struct LinWalkArgs {
    const void *a, *b, *c, *g, *y;   // y: rows that out is multiplied with for the decay's gradient
    Strides3 sa, sb, sc, sg, sy;
    int ra, rb, rc, ry;              // value heads that share a head of that tensor
    LinSeqs seqs;
    int B, H, nslot;
    bool g32, all;                   // all: segments that are alone in their sequence take part as others do
    float scale, inter, into;
    const float *init;               // [N][H] start states of the sequences (NULL: zero), for segments that are alone
    float *final_state;              // [N][H] end states, from segments that are alone (NULL: not wanted)
    float *seg;                      // [B][H][nslot] states of the others: local sums (pass 1), start states (pass 2)
    float *seg_decay;                // [B][H][nslot], written by pass 1
    void *out;                       // [B][H][T][DC], in the inputs' type or (OUTF) float32
    float *dots;                     // [B][H][T]: y_i . (out_i without the term j = i)
};

// OUT: pass 2, the outputs; else pass 1, the segment's own contribution to the state.  TR: states in
// memory have b's channels as rows, else c's.
template <int DA, int DC, bool F32, bool REV, bool TR, bool OUT, bool DOT, bool OUTF>
__global__ __launch_bounds__(256, F32 ? 1 : 2) void lin_walk_kernel(const LinWalkArgs p) {
    using Op = LinOp<F32>;
    using E = typename Op::E;
    using V8 = typename Op::V8;
    constexpr int NA = DA / 32, NC = DC / 32, NDT = DA / 16, NW = 4, NCT = DC / 16 / NW, MP = Op::MP, SP = Op::SP, FB = Op::FB;
    typedef __attribute__((address_space(3))) float lds_f;
    typedef __attribute__((address_space(3))) f32x4 lds_f4;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[(4 * NA * (OUT ? 2 : 1) + 4 * NC + (OUT ? 8 * MP : 0)) * FB];
    // by chunk parity: prefix sums in two floats, weights of the outputs and of the sources, e^{G_last}
    __shared__ __attribute__((aligned(16))) float sg[2 * 320 + 64 + (DOT ? 64 * NW : 0)];
    lds_u8 *sB = lds_base(smem), *sC = sB + 4 * NA * FB, *sA = sC + 4 * NC * FB, *sM = sA + 4 * NA * FB;
    lds_f *sG = (lds_f *)lds_base(sg), *sD = sG + 640, *sDot = sG + 704;
    const int tid0 = threadIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(tid0 >> 6);
    // units in eight runs, one an XCD: heads that share rows are neighbours there
    const unsigned units = (unsigned)p.B * p.H * p.nslot, per = (units + 7) / 8, unit = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= per || unit >= units) return;
    const int h = unit % p.H, slot = unit / p.H % p.nslot, b = unit / p.H / p.nslot;
    int seq, piece;
    if (!p.seqs.find(b, slot, seq, piece)) return;
    const int len = p.seqs.length(seq);
    const bool alone = !p.all && len <= p.seqs.seg;
    if (!OUT && alone) return;
    const int first = p.seqs.start(seq) + piece * p.seqs.seg, rows = max(0, min(p.seqs.seg, len - piece * p.seqs.seg));
    const int nchunk = (rows + 63) / 64;
    const E *ap = reinterpret_cast<const E *>(p.a) + b * p.sa.b + h / p.ra * p.sa.h + (long long)first * p.sa.t;
    const E *bp = reinterpret_cast<const E *>(p.b) + b * p.sb.b + h / p.rb * p.sb.h + (long long)first * p.sb.t;
    const E *cp = reinterpret_cast<const E *>(p.c) + b * p.sc.b + h / p.rc * p.sc.h + (long long)first * p.sc.t;
    const long long g0 = b * p.sg.b + h * p.sg.h + (long long)first * p.sg.t;
    const size_t row0 = ((size_t)b * p.H + h) * p.seqs.T + first, sunit = ((size_t)b * p.H + h) * p.nslot + slot;
    const size_t nstate = ((size_t)seq * p.H + h) * (DA * DC);

    // the lane's 8 rows 32 kb + 8 g .. of its column in tile ct of a state in memory
    auto state_at = [&](int kb, int ct) {
        const int g = tid0 >> 4 & 3, n = tid0 & 15;
        const int d = 32 * kb + 8 * g, c = perm_row(w * NCT + ct, n);
        return TR ? d * DC + c : c * DA + d;
    };
    f32x4 P[NCT][NDT];
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    const float *from = !OUT ? nullptr : alone ? (p.init ? p.init + nstate : nullptr) : p.seg + sunit * (DA * DC);
    float *to = !OUT ? p.seg + sunit * (DA * DC) : alone && p.final_state ? p.final_state + nstate : nullptr;
    // a state that is handed on keeps all 24 bits; one that only feeds outputs does with 16
    const bool whole = to != nullptr;
#pragma unroll
    for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
        for (int kb = 0; kb < NA; ++kb) {
            f32x4 x = zero, y = zero;
            if (from) {
                const float *s = from + state_at(kb, ct);
                if constexpr (TR) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[i] = s[i * DC];
                        y[i] = s[(4 + i) * DC];
                    }
                } else {
                    x = *reinterpret_cast<const f32x4 *>(s);
                    y = *reinterpret_cast<const f32x4 *>(s + 4);
                }
            }
            P[ct][2 * kb] = x;
            P[ct][2 * kb + 1] = y;
        }

    TileStage<F32, DA / 8> ta, tb;
    TileStage<F32, DC / 8> tc;
    float gn = 0.f;
    double total = 0.0;
    auto load = [&](int c, int tid) {
        const int lane = tid & 63;
        if constexpr (OUT) ta.load(ap, p.sa.t, 64 * c, rows, tid);
        tb.load(bp, p.sb.t, 64 * c, rows, tid);
        tc.load(cp, p.sc.t, 64 * c, rows, tid);
        if (w == NW - 1) gn = 64 * c + lane < rows ? load_g(p.g, g0 + (long long)(64 * c + lane) * p.sg.t, p.g32) : 0.f;
    };
    auto decays = [&](int c, int par, int lane) {  // the last wave: it has least to do with the scores
        const double G = wave_scan64(decay_log2(gn)), last = lane64(G, 63);
        const float hi = (float)G, e0 = ex2(hi), e1 = ex2((float)(last - G));
        lds_f *s = sG + 320 * par;
        s[lane] = hi;
        s[64 + lane] = (float)(G - (double)hi);
        s[128 + lane] = p.inter * (REV ? e1 : e0);
        // rows behind the last arrive as zeros, or as earlier rows where rows overlap (strides below a row)
        s[192 + lane] = 64 * c + lane < rows ? p.into * (REV ? e0 : e1) : 0.f;
        if (lane == 0) s[256] = ex2((float)last);
        total += last;
    };
    auto chunk_of = [&](int ci) { return REV ? nchunk - 1 - ci : ci; };
    if (nchunk > 0) {
        load(chunk_of(0), tid0);
        if (w == NW - 1) decays(chunk_of(0), 0, tid0 & 63);
    }
    for (int ci = 0; ci < nchunk; ++ci) {
        const int c = chunk_of(ci);
        const int tid = lane_here(tid0), lane = tid & 63, g = lane >> 4, n = lane & 15;
        const lds_f *sH = sG + 320 * (ci & 1), *sWd = sH + 128, *sWs = sH + 192;
        barrier_lds();  // the last chunk has been read
        if constexpr (OUT) ta.store(sA, NA, 0, tid);
        tb.store(sB, NA, 0, tid);
        tc.store(sC, NC, 0, tid);
        if (ci + 1 < nchunk) load(chunk_of(ci + 1), tid);
        barrier_lds();
        // (tid through lane_here: a chunk's addresses are made in the chunk, or they would fill the registers)
        V8 cf[NCT][2];  // C transposed, the wave's columns
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const int t = w * NCT + ct;
                const lds_u8 *f = sC + (2 * kb * NC + (t >> 1)) * FB;
                cf[ct][kb] = Op::get_t(f, f + NC * FB, t, lane);
            }
        if constexpr (OUT) {
            // scores: six causal fragments of 32 columns, by row tile `it` and column block `jb`
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int f = w + NW * k;
                if (f >= 6) continue;
                const int it = REV ? (f < 4 ? f : f - 4) : (f < 4 ? f : f - 2), jb = REV ? (f < 4 ? 1 : 0) : f < 4 ? 0 : 1;
                V8 af[NA];
#pragma unroll
                for (int kb = 0; kb < NA; ++kb) af[kb] = Op::get(sA + (it * NA + kb) * FB, kb, lane);
                const int i = perm_row(it, n);
                const float ih = sH[i], il = sH[64 + i];
                f32x4 s[2] = {zero, zero};
#pragma unroll
                for (int o = 0; o < 2; ++o) {
#pragma unroll
                    for (int kb = 0; kb < NA; ++kb)
                        s[o] = Op::mma(Op::get(sB + ((2 * jb + o) * NA + kb) * FB, kb, lane), af[kb], s[o]);
                    const int j = perm_row(2 * jb + o, 4 * g);
                    const f32x4 jh = *reinterpret_cast<const lds_f4 *>(sH + j), jl = *reinterpret_cast<const lds_f4 *>(sH + 64 + j);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float e = (ih - jh[x]) + (il - jl[x]);
                        const float m = p.scale * s[o][x] * ex2(REV ? -e : e);
                        const bool self = j + x == i;
                        if (DOT && self) sD[i] = m;
                        s[o][x] = (REV ? j + x < i || 64 * c + j + x >= rows : j + x > i) || (DOT && self) ? 0.f : m;
                    }
                }
                V8 m[MP];
                Op::pieces(s[0], s[1], m);
#pragma unroll
                for (int x = 0; x < MP; ++x) Op::put_lane(sM + ((2 * it + jb) * MP + x) * FB, lane, m[x]);
            }
            __builtin_amdgcn_sched_barrier(0);
            f32x4 O[NCT][4];
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                for (int it = 0; it < 4; ++it) O[ct][it] = zero;
#pragma unroll
            for (int kb = 0; kb < NA; ++kb) {
                V8 pf[NCT][MP];
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) Op::pieces(P[ct][2 * kb], P[ct][2 * kb + 1], pf[ct]);
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                    const V8 af = Op::get(sA + (it * NA + kb) * FB, kb, lane);
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                        for (int x = 0; x < MP; ++x) O[ct][it] = Op::mma(pf[ct][x], af, O[ct][it]);
                }
            }
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const float wd = sWd[perm_row(it, n)];
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) O[ct][it] *= wd;
            }
            barrier_lds();  // M is there
#pragma unroll
            for (int it = 0; it < 4; ++it)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    if (REV ? kb < (it >> 1) : kb > (it >> 1)) continue;
#pragma unroll
                    for (int x = 0; x < MP; ++x) {
                        const V8 m = Op::get_lane(sM + ((2 * it + kb) * MP + x) * FB, lane);
#pragma unroll
                        for (int ct = 0; ct < NCT; ++ct) O[ct][it] = Op::mma(cf[ct][kb], m, O[ct][it]);
                    }
                }
            const int c0 = perm_row(w * NCT, 4 * g);  // the lane's channels c0 .. + 4 NCT
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const int i = perm_row(it, n), row = 64 * c + i;
                if constexpr (DOT) {
                    float d = 0.f;
                    if (row < rows) {
                        const E *y = reinterpret_cast<const E *>(p.y) + b * p.sy.b + h / p.ry * p.sy.h + (long long)(first + row) * p.sy.t + c0;
#pragma unroll
                        for (int ct = 0; ct < NCT; ++ct) {
                            float v[4];
                            ld4(y + 4 * ct, v);
#pragma unroll
                            for (int x = 0; x < 4; ++x) d += O[ct][it][x] * v[x];
                        }
                    }
                    d = col_sum(d);
                    if (g == 0) sDot[64 * w + i] = d;
                    // the term j = i, in float32: rows of C as they lie
                    const float m = sD[i];
                    f32x4 x, y;
                    Op::split(Op::get(sC + (it * NC + (w * NCT >> 1)) * FB, w * NCT >> 1, lane), x, y);
                    if constexpr (NCT == 2) {
                        O[0][it] += m * x;
                        O[1][it] += m * y;
                    } else {
                        O[0][it] += m * (w & 1 ? y : x);
                    }
                }
                if (row < rows) {
                    const size_t at = (row0 + row) * DC + c0;
                    if constexpr (OUTF) {
                        float *o = reinterpret_cast<float *>(p.out) + at;
#pragma unroll
                        for (int ct = 0; ct < NCT; ++ct) *reinterpret_cast<f32x4 *>(o + 4 * ct) = O[ct][it];
                    } else if constexpr (NCT == 2) {
                        Op::store8(reinterpret_cast<E *>(p.out) + at, O[0][it], O[1][it]);
                    } else {
                        st_tile(reinterpret_cast<E *>(p.out) + at, 0, O[0][it]);
                    }
                }
            }
        }
        if (w == NW - 1 && ci + 1 < nchunk) decays(chunk_of(ci + 1), (ci + 1) & 1, lane);
        const float dec = sH[256];
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
            for (int dt = 0; dt < NDT; ++dt) P[ct][dt] *= dec;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            const f32x4 w0 = *reinterpret_cast<const lds_f4 *>(sWs + 32 * kb + 8 * g), w1 = *reinterpret_cast<const lds_f4 *>(sWs + 32 * kb + 8 * g + 4);
            V8 xf[NCT][SP];
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) {
                f32x4 x, y;
                Op::split(cf[ct][kb], x, y);
                x *= w0;
                y *= w1;
                xf[ct][0] = Op::piece(x, y);
                if constexpr (SP > 1) xf[ct][1] = Op::piece(x, y);
                if (SP > 2 && (!OUT || whole)) xf[ct][SP - 1] = Op::piece(x, y);
            }
#pragma unroll
            for (int dt = 0; dt < NDT; ++dt) {
                const lds_u8 *f = sB + (2 * kb * NA + (dt >> 1)) * FB;
                const V8 bt = Op::get_t(f, f + NA * FB, dt, lane);
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                    for (int x = 0; x < SP; ++x)
                        if (!OUT || x < 2 || whole) P[ct][dt] = Op::mma(bt, xf[ct][x], P[ct][dt]);
            }
        }
        if constexpr (DOT) {
            barrier_lds();
            if (tid < 64 && 64 * c + tid < rows) {
                float d = 0.f;
#pragma unroll
                for (int k = 0; k < NW; ++k) d += sDot[64 * k + tid];
                p.dots[row0 + 64 * c + tid] = d;
            }
        }
    }
    if (!OUT && w == NW - 1 && (tid0 & 63) == 0) p.seg_decay[sunit] = ex2((float)total);
    if (!to) return;
#pragma unroll
    for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
        for (int kb = 0; kb < NA; ++kb) {
            float *s = to + state_at(kb, ct);
            const f32x4 x = P[ct][2 * kb], y = P[ct][2 * kb + 1];
            if constexpr (TR) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[i * DC] = x[i];
                    s[(4 + i) * DC] = y[i];
                }
            } else {
                *reinterpret_cast<f32x4 *>(s) = x;
                *reinterpret_cast<f32x4 *>(s + 4) = y;
            }
        }
}

}  // namespace kda
