// The walk of decayed linear attention over the chunks of one segment (formulas: lin_common.h):
//   out_i = scale sum_j D_ij (a_i . b_j) c_j + inter wd_i a_i P,   P <- e^{G_last} P + into sum_j ws_j b_j c_j^T
// forwards (j <= i, D_ij = e^{G_i - G_j}, wd_i = e^{G_i}, ws_j = e^{G_last - G_j}) or, REV, backwards in
// time (j >= i, D_ij = e^{G_j - G_i}, wd and ws change places).
//
// A work-group takes one segment of one head, each of four waves a quarter of c's channels.  Everything but
// the scores is computed transposed: O^T = C^T M^T + P^T A^T has the channels on the accumulator's rows, so
// that a lane stores eight consecutive ones; the scores S^T = B A^T are, as they lie, the B operand of M^T;
// and the state P (rows b's channels, columns c's, DC / 4 columns a wave, in registers throughout) is, as it
// lies, the A operand of P^T A^T.  C's transposed fragments serve O^T unscaled and, times ws in pieces, the
// state.  Scores go round through LDS.
#pragma once
#include "lin_common.h"

namespace kda {

struct LinWalkArgs {
    const void *a, *b, *c, *g, *y;   // y: rows that out is multiplied with for the decay's gradient
    Strides3 sa, sb, sc, sg, sy;
    int ra, rb, rc, ry;              // value heads that share a head of that tensor
    LinSeqs seqs;
    int B, H, nslot, nstate;         // work slots and states of a batch entry's head
    int parts;                       // work-groups that share the columns of a segment's own state (pass 1)
    bool g32, all;                   // all (pass 1): also of segments that are alone in their sequence, into final_state
    float scale, inter, into;
    const float *init;               // [N][H] start states of the sequences (NULL: zero), for segments that are alone
    float *final_state;              // [N][H] end states, from segments that are alone (NULL: not wanted)
    float *seg;                      // [B][H][nstate] states of the others: local sums (pass 1), start states (pass 2)
    float *seg_decay;                // [B][H][nslot], written by pass 1
    void *out;                       // [B][H][T][DC], in the inputs' type or (OUTF) float32
    float *dots;                     // [B][H][T]: y_i . (out_i without the term j = i)
};

// Where a work-group's segment lies, and its rows.
template <typename E> struct LinUnit {
    int b, h, part, seq, first, rows, nchunk;
    bool alone;
    const E *ap, *bp, *cp;
    long long g0;
    size_t row0, sunit, sstate, nstate;  // places of its decay, of its state in seg, and (alone) of its sequence's
    // false: nothing there.  Units in eight runs, one an XCD: parts of a state and heads that share rows are
    // neighbours there.
    __device__ __forceinline__ bool find(const LinWalkArgs &p, int state, int parts = 1) {
        const unsigned all = (unsigned)p.B * p.H * p.nslot * parts, per = (all + 7) / 8, at = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
        if ((blockIdx.x >> 3) >= per || at >= all) return false;
        part = at % parts;
        const unsigned unit = at / parts;
        h = unit % p.H;
        b = unit / p.H / p.nslot;
        const int slot = unit / p.H % p.nslot;
        int piece;
        if (!p.seqs.find(b, slot, seq, piece)) return false;
        const int len = p.seqs.length(seq);
        first = p.seqs.start(seq) + piece * p.seqs.seg;
        alone = len <= p.seqs.seg;
        rows = max(0, min(p.seqs.seg, len - piece * p.seqs.seg));
        nchunk = (rows + 63) / 64;
        ap = reinterpret_cast<const E *>(p.a) + b * p.sa.b + h / p.ra * p.sa.h + (long long)first * p.sa.t;
        bp = reinterpret_cast<const E *>(p.b) + b * p.sb.b + h / p.rb * p.sb.h + (long long)first * p.sb.t;
        cp = reinterpret_cast<const E *>(p.c) + b * p.sc.b + h / p.rc * p.sc.h + (long long)first * p.sc.t;
        g0 = b * p.sg.b + h * p.sg.h + (long long)first * p.sg.t;
        row0 = ((size_t)b * p.H + h) * p.seqs.T + first;
        sunit = ((size_t)b * p.H + h) * p.nslot + slot;
        sstate = ((size_t)b * p.H + h) * p.nstate + p.seqs.state_slot(seq, piece, slot);
        nstate = ((size_t)seq * p.H + h) * state;
        return true;
    }
};

// bf16.  Four waves walk: a quarter of c's channels each, they hold the state and make the outputs; four more
// load the next chunk, sum its log-decays and make its scores.  Tiles, scores and decays are there twice, so
// a chunk takes two barriers (pass 1: one), and neither side waits for the other's latencies:
//   walkers   a_i P                          | + M C, out; state
//   helpers   next tile into LDS, decays     | next scores
// As one group of four waves that did all of it in turn, two work-groups on a CU, a chunk took 17,400 cycles
// of a work-group, half of them waits, and the parts' times added up (4 x 8192 x 16 heads 248 us against 202).
//
// 1 x 65536 x 32 heads of 128 x 128, 256 segments of 128 chunks: pass 1 takes 240 us (its loads of 0.8 GB alone
// 153, its products and pieces alone 205), pass 2 460 (its 1.6 GB alone 290, the rest alone 375).  A SIMD has some
// 1000 vector instructions of 4 cycles a chunk of pass 2, most of them pieces of P and of the weighted C, beside
// 160 MFMAs of 16: vector issue 51 % and matrix units 38 % busy (pass 1: 67 and 44), in two waves a SIMD that go
// each in order.
//
// OUT: pass 2, the outputs; else pass 1, the segment's own contribution to the state.  TR: states in memory
// have b's channels as rows, else c's.
template <int DA, int DC, bool OUT, bool DOT> struct LinPairLds {
    static constexpr int FB = LinOp<false>::FB;
    static constexpr int TILE = (4 * (DA / 32) * (OUT ? 2 : 1) + 4 * (DC / 32)) * FB, MB = 6 * 2 * FB;  // of a chunk: rows, scores
    static constexpr int BYTES = 2 * TILE + (OUT ? 2 * MB : 0);
    // for eight chunks: prefix sums in two floats, weights of the outputs and of the sources, e^{G_last}; the
    // scores of tokens with themselves, by parity; and the walkers' dot products
    static constexpr int FLOATS = 8 * 320 + (DOT ? 2 * 64 + 4 * 64 : 0);
};
template <int DA, int DC, bool REV, bool TR, bool OUT, bool DOT, bool OUTF>
__device__ __forceinline__ void lin_pair(const LinWalkArgs &p, lds_u8 *sT, __attribute__((address_space(3))) float *sG) {
    using Op = LinOp<false>;
    using E = __bf16;
    using V8 = bf16x8;
    using Lds = LinPairLds<DA, DC, OUT, DOT>;
    constexpr int NA = DA / 32, NC = DC / 32, NDT = DA / 16, NCT = DC / 64, FB = Op::FB, TILE = Lds::TILE, MB = Lds::MB;
    typedef __attribute__((address_space(3))) float lds_f;
    typedef __attribute__((address_space(3))) f32x4 lds_f4;
    lds_u8 *sM = sT + 2 * TILE;
    lds_f *sD = sG + 8 * 320, *sDot = sD + 128;
    const int tid = threadIdx.x & 255, lane = tid & 63, g = lane >> 4, n = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool helper = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8) != 0;
    LinUnit<E> u;
    if (!u.find(p, DA * DC, OUT ? 1 : p.parts) || (!OUT && u.alone && !p.all)) return;
    if (!OUT) u.cp += u.part * DC;
    const int nchunk = u.nchunk, rows = u.rows;
    auto chunk_of = [&](int ci) { return REV ? nchunk - 1 - ci : ci; };
    auto tile_b = [&](int par) { return sT + par * TILE; };
    auto tile_c = [&](int par) { return sT + par * TILE + 4 * NA * FB; };
    auto tile_a = [&](int par) { return sT + par * TILE + (4 * NA + 4 * NC) * FB; };
    // place of the fragment (row tile it, column block jb) among the six causal ones
    auto frag = [](int it, int jb) { return REV ? (jb == 1 ? it : 4 + it) : (jb == 0 ? it : 2 + it); };

    if (helper) {
        struct Stage {  // one chunk on its way: two of them, so that a chunk's loads have two chunks' time
            TileStage<false, DA / 8> ta, tb;
            TileStage<false, DC / 8> tc;
            unsigned g;
        } st0, st1;
        double total = 0.0;
        // (of no rows behind the last chunk: were the loads left out there, none could be waited for without
        // those behind it)
        auto load = [&](int ci, Stage &s) {
            const int c = ci < nchunk ? chunk_of(ci) : 0, n = ci < nchunk ? rows : 0;
            if constexpr (OUT) s.ta.load(u.ap, p.sa.t, 64 * c, n, tid);
            s.tb.load(u.bp, p.sb.t, 64 * c, n, tid);
            s.tc.load(u.cp, p.sc.t, 64 * c, n, tid);
            // log-decays of four chunks at a time, one a wave: a scan in float64 is a long chain, and every chunk
            // would wait for it
            if ((ci & 3) == 0 && ci + w < nchunk) {
                const int row = 64 * chunk_of(ci + w) + lane;
                s.g = row < rows ? load_g_bits(p.g, u.g0 + (long long)row * p.sg.t, p.g32) : 0u;
            }
        };
        auto decays = [&](int ci, unsigned bits) {
            if (ci + w >= nchunk) return;
            const double G = wave_scan64(decay_log2(g_value(bits, p.g32))), last = lane64(G, 63);
            const float hi = (float)G, e0 = ex2(hi), e1 = ex2((float)(last - G));
            lds_f *s = sG + 320 * ((ci + w) & 7);
            s[lane] = hi;
            s[64 + lane] = (float)(G - (double)hi);
            s[128 + lane] = p.inter * (REV ? e1 : e0);
            // rows behind the last arrive as zeros, or as earlier rows where rows overlap (strides below a row)
            s[192 + lane] = 64 * chunk_of(ci + w) + lane < rows ? p.into * (REV ? e0 : e1) : 0.f;
            if (lane == 0) s[256] = ex2((float)last);
            total += last;
        };
        auto store = [&](int ci, const Stage &st) {  // and the decays of this chunk and the next three
            const int par = ci & 1;
            if constexpr (OUT) st.ta.store(tile_a(par), NA, 0, tid);
            st.tb.store(tile_b(par), NA, 0, tid);
            st.tc.store(tile_c(par), NC, 0, tid);
            if ((ci & 3) == 0) decays(ci, st.g);
        };
        auto scores = [&](int ci) {
            const int par = ci & 1, left = rows - 64 * chunk_of(ci);
            const lds_u8 *sA = tile_a(par), *sB = tile_b(par);
            const lds_f *sH = sG + 320 * (ci & 7);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int f = w == 0 ? 4 * k : w == 1 ? 1 + 4 * k : w;  // waves 0 and 1 take two of the six
                if (k == 1 && w > 1) break;
                const int it = REV ? (f < 4 ? f : f - 4) : (f < 4 ? f : f - 2), jb = REV ? (f < 4 ? 1 : 0) : f < 4 ? 0 : 1;
                V8 af[NA];
#pragma unroll
                for (int kb = 0; kb < NA; ++kb) af[kb] = Op::get(sA + (it * NA + kb) * FB, kb, lane);
                const int i = perm_row(it, n);
                const float ih = sH[i], il = sH[64 + i];
                f32x4 s[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
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
                        if (DOT && self) sD[64 * par + i] = m;
                        s[o][x] = (REV ? j + x < i || j + x >= left : j + x > i) || (DOT && self) ? 0.f : m;
                    }
                }
                V8 m[2];
                Op::pieces(s[0], s[1], m);
#pragma unroll
                for (int x = 0; x < 2; ++x) Op::put_lane(sM + par * MB + (2 * f + x) * FB, lane, m[x]);
            }
        };
        auto dots = [&](int ci) {  // of a chunk that is done
            const int row = 64 * chunk_of(ci) + tid;
            if (tid < 64 && row < rows) p.dots[u.row0 + row] = (sDot[tid] + sDot[64 + tid]) + (sDot[128 + tid] + sDot[192 + tid]);
        };
        auto step = [&](int ci, Stage &s) {  // s holds the chunk behind ci
            if (DOT && ci > 0) dots(ci - 1);
            if (ci + 1 < nchunk) store(ci + 1, s);
            load(ci + 3, s);
            barrier_lds();
            if constexpr (OUT) {
                if (ci + 1 < nchunk) scores(ci + 1);
                barrier_lds();
            }
        };
        if (nchunk > 0) {
            load(0, st0);
            load(1, st1);
            store(0, st0);
            load(2, st0);
            barrier_lds();
            if constexpr (OUT) {
                scores(0);
                barrier_lds();
            }
        }
        int ci = 0;  // (steps in pairs, or loads in flight would be counted as if every step could be the last)
        for (; ci + 1 < nchunk; ci += 2) {
            step(ci, st1);
            step(ci + 1, st0);
        }
        if (ci < nchunk) step(ci, st1);
        if (DOT && nchunk > 0) dots(nchunk - 1);
        if constexpr (!OUT) {
            typedef __attribute__((address_space(3))) double lds_d;
            lds_d *sum = (lds_d *)sG;
            if (lane == 0) sum[w] = total;
            barrier_lds();
            if (tid == 0 && u.part == 0) p.seg_decay[u.sunit] = ex2((float)((sum[0] + sum[1]) + (sum[2] + sum[3])));
        }
        return;
    }

    // the lane's 8 rows 32 kb + 8 g .. of its column in tile ct of a state in memory
    auto state_at = [&](int kb, int ct) {
        const int d = 32 * kb + 8 * g, c = perm_row(w * NCT + ct, n);
        return TR ? d * DC + c : c * DA + d;
    };
    f32x4 P[NCT][NDT];
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    const float *from = !OUT ? nullptr : u.alone ? (p.init ? p.init + u.nstate : nullptr) : p.seg + u.sstate * (DA * DC);
    float *to = !u.alone ? (OUT ? nullptr : p.seg + (u.sstate * p.parts + u.part) * (DA * DC))
                : p.final_state ? p.final_state + (OUT ? u.nstate : u.nstate * p.parts + u.part * (DA * DC)) : nullptr;
    // a state that can be handed on keeps all 24 bits, whether it is asked for or not, or the outputs made from
    // it would depend on that; one that only feeds outputs does with 16
    const bool whole = !OUT || (!TR && __builtin_amdgcn_readfirstlane(u.alone) != 0);
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
    const int lane0 = lane;
    const E *yp = DOT ? reinterpret_cast<const E *>(p.y) + u.b * p.sy.b + u.h / p.ry * p.sy.h + (long long)u.first * p.sy.t : nullptr;
    // Products in steps of one fragment from LDS, read AHEAD steps before its MFMAs, and beside the MFMAs a
    // share of what the vector unit has to do for the steps to come: the pieces of P for the next 32 of b's
    // channels, those of the weighted C for the next 32 tokens.  The order is fixed step by step: left alone,
    // the scheduler puts each read right before its use.
    typedef __attribute__((ext_vector_type(4))) unsigned u32x4;
    constexpr int AHEAD = 3, RING = AHEAD + 1;
    u32x4 pf[2][NCT][2];  // pieces of P, the current and the next 32 channels
    auto p_part = [&](int kb, int q) {  // q of 2 NCT: half a column tile
        const int ct = q >> 1, h = q & 1;
        f32x4 x = P[ct][2 * kb + h];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            pf[kb & 1][ct][k][2 * h] = Op::take(x, 0);
            pf[kb & 1][ct][k][2 * h + 1] = Op::take(x, 2);
        }
    };
    if (OUT) {
#pragma unroll
        for (int q = 0; q < 2 * NCT; ++q) p_part(0, q);
    }
    if (nchunk > 0) {
        barrier_lds();
        if constexpr (OUT) barrier_lds();
    }
    for (int ci = 0; ci < nchunk; ++ci) {
        const int c = chunk_of(ci), par = ci & 1;
        // (through lane_here: a chunk's addresses are made in the chunk, or they would fill the registers)
        const int lane = lane_here(lane0), g = lane >> 4, n = lane & 15, c0 = perm_row(w * NCT, 4 * g);  // the lane's channels c0 .. + 4 NCT
        const lds_f *sH = sG + 320 * (ci & 7), *sWd = sH + 128, *sWs = sH + 192;
        const lds_u8 *sA = tile_a(par), *sB = tile_b(par), *sC = tile_c(par);
        V8 ring[RING];
        V8 cf[NCT][2];  // C transposed, the wave's columns
        auto get_c = [&]() {
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    const int t = w * NCT + ct;
                    const lds_u8 *f = sC + (2 * kb * NC + (t >> 1)) * FB;
                    cf[ct][kb] = Op::get_t(f, f + NC * FB, t, lane);
                }
        };
        f32x4 ws[2][2];
        u32x4 xf[2][NCT][3];  // pieces of the weighted C, by 32 tokens
        auto x_part = [&](int kb, int q, int np) {  // q of 4 NCT: two tokens of a column tile
            const int ct = q >> 2, i = q & 3;
            const unsigned v = __builtin_bit_cast(u32x4, cf[ct][kb])[i];
            f32x4 x;
            x[0] = __builtin_bit_cast(float, v << 16) * ws[kb][i >> 1][2 * (i & 1)];
            x[1] = __builtin_bit_cast(float, v & 0xffff0000u) * ws[kb][i >> 1][2 * (i & 1) + 1];
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (k < np) xf[kb][ct][k][i] = Op::take(x, 0);
        };
        auto get_b = [&](int k) {  // step k: 32 tokens k / NDT, row tile k % NDT
            const int dt = k % NDT;
            const lds_u8 *f = sB + (k / NDT * 2 * NA + (dt >> 1)) * FB;
            return Op::get_t(f, f + NA * FB, dt, lane);
        };
        auto get_ws = [&]() {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int o = 0; o < 2; ++o) ws[kb][o] = *reinterpret_cast<const lds_f4 *>(sWs + 32 * kb + 8 * g + 4 * o);
        };
        // P <- dec P + B^T (weighted C) in np pieces; the first AHEAD fragments are in the ring, xf[0] is made
        auto state = [&](auto np_) {
            constexpr int np = decltype(np_)::value;
            const float dec = sH[256];
#pragma unroll
            for (int k = 0; k < 2 * NDT; ++k) {
                const int dt = k % NDT;
                if (k + AHEAD < 2 * NDT) ring[(k + AHEAD) % RING] = get_b(k + AHEAD);
                if (k < NDT) {
#pragma unroll
                    for (int q = 0; q < 4 * NCT; ++q)
                        if (q * NDT / (4 * NCT) == k) x_part(1, q, np);
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct) P[ct][dt] *= dec;
                } else if constexpr (OUT) {
#pragma unroll
                    for (int q = 0; q < 2 * NCT; ++q)
                        if (2 + q * (NDT - 2) / (2 * NCT) == dt) p_part(0, q);
                }
#pragma unroll
                for (int x = 0; x < np; ++x)
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct) P[ct][dt] = Op::mma(ring[k % RING], __builtin_bit_cast(V8, xf[k / NDT][ct][x]), P[ct][dt]);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        if constexpr (OUT) {
            bf16x4 y[4][NCT];
            if constexpr (DOT) {
#pragma unroll
                for (int it = 0; it < 4; ++it)
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct) {  // rows behind the last: the last
                        const int row = min(64 * c + perm_row(it, n), rows - 1);
                        y[it][ct] = *reinterpret_cast<const bf16x4 *>(yp + (long long)row * p.sy.t + c0 + 4 * ct);
                    }
            }
            auto get_a = [&](int k) { return Op::get(sA + ((k & 3) * NA + (k >> 2)) * FB, k >> 2, lane); };
            f32x4 O[NCT][4];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) ring[k] = get_a(k);
#pragma unroll
            for (int k = 0; k < 4 * NA; ++k) {
                const int kb = k >> 2, it = k & 3;
                if (k + AHEAD < 4 * NA) ring[(k + AHEAD) % RING] = get_a(k + AHEAD);
                if (kb + 1 < NA) {
#pragma unroll
                    for (int q = 0; q < 2 * NCT; ++q)
                        if (q * 4 / (2 * NCT) == it) p_part(kb + 1, q);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct)
                        O[ct][it] = Op::mma(__builtin_bit_cast(V8, pf[kb & 1][ct][x]), ring[k % RING], kb == 0 && x == 0 ? zero : O[ct][it]);
                __builtin_amdgcn_sched_barrier(0);
            }
            get_c();
            get_ws();
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const float wd = sWd[perm_row(it, n)];
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) O[ct][it] *= wd;
            }
            barrier_lds();
            // six fragments of M in two pieces
            auto m_it = [](int k) { const int f = k >> 1; return REV ? (f < 4 ? f : f - 4) : (f < 4 ? f : f - 2); };
            auto m_kb = [](int k) { const int f = k >> 1; return REV ? (f < 4 ? 1 : 0) : (f < 4 ? 0 : 1); };
            auto get_m = [&](int k) { return Op::get_lane(sM + par * MB + k * FB, lane); };
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) ring[k] = get_m(k);
#pragma unroll
            for (int k = 0; k < 12; ++k) {
                if (k + AHEAD < 12) ring[(k + AHEAD) % RING] = get_m(k + AHEAD);
                else ring[(k + AHEAD) % RING] = get_b(k + AHEAD - 12);  // into the state's steps
#pragma unroll
                for (int q = 0; q < 4 * NCT; ++q)
                    if (q * 12 / (4 * NCT) == k) x_part(0, q, whole ? 3 : 2);
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) O[ct][m_it(k)] = Op::mma(cf[ct][m_kb(k)], ring[k % RING], O[ct][m_it(k)]);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const int i = perm_row(it, n), row = 64 * c + i;
                if constexpr (DOT) {
                    float d = 0.f;
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                        for (int x = 0; x < 4; ++x) d += O[ct][it][x] * (float)y[it][ct][x];
                    d = col_sum(d);
                    if (g == 0) sDot[64 * w + i] = d;
                    // the term j = i, in float32: rows of C as they lie
                    const float m = sD[64 * par + i];
                    f32x4 x, z;
                    Op::split(Op::get(sC + (it * NC + (w * NCT >> 1)) * FB, w * NCT >> 1, lane), x, z);
                    if constexpr (NCT == 2) {
                        O[0][it] += m * x;
                        O[1][it] += m * z;
                    } else {
                        O[0][it] += m * (w & 1 ? z : x);
                    }
                }
                if (row < rows) {
                    const size_t at = (u.row0 + row) * DC + c0;
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
            __builtin_amdgcn_sched_barrier(0);
            if (whole) state(std::integral_constant<int, 3>());
            else state(std::integral_constant<int, 2>());
        } else {
            get_c();
            get_ws();
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) ring[k] = get_b(k);
#pragma unroll
            for (int q = 0; q < 4 * NCT; ++q) x_part(0, q, 3);
            state(std::integral_constant<int, 3>());
        }
        barrier_lds();
    }
    if constexpr (!OUT) barrier_lds();  // the helpers' sums
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

// One walk, or walks that do not depend on each other in one launch, where the next one's work-groups follow
// on a CU as soon as the last one's are done (11 packed documents, 5003 tokens, training step: 102 -> 95 us when they came together).
template <int DA, int DC, bool REV, bool TR, bool OUT, bool DOT, bool OUTF> struct LinWalk {
    static constexpr int BYTES = LinPairLds<DA, DC, OUT, DOT>::BYTES, FLOATS = LinPairLds<DA, DC, OUT, DOT>::FLOATS;
    __device__ __forceinline__ static void run(const LinWalkArgs &p, lds_u8 *sT, __attribute__((address_space(3))) float *sG) {
        lin_pair<DA, DC, REV, TR, OUT, DOT, OUTF>(p, sT, sG);
    }
};
template <int N> struct LinWalkList {
    LinWalkArgs a[N];
};
template <typename... W>
__global__ __launch_bounds__(512, 2) void lin_pair_kernel(const LinWalkList<sizeof...(W)> list) {
    constexpr int N = sizeof...(W);
    constexpr int bytes[N] = {W::BYTES...}, floats[N] = {W::FLOATS...};
    constexpr auto most = [](const int (&x)[N]) {
        int m = 0;
        for (int i = 0; i < N; ++i) m = x[i] > m ? x[i] : m;
        return m;
    };
    __shared__ __attribute__((aligned(1024))) unsigned char smem[most(bytes)];
    __shared__ __attribute__((aligned(16))) float sg[most(floats)];
    // (the list's entry by its number: by the walk, all walks' arguments would be read ahead and kept)
    const LinWalkArgs &p = list.a[N > 1 ? blockIdx.y : 0];
    int i = 0;
    ((void)(i++ == (int)blockIdx.y && (W::run(p, lds_base(smem), (__attribute__((address_space(3))) float *)lds_base(sg)), true)), ...);
}

// float32: tiles fill the LDS once, so one group of four waves does everything in turn, on float32 MFMAs, which run
// at an eighth of bf16's rate.  Parameters as above.  2 x 4096 x 16 heads of 128 x 128: forward 259 us, 104 of them
// the products themselves at a large matrix product's rate (155 TFLOP/s); the rest are loads, scores and barriers
// that nothing hides.
template <int DA, int DC, bool REV, bool TR, bool OUT, bool DOT>
__global__ __launch_bounds__(256, 1) void lin_walk32_kernel(const LinWalkArgs p) {
    using Op = LinOp<true>;
    using V8 = typename Op::V8;
    constexpr int NA = DA / 32, NC = DC / 32, NDT = DA / 16, NW = 4, NCT = DC / 16 / NW, FB = Op::FB;
    typedef __attribute__((address_space(3))) float lds_f;
    typedef __attribute__((address_space(3))) f32x4 lds_f4;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[(4 * NA * (OUT ? 2 : 1) + 4 * NC + (OUT ? 8 : 0)) * FB];
    // by chunk parity: prefix sums in two floats, weights of the outputs and of the sources, e^{G_last}
    __shared__ __attribute__((aligned(16))) float sg[2 * 320 + 64 + (DOT ? 64 * NW : 0)];
    lds_u8 *sB = lds_base(smem), *sC = sB + 4 * NA * FB, *sA = sC + 4 * NC * FB, *sM = sA + 4 * NA * FB;
    lds_f *sG = (lds_f *)lds_base(sg), *sD = sG + 640, *sDot = sG + 704;
    const int tid0 = threadIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(tid0 >> 6);
    LinUnit<float> u;
    if (!u.find(p, DA * DC) || (!OUT && u.alone && !p.all)) return;
    const int rows = u.rows, nchunk = u.nchunk;

    // the lane's 8 rows 32 kb + 8 g .. of its column in tile ct of a state in memory
    auto state_at = [&](int kb, int ct) {
        const int g = tid0 >> 4 & 3, n = tid0 & 15;
        const int d = 32 * kb + 8 * g, c = perm_row(w * NCT + ct, n);
        return TR ? d * DC + c : c * DA + d;
    };
    f32x4 P[NCT][NDT];
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    const float *from = !OUT ? nullptr : u.alone ? (p.init ? p.init + u.nstate : nullptr) : p.seg + u.sstate * (DA * DC);
    float *to = !u.alone ? (OUT ? nullptr : p.seg + u.sstate * (DA * DC)) : p.final_state ? p.final_state + u.nstate : nullptr;
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

    const float *yp = DOT ? reinterpret_cast<const float *>(p.y) + u.b * p.sy.b + u.h / p.ry * p.sy.h + (long long)u.first * p.sy.t : nullptr;
    TileStage<true, DA / 8> ta, tb;
    TileStage<true, DC / 8> tc;
    float gn = 0.f;
    double total = 0.0;
    auto load = [&](int c, int tid) {
        const int lane = tid & 63;
        if constexpr (OUT) ta.load(u.ap, p.sa.t, 64 * c, rows, tid);
        tb.load(u.bp, p.sb.t, 64 * c, rows, tid);
        tc.load(u.cp, p.sc.t, 64 * c, rows, tid);
        if (w == NW - 1) gn = 64 * c + lane < rows ? load_g(p.g, u.g0 + (long long)(64 * c + lane) * p.sg.t, p.g32) : 0.f;
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
                Op::put_lane(sM + (2 * it + jb) * FB, lane, V8{s[0], s[1]});
            }
            __builtin_amdgcn_sched_barrier(0);
            f32x4 O[NCT][4];
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
                for (int it = 0; it < 4; ++it) O[ct][it] = zero;
#pragma unroll
            for (int kb = 0; kb < NA; ++kb) {
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                    const V8 af = Op::get(sA + (it * NA + kb) * FB, kb, lane);
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct) O[ct][it] = Op::mma(V8{P[ct][2 * kb], P[ct][2 * kb + 1]}, af, O[ct][it]);
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
                    const V8 m = Op::get_lane(sM + (2 * it + kb) * FB, lane);
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct) O[ct][it] = Op::mma(cf[ct][kb], m, O[ct][it]);
                }
            const int c0 = perm_row(w * NCT, 4 * g);  // the lane's channels c0 .. + 4 NCT
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const int i = perm_row(it, n), row = 64 * c + i;
                if constexpr (DOT) {
                    float d = 0.f;
                    if (row < rows) {
                        const float *y = yp + (long long)row * p.sy.t + c0;
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
                    const V8 x = Op::get(sC + (it * NC + (w * NCT >> 1)) * FB, w * NCT >> 1, lane);
                    if constexpr (NCT == 2) {
                        O[0][it] += m * x.a;
                        O[1][it] += m * x.b;
                    } else {
                        O[0][it] += m * (w & 1 ? x.b : x.a);
                    }
                }
                if (row < rows) {
                    float *o = reinterpret_cast<float *>(p.out) + (u.row0 + row) * DC + c0;
#pragma unroll
                    for (int ct = 0; ct < NCT; ++ct) *reinterpret_cast<f32x4 *>(o + 4 * ct) = O[ct][it];
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
            V8 xf[NCT];
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) xf[ct] = V8{cf[ct][kb].a * w0, cf[ct][kb].b * w1};
#pragma unroll
            for (int dt = 0; dt < NDT; ++dt) {
                const lds_u8 *f = sB + (2 * kb * NA + (dt >> 1)) * FB;
                const V8 bt = Op::get_t(f, f + NA * FB, dt, lane);
#pragma unroll
                for (int ct = 0; ct < NCT; ++ct) P[ct][dt] = Op::mma(bt, xf[ct], P[ct][dt]);
            }
        }
        if constexpr (DOT) {
            barrier_lds();
            if (tid < 64 && 64 * c + tid < rows) {
                float d = 0.f;
#pragma unroll
                for (int k = 0; k < NW; ++k) d += sDot[64 * k + tid];
                p.dots[u.row0 + 64 * c + tid] = d;
            }
        }
    }
    if (!OUT && w == NW - 1 && (tid0 & 63) == 0) p.seg_decay[u.sunit] = ex2((float)total);
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
