// Expanded latent attention, backward.  With p_ij recomputed from the kept log-sum-exp and
// delta_i = sum_j p_ij (dout_i . v_j) = dout_i . out_i:
//   dp_ij = dout_i . v_j,  ds_ij = p_ij (dp_ij - delta_i),
//   dq_i = scale sum_j ds_ij key_j,  dkey_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij dout_i,
// key_j = [k_j, k_rope_j]; k_rope's gradient is summed over the heads.
//
// Two kernels, so that no sum needs atomics: one walks the keys of 128 queries (dq, and delta on the
// way), one the queries of 128 keys (dk, dv), seven products for five.  The other side comes in tiles
// of 32 rows through LDS.  Four waves hold their own side's operands and make p and ds, four others
// hold the accumulators and take p and ds as operands, a tile behind: by themselves the operands (80
// registers a lane) and the accumulators (160) leave two waves a SIMD, which fill each other's waits,
// where one wave with both (340) spent 9,900 cycles on a 64 x 128 tile whose matrix work is 2,560.
//
// delta from the kept output carries the output's rounding, 2^-9 of |dout| |out|, and ds is what is left
// of p (dp - delta): little where a query sees few keys or one of them has most of p.  (One key: ds = 0,
// which is set, as p is 1 but for the rounding of the log-sum-exp.  8 keys, bf16: dq off by 2.7e-3 from this alone, where rounding ds costs 1.4e-3.)  So a tile of queries
// that see at most kExactKeys keys walks them once more, first, for the sum itself; and every tile adds
// up its ds, whose sum would be 0, so that the delta left for dk and dv is the sum in float32 in any
// case.  At 256 keys the rounding has fallen to a tenth of ds's own and a second walk would be 60 % of
// the kernel's work.
//
// What is handed over is rounded to the inputs' type as the MFMA takes it in either case.  Sums of a few
// terms keep all of a term's rounding (dk 2.8e-3 off where the outputs' own rounding leaves 1.8e-3), so
// the ds of a sequence of up to kExactKeys keys are two bf16 pieces, with a second product, which costs
// so short a sequence nothing (and a long one, whose waves branch around it, 1 to 3 %).  The rotary
// part's gradient goes to a float32 partial per head, which a third kernel sums.  16 heads x 4096
// queries and keys, 128 + 64 channels: dq 179 us, dk and dv 212 us, matrix units busy 38 and 41 % of
// the time, the LDS 47 and 49 %; one kind of wave, 64-row tiles: 270 and 325 us.
#pragma once
#include "latent_common.h"

namespace kda {

constexpr int kExactKeys = 256;

struct LatentBwdArgs {
    const void *q, *k, *kr, *v, *out, *dout;
    Strides3 sq, sk, skr, sv, sdo;
    AttnSeqs seqs;
    int H, NB, ntile;          // heads; batch entries; tiles of this kernel's side per batch entry
    float scale;
    const float *lse;          // [B][H][T]
    float *delta;              // [B][H][T]
    void *dq;                  // [B][H][T][dn + dr]
    void *dk, *dv;             // [B][H][S][dn]
    float *dkr;                // [B][H][S][dr] partials
};

// LDS of a 512-thread work-group: three tiles, and what the four makers hand over, twice
template <bool F32, int FRAGS, int HAND> struct LatentBwdLds {
    static constexpr int TILE = FRAGS * AttnOp<F32>::FB, EX = 3 * TILE, EXB = 4 * HAND * AttnOp<F32>::FB, BYTES = EX + 2 * EXB;
};

// s = X a, d = Y c: rows 0 .. 31 of a tile (X: NA column blocks from f on, Y: NC from e on) against NX
// operand columns a lane.  A group's fragments are read while the group before is multiplied; left to
// itself the compiler waits for each one it reads.
template <typename Op, int NA, int NC, int NX>
__device__ __forceinline__ void tile_products(const lds_u8 *f, const lds_u8 *e, int lane, const typename Op::V8 (&a)[NX][NA],
                                              const typename Op::V8 (&c)[NX][NC], f32x4 (&s)[2][NX], f32x4 (&d)[2][NX]) {
    typename Op::V8 fa[2][NA], fc[2][NC];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int x = 0; x < NX; ++x) s[t][x] = d[t][x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < NA; ++kb) fa[0][kb] = Op::get(f + kb * Op::FB, kb, lane);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int kb = 0; kb < NC; ++kb) fc[t][kb] = Op::get(e + (t * NC + kb) * Op::FB, kb, lane);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int kb = 0; kb < NA; ++kb)
#pragma unroll
            for (int x = 0; x < NX; ++x) s[t][x] = Op::mma(fa[t][kb], a[x][kb], s[t][x]);
        if (t == 0) {
#pragma unroll
            for (int kb = 0; kb < NA; ++kb) fa[1][kb] = Op::get(f + (NA + kb) * Op::FB, kb, lane);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int kb = 0; kb < NC; ++kb)
#pragma unroll
            for (int x = 0; x < NX; ++x) d[t][x] = Op::mma(fc[t][kb], c[x][kb], d[t][x]);
    }
}

template <int DN, int DR, bool F32>
__global__ __launch_bounds__(512) void latent_dq_kernel(const LatentBwdArgs p) {
    using Op = AttnOp<F32>;
    using E = typename Op::E;
    using V8 = typename Op::V8;
    constexpr int NKB = (DN + DR) / 32, NDB = DN / 32, NT = (DN + DR) / 16, NQ = F32 ? 1 : 2, BM = 64 * NQ;
    constexpr int HAND = F32 ? NQ : 2 * NQ;  // ds, and what rounding left of it
    using S = LatentBwdLds<F32, 2 * NKB + 2 * NDB, HAND>;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[S::BYTES];
    lds_u8 *sx = lds_base(smem);
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, n = lane & 15;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6), w = wid & 3;
    const int unit = (blockIdx.x >> 3) / p.ntile * 8 + (blockIdx.x & 7);
    const int slot = p.ntile - 1 - (blockIdx.x >> 3) % p.ntile;
    if (unit >= p.NB * p.H) return;
    const int b = unit / p.H, h = unit % p.H;
    int seq, tile, q0, nq, k0, nk;
    if (!p.seqs.template find<BM>(p.seqs.cu_q, p.seqs.T, b, slot, seq, tile)) return;
    AttnSeqs::range(p.seqs.cu_q, seq, p.seqs.T, q0, nq);
    AttnSeqs::range(p.seqs.cu_k, seq, p.seqs.S, k0, nk);
    if (tile * BM >= nq) return;
    const int qw = tile * BM + 16 * NQ * w, shift = nk - nq;
    const E *kp = reinterpret_cast<const E *>(p.k) + b * p.sk.b + h * p.sk.h + (long long)k0 * p.sk.t;
    const E *rp = reinterpret_cast<const E *>(p.kr) + b * p.skr.b + (long long)k0 * p.skr.t;
    const E *vp = reinterpret_cast<const E *>(p.v) + b * p.sv.b + h * p.sv.h + (long long)k0 * p.sv.t;
    const size_t row0 = (size_t)(b * p.H + h) * p.seqs.T + q0;
    const int nkey = max(0, min(nk, min(tile * BM + BM - 1, nq - 1) + shift + 1)), ntk = (nkey + 31) / 32;
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

    TileStage<F32, DN / 8, 32, 512> stk, stv;
    TileStage<F32, DR / 8, 32, 512> str;
    auto load = [&](int kt) {  // behind the last tile it loads nothing
        stk.load(kp, p.sk.t, 32 * kt, nk, tid);
        str.load(rp, p.skr.t, 32 * kt, nk, tid);
        stv.load(vp, p.sv.t, 32 * kt, nk, tid);
    };
    auto store = [&](int buf) {
        lds_u8 *to = sx + buf * S::TILE;
        stk.store(to, NKB, 0, tid);
        str.store(to, NKB, NDB, tid);
        stv.store(to + 2 * NKB * Op::FB, NDB, 0, tid);
    };
    const bool exact = nk <= kExactKeys;
    const int pass0 = nkey <= kExactKeys ? 0 : 1;  // pass 0: delta alone

    // step kt: tile kt + 1 to LDS; p and ds of tile kt; the products of tile kt - 1
    if (wid < 4) {
        const E *qp = reinterpret_cast<const E *>(p.q) + b * p.sq.b + h * p.sq.h + (long long)q0 * p.sq.t + 8 * g;
        const E *dp_ = reinterpret_cast<const E *>(p.dout) + b * p.sdo.b + h * p.sdo.h + (long long)q0 * p.sdo.t + 8 * g;
        const E *op = reinterpret_cast<const E *>(p.out) + row0 * DN + 8 * g;
        const float c = p.scale * kLog2e;
        V8 qf[NQ][NKB], df[NQ][NDB];
        float lse[NQ], delta[NQ], rest[NQ];  // rest: sum of ds over the keys
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            const int r = min(qw + 16 * x + n, nq - 1);
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) qf[x][kb] = Op::load(qp + (long long)r * p.sq.t + 32 * kb);
            float d = 0.f;
#pragma unroll
            for (int kb = 0; kb < NDB; ++kb) {
                df[x][kb] = Op::load(dp_ + (long long)r * p.sdo.t + 32 * kb);
                float a[8], o[8];
                ld8(dp_ + (long long)r * p.sdo.t + 32 * kb, a);
                ld8(op + (size_t)r * DN + 32 * kb, o);
#pragma unroll
                for (int j = 0; j < 8; ++j) d = fmaf(a[j], o[j], d);
            }
            delta[x] = pass0 == 0 ? 0.f : col_sum(d);
            const float e = p.lse[row0 + r];
            lse[x] = e == -INFINITY ? 0.f : e * kLog2e;  // nothing seen: no key below the mask either
        }
        for (int pass = pass0; pass < 2; ++pass) {
#pragma unroll
            for (int x = 0; x < NQ; ++x) rest[x] = 0.f;
            barrier_lds();  // the pass before has read its tiles
            load(0);
            store(0);
            load(1);
            int buf = 0;
            for (int kt = 0; kt <= ntk; ++kt) {
                barrier_lds();
                const int nb = buf == 2 ? 0 : buf + 1;
                store(nb);
                load(kt + 2);
                if (kt < ntk) {
                    const lds_u8 *sk = sx + buf * S::TILE, *sv = sk + 2 * NKB * Op::FB;
                    const int first = 32 * kt;
                    const bool edge = first + 32 > nk || first + 31 > qw + shift;
                    f32x4 s[2][NQ], d[2][NQ];
                    tile_products<Op>(sk, sv, lane, qf, df, s, d);
                    if (edge)  // one branch a tile, not one an element
#pragma unroll
                        for (int x = 0; x < NQ; ++x) {
                            const int see = min(nk - 1, qw + 16 * x + n + shift) - first - 8 * g;
#pragma unroll
                            for (int t = 0; t < 2; ++t)
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    s[t][x][i] = perm_row(t, i) > see ? -INFINITY : s[t][x][i];
                                    d[t][x][i] = see + first + 8 * g == 0 ? delta[x] : d[t][x][i];  // one key: ds = 0
                                }
                        }
#pragma unroll
                    for (int x = 0; x < NQ; ++x) {
#pragma unroll
                        for (int t = 0; t < 2; ++t)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float pr = ex2(fmaf(s[t][x][i], c, -lse[x]));
                                s[t][x][i] = pr * (d[t][x][i] - delta[x]);
                                rest[x] += s[t][x][i];
                            }
                        lds_u8 *to = sx + S::EX + (kt & 1) * S::EXB + (w * HAND + x) * Op::FB;
                        const V8 r = Op::pair(s[0][x], s[1][x]);
                        Op::put_lane(to, lane, r);
                        if constexpr (!F32)
                            if (exact) Op::put_lane(to + NQ * Op::FB, lane, Op::rest(s[0][x], s[1][x], r));
                    }
                }
                buf = nb;
            }
#pragma unroll
            for (int x = 0; x < NQ; ++x) delta[x] += col_sum(rest[x]);
        }
#pragma unroll
        for (int x = 0; x < NQ; ++x)
            if (g == 0 && qw + 16 * x + n < nq) p.delta[row0 + qw + 16 * x + n] = delta[x];
        return;
    }
    f32x4 dq[NT][NQ];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int x = 0; x < NQ; ++x) dq[t][x] = zero;
    for (int pass = pass0; pass < 2; ++pass) {
        barrier_lds();
        load(0);
        store(0);
        load(1);
        int buf = 0;
        for (int kt = 0; kt <= ntk; ++kt) {
            barrier_lds();
            const int nb = buf == 2 ? 0 : buf + 1, pb = buf == 0 ? 2 : buf - 1;
            store(nb);
            load(kt + 2);
            if (kt > 0 && pass > 0) {
                const lds_u8 *sk = sx + pb * S::TILE;
                auto add = [&](const lds_u8 *from) {
                    V8 sf[NQ];
#pragma unroll
                    for (int x = 0; x < NQ; ++x) sf[x] = Op::get_lane(from + (w * HAND + x) * Op::FB, lane);
                    // four column tiles' fragments are read while the four before are multiplied
                    V8 f4[2][4];
                    auto read = [&](int j) {
#pragma unroll
                        for (int t = 4 * j; t < min(4 * j + 4, NT); ++t) {
                            const lds_u8 *f0 = sk + (t >> 1) * Op::FB;
                            f4[j & 1][t & 3] = Op::get_t(f0, f0 + NKB * Op::FB, t, lane);
                        }
                    };
                    read(0);
#pragma unroll
                    for (int j = 0; j < (NT + 3) / 4; ++j) {
                        read(j + 1);
                        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                        for (int t = 4 * j; t < min(4 * j + 4, NT); ++t)
#pragma unroll
                            for (int x = 0; x < NQ; ++x) dq[t][x] = Op::mma(f4[j & 1][t & 3], sf[x], dq[t][x]);
                    }
                };
                const lds_u8 *ex = sx + S::EX + ((kt - 1) & 1) * S::EXB;
                add(ex);
                if constexpr (!F32)
                    if (exact) add(ex + NQ * Op::FB);
            }
            buf = nb;
        }
    }
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        const int r = qw + 16 * x + n;
        if (r >= nq) continue;
#pragma unroll
        for (int t = 0; t < NT; t += 2) {
            f32x4 a = dq[t][x], d = dq[t + 1][x];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] *= p.scale;
                d[i] *= p.scale;
            }
            Op::store8(reinterpret_cast<E *>(p.dq) + (row0 + r) * (DN + DR) + 16 * t + 8 * g, a, d);
        }
    }
}

template <int DN, int DR, bool F32>
__global__ __launch_bounds__(512) void latent_dkv_kernel(const LatentBwdArgs p) {
    using Op = AttnOp<F32>;
    using E = typename Op::E;
    using V8 = typename Op::V8;
    constexpr int NKB = (DN + DR) / 32, NDB = DN / 32, NT = (DN + DR) / 16, NV = DN / 16, NK = F32 ? 1 : 2, BN = 64 * NK;
    constexpr int HAND = F32 ? 2 * NK : 3 * NK;  // p, ds, and what rounding left of ds
    using S = LatentBwdLds<F32, 2 * NKB + 2 * NDB, HAND>;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[S::BYTES];
    __shared__ __attribute__((aligned(16))) float sl[3][32], sd[3][32];
    lds_u8 *sx = lds_base(smem);
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, n = lane & 15;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6), w = wid & 3;
    const int unit = (blockIdx.x >> 3) / p.ntile * 8 + (blockIdx.x & 7), slot = (blockIdx.x >> 3) % p.ntile;
    if (unit >= p.NB * p.H) return;
    const int b = unit / p.H, h = unit % p.H;
    int seq, tile, q0, nq, k0, nk;
    if (!p.seqs.template find<BN>(p.seqs.cu_k, p.seqs.S, b, slot, seq, tile)) return;
    AttnSeqs::range(p.seqs.cu_q, seq, p.seqs.T, q0, nq);
    AttnSeqs::range(p.seqs.cu_k, seq, p.seqs.S, k0, nk);
    if (tile * BN >= nk) return;
    const int kw = tile * BN + 16 * NK * w, shift = nk - nq;
    const E *qp = reinterpret_cast<const E *>(p.q) + b * p.sq.b + h * p.sq.h + (long long)q0 * p.sq.t;
    const E *dp_ = reinterpret_cast<const E *>(p.dout) + b * p.sdo.b + h * p.sdo.h + (long long)q0 * p.sdo.t;
    const size_t qrow = (size_t)(b * p.H + h) * p.seqs.T + q0;
    const bool exact = nk <= kExactKeys;
    // queries that see the tile's first key stand at its index minus shift, or later
    const int t_first = max(0, tile * BN - shift) / 32, ntq = max(0, (nq + 31) / 32 - t_first);
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

    TileStage<F32, DN / 8, 32, 512> stq, sto;
    TileStage<F32, DR / 8, 32, 512> str;
    float rl = 0.f, rd = 0.f;
    auto load = [&](int i) {  // behind the last tile it loads nothing
        const int row = 32 * (t_first + i);
        stq.load(qp, p.sq.t, row, nq, tid);
        str.load(qp + DN, p.sq.t, row, nq, tid);
        sto.load(dp_, p.sdo.t, row, nq, tid);
        if (tid < 32 && nq > 0) {
            const int r = min(row + tid, nq - 1);
            rl = p.lse[qrow + r];
            rd = p.delta[qrow + r];
        }
    };
    auto store = [&](int buf) {
        lds_u8 *to = sx + buf * S::TILE;
        stq.store(to, NKB, 0, tid);
        str.store(to, NKB, NDB, tid);
        sto.store(to + 2 * NKB * Op::FB, NDB, 0, tid);
        if (tid < 32) {
            sl[buf][tid] = rl == -INFINITY ? 0.f : rl * kLog2e;
            sd[buf][tid] = rd;
        }
    };
    load(0);
    store(0);
    load(1);

    // step i: tile i + 1 to LDS; p and ds of tile i; the products of tile i - 1
    if (wid < 4) {
        const E *kp = reinterpret_cast<const E *>(p.k) + b * p.sk.b + h * p.sk.h + (long long)k0 * p.sk.t + 8 * g;
        const E *rp = reinterpret_cast<const E *>(p.kr) + b * p.skr.b + (long long)k0 * p.skr.t + 8 * g;
        const E *vp = reinterpret_cast<const E *>(p.v) + b * p.sv.b + h * p.sv.h + (long long)k0 * p.sv.t + 8 * g;
        const float c = p.scale * kLog2e;
        V8 kf[NK][NKB], vf[NK][NDB];
#pragma unroll
        for (int x = 0; x < NK; ++x) {
            const int r = min(kw + 16 * x + n, nk - 1);
#pragma unroll
            for (int kb = 0; kb < NDB; ++kb) {
                kf[x][kb] = Op::load(kp + (long long)r * p.sk.t + 32 * kb);
                vf[x][kb] = Op::load(vp + (long long)r * p.sv.t + 32 * kb);
            }
#pragma unroll
            for (int kb = NDB; kb < NKB; ++kb) kf[x][kb] = Op::load(rp + (long long)r * p.skr.t + 32 * (kb - NDB));
        }
        int buf = 0;
        for (int it = 0; it <= ntq; ++it) {
            barrier_lds();
            const int nb = buf == 2 ? 0 : buf + 1;
            store(nb);
            load(it + 2);
            if (it < ntq) {
                const lds_u8 *sq = sx + buf * S::TILE, *so = sq + 2 * NKB * Op::FB;
                const int first = 32 * (t_first + it);
                const bool edge = first + 32 > nq || first + shift < kw + 16 * NK - 1;
                f32x4 s[2][NK], d[2][NK], l4[2], d4[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    l4[t] = *reinterpret_cast<const f32x4 *>(sl[buf] + perm_row(t, 4 * g));
                    d4[t] = *reinterpret_cast<const f32x4 *>(sd[buf] + perm_row(t, 4 * g));
#pragma unroll
                    for (int x = 0; x < NK; ++x) s[t][x] = d[t][x] = zero;
#pragma unroll
                    for (int kb = 0; kb < NKB; ++kb) {
                        const V8 qf = Op::get(sq + (t * NKB + kb) * Op::FB, kb, lane);
#pragma unroll
                        for (int x = 0; x < NK; ++x) s[t][x] = Op::mma(qf, kf[x][kb], s[t][x]);
                    }
#pragma unroll
                    for (int kb = 0; kb < NDB; ++kb) {
                        const V8 of = Op::get(so + (t * NDB + kb) * Op::FB, kb, lane);
#pragma unroll
                        for (int x = 0; x < NK; ++x) d[t][x] = Op::mma(of, vf[x][kb], d[t][x]);
                    }
                }
                if (edge)  // one branch a tile, not one an element
#pragma unroll
                    for (int x = 0; x < NK; ++x) {
                        const int seen = kw + 16 * x + n - shift - first - 8 * g, none = nq - first - 8 * g;  // rows seen .. none - 1
                        const int lone = -shift - first - 8 * g;  // the row that sees one key
#pragma unroll
                        for (int t = 0; t < 2; ++t)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                s[t][x][i] = (perm_row(t, i) >= none) | (perm_row(t, i) < seen) ? -INFINITY : s[t][x][i];
                                d[t][x][i] = perm_row(t, i) == lone ? d4[t][i] : d[t][x][i];
                            }
                    }
#pragma unroll
                for (int x = 0; x < NK; ++x) {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float pr = ex2(fmaf(s[t][x][i], c, -l4[t][i]));
                            s[t][x][i] = pr;
                            d[t][x][i] = pr * (d[t][x][i] - d4[t][i]);
                        }
                    lds_u8 *to = sx + S::EX + (it & 1) * S::EXB + (w * HAND + x) * Op::FB;
                    const V8 r = Op::pair(d[0][x], d[1][x]);
                    Op::put_lane(to, lane, Op::pair(s[0][x], s[1][x]));
                    Op::put_lane(to + NK * Op::FB, lane, r);
                    if constexpr (!F32)
                        if (exact) Op::put_lane(to + 2 * NK * Op::FB, lane, Op::rest(d[0][x], d[1][x], r));
                }
            }
            buf = nb;
        }
        return;
    }
    f32x4 dk[NT][NK], dv[NV][NK];
#pragma unroll
    for (int x = 0; x < NK; ++x) {
#pragma unroll
        for (int t = 0; t < NT; ++t) dk[t][x] = zero;
#pragma unroll
        for (int t = 0; t < NV; ++t) dv[t][x] = zero;
    }
    int buf = 0;
    for (int it = 0; it <= ntq; ++it) {
        barrier_lds();
        const int nb = buf == 2 ? 0 : buf + 1, pb = buf == 0 ? 2 : buf - 1;
        store(nb);
        load(it + 2);
        if (it > 0) {
            const lds_u8 *sq = sx + pb * S::TILE, *so = sq + 2 * NKB * Op::FB;
            const lds_u8 *ex = sx + S::EX + ((it - 1) & 1) * S::EXB + w * HAND * Op::FB;
            V8 pf[NK];
#pragma unroll
            for (int x = 0; x < NK; ++x) pf[x] = Op::get_lane(ex + x * Op::FB, lane);
#pragma unroll
            for (int t = 0; t < NV; ++t) {
                const lds_u8 *f0 = so + (t >> 1) * Op::FB;
                const V8 of = Op::get_t(f0, f0 + NDB * Op::FB, t, lane);
#pragma unroll
                for (int x = 0; x < NK; ++x) dv[t][x] = Op::mma(of, pf[x], dv[t][x]);
            }
            auto add = [&](const lds_u8 *from) {
                V8 sf[NK];
#pragma unroll
                for (int x = 0; x < NK; ++x) sf[x] = Op::get_lane(from + x * Op::FB, lane);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const lds_u8 *f0 = sq + (t >> 1) * Op::FB;
                    const V8 qf = Op::get_t(f0, f0 + NKB * Op::FB, t, lane);
#pragma unroll
                    for (int x = 0; x < NK; ++x) dk[t][x] = Op::mma(qf, sf[x], dk[t][x]);
                }
            };
            add(ex + NK * Op::FB);
            if constexpr (!F32)
                if (exact) add(ex + 2 * NK * Op::FB);
        }
        buf = nb;
    }
#pragma unroll
    for (int x = 0; x < NK; ++x) {
        const int r = kw + 16 * x + n;
        if (r >= nk) continue;
        const size_t row = (size_t)(b * p.H + h) * p.seqs.S + k0 + r;
#pragma unroll
        for (int t = 0; t < NV; t += 2)
            Op::store8(reinterpret_cast<E *>(p.dv) + row * DN + 16 * t + 8 * g, dv[t][x], dv[t + 1][x]);
#pragma unroll
        for (int t = 0; t < NT; t += 2) {
            f32x4 a = dk[t][x], d = dk[t + 1][x];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] *= p.scale;
                d[i] *= p.scale;
            }
            if (t < NV) {
                Op::store8(reinterpret_cast<E *>(p.dk) + row * DN + 16 * t + 8 * g, a, d);
            } else {
                float *to = p.dkr + row * DR + 16 * (t - NV) + 8 * g;
                *reinterpret_cast<f32x4 *>(to) = a;
                *reinterpret_cast<f32x4 *>(to + 4) = d;
            }
        }
    }
}

// Sum of the heads' partials of the rotary key part: part [B][H][S][DR] -> out [B][S][DR], keys that
// no sequence covers as zeros.
template <typename E>
__global__ __launch_bounds__(256) void latent_dkr_kernel(const float *part, AttnSeqs seqs, int H, int DR, E *out) {
    const int b = blockIdx.y;
    const long long n = (long long)seqs.S * DR, at = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;
    if (at >= n) return;
    const int row = (int)(at / DR);
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    bool covered = true;
    if (seqs.cu_k) {
        const int lo = AttnSeqs::clip(seqs.cu_k[0], seqs.S), hi = AttnSeqs::clip(seqs.cu_k[seqs.N], seqs.S);
        covered = row >= lo && row < hi;
    }
    if (covered)
        for (int h = 0; h < H; ++h) s += *reinterpret_cast<const f32x4 *>(part + ((long long)b * H + h) * n + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) out[b * n + at + i] = from_f<E>(s[i]);
}

// Rows of to [H][total][width] that no sequence of a packed stream covers, as zeros.
template <typename E>
__global__ __launch_bounds__(256) void latent_uncovered_kernel(const int *cu, int N, int total, int width, E *to) {
    const int lo = AttnSeqs::clip(cu[0], total), hi = max(lo, AttnSeqs::clip(cu[N], total));
    const long long n = (long long)(lo + total - hi) * width;
    for (long long i = blockIdx.x * 256 + threadIdx.x; i < n; i += 256 * gridDim.x) {
        const long long row = i / width;
        to[((long long)blockIdx.y * total + (row < lo ? row : hi + row - lo)) * width + i % width] = (E)0.f;
    }
}

}  // namespace kda
