// Expanded latent attention, backward.  With p_ij recomputed from the kept log-sum-exp and
// delta_i = dout_i . out_i:
//   dp_ij = dout_i . v_j,  ds_ij = p_ij (dp_ij - delta_i),
//   dq_i = scale sum_j ds_ij key_j,  dkey_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij dout_i,
// key_j = [k_j, k_rope_j]; k_rope's gradient is summed over the heads.
//
// Two kernels, so that no sum needs atomics: one walks the keys of 128 queries (dq, and delta on the
// way), one the queries of 128 keys (dk, dv), seven products for five.  Both hold their own side's
// operands and their accumulators in registers (up to 340 a lane, one wave per SIMD, bf16) and stage
// the other side 64 rows at a time through 40 KiB of LDS.  The rotary part's gradient goes to a
// float32 partial per head, which a third kernel sums.
#pragma once
#include "latent_common.h"

namespace kda {

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

template <int DN, int DR, bool F32>
__global__ __launch_bounds__(256, 1) void latent_dq_kernel(const LatentBwdArgs p) {
    using Op = AttnOp<F32>;
    using E = typename Op::E;
    using V8 = typename Op::V8;
    constexpr int NKB = (DN + DR) / 32, NDB = DN / 32, NT = (DN + DR) / 16, NQ = F32 ? 1 : 2, BM = 64 * NQ;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[(4 * NKB + 4 * NDB) * Op::FB];
    lds_u8 *sk = lds_base(smem), *sv = sk + 4 * NKB * Op::FB;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, n = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
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
    const E *qp = reinterpret_cast<const E *>(p.q) + b * p.sq.b + h * p.sq.h + (long long)q0 * p.sq.t + 8 * g;
    const E *dp_ = reinterpret_cast<const E *>(p.dout) + b * p.sdo.b + h * p.sdo.h + (long long)q0 * p.sdo.t + 8 * g;
    const size_t row0 = (size_t)(b * p.H + h) * p.seqs.T + q0;
    const E *op = reinterpret_cast<const E *>(p.out) + row0 * DN + 8 * g;
    const int nkey = max(0, min(nk, min(tile * BM + BM - 1, nq - 1) + shift + 1)), ntk = (nkey + 63) / 64;
    const float c = p.scale * kLog2e;

    V8 qf[NQ][NKB], df[NQ][NDB];
    float lse[NQ], delta[NQ];
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
        delta[x] = col_sum(d);
        const float e = p.lse[row0 + r];
        lse[x] = e == -INFINITY ? 0.f : e * kLog2e;  // nothing seen: no key below the mask either
        if (g == 0 && qw + 16 * x + n < nq) p.delta[row0 + r] = delta[x];
    }
    f32x4 dq[NT][NQ];
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int x = 0; x < NQ; ++x) dq[t][x] = zero;
    TileStage<F32, DN / 8> stk, stv;
    TileStage<F32, DR / 8> str;
    if (ntk > 0) {
        stk.load(kp, p.sk.t, 0, nk, tid);
        str.load(rp, p.skr.t, 0, nk, tid);
        stv.load(vp, p.sv.t, 0, nk, tid);
    }
    for (int kt = 0; kt < ntk; ++kt) {
        barrier_lds();
        stk.store(sk, NKB, 0, tid);
        str.store(sk, NKB, NDB, tid);
        stv.store(sv, NDB, 0, tid);
        barrier_lds();
        stk.load(kp, p.sk.t, 64 * kt + 64, nk, tid);  // behind the last tile it loads nothing
        str.load(rp, p.skr.t, 64 * kt + 64, nk, tid);
        stv.load(vp, p.sv.t, 64 * kt + 64, nk, tid);
        const int first = 64 * kt;
        const bool edge = first + 64 > nk || first + 63 > qw + shift;
#pragma unroll
        for (int hb = 0; hb < 2; ++hb) {  // 32 keys: the k of one MFMA
            f32x4 s[2][NQ], d[2][NQ];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int x = 0; x < NQ; ++x) s[t][x] = d[t][x] = zero;
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb) {
                    const V8 kf = Op::get(sk + ((2 * hb + t) * NKB + kb) * Op::FB, kb, lane);
#pragma unroll
                    for (int x = 0; x < NQ; ++x) s[t][x] = Op::mma(kf, qf[x][kb], s[t][x]);
                }
#pragma unroll
                for (int kb = 0; kb < NDB; ++kb) {
                    const V8 vf = Op::get(sv + ((2 * hb + t) * NDB + kb) * Op::FB, kb, lane);
#pragma unroll
                    for (int x = 0; x < NQ; ++x) d[t][x] = Op::mma(vf, df[x][kb], d[t][x]);
                }
            }
            V8 sf[NQ];
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                const int see = min(nk - 1, qw + 16 * x + n + shift) - first - 8 * g;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (edge && perm_row(2 * hb + t, i) > see) s[t][x][i] = -INFINITY;
                        const float pr = ex2(fmaf(s[t][x][i], c, -lse[x]));
                        s[t][x][i] = pr * (d[t][x][i] - delta[x]);
                    }
                sf[x] = Op::pair(s[0][x], s[1][x]);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const lds_u8 *f0 = sk + (2 * hb * NKB + (t >> 1)) * Op::FB;
                const V8 kf = Op::get_t(f0, f0 + NKB * Op::FB, t, lane);
#pragma unroll
                for (int x = 0; x < NQ; ++x) dq[t][x] = Op::mma(kf, sf[x], dq[t][x]);
            }
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
__global__ __launch_bounds__(256, 1) void latent_dkv_kernel(const LatentBwdArgs p) {
    using Op = AttnOp<F32>;
    using E = typename Op::E;
    using V8 = typename Op::V8;
    constexpr int NKB = (DN + DR) / 32, NDB = DN / 32, NT = (DN + DR) / 16, NV = DN / 16, NK = F32 ? 1 : 2, BN = 64 * NK;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[(4 * NKB + 4 * NDB) * Op::FB];
    __shared__ __attribute__((aligned(16))) float sl[64], sd[64];
    lds_u8 *sq = lds_base(smem), *so = sq + 4 * NKB * Op::FB;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, n = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int unit = (blockIdx.x >> 3) / p.ntile * 8 + (blockIdx.x & 7), slot = (blockIdx.x >> 3) % p.ntile;
    if (unit >= p.NB * p.H) return;
    const int b = unit / p.H, h = unit % p.H;
    int seq, tile, q0, nq, k0, nk;
    if (!p.seqs.template find<BN>(p.seqs.cu_k, p.seqs.S, b, slot, seq, tile)) return;
    AttnSeqs::range(p.seqs.cu_q, seq, p.seqs.T, q0, nq);
    AttnSeqs::range(p.seqs.cu_k, seq, p.seqs.S, k0, nk);
    if (tile * BN >= nk) return;
    const int kw = tile * BN + 16 * NK * w, shift = nk - nq;
    const E *kp = reinterpret_cast<const E *>(p.k) + b * p.sk.b + h * p.sk.h + (long long)k0 * p.sk.t + 8 * g;
    const E *rp = reinterpret_cast<const E *>(p.kr) + b * p.skr.b + (long long)k0 * p.skr.t + 8 * g;
    const E *vp = reinterpret_cast<const E *>(p.v) + b * p.sv.b + h * p.sv.h + (long long)k0 * p.sv.t + 8 * g;
    const E *qp = reinterpret_cast<const E *>(p.q) + b * p.sq.b + h * p.sq.h + (long long)q0 * p.sq.t;
    const E *dp_ = reinterpret_cast<const E *>(p.dout) + b * p.sdo.b + h * p.sdo.h + (long long)q0 * p.sdo.t;
    const size_t qrow = (size_t)(b * p.H + h) * p.seqs.T + q0;
    const float c = p.scale * kLog2e;
    // queries that see the tile's first key stand at its index minus shift, or later
    const int t_first = max(0, tile * BN - shift) / 64, t_end = (nq + 63) / 64;

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
    f32x4 dk[NT][NK], dv[NV][NK];
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < NK; ++x) {
#pragma unroll
        for (int t = 0; t < NT; ++t) dk[t][x] = zero;
#pragma unroll
        for (int t = 0; t < NV; ++t) dv[t][x] = zero;
    }
    TileStage<F32, DN / 8> stq, sto;
    TileStage<F32, DR / 8> str;
    float rl = 0.f, rd = 0.f;
    auto load = [&](int qt) {
        stq.load(qp, p.sq.t, 64 * qt, nq, tid);
        str.load(qp + DN, p.sq.t, 64 * qt, nq, tid);
        sto.load(dp_, p.sdo.t, 64 * qt, nq, tid);
        if (tid < 64) {
            const int r = min(64 * qt + tid, nq - 1);
            const float e = p.lse[qrow + r];
            rl = e == -INFINITY ? 0.f : e * kLog2e;
            rd = p.delta[qrow + r];
        }
    };
    if (t_first < t_end) load(t_first);
    for (int qt = t_first; qt < t_end; ++qt) {
        barrier_lds();
        stq.store(sq, NKB, 0, tid);
        str.store(sq, NKB, NDB, tid);
        sto.store(so, NDB, 0, tid);
        if (tid < 64) {
            sl[tid] = rl;
            sd[tid] = rd;
        }
        barrier_lds();
        load(qt + 1);  // behind the last tile it loads nothing
        const int first = 64 * qt;
        const bool edge = first + 64 > nq || first + shift < kw + 16 * NK - 1;
#pragma unroll
        for (int hb = 0; hb < 2; ++hb) {
            f32x4 s[2][NK], d[2][NK];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int x = 0; x < NK; ++x) s[t][x] = d[t][x] = zero;
#pragma unroll
                for (int kb = 0; kb < NKB; ++kb) {
                    const V8 qf = Op::get(sq + ((2 * hb + t) * NKB + kb) * Op::FB, kb, lane);
#pragma unroll
                    for (int x = 0; x < NK; ++x) s[t][x] = Op::mma(qf, kf[x][kb], s[t][x]);
                }
#pragma unroll
                for (int kb = 0; kb < NDB; ++kb) {
                    const V8 of = Op::get(so + ((2 * hb + t) * NDB + kb) * Op::FB, kb, lane);
#pragma unroll
                    for (int x = 0; x < NK; ++x) d[t][x] = Op::mma(of, vf[x][kb], d[t][x]);
                }
            }
            V8 pf[NK], sf[NK];
            f32x4 l4[2], d4[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                l4[t] = *reinterpret_cast<const f32x4 *>(sl + perm_row(2 * hb + t, 4 * g));
                d4[t] = *reinterpret_cast<const f32x4 *>(sd + perm_row(2 * hb + t, 4 * g));
            }
#pragma unroll
            for (int x = 0; x < NK; ++x) {
                const int seen = kw + 16 * x + n - shift - first - 8 * g, none = nq - first - 8 * g;  // rows seen .. none - 1
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = perm_row(2 * hb + t, i);
                        if (edge && (row >= none || row < seen)) s[t][x][i] = -INFINITY;
                        const float pr = ex2(fmaf(s[t][x][i], c, -l4[t][i]));
                        s[t][x][i] = pr;
                        d[t][x][i] = pr * (d[t][x][i] - d4[t][i]);
                    }
                pf[x] = Op::pair(s[0][x], s[1][x]);
                sf[x] = Op::pair(d[0][x], d[1][x]);
            }
#pragma unroll
            for (int t = 0; t < NV; ++t) {
                const lds_u8 *f0 = so + (2 * hb * NDB + (t >> 1)) * Op::FB;
                const V8 of = Op::get_t(f0, f0 + NDB * Op::FB, t, lane);
#pragma unroll
                for (int x = 0; x < NK; ++x) dv[t][x] = Op::mma(of, pf[x], dv[t][x]);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const lds_u8 *f0 = sq + (2 * hb * NKB + (t >> 1)) * Op::FB;
                const V8 qf = Op::get_t(f0, f0 + NKB * Op::FB, t, lane);
#pragma unroll
                for (int x = 0; x < NK; ++x) dk[t][x] = Op::mma(qf, sf[x], dk[t][x]);
            }
        }
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
// no sequence covers as zeros; and those keys' rows of dk, dv, those queries' rows of dq as zeros.
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
