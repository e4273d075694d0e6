"""The gradient by the log-decays of linear attention in float64, pair of tokens by pair, and how far a kernel's
may be off.

With X_ij = scale e^{F_i - F_j} (q_i . k_j) (do_i . v_j), the part that token j has in the loss by way of token i
(i > j), first_i = scale e^{F_i} do_i S_0 q_i, end_j = e^{F_last - F_j} v_j R k_j and R the end state's gradient,

  dg_t = sum_{i >= t > j} X_ij + sum_{i >= t} first_i + sum_{j < t} end_j + e^{F_last} <S_0, R>.

The value is taken from this sum as it stands.  The kernels have it as a sum over the tokens u >= t of a row's
and a column's total, row_u = q_u . dq_u and col_u = k_u . dk_u (the pair of a token with itself left out of both),
up to a segment's end, plus <R, S> there, so their error is that of all rows and columns behind t.

Error.  It is made of many independent roundings, so sizes are added as squares.  A pair's part of a row or
a column is a product of two sums over channels, and its size is the larger of what they are and what they are
by the squares of their terms:
  m2_ij = max((q_i . k_j)^2, q_i^2 . k_j^2) max((do_i . v_j)^2, do_i^2 . v_j^2) (scale D_ij)^2,
and as much for the pairs with the start and the end state.  Relative to that size a pair is off
 - with bf16 inputs, twice, by 2^-16: scores (inside a chunk) or the weighted operand and the state (from chunk to
   chunk) enter a product in two bf16 pieces, each of which is off by 2^-8 of what it is made of;
 - by the roundings of 2 d + T + 64 float32 additions at most, 2^-24 each, in quadrature;
 - by its decay, whose exponent x is a float32 (x 2^-24) and which is a product of T / 64 + 2 exponentials at
   most, two steps of 2^-24 each: so x is counted with D, against a rate that is above 16 2^-24.
A rounding that is off by e at most is off by e / sqrt(3) on average.  So `rms`, the sum of the squares of all these e,
bounds the error in norm, and 6 times it, ten standard deviations, each element's; then dg is rounded to its type."""
import torch

from tests.lin_util import BF, HALF


def parts(q, k, v, g, scale, S0, do, R):
    """X, first, end, last <S_0, R>, and the squares of their sizes, exponents counted in."""
    q, k, v, g, do = (t.double() for t in (q, k, v, g, do))
    T, dk, dv = q.shape[0], q.shape[1], v.shape[1]
    S0, R = (torch.zeros(dv, dk, dtype=torch.float64) if t is None else t.double() for t in (S0, R))
    F = g.clamp(min=-1000).cumsum(0)
    low = torch.ones(T, T, dtype=torch.bool).tril(-1)
    x = (F[None] - F[:, None]).masked_fill(~low, float("inf"))
    near = lambda x: torch.where(x == float("inf"), 0.0, torch.exp(-x) * (1 + x / 16))  # a decay, with its exponent
    larger = lambda a, b: torch.maximum(a.square(), b)
    qk, dov = q @ k.T, do @ v.T
    X = scale * torch.exp(-x) * qk * dov
    X2 = (scale * near(x)).square() * larger(qk, q.square() @ k.square().T) * larger(dov, do.square() @ v.square().T)
    a, b = ((do @ S0) * q).sum(-1), ((v @ R) * k).sum(-1)
    first, first2 = scale * torch.exp(F) * a, (scale * near(-F)).square() * larger(a, ((do.square() @ S0.square()) * q.square()).sum(-1))
    w = F[-1] - F
    end, end2 = torch.exp(w) * b, near(-w).square() * larger(b, ((v.square() @ R.square()) * k.square()).sum(-1))
    both = (S0 * R).sum()
    return X, first, end, torch.exp(F[-1]) * both, X2, first2, end2, near(-F[-1]).square() * larger(both, (S0.square() * R.square()).sum())


def dg(q, k, v, g, scale, dtype, gdtype, S0, do, R):
    """(value, bound of each element, rms error) of one value head of one sequence of T >= 1 tokens."""
    X, first, end, both, X2, first2, end2, both2 = parts(q, k, v, g, scale, S0, do, R)
    T, d = q.shape[0], q.shape[1] + v.shape[1]
    from_t = lambda z: z.flip(0).cumsum(0).flip(0)
    before = torch.cat([torch.zeros(T, 1, dtype=torch.float64), X.cumsum(1)[:, :-1]], 1)  # [i, t]: sum over j < t
    value = torch.diagonal(from_t(before)) + from_t(first) + torch.cat([torch.zeros(1), end.cumsum(0)[:-1]]) + both
    rate32 = ((2 * d + T + 64) ** 0.5 + 2 * (T / 64 + 2) ** 0.5) * 2.0 ** -24
    rate = rate32 + (2 ** 0.5 * 2.0 ** -16 if dtype == BF else 0.0)
    rms = rate * (from_t(X2.sum(1) + first2 + X2.sum(0) + end2) + end2.sum() + both2).sqrt()
    return value, HALF[gdtype] * value.abs() * 1.01 + 6 * rms + 1e-30, rms


def shares(got, ref, dtype_g):
    """(the worst element's share of its bound, the norm's of its own)."""
    value, bound, rms = ref
    e = got.double().cpu() - value
    return float((e.abs() / bound).max()), float(e.norm() / (HALF[dtype_g] * value.norm() * 1.01 + rms.norm() + 1e-30))


def check(got, ref, gdtype, what):
    assert torch.isfinite(got).all(), "non-finite " + what
    worst, norm = shares(got, ref, gdtype)
    value, _, rms = ref
    print("  %s: worst share of the bound %.3f, of the norm's %.3f; rms error allowed %.1e of dg's" % (
        what, worst, norm, float(rms.norm() / value.norm().clamp(min=1e-30))), flush=True)
    assert worst <= 1.0 and norm <= 1.0, "%s: %.3f and %.3f of the bounds" % (what, worst, norm)
