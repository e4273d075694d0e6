"""Float64 reference of decayed linear attention for the tests, pair of tokens by pair of tokens, and the
error bounds of its kernels.

With F the sum of the log-decays, out_i = scale (sum_{j <= i} e^{F_i - F_j} (q_i . k_j) v_j + e^{F_i} S_0 q_i).

Bounds.  A result is a sum of terms; `size` is that sum with every factor by magnitude.  Each term is off
by what its factors are carried with: 2^-16 where bf16 inputs' scores and states enter a product again in
two pieces, nothing but float32's own rounding in the state (three pieces hold all 24 bits) and with
float32 inputs.  Every term passes sums of dk + dv + T + 64 float32 additions at most (each off by 2^-24
of what is summed so far, so by `size`), and a decay that is a product of up to T / 64 + 2 exponentials:
a few steps of 2^-24 each, and 2^-24 of its exponent, which is at most 0.54 / e of the undecayed term.
Then the result is rounded to its type."""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative
BF = torch.bfloat16


def inputs(B, Hk, H, T, dk, dv, dtype, seed, packed=False, rate=-3.0, g32=False):
    """q, k, v, g of a batch [B,H,T,d], or of a packed stream [H,T,d]."""
    gen = torch.Generator().manual_seed(seed)
    lead = (lambda h: (h, T)) if packed else (lambda h: (B, h, T))
    q, k, v = (torch.randn(*lead(h), d, generator=gen).to(dtype) for h, d in ((Hk, dk), (Hk, dk), (H, dv)))
    g = -torch.exp(torch.randn(*lead(H), generator=gen) * 1.5 + rate)
    return q, k, v, g if g32 else g.to(dtype)


def rel(dtype, T, d, pieces=True):
    return (2.0 ** -16 if pieces and dtype == BF else 0.0) + (2 * d + T + 64 + 8 * (T // 64 + 2)) * 2.0 ** -24


def one(q, k, v, g, scale, dtype, gdtype, S0=None, dout=None, dfinal=None):
    """One value head of one sequence: {name: (value, bound)} for out, final_state and, with dout, the
    gradients (dq and dk of this value head alone, their bounds without the last rounding)."""
    q, k, v, g = (t.double() for t in (q, k, v, g))
    T, dk, dv = q.shape[0], q.shape[1], v.shape[1]
    S0 = torch.zeros(dv, dk, dtype=torch.float64) if S0 is None else S0.double()
    F = g.clamp(min=-1000).cumsum(0) if T else g
    low = torch.ones(T, T, dtype=torch.bool).tril()
    D = torch.exp((F[:, None] - F[None]).masked_fill(~low, float("-inf")))
    # a decay's own error grows with its exponent x: x e^-x <= 0.37 for every pair
    D1 = D + 0.4 * low
    e, e1 = torch.exp(F)[:, None], torch.exp(F)[:, None] + 0.4
    w = torch.exp(F[-1] - F)[:, None] if T else e
    last = torch.exp(F[-1]) if T else torch.ones(())
    r, rs = rel(dtype, T, dk + dv), rel(dtype, T, dk + dv, pieces=False)
    M, N0 = scale * (q @ k.T) * D, None
    Ma = abs(scale) * (q.abs() @ k.abs().T) * D1
    out = M @ v + scale * e * (q @ S0.T)
    size = Ma @ v.abs() + abs(scale) * e1 * (q.abs() @ S0.abs().T)
    S = last * S0 + (w * v).T @ k
    Sa = S0.abs() + ((w + 0.4) * v.abs()).T @ k.abs() if T else S0.abs()
    got = {"out": (out, HALF[dtype] * out.abs() * 1.01 + r * size + 1e-30), "final_state": (S, HALF[torch.float32] * S.abs() + rs * Sa + 1e-30)}
    if dout is None:
        return got
    do = dout.double()
    R = torch.zeros_like(S0) if dfinal is None else dfinal.double()
    N, Na = scale * (do @ v.T) * D, abs(scale) * (do.abs() @ v.abs().T) * D1
    dq = N @ k + scale * e * (do @ S0)
    dqa = Na @ k.abs() + abs(scale) * e1 * (do.abs() @ S0.abs())
    dk_ = N.T @ q + w * (v @ R)
    dka = Na.T @ q.abs() + (w + 0.4) * (v.abs() @ R.abs())
    dv_ = M.T @ do + w * (k @ R.T)
    dva = Ma.T @ do.abs() + (w + 0.4) * (k.abs() @ R.abs().T)
    ds = last * R + scale * (e * do).T @ q
    dsa = R.abs() + abs(scale) * (e1 * do.abs()).T @ q.abs()
    # pairs of different tokens; those with the start state and with the end state
    X = M * (do @ v.T)
    X = X - torch.diag(torch.diagonal(X))
    first = scale * e[:, 0] * ((q @ S0.T) * do).sum(-1)
    end = w[:, 0] * ((k @ R.T) * v).sum(-1)
    through = X.sum(1) + first - X.sum(0) - end
    both = last * (S0 * R).sum() + end.sum()  # what passes over the sequence's end
    dg = through.flip(0).cumsum(0).flip(0) + both
    rows = (q.abs() * dqa).sum(-1) + (k.abs() * dka).sum(-1)
    dga = rows.sum() + (Sa * R.abs()).sum() + sum((Sa * dsa).sum() for _ in range(1))
    got.update(dq=(dq, r * dqa + 1e-30), dk=(dk_, r * dka + 1e-30), dv=(dv_, HALF[dtype] * dv_.abs() * 1.01 + r * dva + 1e-30),
               dinitial_state=(ds, HALF[torch.float32] * ds.abs() + rs * dsa + 1e-30),
               dg=(dg, HALF[gdtype] * dg.abs() * 1.01 + r * dga + 1e-30))
    return got


def check(got, ref, bound, what, dtype=None):
    """Element by element against the bound; with a type also in norm: independent roundings of half a
    step at most leave a relative norm below half a step, and 2^-13 covers all the rest."""
    got, ref = got.double().cpu(), ref.double()
    assert got.shape == ref.shape, what
    assert torch.isfinite(got).all(), "non-finite %s" % what
    d = (got - ref).abs()
    worst = float((d / bound).max()) if d.numel() else 0.0
    norm = float(d.norm() / ref.norm().clamp(min=1e-30)) if d.numel() else 0.0
    print("  %s: worst share of the bound %.3f, relative norm %.2e" % (what, worst, norm), flush=True)
    assert worst <= 1.0, "%s: %.3f of the bound" % (what, worst)
    if dtype is not None and d.numel() > 64:
        most = HALF[dtype] + 2.0 ** -13 if dtype == BF else 2.0 ** -15
        assert norm <= most, "%s: relative norm %.2e" % (what, norm)


def check_sequence(x, what, H, r, ref, dtype, gdtype):
    """x: {name: tensor} of one sequence ([H,T,..], states [H,..]) against ref(h) -> one(...)."""
    sums = {}
    for h in range(H):
        want = ref(h)
        for n, (value, bound) in want.items():
            if n in ("dq", "dk"):
                a, c = sums.get((n, h // r), (0.0, 0.0))
                sums[n, h // r] = (a + value, c + bound)
            elif x.get(n) is not None:
                # dg's terms cancel: no bound in its norm
                check(x[n][h], value, bound, "%s%s %d" % (what, n, h), None if n == "dg" else torch.float32 if "state" in n else dtype)
    for (n, h), (value, bound) in sums.items():
        if x.get(n) is not None:
            check(x[n][h], value, bound + HALF[dtype] * value.abs() * 1.01, "%s%s %d" % (what, n, h), dtype)
