"""Float64 reference of the gated delta rule for the tests, and the error bounds of its kernels.

The reference runs the token recurrence; the bounds come from the chunked form in float64, whose
intermediate values (start states P, M, U) say how large the rounded operands are."""
import numpy as np
import torch

U16 = 2.0 ** -11   # fp16, rounded to nearest; twice that where it is cut off
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative


def inputs(B, Hk, H, T, dk, dv, dtype, seed, packed=False, rate=-3.0, unit=True):
    """q, k, v, g, beta of a batch [B,H,T,d], or of a packed stream [H,T,d]."""
    gen = torch.Generator().manual_seed(seed)
    lead = (lambda h: (h, T)) if packed else (lambda h: (B, h, T))
    def unit_rows(*s):
        x = torch.randn(*s, generator=gen, dtype=torch.float64)
        return (x / x.norm(dim=-1, keepdim=True) if unit else x * 0.3).to(dtype)
    q, k = unit_rows(*lead(Hk), dk), unit_rows(*lead(Hk), dk)
    v = torch.randn(*lead(H), dv, generator=gen).to(dtype)
    g = (-torch.exp(torch.randn(*lead(H), generator=gen) * 1.5 + rate)).to(dtype)
    beta = torch.sigmoid(torch.randn(*lead(H), generator=gen)).to(dtype)
    return q, k, v, g, beta


def recurrent(q, k, v, g, beta, scale, S0=None):
    """Token recurrence in float64 on [B,H,T,d] (q, k with Hk heads): out, final state, and each
    token's state norm per value channel (for the bounds)."""
    q, k, v, g, beta = (t.double() for t in (q, k, v, g, beta))
    B, H, T, dv = v.shape
    r = H // k.shape[1]
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    S = torch.zeros(B, H, dv, k.shape[-1], dtype=torch.float64) if S0 is None else S0.double().clone()
    out = torch.zeros(B, H, T, dv, dtype=torch.float64)
    for t in range(T):
        S = torch.exp(g[:, :, t])[..., None, None] * S
        w = beta[:, :, t, None] * (v[:, :, t] - torch.einsum("bhvk,bhk->bhv", S, k[:, :, t]))
        S = S + torch.einsum("bhv,bhk->bhvk", w, k[:, :, t])
        out[:, :, t] = scale * torch.einsum("bhvk,bhk->bhv", S, q[:, :, t])
    return out, S


def chunk_terms(q, k, v, g, beta, scale, S0=None):
    """What the kernels round, summed by magnitude, for one sequence [H,T,d]: a bound on |out| terms
    [H,T,dv] split as (|e^G q| |P|, |M| |U|), and on the state's terms [H,dv,dk] at the end."""
    q, k, v, g, beta = (t.double() for t in (q, k, v, g, beta))
    H, T, dv = v.shape
    r = H // k.shape[0]
    q, k = q.repeat_interleave(r, 0), k.repeat_interleave(r, 0)
    P = torch.zeros(H, k.shape[-1], dv, dtype=torch.float64) if S0 is None else S0.double().transpose(-1, -2).clone()
    inter, intra = torch.zeros_like(v), torch.zeros_like(v)
    size = P.abs()
    for t in range(0, T, 64):
        s = slice(t, min(T, t + 64))
        kc, qc, G = k[:, s], q[:, s], g[:, s].clamp(min=-1000).cumsum(-1)
        D = torch.exp((G[:, :, None] - G[:, None]).tril()) * torch.ones_like(G[0, :, None] - G[0, None]).tril()
        A = (beta[:, s, None] * (kc @ kc.transpose(-1, -2)) * D).tril(-1)
        Tm = torch.linalg.inv(torch.eye(A.shape[-1], dtype=torch.float64) + A)
        eG, eL = torch.exp(G)[..., None], torch.exp(G[:, -1:] - G)[..., None]
        X = beta[:, s, None] * (v[:, s] - eG * (kc @ P))
        Xs = beta[:, s, None] * (v[:, s].abs() + eG * (kc.abs() @ P.abs()))
        U, Us = Tm @ X, Tm.abs() @ Xs
        M = scale * (qc @ kc.transpose(-1, -2)) * D
        inter[:, s] = abs(scale) * eG * (qc.abs() @ P.abs())
        intra[:, s] = M.abs() @ U.abs()
        last = torch.exp(G[:, -1])[:, None, None]
        size = last * size + kc.abs().transpose(-1, -2) @ (eL * Us)
        P = last * P + kc.transpose(-1, -2) @ (eL * U)
    return inter, intra, size.transpose(-1, -2)


def check(got, ref, bound, what):
    got, ref = got.double().cpu(), ref.double()
    assert got.shape == ref.shape, what
    assert torch.isfinite(got).all(), "non-finite %s" % what
    d = (got - ref).abs()
    worst = float((d / bound.clamp(min=1e-300)).max()) if d.numel() else 0.0
    rel = float(d.norm() / ref.norm().clamp(min=1e-300)) if d.numel() else 0.0
    print("  %s: worst share of the bound %.3f, relative norm %.2e" % (what, worst, rel), flush=True)
    assert worst <= 1.0, "%s: %.3f of the bound" % (what, worst)


def out_bound(ref, inter, intra, dtype):
    """|out - exact|: one rounding to the output's type; bf16 inputs: P cut to fp16 (2 U16), M and U
    rounded to fp16 (U16 each), the float32 sums far below; float32 inputs: operands keep 22 bits cut
    off (2^-21 each, four of them on a term's way), sums of up to 192 terms in float32."""
    if dtype == torch.bfloat16:
        return HALF[dtype] * ref.abs() + 1.01 * (2 * U16 * inter + 2 * U16 * intra) + 1e-30
    return HALF[dtype] * ref.abs() + (4 * 2.0 ** -21 + 192 * 2.0 ** -24) * (inter + intra) * 4 + 1e-30


def state_bound(size):
    """|final state - exact|: P, X, T, U each keep 22 bits cut off, float32 sums of up to 192 terms,
    carried over the chunks with the terms' own magnitudes; the factor 4 covers that an error in one
    chunk passes through the next ones' K P and T."""
    return 4 * (4 * 2.0 ** -21 + 192 * 2.0 ** -24) * size + 1e-30
