"""The reference of the log-decays' gradient (lin_decay_util.py) against differences in float64, and what its
bounds notice: every planted mistake here is in the reference's own sum."""
import pytest
import torch

from tests import lin_decay_util as D
from tests import lin_util as U

BF, F32 = torch.bfloat16, torch.float32


def case(T, dk, dv, dtype, kind, seed=5):
    q, k, v, g = (t[0, 0] for t in U.inputs(1, 1, 1, T, dk, dv, dtype, seed, rate={"far": -6.0}.get(kind, -3.0)))
    do = U.inputs(1, 1, 1, T, dk, dv, dtype, seed + 1)[2][0, 0]
    gen = torch.Generator().manual_seed(seed)
    s0, df = (torch.randn(dv, dk, generator=gen) if kind != "no states" else None for _ in range(2))
    if kind == "strong":
        g = (-20 * torch.rand(T, generator=gen)).to(dtype)
    return q, k, v, g, s0, do, df


def test_value_against_differences_and_the_other_reference():
    q, k, v, g, s0, do, df = case(90, 64, 64, F32, "states")
    value, *_ = D.dg(q, k, v, g, 0.1, F32, F32, s0, do, df)
    x = [t.double() for t in (q, k, v)]
    gd = g.double()

    def loss(g):
        o = U.one(*x, g, 0.1, F32, F32, s0)
        return float((o["out"][0] * do.double()).sum() + (o["final_state"][0] * df.double()).sum())

    for t in (0, 1, 30, 63, 64, 88, 89):
        h = torch.zeros(90, dtype=torch.float64)
        h[t] = 1e-4 * abs(float(gd[t])) + 1e-6
        slope = (loss(gd + h) - loss(gd - h)) / (2 * float(h[t]))
        assert abs(slope - float(value[t])) <= 1e-6 * (1 + float(value.abs().max())), t
    other = U.one(q, k, v, g, 0.1, F32, F32, s0, do, df)["dg"][0]
    assert float((other - value).abs().max()) <= 1e-9 * float(value.abs().max())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,dk,dv,kind", [(64, 64, 128, "states"), (257, 128, 128, "states"), (700, 128, 128, "no states"), (1030, 64, 128, "states"),
                                          (1030, 64, 64, "far"), (700, 64, 64, "strong"), (330, 64, 64, "strong")])
def test_mistakes_are_noticed(T, dk, dv, kind, dtype):
    q, k, v, g, s0, do, df = case(T, dk, dv, dtype, kind)
    ref = D.dg(q, k, v, g, 0.1, dtype, dtype, s0, do, df)
    X, first, end, both, *_ = D.parts(q, k, v, g, 0.1, s0, do, df)
    value = ref[0]
    assert max(D.shares(value.to(dtype), ref, dtype)) <= 1.0  # rounded, and nothing else
    from_t = lambda z: z.flip(0).cumsum(0).flip(0)
    row, col = X.sum(1) + first, X.sum(0) + end
    segment = torch.arange(T) // 64
    wrong = {"zeros": 0 * value, "sign": -value, "a token late": torch.cat([value[:1], value[:-1]]), "off by a little": value * (1.001 if dtype == F32 else 1.02),
             "no rows": value - from_t(row), "no columns": value + from_t(col)}
    if T > 64:
        # one segment without what passes over its end (the end that most passes over), or with its neighbour's
        t1 = max(range(64, T, 64), key=lambda t: abs(float(value[t])))
        inside, over = segment == t1 // 64 - 1, float(value[t1])
        wrong["no tail"] = torch.where(inside, value - over, value)
        wrong["a neighbour's tail"] = torch.where(inside, value - over + float(value[t1 - 64]), value)
        # a chunk whose rows, or columns, are the one's in front of it
        for name, z in (("rows", row), ("columns", -col)):
            there = torch.zeros(T, dtype=torch.float64)
            there[64:128] = (torch.roll(z, 64) - z)[64:128]
            wrong["a chunk's " + name] = value + torch.where(segment <= 1, from_t(there), 0.0)
    if kind not in ("no states", "strong"):  # (strong decays leave nothing of a state behind the first token)
        wrong["no start state"] = value - from_t(first) - both
        wrong["no end state"] = value - torch.cat([torch.zeros(1), end.cumsum(0)[:-1]]) - both
    for name, x in wrong.items():
        worst, norm = D.shares(x.to(dtype), ref, dtype)
        print("  %s: %.1f, %.1f" % (name, worst, norm))
        assert worst > 1.0, name
