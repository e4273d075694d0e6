"""Decayed linear attention of packed streams with many more documents than segments: documents of one
segment, which have no state in the workspace, beside long ones.  Bounds as in lin_util.py."""
import pytest
import torch

import chunked_gated_linear_bounded_amd as kda
from tests import lin_util as U

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.lib()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,dk,dv,lens", [
    # segments of one chunk: starts anywhere in one, lengths of just more than one
    (2, 64, 128, [3, 65, 65, 1, 0, 0, 64, 128, 129, 2] + [1] * 20 + [300, 65] + [0] * 9 + [66, 7]),
    (1, 128, 64, [7] * 60 + [700]), (1, 64, 64, [65] * 3 + [0] * 30),
    # and of several (a full card)
    (32, 64, 64, [1] * 40 + [700, 64, 1500] + [9] * 50 + [130, 520, 259, 257] + [0] * 20),
    (40, 64, 64, [65] * 5 + [1100, 3, 900, 130]),
])
def test_more_documents_than_segments(H, dk, dv, lens, dtype):
    """With and without start states and end states, from a workspace of NaN of exactly the size asked for; each
    document against float64, and the same bits as alone in the stream where its segments are the same."""
    cu = [2]
    for n in lens:
        cu.append(cu[-1] + n)
    T, N = cu[-1] + 5, len(lens)
    q, k, v, g = U.inputs(0, 1, H, T, dk, dv, dtype, 91, packed=True)
    do = U.inputs(0, 1, H, T, dk, dv, dtype, 92, packed=True)[2]
    gen = torch.Generator().manual_seed(93)
    s0, df = (torch.randn(N, H, dv, dk, generator=gen) for _ in range(2))
    x, dd, c = [t.cuda() for t in (q, k, v, g)], do.cuda(), torch.tensor(cu, dtype=torch.int32).cuda()
    need = lambda **kw: kda.lin_workspace_bytes(N, 1, H, T, dk, dv, dtype, packed=True, **kw)
    room = torch.empty(need(backward=True) + 4096, dtype=torch.uint8, device="cuda")

    def ws(**kw):
        room.fill_(255)
        return room[:need(**kw)]

    for init, end in ((s0, df), (None, df), (s0, None), (None, None)):
        i, e = (None if t is None else t.cuda() for t in (init, end))
        w = ws()
        out, fs = kda.lin_chunk_fwd_varlen(*x, c, scale=0.1, initial_state=i, return_final_state=True, workspace=w)
        torch.cuda.synchronize()
        assert bool((room[w.numel():] == 255).all())
        w = ws(backward=True, end_state=end is not None)
        d = kda.lin_chunk_bwd_varlen(*x, dd, c, scale=0.1, initial_state=i, dfinal_state=e, workspace=w)
        torch.cuda.synchronize()
        assert bool((room[w.numel():] == 255).all())
        for n in (range(N) if init is not None and end is not None else sorted(range(N), key=lambda n: -lens[n])[:4]):
            s = slice(cu[n], cu[n + 1])
            for h in {0, H - 1}:
                got = {"out": out[h:h + 1, s], "final_state": fs[n, h:h + 1], "dinitial_state": d["dinitial_state"][n, h:h + 1],
                       **{m: d[m][h:h + 1, s] for m in ("dv", "dg")}, **({m: d[m][:, s] for m in ("dq", "dk")} if H == 1 else {})}
                U.check_sequence(got, "%d %d " % (n, h), 1, 1, lambda _: U.one(
                    q[0, s], k[0, s], v[h, s], g[h, s], 0.1, dtype, dtype, None if init is None else init[n, h], do[h, s],
                    None if end is None else end[n, h]), dtype, dtype)
