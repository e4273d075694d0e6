"""What the bounds of drafted tokens' outputs notice on histories of latent_pieces_util.py: mistakes planted in
the reference."""
import pytest
import torch

from tests import latent_pieces_util as P
from tests.test_gpu_latent_serving import BF, F32, attend

SCALE = 0.07


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,rows_a_piece", [(20011, 128), (20011, 64), (9001, 64), (3000, 320)])
def test_a_lost_piece_is_noticed(n, rows_a_piece, dtype):
    gen = torch.Generator().manual_seed(3)
    rows, q = P.history(n, 512, dtype, gen), P.queries(1, 1, 8, 512, dtype, gen)[0, 0]
    ref, tol, lref, _ = attend(q, rows, SCALE, 512, dtype)
    ltol = P.lse_bound(q, rows, SCALE, lref)
    worst = lambda got: (float(((got[0] - ref).abs() / (tol + 1e-30)).max()), float(((got[1] - lref).abs() / (ltol + 1e-30)).max()))
    assert max(worst((ref.to(dtype).double(), lref.float().double()))) <= 1.0
    pieces = -(-n // rows_a_piece)
    s = q.double() @ rows.double().T * SCALE

    def joined(weights):  # of each piece, beside its own
        p = torch.exp(s - s.max(-1, keepdim=True).values) * torch.repeat_interleave(weights, rows_a_piece)[:n]
        return p @ rows[:, :512].double() / p.sum(-1, keepdim=True), torch.log(p.sum(-1)) + s.max(-1).values

    for i in sorted({0, 1, 62, 63, 64, 65, 127, 128, pieces - 2, pieces - 1}):
        if not 0 <= i < pieces:
            continue
        for w in (0.0, 2.0):  # lost; twice
            weights = torch.ones(pieces, dtype=torch.float64)
            weights[i] = w
            out, lse = worst(joined(weights))
            print("  piece %d times %g: %.1f, %.1f" % (i, w, out, lse))
            assert out > 4.0 and (lse > 1.0 or i == pieces - 1)  # (the last one may be a few rows)
