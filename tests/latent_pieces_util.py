"""Histories of the paged latent cache in which every tile of 64 rows shows in the result by itself.

Tile k's rows have a one in channel k of the latent and zeros beside it, and the queries' absorbed part is zero: so
scores come from the rotary parts alone, and out's channel k is the softmax's mass of tile k.  A tile, or a
piece of several, that is lost, taken twice or weighted as another leaves its own channels off by their whole size,
where with random rows it moves every channel by less than bf16's rounding."""
import torch


def history(n, dc, dtype, gen):
    """[n, dc + 64] rows."""
    assert n <= 64 * dc
    rows = torch.zeros(n, dc + 64)
    rows[torch.arange(n), torch.arange(n) // 64] = 1
    rows[:, dc:] = torch.randn(n, 64, generator=gen)
    return rows.to(dtype)


def queries(B, T, H, dc, dtype, gen):
    q = torch.zeros(B, T, H, dc + 64)
    q[..., dc:] = torch.randn(B, T, H, 64, generator=gen) * 2
    return q.to(dtype)


def lse_bound(q, rows, scale, lse):
    """A sum of exponentials is off by no more than its terms are: by a score's error, a float32 sum of D products
    (2^-24 of their size each, twice for what is subtracted from it), by 2^-21 for the exponential and the sum; and
    the result is a float32 made of two."""
    size = float((q.double().abs() @ rows.double().abs().T).max()) * scale if rows.shape[0] else 0.0
    return 2 * q.shape[-1] * 2.0 ** -24 * size + 2.0 ** -21 + 2.0 ** -22 * torch.where(torch.isinf(lse), 0.0, lse.abs())
