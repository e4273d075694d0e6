"""LinChunkFunction's own decisions, without a GPU: what it refuses under a capture."""
import pytest
import torch

import chunked_gated_linear_bounded_amd as kda


def test_leaves_may_be_captured_where_nothing_is_differentiated(monkeypatch):
    """Parameters in a capture under no_grad or inference_mode go as far as the check of the device; with
    gradients enabled they are refused in every place."""
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    x, g, s0 = torch.zeros(1, 2, 8, 64), torch.zeros(1, 2, 8), torch.zeros(1, 2, 64, 64)
    leaf = lambda t: t.clone().requires_grad_()
    places = [(leaf(x), x, x, g, 1.0, s0), (x, leaf(x), x, g, 1.0, s0), (x, x, leaf(x), g, 1.0, s0), (x, x, x, leaf(g), 1.0, s0),
              (x, x, x, g, 1.0, leaf(s0))]
    for args in places:
        for context in (torch.no_grad, torch.inference_mode):
            with context(), pytest.raises(ValueError, match="GPU"):
                kda.LinChunkFunction.apply(*args)
        with pytest.raises(RuntimeError, match="leaf"):
            kda.LinChunkFunction.apply(*args)


def test_gradients_that_nobody_asked_for_are_not_made(monkeypatch):
    """The backward is given the end state's gradient only where there is one, and zeros in dout's place where
    the output was not used."""
    from chunked_gated_linear_bounded_amd import lin
    seen = []

    def fwd(q, k, v, g, cu, scale, out, fs, want, s0, ws, stream):
        return v * 1, torch.ones(v.shape[0], v.shape[1], v.shape[3], q.shape[3])

    def bwd(q, k, v, g, dout, cu, scale, s0, dfinal, ws, stream, want_dg, want_dinitial):
        seen.append((dout, dfinal, want_dg, want_dinitial))
        return dict(dq=q * 1, dk=k * 1, dv=v * 1, dg=g * 1 if want_dg else None, dinitial_state=None)

    monkeypatch.setattr(lin, "_fwd", fwd)
    monkeypatch.setattr(lin, "_bwd", bwd)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    x, g = torch.randn(1, 2, 8, 64), torch.randn(1, 2, 8)
    leaf = lambda t: t.clone().requires_grad_()
    out, fs = kda.LinChunkFunction.apply(leaf(x), x, x, leaf(g))
    out.sum().backward()
    out, fs = kda.LinChunkFunction.apply(leaf(x), x, x, g)
    fs.sum().backward()
    out, fs = kda.LinChunkFunction.apply(leaf(x), x, x, g)
    (out.sum() + fs.transpose(-1, -2).mul(2).sum()).backward()
    (d0, f0, g0, _), (d1, f1, g1, _), (d2, f2, _, _) = seen
    assert f0 is None and bool((d0 == 1).all()) and g0 and not g1
    assert d1.shape == x.shape and bool((d1 == 0).all()) and bool((f1 == 1).all())
    assert bool((d2 == 1).all()) and bool((f2 == 2).all()) and f2.is_contiguous()
    # neither used: nothing to do
    q = leaf(x)
    out, fs = kda.LinChunkFunction.apply(q, x, x, g)
    assert torch.autograd.grad((q * 2).sum(), q)[0] is not None and len(seen) == 3
