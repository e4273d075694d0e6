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
