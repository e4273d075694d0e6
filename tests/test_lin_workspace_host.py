"""Workspace of decayed linear attention, without a GPU: what it grows with."""
import pytest
import torch

import chunked_gated_linear_bounded_amd as kda

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,T,dk,dv", [(32, 65536, 128, 128), (4, 5000, 64, 128), (1, 1 << 20, 64, 64)])
def test_short_documents_have_no_states(H, T, dk, dv, dtype):
    """A document more in the stream takes no state more, beyond one in every 32 tokens, but with dfinal_state and dg
    the one that its gradient is multiplied with."""
    state, fwd = dk * dv * 4, lambda n: kda.lin_workspace_bytes(n, H, H, T, dk, dv, dtype, packed=True)
    bwd = lambda n, e: kda.lin_workspace_bytes(n, H, H, T, dk, dv, dtype, packed=True, backward=True, end_state=e)
    room = lambda n: 16 * H * (T // 64 + n) + 4096  # decays, of any number of segments
    many = min(T // 2, 20000)  # (2^24 pieces of 4 KiB of states are refused)
    dots = 2 * H * T * 4 + 4096
    for n in (1, 9, 100, many):
        assert fwd(n) <= 2 * fwd(1) + room(n), n
        assert bwd(n, False) - dots <= 2 * (bwd(1, False) - dots) + room(n), n
        assert 0 <= bwd(n, True) - bwd(n, False) - n * H * state < 256
        assert fwd(n) <= H * (T // 32 + 1) * state + room(n)
    # as many states as there can be segments, while that is fewer (decays begin and end at multiples of 16 bytes)
    assert abs(fwd(2) - fwd(1) - H * (state + 4)) < 16


def test_batches_of_one_segment_have_no_states():
    H, T, d = 8, 100, 128
    a, b = (kda.lin_workspace_bytes(n, H, H, T, d, d, BF, backward=True, end_state=False) for n in (1, 1001))
    assert b - a < 1000 * H * (2 * T * 4 + 16) + 4096
    # a caller that does not say gets enough for either
    assert kda.lin_workspace_bytes(3, H, H, T, d, d, BF, backward=True) >= kda.lin_workspace_bytes(3, H, H, T, d, d, BF, backward=True, end_state=False)


def test_the_call_asks_for_what_the_query_says():
    """One byte less is refused, whichever gradients are asked for; a smaller workspace does where dfinal_state or dg
    is left out (T = 0: nothing is launched)."""
    FAKE, E_WS, OK = 0x100000, -6, 0
    N, H, T, d = 3, 2, 200, 64

    def call(ws, df, dg, T):
        x = [FAKE, None] * 5
        return kda.lib().kda_lin_chunk_bwd(*x, None, N, H, H, T, d, d, 0, 0, 1.0, None, FAKE if df else None, FAKE, FAKE, FAKE, FAKE if dg else None,
                                           None, FAKE, ws, None)

    for df, dg in ((False, False), (False, True), (True, False), (True, True)):
        need = kda.lin_workspace_bytes(N, H, H, T, d, d, BF, backward=True, end_state=df and dg)
        assert call(need - 1, df, dg, T) == E_WS
        none = kda.lin_workspace_bytes(N, H, H, 0, d, d, BF, backward=True, end_state=df and dg)
        assert call(none - 1, df, dg, 0) == E_WS and call(none, df, dg, 0) == OK


@pytest.mark.parametrize("B,Hk,H,T,forward,backward", [
    (1, 1, 1, (1 << 28) - 64, True, True), (1, 1, 1, 1 << 28, True, False), (1, 1, 128, (1 << 21) + 64, True, False),
    (1, 64, 128, (1 << 21) - 64, True, True),                            # shared key heads
    (2, 64, 64, 1 << 21, True, False), (1, 1, 1, (1 << 31) - (1 << 19) - 1, True, False), (1, 1, 1, (1 << 31) - (1 << 19), False, False),
])
def test_limits_of_the_forward_are_its_own(B, Hk, H, T, forward, backward):
    """What only the backward's launches cannot take, the forward does."""
    FAKE, E_SHAPE, E_WS = 0x100000, -2, -6
    d = 64
    assert (kda.lin_workspace_bytes(B, Hk, H, T, d, d, BF) > 0) == forward
    assert (kda.lin_workspace_bytes(B, Hk, H, T, d, d, BF, backward=True) > 0) == backward
    x = [FAKE, None] * 4
    st = kda.lib().kda_lin_chunk_fwd(*x, None, B, Hk, H, T, d, d, 0, 0, 1.0, None, FAKE, None, None, 0, None)
    assert st == (E_WS if forward else E_SHAPE)
    st = kda.lib().kda_lin_chunk_bwd(*x, FAKE, None, None, B, Hk, H, T, d, d, 0, 0, 1.0, None, None, FAKE, FAKE, FAKE, FAKE, None, None, 0, None)
    assert st == (E_WS if backward else E_SHAPE)
