"""Problems whose launches would take 2^32 work-items or more in x are refused on the host, as a shape,
and those just below are not: the gated delta rule's and latent attention's entry points, without a GPU."""
import pytest
import torch

import chunked_gated_linear_bounded_amd as kda

FAKE = 0x100000  # aligned, never dereferenced
E_SHAPE = -2
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("N,H,T,dk,dv,dtype,packed,backward,fits", [
    # 512 threads for every 32 value columns of a sequence and head
    (1 << 21, 1, 64, 64, 128, BF, True, False, False), ((1 << 21) - 8, 1, 64, 64, 128, BF, True, False, True),
    (1 << 17, 16, 64, 128, 128, F32, True, False, False), (1 << 17, 16, 64, 128, 128, BF, True, True, False),
    # the reverse pass in float32 at dk = 128: for every 16
    (1 << 20, 1, 64, 128, 128, F32, True, True, False), ((1 << 20) - 8, 1, 64, 128, 128, F32, True, True, True),
    # 256 threads a chunk, 512 in the gradient stage
    (1, 1, 1 << 30, 64, 64, BF, False, False, False), (1, 1, (1 << 30) - 64, 64, 64, BF, False, False, True),
    (1, 1, 1 << 29, 64, 64, BF, False, True, False), (1, 1, (1 << 29) - 64, 64, 64, BF, False, True, True),
])
def test_gdr_chunks(N, H, T, dk, dv, dtype, packed, backward, fits):
    assert (kda.gdr_workspace_bytes(N, 1, H, T, dk, dv, dtype, packed=packed, backward=backward) > 0) == fits
    if not fits and not backward:
        st = kda.lib().kda_gdr_chunk_fwd(FAKE, None, FAKE, None, FAKE, None, FAKE, None, FAKE, None, FAKE if packed else None, N, 1, H,
                                         T, dk, dv, int(dtype == F32), 1.0, None, FAKE, None, FAKE, 1 << 50, None)
        assert st == E_SHAPE


def test_gdr_one_token():
    a = [FAKE] * 5 + [1 << 21, 1, 1, 128, 128, 0, 1.0, FAKE, FAKE, None]
    assert kda.lib().kda_gdr_decode_step(*a) == E_SHAPE


@pytest.mark.parametrize("N,H,T,dtype,fits", [
    (65536, 128, 65536, BF, False), (65000, 128, 65000, BF, True), (65000, 128, 66000, F32, False), # one head: eight units of 2^20 tiles of 128 rows, 512 threads each
    (1, 1, 1 << 27, BF, False), (1, 1, (1 << 27) - 128, BF, True),
])
def test_latent_backward(N, H, T, dtype, fits):
    assert (kda.latent_bwd_workspace_bytes(N, H, T, T, 128, 64, dtype, packed=N > 1) > 0) == fits


def test_latent_forward_and_one_token():
    fwd = [FAKE, None] * 4 + [FAKE, FAKE, 1 << 17, 128, 1 << 17, 1 << 17, 128, 64, 0, 0.1, FAKE, FAKE, None]
    assert kda.lib().kda_latent_attn_fwd(*fwd) == E_SHAPE
    one = [FAKE] * 4 + [65535, 65535, 50, 64, 20, 512, 64, 0, 0.1, FAKE, FAKE, FAKE, 1 << 50, None]
    assert kda.lib().kda_latent_decode_step(*one) == E_SHAPE
    assert kda.latent_decode_workspace_bytes(65535, 65535, 64, 20, 512, 64, BF) == 0
