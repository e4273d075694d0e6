"""The gated delta rule on the GPU where the magnitudes inside a chunk are uneven: keys that end before
the chunk does, betas and keys far from one, value channels that are zero or hold an infinity.  The
bounds are those of gdr_util.py and test_gpu_gdr_bwd.py."""
import pytest
import torch

import chunked_gated_linear_bounded_amd as kda
from gdr_util import check, chunk_terms, inputs, out_bound, recurrent, state_bound
from test_gpu_gdr_bwd import NAMES, compare, reference

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
# sequences, key heads, value heads, dv: one and two column tiles a work-group at dk = 128
SIZES = [(1, 1, 2, 64), (3, 4, 12, 128)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.lib()


def _floor(q, k, v, g, beta, scale):
    """Besides their 11 or 22 bits the fp16 pieces of a block are multiples of 2^-24, with the block's
    bound at 2^13 or above: a value is off by up to 2^-37 of that bound.  For out = M U + ... that is
    2^-37 (max|M| sum_j |U_j| + (|T|_inf max|X|) sum_j |M_ij|), which counts where a token's own decays
    from its chunk's largest are below 2^-13; the inputs of one sequence, [H,T,dv]."""
    q, k, v, g, beta = (t.double() for t in (q, k, v, g, beta))
    r = v.shape[0] // k.shape[0]
    q, k = q.repeat_interleave(r, 0), k.repeat_interleave(r, 0)
    P, floor = torch.zeros(v.shape[0], k.shape[-1], v.shape[-1], dtype=torch.float64), torch.zeros_like(v)
    for t in range(0, v.shape[1], 64):
        s = slice(t, min(v.shape[1], t + 64))
        kc, G = k[:, s], g[:, s].cumsum(-1)
        D = torch.exp((G[:, :, None] - G[:, None]).tril()).tril()
        T = torch.linalg.inv(torch.eye(G.shape[-1], dtype=torch.float64) + (beta[:, s, None] * (kc @ kc.mT) * D).tril(-1))
        X = beta[:, s, None] * (v[:, s] - torch.exp(G)[..., None] * (kc @ P))
        U, M = T @ X, scale * (q[:, s] @ kc.mT) * D
        most = T.abs().sum(-1).amax(-1) * X.abs().amax((-1, -2))
        floor[:, s] = 2.0 ** -37 * (M.abs().amax((-1, -2))[:, None, None] * U.abs().sum(1, keepdim=True)
                                    + most[:, None, None] * M.abs().sum(-1, keepdim=True))
        P = torch.exp(G[:, -1])[:, None, None] * P + kc.mT @ (torch.exp(G[:, -1:] - G)[..., None] * U)
    return floor


def _check_fwd(x, out, fs, scale, channels=slice(None)):
    """`channels`: the value channels that are compared."""
    ref, S = recurrent(*x, scale)
    for b in range(ref.shape[0]):
        inter, intra, size = chunk_terms(*(t[b] for t in x), scale)
        bound = out_bound(ref[b], inter, intra, x[0].dtype) + _floor(*(t[b] for t in x), scale)
        check(out[b][..., channels], ref[b][..., channels], bound[..., channels], "out %d" % b)
        check(fs[b][:, channels], S[b][:, channels], state_bound(size)[:, channels], "state %d" % b)


def _fwd_and_grads(x, dout, scale, skip=()):
    """Forward against the recurrence, gradients (no start state) against its adjoint."""
    dtype, (B, H, T, dv), dk = x[0].dtype, x[2].shape, x[0].shape[-1]
    d = [t.cuda() for t in x]
    out, fs = kda.gdr_chunk_fwd(*d, scale=scale, return_final_state=True)
    _check_fwd(x, out, fs, scale)
    got = kda.gdr_chunk_bwd(*d, dout.cuda(), scale=scale)
    for name, ref in zip(NAMES, reference(x, dout, scale, torch.zeros(B, H, dv, dk), None)):
        if name not in skip:
            compare(got[name], ref, dtype, name)


def _tail(sizes, dtype, decay):
    """Keys and values stop after 30 tokens of the first chunk while the state goes on decaying, and no
    value comes afterwards: what follows is as small as the state is then."""
    B, Hk, H, dv = sizes
    x = inputs(B, Hk, H, 150, 128, dv, dtype, 71, rate=-6.0)
    x[1][:, :, 30:64] = 0.0
    x[2][:, :, 30:] = 0.0
    x[3][:, :, 30:64] = decay
    dout = torch.randn(B, H, 150, dv, generator=torch.Generator().manual_seed(3)).to(dtype)
    dout[:, :, :64] = 0.0  # the gradients of q, g and beta are then as small as the state, too
    return x, dout


@pytest.mark.parametrize("decay", [-0.1, -0.2, -0.5, -1.0])
@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_keys_end_before_the_chunk(dtype, sizes, decay):
    _fwd_and_grads(*_tail(sizes, dtype, decay), 128 ** -0.5)


@pytest.mark.parametrize("T", [64, 150])
@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradients_begin_inside_the_chunk(dtype, sizes, T):
    """The mirror image: no queries, keys and gradients in the first 34 tokens, over which the state
    decays, so that the start state's gradient is as small as that decay."""
    B, Hk, H, dv = sizes
    x = inputs(B, Hk, H, T, 128, dv, dtype, 72, rate=-6.0)
    x[0][:, :, :34] = 0.0
    x[1][:, :, :34] = 0.0
    x[3][:, :, :34] = -0.5
    gen = torch.Generator().manual_seed(4)
    dout = torch.randn(B, H, T, dv, generator=gen).to(dtype)
    dout[:, :, :34] = 0.0
    S0 = torch.randn(B, H, dv, 128, generator=gen) * 0.5
    got = kda.gdr_chunk_bwd(*(t.cuda() for t in x), dout.cuda(), scale=128 ** -0.5, initial_state=S0.cuda())
    ref = reference(x, dout, 128 ** -0.5, S0, None)
    for name, t in zip(NAMES, ref):
        compare(got[name], t, dtype, name)


@pytest.mark.parametrize("norm", [0.3, 1e-3, 300.0])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_beta_far_from_one(dtype, norm):
    """Keys of another norm, and betas that keep beta |k|^2 below one: up to 10, to 9e5, to 1e-5."""
    x = list(inputs(2, 2, 4, 150, 128, 64, dtype, 81))
    x[1] = (x[1].double() * norm).to(dtype)
    x[4] = (x[4].double() * 0.9 / norm ** 2).to(dtype)
    dout = torch.randn(2, 4, 150, 64, generator=torch.Generator().manual_seed(4)).to(dtype)
    _fwd_and_grads(x, dout, 128 ** -0.5)


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_zero_channels(dtype, sizes):
    """Heads padded with zero channels (values and gradients of 16 or 32 columns), beside small values
    and small gradients."""
    B, Hk, H, dv = sizes
    x = inputs(B, Hk, H, 150, 128, dv, dtype, 91)
    dout = torch.randn(B, H, 150, dv, generator=torch.Generator().manual_seed(5)).to(dtype)
    for t in (x[2], dout):
        t *= 2.0 ** -20
        t[..., -32:] = 0.0
    _fwd_and_grads(x, dout, 128 ** -0.5)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_bad_value_stays_in_its_channel(dtype, sizes, bad):
    """An infinity or NaN in one channel of v reaches that channel of the outputs and of the state, from
    its chunk on, and no other; one in dout that channel of dv and of the start state's gradient."""
    B, Hk, H, dv = sizes
    x = list(inputs(B, Hk, H, 150, 128, dv, dtype, 101))
    x[2] *= 8.0
    dout = (8.0 * torch.randn(B, H, 150, dv, generator=torch.Generator().manual_seed(6))).to(dtype)
    rest = [c for c in range(dv) if c != 5]
    d = [t.cuda() for t in x]
    d[2] = d[2].clone()
    d[2][:, :, 70, 5] = bad
    out, fs = kda.gdr_chunk_fwd(*d, return_final_state=True)
    _check_fwd(x, out, fs, 1.0, rest)
    assert torch.isfinite(out[:, :, :64]).all() and not torch.isfinite(out[:, :, 70:, 5]).any()
    assert not torch.isfinite(fs[:, :, 5]).all(-1).any()
    ref = reference(x, dout, 1.0, torch.zeros(B, H, dv, 128), None)
    dirty = dout.cuda()
    dirty[:, :, 70, 5] = bad
    got = kda.gdr_chunk_bwd(*(t.cuda() for t in x), dirty)
    compare(got["dv"][..., rest], ref[2][..., rest], dtype, "dv")
    compare(got["dinitial_state"][:, :, rest], ref[5][:, :, rest], dtype, "dinitial_state")
    assert not torch.isfinite(got["dv"][:, :, 70, 5]).any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_bad_query_stays_in_its_row(dtype):
    x = list(inputs(1, 1, 2, 150, 128, 64, dtype, 111))
    x[0] *= 64.0
    d = [t.cuda() for t in x]
    d[0] = d[0].clone()
    d[0][:, :, 70, 3] = float("inf")
    out, fs = kda.gdr_chunk_fwd(*d, return_final_state=True)
    assert not torch.isfinite(out[:, :, 70]).any()
    out[:, :, 70] = recurrent(*x, 1.0)[0][:, :, 70].to(out)
    _check_fwd(x, out, fs, 1.0)


def test_second_derivatives_are_refused():
    """The gradients carry no graph of their own: a penalty on one is an error, not a term left out."""
    x = [t.cuda().requires_grad_() for t in inputs(1, 1, 1, 64, 64, 64, F32, 121)]
    a = [t.cuda().requires_grad_() for t in inputs(1, 1, 1, 64, 64, 64, F32, 122)]
    for leaf, out in ((x, kda.GdrChunkFunction.apply(*x)[0]), (a, kda.KdaChunkFunction.apply(*a[:3], a[0] * 1.0, a[4])[0])):
        first = torch.autograd.grad(out.square().sum(), leaf[2], create_graph=True)[0]
        with pytest.raises(RuntimeError):
            (first.square().sum() + leaf[0].sum()).backward()


def _loose(t, dims):
    """t with a stride of 13 in dimensions of one, which no row's start depends on."""
    t = t.cuda().contiguous()
    assert all(t.shape[i] == 1 for i in dims)
    return t.as_strided(t.shape, [13 if i in dims else s for i, s in enumerate(t.stride())])


@pytest.mark.parametrize("T,dims", [(70, (0, 1)), (1, (0, 2))])
def test_strides_of_dimensions_of_one(T, dims):
    H = 1 if 1 in dims else 3
    x = inputs(1, H, H, T, 64, 64, BF, 131)
    dout = torch.randn(1, H, T, 64, generator=torch.Generator().manual_seed(7)).to(BF)
    a, b = [t.cuda() for t in x], [_loose(t, dims) for t in x]
    want, got = kda.gdr_chunk_fwd(*a, return_final_state=True), kda.gdr_chunk_fwd(*b, return_final_state=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    want, got = kda.gdr_chunk_bwd(*a, dout.cuda()), kda.gdr_chunk_bwd(*b, _loose(dout, dims))
    assert all(torch.equal(got[n], want[n]) for n in NAMES)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strided_gradient(dtype):
    """dout as a model has it, [B,T,H,d] seen as [B,H,T,d] and a slice of wider rows."""
    x = inputs(2, 2, 4, 70, 128, 64, dtype, 141)
    wide = torch.randn(2, 70, 4, 96, generator=torch.Generator().manual_seed(8)).to(dtype).cuda()
    dout = wide[..., 16:80].transpose(1, 2)
    assert not dout.is_contiguous()
    d = [t.cuda() for t in x]
    want, got = kda.gdr_chunk_bwd(*d, dout.contiguous()), kda.gdr_chunk_bwd(*d, dout)
    assert all(torch.equal(got[n], want[n]) for n in NAMES)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_factors_of_a_bound_far_apart(dtype):
    """A state of 1e30 that decays by e^-80 at a chunk's first token, keys of 1e6 with betas of 1e-12, no
    values: every term is of ordinary size, though products of some of a bound's factors leave float's
    range.  (Spread over the chunk, that decay would leave the state below 2^-37 of what its first tokens
    wrote.)"""
    x = list(inputs(1, 1, 2, 130, 64, 64, dtype, 151))
    x[1] = (x[1].double() * 1e6).to(dtype)
    x[2] = torch.zeros_like(x[2])
    x[3] = torch.full_like(x[3], -0.01)
    x[3][:, :, 0] = -80.0
    x[4] = (x[4].double() * 0.9e-12).to(dtype)
    S0 = torch.randn(1, 2, 64, 64, generator=torch.Generator().manual_seed(9)) * 1e30
    dfin = torch.randn(1, 2, 64, 64, generator=torch.Generator().manual_seed(10))
    d = [t.cuda() for t in x]
    _, fs = kda.gdr_chunk_fwd(*d, return_final_state=True, initial_state=S0.cuda())
    _, S = recurrent(*x, 1.0, S0)
    check(fs[0], S[0], state_bound(chunk_terms(*(t[0] for t in x), 1.0, S0[0])[2]), "state")
    got = kda.gdr_chunk_bwd(*d, torch.zeros_like(d[2]), initial_state=S0.cuda(), dfinal_state=dfin.cuda())
    ref = reference(x, torch.zeros_like(x[2]), 1.0, S0, dfin)
    compare(got["dinitial_state"], ref[5], dtype, "dinitial_state")
