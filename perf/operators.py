"""Workloads of the gated delta rule and of latent attention.

Two token mixers that hybrid language models interleave:

* the gated delta rule, S_t = e^g S_{t-1} (I - b k k^T) + b v k^T, o_t = scale S_t q_t with one
  log-decay per token and value head: chunked forward ("gdr_fwd"), forward and backward of a
  training step ("gdr_train"), and the one-token step of decoding ("gdr_decode");
* attention whose keys and values come from one latent vector per token: the expanded form with a
  rotary key part shared by the heads, as prefill ("latent_fwd") and as a training step
  ("latent_train"), and the absorbed form, one token against a paged cache of latents
  ("latent_decode").

`run` computes a case with elementary torch operations in float32 (own = False), or through the
package's entry points (own = True).  `exact` computes it in float64 from the definitions: the token
recurrence and its adjoint, and softmax sequence by sequence.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------- the cases


def listed():
    return [
        # a short first turn, one user: latency of the chunked form, state handed to decoding
        dict(name="gdr_fwd_short", kind="gdr_fwd", io="bf16", B=1, Hk=8, H=16, T=37, dk=128, dv=128, packed=False, s0=False),
        # the 8k training batch of the benchmark's sequence lengths, forward only
        dict(name="gdr_fwd_8k", kind="gdr_fwd", io="bf16", B=4, Hk=16, H=16, T=8192, dk=128, dv=128, packed=False, s0=False),
        # the 64k sequence of the benchmark: few heads, a long chain of chunks
        dict(name="gdr_fwd_64k", kind="gdr_fwd", io="bf16", B=1, Hk=16, H=32, T=65536, dk=128, dv=128, packed=False, s0=True),
        # float32 documents of ragged lengths, each continuing from a state
        dict(name="gdr_fwd_packed_fp32", kind="gdr_fwd", io="fp32", B=7, Hk=2, H=4, T=3001, dk=64, dv=64, packed=True, s0=True),
        # a training step on full sequences, key heads shared by two value heads
        dict(name="gdr_train_4k", kind="gdr_train", io="bf16", B=2, Hk=8, H=16, T=4096, dk=128, dv=128, packed=False, s0=False),
        # a training step on packed documents with unequal head sizes
        dict(name="gdr_train_packed", kind="gdr_train", io="bf16", B=11, Hk=4, H=4, T=5003, dk=64, dv=128, packed=True, s0=True),
        # decoding for one user and for a full batch
        dict(name="gdr_decode_1", kind="gdr_decode", io="bf16", B=1, Hk=16, H=32, T=1, dk=128, dv=128, packed=False, s0=True),
        dict(name="gdr_decode_256", kind="gdr_decode", io="bf16", B=256, Hk=16, H=32, T=1, dk=128, dv=128, packed=False, s0=True),
        # prompts of ragged lengths behind cached prefixes, one call
        dict(name="latent_fwd_packed", kind="latent_fwd", io="bf16", B=6, H=32, T=4013, S=6007, dn=128, dr=64, dv=128, packed=True),
        # a training step on full sequences
        dict(name="latent_train_4k", kind="latent_train", io="bf16", B=1, H=16, T=4096, S=4096, dn=128, dr=64, dv=128, packed=False),
        # decoding for a few users with short histories, few heads (a tensor-parallel shard)
        dict(name="latent_decode_few", kind="latent_decode", io="bf16", B=3, H=16, S=700, dc=512, dr=64, page=64),
        # decoding for a batch with long histories, all heads
        dict(name="latent_decode_long", kind="latent_decode", io="bf16", B=48, H=128, S=12000, dc=512, dr=64, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["gdr_fwd", "gdr_train", "gdr_decode", "latent_fwd", "latent_train", "latent_decode"])
    io = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if kind.startswith("gdr"):
        Hk = rng.choice([1, 2, 4, 8, 16])
        H = Hk * rng.choice([1, 1, 2, 4])
        dk, dv = rng.choice([64, 128, 128]), rng.choice([64, 128, 128])
        if kind == "gdr_decode":
            return dict(kind=kind, io=io, B=_log(rng, 1, min(256, 8192 // H)), Hk=Hk, H=H, T=1, dk=dk, dv=dv, packed=False, s0=True)
        # tokens times value heads up to 2^20 (a training step: 2^17)
        most = 1 << (20 if kind == "gdr_fwd" else 17)
        packed = rng.random() < 0.4
        B = _log(rng, 1, 16) if packed else rng.choice([1, 1, 2, 4])
        T = _log(rng, 1, max(2, min(32768 if kind == "gdr_fwd" else 8192, most // (H * (1 if packed else B)))))
        return dict(kind=kind, io=io, B=B, Hk=Hk, H=H, T=T, dk=dk, dv=dv, packed=packed, s0=rng.random() < 0.5)
    if kind == "latent_decode":
        S = _log(rng, 1, 20000)
        return dict(kind=kind, io=io, B=max(1, min(_log(rng, 1, 128), 400000 // S)), H=rng.choice([1, 5, 8, 16, 32, 64, 128]), S=S,
                    dc=rng.choice([256, 512, 512]), dr=64, page=rng.choice([16, 64, 128]))
    packed = rng.random() < 0.5
    H = _log(rng, 1, 32)
    B = _log(rng, 1, 12) if packed else rng.choice([1, 1, 2])
    dn, dr = rng.choice([(128, 64), (128, 64), (64, 32)])
    # pairs of a query and a key up to those of the listed cases
    T = _log(rng, 1, int(min(6000 if io == "bf16" else 2000, (2.5e8 / (H * (1 if packed else B))) ** 0.5)))
    S = T if kind == "latent_train" else T + rng.choice([0, 0, rng.randrange(0, 2000)])
    return dict(kind=kind, io=io, B=B, H=H, T=T, S=S, dn=dn, dr=dr, dv=dn, packed=packed)


# ------------------------------------------------------------------------------------- the inputs


def _lengths(case, total, seed):
    """B lengths that add up to total, ragged; some may be 0 where there are few tokens."""
    n = case["B"]
    gen = torch.Generator().manual_seed(seed * 7919 + n)
    cuts = torch.randint(0, total + 1, (n - 1,), generator=gen).sort().values.tolist()
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _cu(lengths):
    return torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), dtype=torch.int32)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed * 1000003 + 17)
    dt = _DT[case["io"]]

    def normal(*shape, s=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * s).to(dt)

    st = {"case": dict(case)}
    if case["kind"].startswith("gdr"):
        B, Hk, H, T, dk, dv = (case[n] for n in ("B", "Hk", "H", "T", "dk", "dv"))
        one = case["kind"] == "gdr_decode"
        lead = (lambda h: (h, T)) if case["packed"] else (lambda h: (B, h)) if one else (lambda h: (B, h, T))
        # unit keys and queries, betas in (0, 1), and log-decays as softplus gates give them: most
        # of them slow, a few that forget at once
        for n in ("q", "k"):
            x = torch.randn(*lead(Hk), dk, generator=gen, device=dev)
            st[n] = (x / x.norm(dim=-1, keepdim=True)).to(dt)
        st["v"] = normal(*lead(H), dv)
        rate = torch.exp(torch.randn(*lead(H), generator=gen, device=dev) * 1.5 - 3.0)
        st["g"] = (-rate).to(dt)
        st["beta"] = torch.sigmoid(torch.randn(*lead(H), generator=gen, device=dev)).to(dt)
        st["scale"] = dk ** -0.5
        if case["packed"]:
            st["cu"] = _cu(_lengths(case, T, seed)).to(dev)
        st["s0"] = torch.randn(B, H, dv, dk, generator=gen, device=dev) * 0.3 if case["s0"] else None
        if case["kind"] == "gdr_train":
            st["dout"] = normal(*lead(H), dv)
        return st
    if case["kind"] == "latent_decode":
        B, H, S, dc, dr, page = (case[n] for n in ("B", "H", "S", "dc", "dr", "page"))
        host = torch.Generator().manual_seed(seed * 104729 + S)
        lengths = torch.randint((S + 1) // 2, S + 1, (B,), generator=host)
        lengths[0] = S
        pages = -(-S // page)
        st["lengths"] = lengths.to(torch.int32).to(dev)
        st["table"] = torch.randperm(B * pages, generator=host).reshape(B, pages).to(torch.int32).to(dev)
        st["cache"] = normal(B * pages, page, dc + dr)
        st["q"] = normal(B, H, dc + dr, s=0.5)
        st["scale"] = (128 + dr) ** -0.5
        return st
    B, H, T, S, dn, dr, dv = (case[n] for n in ("B", "H", "T", "S", "dn", "dr", "dv"))
    if case["packed"]:
        # the query block of a sequence stands behind a prefix: its keys are at least as many
        tq = _lengths(case, T, seed)
        pre = _lengths(case, S - T, seed + 1)
        st["cu_q"], st["cu_k"] = _cu(tq).to(dev), _cu([a + b for a, b in zip(tq, pre)]).to(dev)
        bq, bk = (), ()
    else:
        bq, bk = (B,), (B,)
    st["q"] = normal(*bq, H, T, dn + dr)
    # keys and values lie as the up-projection of the latents leaves them, the heads inside a token
    kv = normal(*bk, S, H, dn + dv)
    st["k"], st["v"] = kv[..., :dn].transpose(-3, -2), kv[..., dn:].transpose(-3, -2)
    st["k_rope"] = normal(*bk, S, dr)
    st["scale"] = (dn + dr) ** -0.5
    if case["kind"] == "latent_train":
        st["dout"] = normal(*bq, H, T, dv)
    return st


# ------------------------------------------------------------------------------------- one pass


def run(st):
    kind = st["case"]["kind"]
    if own:
        return _own(st)
    if kind == "gdr_decode":
        return _plain_decode_step(st)
    if kind == "latent_decode":
        return _plain_latent_decode(st)
    return (_plain_gdr if kind.startswith("gdr") else _plain_latent)(st)


def _own(st):
    import chunked_gated_linear_bounded_amd as kda

    kind, packed = st["case"]["kind"], st["case"].get("packed")
    if kind == "gdr_decode":
        out = kda.gdr_decode_step(st["q"], st["k"], st["v"], st["g"], st["beta"], st["s0"], scale=st["scale"])
        return {"out": out, "state": st["s0"]}
    if kind == "latent_decode":
        out, lse = kda.latent_decode_step(st["q"], st["cache"], st["table"], st["lengths"], st["scale"], dc=st["case"]["dc"],
                                          return_lse=True)
        return {"out": out, "lse": lse}
    if kind.startswith("gdr"):
        x = [st[n] for n in ("q", "k", "v", "g", "beta")]
        if packed:
            out, fs = kda.gdr_chunk_fwd_varlen(*x, st["cu"], scale=st["scale"], initial_state=st["s0"], return_final_state=True)
        else:
            out, fs = kda.gdr_chunk_fwd(*x, scale=st["scale"], initial_state=st["s0"], return_final_state=True)
        if kind == "gdr_fwd":
            return {"out": out, "final_state": fs}
        if packed:
            g = kda.gdr_chunk_bwd_varlen(*x, st["dout"], st["cu"], scale=st["scale"], initial_state=st["s0"],
                                         want_dinitial=st["s0"] is not None)
        else:
            g = kda.gdr_chunk_bwd(*x, st["dout"], scale=st["scale"], initial_state=st["s0"], want_dinitial=st["s0"] is not None)
        return {"out": out, **{n: g[n] for n in ("dq", "dk", "dv", "dg", "dbeta", "dinitial_state") if g[n] is not None}}
    x = [st[n] for n in ("q", "k", "v", "k_rope")]
    if packed:
        out, lse = kda.latent_attn_fwd_varlen(*x, st["cu_q"], st["cu_k"], st["scale"], return_lse=True)
    else:
        out, lse = kda.latent_attn_fwd(*x, st["scale"], return_lse=True)
    if kind == "latent_fwd":
        return {"out": out, "lse": lse}
    if packed:
        g = kda.latent_attn_bwd_varlen(*x, out, lse, st["dout"], st["cu_q"], st["cu_k"], st["scale"])
    else:
        g = kda.latent_attn_bwd(*x, out, lse, st["dout"], st["scale"])
    return {"out": out, **{n: g[n] for n in ("dq", "dk", "dv", "dk_rope")}}


# ------------------------------------------------------------------------------------- plain forms


def _pad_index(cu, T):
    """Rows of a packed stream as [N, longest] indexes, and which of them are tokens."""
    cu = cu.long()
    lens = cu[1:] - cu[:-1]
    at = torch.arange(int(lens.max()), device=cu.device)
    real = at[None] < lens[:, None]
    return torch.where(real, cu[:-1, None] + at[None], 0), real


def _gdr_chunks(q, k, v, g, beta, scale, s0):
    """The chunked form on [B,H,T,*] in float32, 64 tokens a chunk; the state as [B,H,dk,dv]."""
    B, H, T, dk = k.shape
    C = 64
    n = max(1, -(-T // C))
    pad = n * C - T
    grow = torch.nn.functional.pad
    q, k, v = (grow(x, (0, 0, 0, pad)).reshape(B, H, n, C, -1) for x in (q * scale, k, v))
    g, beta = (grow(x, (0, pad)).reshape(B, H, n, C) for x in (g, beta))
    G = g.cumsum(-1)
    low = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    decay = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, float("-inf")))
    eye = torch.eye(C, device=q.device)
    X = -(beta[..., None] * (k @ k.transpose(-1, -2)) * decay) * (1 - eye)
    Tm = eye + X
    for _ in range(5):  # (I - X)^-1 = (I + X)(I + X^2)(I + X^4) ..., X^64 = 0
        X = X @ X
        Tm = Tm + Tm @ X
    eG = torch.exp(G)[..., None]
    W, U = Tm @ (beta[..., None] * eG * k), Tm @ (beta[..., None] * v)
    M, Qg = (q @ k.transpose(-1, -2)) * decay, q * eG
    Kg, last = (k * torch.exp(G[..., -1:] - G)[..., None]).transpose(-1, -2), torch.exp(G[..., -1])[..., None, None]
    P, outs = s0, []
    for c in range(n):
        u = U[:, :, c] - W[:, :, c] @ P
        outs.append(Qg[:, :, c] @ P + M[:, :, c] @ u)
        P = last[:, :, c] * P + Kg[:, :, c] @ u
    return torch.stack(outs, 2).reshape(B, H, n * C, -1)[:, :, :T], P


def _plain_gdr(st):
    case, train = st["case"], st["case"]["kind"] == "gdr_train"
    dt, names = st["q"].dtype, ("q", "k", "v", "g", "beta")
    leaf = [st[n].float().requires_grad_(train) for n in names]
    if case["packed"]:
        at, real = _pad_index(st["cu"], case["T"])
        x = [(t[:, at].transpose(0, 1) * (real[:, None, :, None] if t.dim() == 3 else real[:, None])) for t in leaf]
    else:
        x = leaf
    r = case["H"] // case["Hk"]
    q, k = (t.repeat_interleave(r, dim=1) for t in x[:2])
    if st["s0"] is not None:
        leaf.append(st["s0"].detach().requires_grad_(train))
    with torch.set_grad_enabled(train):
        s0 = leaf[5].transpose(-1, -2) if st["s0"] is not None else q.new_zeros(case["B"], case["H"], case["dk"], case["dv"])
        out, P = _gdr_chunks(q, k, *x[2:5], st["scale"], s0)
        if case["packed"]:
            out = out.transpose(0, 1)[:, real]
    if not train:
        return {"out": out.to(dt), "final_state": P.transpose(-1, -2).contiguous()}
    grads = torch.autograd.grad(out, leaf, st["dout"].float())
    got = {"out": out.detach().to(dt), **{"d" + n: t.to(dt) for n, t in zip(names, grads)}}
    return {**got, "dinitial_state": grads[5]} if st["s0"] is not None else got


def _plain_decode_step(st):
    r = st["case"]["H"] // st["case"]["Hk"]
    q, k = (st[n].float().repeat_interleave(r, dim=1) for n in ("q", "k"))
    v, g, beta = (st[n].float() for n in ("v", "g", "beta"))
    S = st["s0"].mul_(torch.exp(g)[..., None, None])
    write = beta[..., None] * (v - (S * k[..., None, :]).sum(-1))
    S.add_(write[..., :, None] * k[..., None, :])
    return {"out": (st["scale"] * (S * q[..., None, :]).sum(-1)).to(st["q"].dtype), "state": S}


def _plain_latent(st):
    case, train = st["case"], st["case"]["kind"] == "latent_train"
    dt, names = st["q"].dtype, ("q", "k", "v", "k_rope")
    leaf = [st[n].float().requires_grad_(train) for n in names]
    T, S, dn = case["T"], case["S"], case["dn"]
    iq, ik = torch.arange(T, device=leaf[0].device), torch.arange(S, device=leaf[0].device)
    if case["packed"]:
        cq, ck = st["cu_q"].long(), st["cu_k"].long()
        nq, nk = torch.searchsorted(cq[1:], iq, right=True), torch.searchsorted(ck[1:], ik, right=True)
        pos = iq - cq[1:][nq] + ck[1:][nq]  # the last query stands at the last key
        seen = (nq[:, None] == nk[None]) & (ik[None] <= pos[:, None])
    else:
        seen = ik[None] <= (iq + S - T)[:, None]
    with torch.set_grad_enabled(train):
        q, k, v, k_rope = leaf
        s = q[..., :dn] @ k.transpose(-1, -2) + q[..., dn:] @ k_rope.unsqueeze(-3).transpose(-1, -2)
        s = (s * st["scale"]).masked_fill(~seen, float("-inf"))
        most = s.detach().amax(-1, keepdim=True)
        p = torch.exp(s - most)
        total = p.sum(-1, keepdim=True)
        out = (p / total) @ v
    if not train:
        return {"out": out.to(dt), "lse": (most + torch.log(total)).squeeze(-1)}
    del s, p
    grads = torch.autograd.grad(out, leaf, st["dout"].float())
    return {"out": out.detach().to(dt), **{"d" + n: t.to(dt) for n, t in zip(names, grads)}}


def _plain_latent_decode(st):
    case = st["case"]
    rows = st["cache"].float()[st["table"].long()].reshape(case["B"], -1, case["dc"] + case["dr"])
    s = (st["q"].float() @ rows.transpose(-1, -2)) * st["scale"]
    seen = torch.arange(rows.shape[1], device=s.device)[None] < st["lengths"][:, None]
    s = s.masked_fill(~seen[:, None], float("-inf"))
    most = s.amax(-1, keepdim=True)
    p = torch.exp(s - most)
    total = p.sum(-1, keepdim=True)
    out = (p / total) @ rows[..., : case["dc"]]
    return {"out": out.to(st["q"].dtype), "lse": (most + torch.log(total)).squeeze(-1)}


# ------------------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "latent_decode":
        return _exact_latent_decode(st)
    return (_exact_gdr if case["kind"].startswith("gdr") else _exact_latent)(st)


def _exact_gdr(st):
    """Token by token, and for gradients the adjoint of the token step, a few heads at a time."""
    case, kind = st["case"], st["case"]["kind"]
    H, dk, dv = case["H"], case["dk"], case["dv"]
    r = H // case["Hk"]
    q, k, v, g, beta = (st[n].double() for n in ("q", "k", "v", "g", "beta"))
    if kind == "gdr_decode":
        q, k, v, g, beta = (t.unsqueeze(2) for t in (q, k, v, g, beta))
    train = kind == "gdr_train"
    d = st["dout"].double() if train else v
    if case["packed"]:
        at, real = _pad_index(st["cu"], case["T"])
        q, k, v, g, beta, d = (t[:, at].transpose(0, 1) * (real[:, None, :, None] if t.dim() == 3 else real[:, None])
                               for t in (q, k, v, g, beta, d))
    q, k = (t.repeat_interleave(r, dim=1) for t in (q, k))
    B, T = v.shape[0], v.shape[2]
    S0 = st["s0"].double() if st["s0"] is not None else v.new_zeros(B, H, dv, dk)
    out, grads = torch.empty_like(v), [torch.zeros_like(t) for t in (q, k, v, g, beta)]
    end, start = torch.empty_like(S0), torch.empty_like(S0)
    step = max(1, min(H, int(24e9 // (8.0 * dk * dv * B * T)))) if train else H
    if train and 8.0 * dk * dv * B * T * step > 100e9 or -(-H // step) * T * (12 if train else 4) * 1e-5 > 20:
        return None
    for h in range(0, H, step):
        hs = slice(h, h + step)
        S, kept = S0[:, hs].clone(), []
        for t in range(T):
            if train:
                kept.append(S)
            kt = k[:, hs, t]
            S = torch.exp(g[:, hs, t])[..., None, None] * S
            w = beta[:, hs, t, None] * (v[:, hs, t] - (S @ kt[..., None])[..., 0])
            S = S + w[..., None] * kt[..., None, :]
            out[:, hs, t] = st["scale"] * (S @ q[:, hs, t, :, None])[..., 0]
        end[:, hs] = S
        if not train:
            continue
        dS = torch.zeros_like(S)
        for t in range(T - 1, -1, -1):
            kt, b, dec = k[:, hs, t], beta[:, hs, t, None], torch.exp(g[:, hs, t])[..., None, None]
            before = dec * kept.pop()
            y = v[:, hs, t] - (before @ kt[..., None])[..., 0]
            after = before + (b * y)[..., None] * kt[..., None, :]
            do = st["scale"] * d[:, hs, t]
            grads[0][:, hs, t] = (do[..., None, :] @ after)[..., 0, :]
            dS = dS + do[..., None] * q[:, hs, t, None, :]
            dw = (dS @ kt[..., None])[..., 0]
            dy = b * dw
            grads[1][:, hs, t] = ((b * y)[..., None, :] @ dS)[..., 0, :] - (dy[..., None, :] @ before)[..., 0, :]
            grads[2][:, hs, t] = dy
            grads[4][:, hs, t] = (dw * y).sum(-1)
            dS = dS - dy[..., None] * kt[..., None, :]
            grads[3][:, hs, t] = (dS * before).sum((-1, -2))
            dS = dS * dec
        start[:, hs] = dS
    if kind == "gdr_decode":
        return {"out": out[:, :, 0], "state": end}
    grads[0], grads[1] = (t.unflatten(1, (H // r, r)).sum(2) for t in grads[:2])
    if case["packed"]:
        out, *grads = (t.transpose(0, 1)[:, real] for t in (out, *grads))
    if not train:
        return {"out": out, "final_state": end}
    got = {"out": out, **dict(zip(("dq", "dk", "dv", "dg", "dbeta"), grads))}
    return {**got, "dinitial_state": start} if st["s0"] is not None else got


def _exact_latent(st):
    """Softmax sequence by sequence and head by head."""
    case, train = st["case"], st["case"]["kind"] == "latent_train"
    B, H, dn = case["B"], case["H"], case["dn"]
    q, k, v, k_rope = (st[n].double() for n in ("q", "k", "v", "k_rope"))
    d = st["dout"].double() if train else None
    out, lse = q.new_zeros(*q.shape[:-1], case["dv"]), q.new_zeros(q.shape[:-1])
    dq, dk, dv, dr = (torch.zeros_like(t) for t in (q, k, v, k_rope))
    cq, ck = (st["cu_q"].tolist(), st["cu_k"].tolist()) if case["packed"] else (None, None)
    for n in range(B):
        for h in range(H):
            a = (h, slice(cq[n], cq[n + 1])) if case["packed"] else (n, h)
            b = (h, slice(ck[n], ck[n + 1])) if case["packed"] else (n, h)
            c = b[1:] if case["packed"] else (n,)
            key = torch.cat([k[b], k_rope[c]], -1)
            T, S = q[a].shape[0], key.shape[0]
            if not T:
                continue
            s = (q[a] @ key.T * st["scale"]).masked_fill(torch.ones(T, S, dtype=torch.bool, device=q.device).triu(S - T + 1), -math.inf)
            lse[a] = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[a][:, None])
            out[a] = p @ v[b]
            if train:
                ds = p * (d[a] @ v[b].T - (d[a] * out[a]).sum(-1, keepdim=True)) * st["scale"]
                dv[b] = p.T @ d[a]
                dq[a] = ds @ key
                dkey = ds.T @ q[a]
                dk[b] = dkey[:, :dn]
                dr[c] += dkey[:, dn:]
    if not train:
        return {"out": out, "lse": lse}
    return {"out": out, "dq": dq, "dk": dk, "dv": dv, "dk_rope": dr}


def _exact_latent_decode(st):
    case = st["case"]
    out, lse = [], []
    for b, n in enumerate(st["lengths"].tolist()):
        at = torch.arange(n, device="cuda")
        rows = st["cache"][st["table"][b].long()[at // case["page"]], at % case["page"]].double()
        s = st["q"][b].double() @ rows.T * st["scale"]
        out.append(torch.softmax(s, -1) @ rows[:, : case["dc"]])
        lse.append(torch.logsumexp(s, -1))
    return {"out": torch.stack(out), "lse": torch.stack(lse)}


# ------------------------------------------------------------------------------------- the work


def work(case):
    e, kind = 2 if case["io"] == "bf16" else 4, case["kind"]
    if kind.startswith("gdr"):
        H, Hk, dk, dv = (case[n] for n in ("H", "Hk", "dk", "dv"))
        tokens = case["T"] * (1 if case["packed"] else case["B"])
        rows = tokens * (2 * Hk * dk + H * (dv + 2)) * e  # q, k, v, g, beta
        state = case["B"] * H * dk * dv * 4
        if kind == "gdr_decode":
            return {"bytes": rows + tokens * H * dv * e + 2 * state, "flops": 7.0 * tokens * H * dk * dv}
        # products of a 64-token chunk, the causal ones at half: K K^T, Q K^T, the solve, the two
        # corrections; then three with the state
        C = 64
        flops = tokens * H * (C * (2 * dk + 2 * dv + C / 3) + 6 * dk * dv)
        bytes_ = rows + tokens * H * dv * e + state * (2 if case["s0"] else 1)
        if kind == "gdr_fwd":
            return {"bytes": bytes_, "flops": flops}
        return {"bytes": 2 * rows + 2 * tokens * H * dv * e + rows + state * (1 if case["s0"] else 0),
                "flops": flops + tokens * H * (C * (5 * dk + 5 * dv) + 12 * dk * dv)}
    if kind == "latent_decode":
        # the lengths lie between half of S and S
        B, H, S, d, dc = case["B"], case["H"], case["S"], case["dc"] + case["dr"], case["dc"]
        rows = (0.75 * (B - 1) + 1) * S
        return {"bytes": rows * d * e + B * H * (d + dc) * e + B * H * 4, "flops": 2.0 * rows * H * (d + dc)}
    H, T, S, dn, dr, dv = (case[n] for n in ("H", "T", "S", "dn", "dr", "dv"))
    n = 1 if case["packed"] else case["B"]
    q, kv = n * H * T * (dn + dr) * e, n * S * (H * (dn + dv) + dr) * e
    out = n * H * T * dv * e
    pairs = n * H * T * (S - T / 2)
    if case["packed"]:  # B uneven sequences: the mean of the sum of squares of B random parts
        pairs *= 2 / (case["B"] + 1)
    fwd = 2.0 * pairs * (dn + dr + dv)
    if kind == "latent_fwd":
        return {"bytes": q + kv + out + n * H * T * 4, "flops": fwd}
    return {"bytes": 3 * (q + kv) + 3 * out, "flops": fwd + 2.0 * pairs * (3 * (dn + dr) + 2 * dv)}
