"""Workloads of decayed linear attention, of writing the paged latent cache, and of attention of drafted
tokens over it.

What a model that interleaves linear layers with latent attention runs, in prefill, training and
speculative decoding:

* linear attention with one decay per token and head, S_t = e^g S_{t-1} + v k^T, o_t = scale S_t q_t:
  chunked forward ("lin_fwd"), forward and backward of a training step ("lin_train"), and the one-token
  step ("lin_decode");
* writing new tokens into a paged cache of latent rows, the latent normalised and the rotary parts of
  key and queries rotated on the way ("append");
* attention of the drafted tokens of a speculative step over that cache, the committed rows visible to
  all of them and the drafted rows by a tree ("tree").

`run` computes a case with elementary torch operations in float32 (own = False), or through the
package's entry points (own = True).  `exact` computes it in float64 from the definitions.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------- the cases


def listed():
    return [
        # a short turn of one user behind a kept state: latency of the chunked form
        dict(name="lin_fwd_short", kind="lin_fwd", io="bf16", B=1, Hk=16, H=16, T=37, dk=128, dv=128, packed=False, s0=True, decay="token"),
        # a batch of 8k sequences, every head with a constant decay in float32
        dict(name="lin_fwd_8k", kind="lin_fwd", io="bf16", B=4, Hk=16, H=16, T=8192, dk=128, dv=128, packed=False, s0=False, decay="head"),
        # one 64k prompt, key heads shared by two value heads
        dict(name="lin_fwd_64k", kind="lin_fwd", io="bf16", B=1, Hk=16, H=32, T=65536, dk=128, dv=128, packed=False, s0=True, decay="token"),
        # float32 documents of ragged lengths, each continuing from a state
        dict(name="lin_fwd_packed_fp32", kind="lin_fwd", io="fp32", B=7, Hk=2, H=4, T=3001, dk=64, dv=64, packed=True, s0=True, decay="token"),
        # a training step on full sequences
        dict(name="lin_train_4k", kind="lin_train", io="bf16", B=2, Hk=8, H=16, T=4096, dk=128, dv=128, packed=False, s0=False, decay="token"),
        # a training step on packed documents with unequal head sizes
        dict(name="lin_train_packed", kind="lin_train", io="bf16", B=11, Hk=4, H=4, T=5003, dk=64, dv=128, packed=True, s0=True, decay="token"),
        # decoding for a full batch
        dict(name="lin_decode_256", kind="lin_decode", io="bf16", B=256, Hk=16, H=32, T=1, dk=128, dv=128, packed=False, s0=True, decay="token"),
        # one token for each of a few users, all heads' queries
        dict(name="append_one", kind="append", io="bf16", B=5, T=1, H=128, S=700, dc=512, dr=64, page=64, packed=False, norm=True, interleaved=True),
        # prompts of ragged lengths behind cached prefixes
        dict(name="append_prompts", kind="append", io="bf16", B=9, T=16411, H=64, S=2500, dc=512, dr=64, page=64, packed=True, norm=True, interleaved=True),
        # few drafted tokens for a few users with short histories, few heads (a tensor-parallel shard)
        dict(name="tree_few", kind="tree", io="bf16", B=3, T=5, H=16, S=700, dc=512, dr=64, page=64),
        # a verification step of a batch with long histories, all heads
        dict(name="tree_batch", kind="tree", io="bf16", B=24, T=8, H=128, S=9000, dc=512, dr=64, page=64),
        # wide trees for a few users
        dict(name="tree_wide", kind="tree", io="bf16", B=4, T=61, H=128, S=5000, dc=512, dr=64, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["lin_fwd", "lin_train", "lin_decode", "append", "tree", "tree"])
    io = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if kind.startswith("lin"):
        Hk = rng.choice([1, 2, 4, 8, 16])
        H = Hk * rng.choice([1, 1, 2, 4])
        dk, dv = rng.choice([64, 128, 128]), rng.choice([64, 128, 128])
        decay = rng.choice(["token", "token", "head"])
        if kind == "lin_decode":
            return dict(kind=kind, io=io, B=_log(rng, 1, min(256, 8192 // H)), Hk=Hk, H=H, T=1, dk=dk, dv=dv, packed=False, s0=True, decay=decay)
        # tokens times value heads up to 2^20 (a training step: 2^17)
        most = 1 << (20 if kind == "lin_fwd" else 17)
        packed = rng.random() < 0.4
        B = _log(rng, 1, 16) if packed else rng.choice([1, 1, 2, 4])
        T = _log(rng, 1, max(2, min(32768 if kind == "lin_fwd" else 8192, most // (H * (1 if packed else B)))))
        return dict(kind=kind, io=io, B=B, Hk=Hk, H=H, T=T, dk=dk, dv=dv, packed=packed, s0=rng.random() < 0.5, decay=decay)
    dc, page = rng.choice([256, 512, 512]), rng.choice([16, 64, 128])
    if kind == "append":
        packed = rng.random() < 0.5
        B = _log(rng, 1, 32 if packed else 200)
        T = _log(rng, 1, 16000) if packed else _log(rng, 1, 64)
        H = rng.choice([1, 5, 16, 64, 128])
        while T * H * (1 if packed else B) > 1000000:
            H = max(1, H // 2)
        return dict(kind=kind, io=io, B=B, T=T, H=H, S=_log(rng, 1, 3000), dc=dc, dr=64, page=page, packed=packed,
                    norm=rng.random() < 0.7, interleaved=rng.random() < 0.5)
    H, T, S = rng.choice([1, 5, 8, 16, 32, 64, 128]), _log(rng, 1, 64), _log(rng, 1, 16000)
    # products up to half of the listed ones' (float32: a tenth of that), and at most 300,000 rows of cache
    most = (1.1e8 if io == "bf16" else 1.1e7) / max(16, T * H)
    S = max(1, min(S, int(most)))
    return dict(kind=kind, io=io, B=max(1, min(_log(rng, 1, 64), 300000 // S, int(most / S))), T=T, H=H, S=S, dc=dc, dr=64, page=page)


# ------------------------------------------------------------------------------------- the inputs


def _lengths(n, total, seed):
    """n lengths that add up to total, ragged; some may be 0 where there are few tokens."""
    gen = torch.Generator().manual_seed(seed * 7919 + n)
    cuts = torch.randint(0, total + 1, (n - 1,), generator=gen).sort().values.tolist()
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _cu(lengths):
    return torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), dtype=torch.int32)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed * 1000003 + 29)
    host = torch.Generator().manual_seed(seed * 104729 + 7)
    dt = _DT[case["io"]]

    def normal(*shape, s=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * s).to(dt)

    st = {"case": dict(case)}
    if case["kind"].startswith("lin"):
        B, Hk, H, T, dk, dv = (case[n] for n in ("B", "Hk", "H", "T", "dk", "dv"))
        one = case["kind"] == "lin_decode"
        lead = (lambda h: (h, T)) if case["packed"] else (lambda h: (B, h)) if one else (lambda h: (B, h, T))
        # activations of order one; log-decays as softplus gates give them (most of them slow, a few that
        # forget at once), or one constant per head from 1/2 down to 1/256, in float32 and expanded
        st["q"], st["k"], st["v"] = normal(*lead(Hk), dk), normal(*lead(Hk), dk), normal(*lead(H), dv)
        if case["decay"] == "token":
            st["g"] = (-torch.exp(torch.randn(*lead(H), generator=gen, device=dev) * 1.5 - 3.0)).to(dt)
        else:
            slope = -torch.exp2(-torch.linspace(1.0, 8.0, H, device=dev))
            st["g"] = (slope if one else slope[:, None]).expand(*lead(H))
            if one:
                st["g"] = st["g"].contiguous()
        st["scale"] = dk ** -0.5
        if case["packed"]:
            st["cu"] = _cu(_lengths(B, T, seed)).to(dev)
        st["s0"] = torch.randn(B, H, dv, dk, generator=gen, device=dev) if case["s0"] else None
        if case["kind"] == "lin_train":
            st["dout"] = normal(*lead(H), dv)
        return st
    B, T, H, S, dc, dr, page = (case[n] for n in ("B", "T", "H", "S", "dc", "dr", "page"))
    if case["kind"] == "append":
        # S: the longest history; new tokens stand behind it
        new = _lengths(B, T, seed) if case["packed"] else [T] * B
        old = torch.randint((S + 1) // 2, S + 1, (B,), generator=host).tolist()
        rows = [a + b for a, b in zip(new, old)]
        pages = -(-max(rows) // page)
        total = (T * (1 if case["packed"] else B) + B * S) // page + B
        order, at = torch.randperm(total, generator=host).to(torch.int32), 0
        table = torch.zeros(B, pages, dtype=torch.int32)
        for b, r in enumerate(rows):
            n = -(-r // page)
            table[b, :n] = order[at:at + n]
            at += n
        st["table"], st["lengths"] = table.to(dev), torch.tensor(rows, dtype=torch.int32).to(dev)
        st["cache"] = normal(total, page, dc + dr)
        lead = (T,) if case["packed"] else (B, T)
        if case["packed"]:
            st["cu"] = _cu(new).to(dev)
        # the down projection leaves latent and rotary key side by side
        both = normal(*lead, dc + dr, s=2.0)
        st["latent"], st["k_rope"] = both[..., :dc], both[..., dc:]
        # the queries' rotary part comes behind their other part, and goes behind the absorbed one
        st["q_rope"] = normal(*lead, H, 128 + dr)[..., 128:]
        st["q"] = normal(*lead, H, dc + dr)
        st["freqs"] = (10000.0 ** (-torch.arange(0, dr, 2, dtype=torch.float64) / dr)).to(torch.float32).to(dev)
        st["weight"] = (1.0 + 0.1 * torch.randn(dc, generator=gen, device=dev)).to(dt) if case["norm"] else None
        st["eps"] = 1e-6
        return st
    # lengths between half of S and S rows of history, then the drafted rows
    lengths = torch.randint((S + 1) // 2, S + 1, (B,), generator=host)
    lengths[0] = S
    lengths += T
    pages = -(-(S + T) // page)
    st["lengths"] = lengths.to(torch.int32).to(dev)
    st["table"] = torch.randperm(B * pages, generator=host).reshape(B, pages).to(torch.int32).to(dev)
    st["cache"] = normal(B * pages, page, dc + dr)
    st["q"] = normal(B, T, H, dc + dr, s=0.5)
    # a random tree: every node's parent is the last token (no bit) or an earlier node
    mask = torch.zeros(B, T, dtype=torch.int64)
    for b in range(B):
        parent = [int(torch.randint(-1, max(i, 1), (1,), generator=host)) if i else -1 for i in range(T)]
        for i, p in enumerate(parent):
            bit = 1 << i if i < 63 else -(1 << 63)
            mask[b, i] = (int(mask[b, p]) if p >= 0 else 0) | bit
    st["mask"] = mask.to(dev)
    st["scale"] = (128 + dr) ** -0.5
    return st


# ------------------------------------------------------------------------------------- one pass


def run(st):
    kind = st["case"]["kind"]
    if own:
        return _own(st)
    if kind == "append":
        return _plain_append(st)
    if kind == "tree":
        return _plain_tree(st)
    return _plain_decode(st) if kind == "lin_decode" else _plain_lin(st)


def _own(st):
    import chunked_gated_linear_bounded_amd as kda

    case = st["case"]
    kind, packed = case["kind"], case.get("packed")
    if kind == "append":
        more = dict(norm_weight=st["weight"], eps=st["eps"], interleaved=case["interleaved"], q_rope=st["q_rope"], q=st["q"])
        x = [st[n] for n in ("latent", "k_rope", "cache", "table", "lengths", "freqs")]
        if packed:
            kda.latent_append_varlen(*x, st["cu"], **more)
        else:
            kda.latent_append(*x, **more)
        return {"cache": st["cache"], "q": st["q"]}
    if kind == "tree":
        out, lse = kda.latent_tree_step(st["q"], st["cache"], st["table"], st["lengths"], st["mask"], st["scale"], dc=case["dc"],
                                        return_lse=True)
        return {"out": out, "lse": lse}
    x = [st[n] for n in ("q", "k", "v", "g")]
    if kind == "lin_decode":
        out = kda.lin_decode_step(*x, st["s0"], scale=st["scale"])
        return {"out": out, "state": st["s0"]}
    if packed:
        out, fs = kda.lin_chunk_fwd_varlen(*x, st["cu"], scale=st["scale"], initial_state=st["s0"], return_final_state=True)
    else:
        out, fs = kda.lin_chunk_fwd(*x, scale=st["scale"], initial_state=st["s0"], return_final_state=True)
    if kind == "lin_fwd":
        return {"out": out, "final_state": fs}
    more = dict(scale=st["scale"], initial_state=st["s0"], want_dg=case["decay"] == "token", want_dinitial=st["s0"] is not None)
    d = kda.lin_chunk_bwd_varlen(*x, st["dout"], st["cu"], **more) if packed else kda.lin_chunk_bwd(*x, st["dout"], **more)
    return {"out": out, **{n: d[n] for n in ("dq", "dk", "dv", "dg", "dinitial_state") if d[n] is not None}}


# ------------------------------------------------------------------------------------- plain forms


def _pad_index(cu, T):
    """Rows of a packed stream as [N, longest] indexes, and which of them are tokens."""
    cu = cu.long()
    lens = cu[1:] - cu[:-1]
    at = torch.arange(max(1, int(lens.max())), device=cu.device)
    real = at[None] < lens[:, None]
    return torch.where(real, cu[:-1, None] + at[None], 0), real


def _decays(G):
    """e^(G_i - G_j) for j <= i, else 0, over the last dimension."""
    n = G.shape[-1]
    low = torch.ones(n, n, dtype=torch.bool, device=G.device).tril()
    return torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, float("-inf")))


def _lin_chunks(q, k, v, g, scale, s0):
    """The chunked form on [B,H,T,*] in float32, 64 tokens a chunk, the chunks' states by one product with
    the decays between chunks; states as [B,H,dk,dv]."""
    B, H, T, dk = k.shape
    C = 64
    n = max(1, -(-T // C))
    grow = torch.nn.functional.pad
    q, k, v = (grow(x, (0, 0, 0, n * C - T)).reshape(B, H, n, C, -1) for x in (q * scale, k, v))
    G = grow(g, (0, n * C - T)).reshape(B, H, n, C).cumsum(-1)
    local = (k * torch.exp(G[..., -1:] - G)[..., None]).transpose(-1, -2) @ v
    # states behind each chunk, from the start state and all chunks up to it
    F = grow(G[..., -1].double().cumsum(-1), (1, 0))
    ends = (_decays(F).to(G.dtype) @ torch.cat([s0[:, :, None], local], 2).flatten(-2)).unflatten(-1, local.shape[-2:])
    out = ((q @ k.transpose(-1, -2)) * _decays(G)) @ v + (q * torch.exp(G)[..., None]) @ ends[:, :, :-1]
    return out.reshape(B, H, n * C, -1)[:, :, :T], ends[:, :, -1]


def _plain_lin(st):
    case, train = st["case"], st["case"]["kind"] == "lin_train"
    dt, names = st["q"].dtype, ("q", "k", "v", "g")
    leaf = [st[n].detach().float().requires_grad_(train) for n in names]
    with torch.set_grad_enabled(train):
        x = leaf
        if case["packed"]:
            at, real = _pad_index(st["cu"], case["T"])
            x = [(t[:, at].transpose(0, 1) * (real[:, None, :, None] if t.dim() == 3 else real[:, None])) for t in leaf]
        r = case["H"] // case["Hk"]
        q, k = (t.repeat_interleave(r, dim=1) for t in x[:2])
        if st["s0"] is not None:
            leaf.append(st["s0"].detach().requires_grad_(train))
        s0 = leaf[4].transpose(-1, -2) if st["s0"] is not None else q.new_zeros(case["B"], case["H"], case["dk"], case["dv"])
        out, P = _lin_chunks(q, k, x[2], x[3], st["scale"], s0)
        if case["packed"]:
            out = out.transpose(0, 1)[:, real]
    if not train:
        return {"out": out.to(dt), "final_state": P.transpose(-1, -2).contiguous()}
    # a constant decay per head is no parameter
    by = {"d" + n: t for n, t in zip(names, leaf) if n != "g" or case["decay"] == "token"}
    if st["s0"] is not None:
        by["dinitial_state"] = leaf[4]
    grads = torch.autograd.grad(out, list(by.values()), st["dout"].float())
    return {"out": out.detach().to(dt), **{n: t if n == "dinitial_state" else t.to(dt) for n, t in zip(by, grads)}}


def _plain_decode(st):
    r = st["case"]["H"] // st["case"]["Hk"]
    q, k = (st[n].float().repeat_interleave(r, dim=1) for n in ("q", "k"))
    S = st["s0"].mul_(torch.exp(st["g"].float())[..., None, None])
    S.add_(st["v"].float()[..., :, None] * k[..., None, :])
    return {"out": (st["scale"] * (S * q[..., None, :]).sum(-1)).to(st["q"].dtype), "state": S}


def _rotate(x, angle, interleaved):
    """Pairs of the last dimension turned by the angles, in float32."""
    c, s = torch.cos(angle).float(), torch.sin(angle).float()
    x = x.float()
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * c - b * s, a * s + b * c], -1)


def _plain_append(st):
    case = st["case"]
    page, dc, dt = case["page"], case["dc"], st["cache"].dtype
    last = st["lengths"].long()
    if case["packed"]:
        cu, t = st["cu"].long(), torch.arange(case["T"], device=last.device)
        seq = torch.searchsorted(cu[1:], t, right=True)
        row = last[seq] - cu[1:][seq] + t
    else:
        seq = torch.arange(case["B"], device=last.device)[:, None].expand(-1, case["T"])
        row = last[:, None] - case["T"] + torch.arange(case["T"], device=last.device)[None]
    angle = row[..., None].double() * st["freqs"].double()
    c = st["latent"].float()
    if st["weight"] is not None:
        c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + st["eps"]) * st["weight"].float()
    new = torch.cat([c, _rotate(st["k_rope"], angle, case["interleaved"])], -1)
    st["cache"][st["table"][seq, row // page].long(), row % page] = new.to(dt)
    st["q"][..., dc:] = _rotate(st["q_rope"], angle[..., None, :], case["interleaved"]).to(dt)
    return {"cache": st["cache"], "q": st["q"]}


def _plain_tree(st):
    case = st["case"]
    B, T, H, dc = case["B"], case["T"], case["H"], case["dc"]
    rows = st["cache"].float()[st["table"].long()].reshape(B, -1, dc + case["dr"])
    s = (st["q"].float().reshape(B, T * H, -1) @ rows.transpose(-1, -2)).mul_(st["scale"]).unflatten(1, (T, H))
    j = torch.arange(rows.shape[1], device=s.device)
    node = j[None] - (st["lengths"].long()[:, None] - T)  # the drafted node of a row; below 0: a committed row
    bit = (st["mask"][:, :, None] >> node[:, None].clamp(0, 63)) & 1
    seen = (node < 0)[:, None] | ((node < T)[:, None] & (bit == 1))
    s.masked_fill_(~seen[:, :, None], float("-inf"))
    most = s.amax(-1, keepdim=True)
    p = torch.exp_(s.sub_(most))
    total = p.sum(-1, keepdim=True)
    out = (p.flatten(1, 2) @ rows[..., :dc]).unflatten(1, (T, H)) / total
    return {"out": out.to(st["q"].dtype), "lse": (most + torch.log(total)).squeeze(-1)}


# ------------------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "append":
        return _exact_append(st)
    if case["kind"] == "tree":
        return _exact_tree(st)
    return _exact_grads(st) if case["kind"] == "lin_train" else _exact_lin(st)


def _exact_lin(st):
    """Token by token."""
    case = st["case"]
    H, T = case["H"], case["T"]
    r = H // case["Hk"]
    q, k, v, g = (st[n].double() for n in ("q", "k", "v", "g"))
    if case["kind"] == "lin_decode":
        q, k, v, g = (t.unsqueeze(2) for t in (q, k, v, g))
    if case["packed"]:
        at, real = _pad_index(st["cu"], T)
        q, k, v, g = (t[:, at].transpose(0, 1) * (real[:, None, :, None] if t.dim() == 3 else real[:, None]) for t in (q, k, v, g))
    q, k = (t.repeat_interleave(r, dim=1) for t in (q, k))
    S = st["s0"].double() if st["s0"] is not None else v.new_zeros(case["B"], H, case["dv"], case["dk"])
    out = torch.empty_like(v)
    for t in range(v.shape[2]):
        S = torch.exp(g[:, :, t])[..., None, None] * S + v[:, :, t, :, None] * k[:, :, t, None, :]
        out[:, :, t] = st["scale"] * (S @ q[:, :, t, :, None])[..., 0]
    if case["kind"] == "lin_decode":
        return {"out": out[:, :, 0], "state": S}
    if case["packed"]:
        out = out.transpose(0, 1)[:, real]
    return {"out": out, "final_state": S}


def _exact_grads(st):
    """Every pair of tokens of a sequence and head: X_ij = scale e^(F_i - F_j) (q_i . k_j), F the sum of
    the log-decays; a log-decay's gradient is the sum over the pairs that it lies between."""
    case = st["case"]
    H, r, scale = case["H"], case["H"] // case["Hk"], st["scale"]
    q, k, v, g, d = (st[n].double() for n in ("q", "k", "v", "g", "dout"))
    cu = st["cu"].tolist() if case["packed"] else None
    out, dq, dk, dv, dg = (torch.zeros_like(t) for t in (v, q, k, v, g))
    ds0 = None if st["s0"] is None else torch.zeros(st["s0"].shape, dtype=torch.float64, device=q.device)
    for n in range(case["B"]):
        for h in range(H):
            a = (h, slice(cu[n], cu[n + 1])) if cu else (n, h)
            b = (h // r, slice(cu[n], cu[n + 1])) if cu else (n, h // r)
            F = g[a].cumsum(-1)
            T = F.shape[0]
            if not T:
                continue
            D = scale * torch.exp((F[:, None] - F[None]).masked_fill(torch.ones(T, T, dtype=torch.bool, device=q.device).triu(1), -math.inf))
            M, N = (q[b] @ k[b].T) * D, (d[a] @ v[a].T) * D
            out[a], dv[a] = M @ v[a], M.T @ d[a]
            dq[b] += N @ k[b]
            dk[b] += N.T @ q[b]
            X = M * (d[a] @ v[a].T)
            X.fill_diagonal_(0.0)
            through = X.sum(1) - X.sum(0)
            if ds0 is not None:
                S, e = st["s0"][n, h].double(), scale * torch.exp(F)[:, None]
                first = e * (q[b] @ S.T)
                out[a] += first
                dq[b] += e * (d[a] @ S)
                ds0[n, h] = (e * d[a]).T @ q[b]
                through = through + (first * d[a]).sum(-1)
            dg[a] = through.flip(0).cumsum(0).flip(0)
    got = {"out": out, "dq": dq, "dk": dk, "dv": dv}
    if case["decay"] == "token":
        got["dg"] = dg
    return got if ds0 is None else {**got, "dinitial_state": ds0}


def _exact_append(st):
    """Token by token of each sequence, pairs as complex numbers."""
    case = st["case"]
    page, dc, dr = case["page"], case["dc"], case["dr"]
    cache, q = st["cache"].double(), st["q"].double()
    table = st["table"].long()

    def turn(x, row):
        z = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), row.double()[:, None] * st["freqs"].double()[None])
        z = z if x.dim() == 2 else z[:, None]
        x = x.double()
        if case["interleaved"]:
            return torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (dr // 2, 2)).contiguous()) * z).flatten(-2)
        y = torch.complex(x[..., :dr // 2], x[..., dr // 2:]) * z
        return torch.cat([y.real, y.imag], -1)

    for b, n in enumerate(st["lengths"].tolist()):
        at = slice(int(st["cu"][b]), int(st["cu"][b + 1])) if case["packed"] else b
        c = st["latent"][at].double()
        row = torch.arange(n - c.shape[0], n, device=c.device)
        if st["weight"] is not None:
            c = c / torch.sqrt((c * c).mean(-1, keepdim=True) + st["eps"]) * st["weight"].double()
        cache[table[b][row // page], row % page] = torch.cat([c, turn(st["k_rope"][at], row)], -1)
        q[at, ..., dc:] = turn(st["q_rope"][at], row)
    return {"cache": cache, "q": q}


def _exact_tree(st):
    """Softmax sequence by sequence and node by node."""
    case = st["case"]
    T, dc = case["T"], case["dc"]
    out, lse = [], []
    for b, n in enumerate(st["lengths"].tolist()):
        at = torch.arange(n, device="cuda")
        rows = st["cache"][st["table"][b].long()[at // case["page"]], at % case["page"]].double()
        for i in range(T):
            bits = int(st["mask"][b, i])
            use = [n - T + j for j in range(T) if bits >> j & 1]
            sub = torch.cat([rows[:n - T], rows[use]])
            s = st["q"][b, i].double() @ sub.T * st["scale"]
            out.append(torch.softmax(s, -1) @ sub[:, :dc])
            lse.append(torch.logsumexp(s, -1))
    lead = (case["B"], T)
    return {"out": torch.stack(out).unflatten(0, lead), "lse": torch.stack(lse).unflatten(0, lead)}


# ------------------------------------------------------------------------------------- the work


def work(case):
    e, kind = 2 if case["io"] == "bf16" else 4, case["kind"]
    if kind.startswith("lin"):
        H, Hk, dk, dv = (case[n] for n in ("H", "Hk", "dk", "dv"))
        tokens = case["T"] * (1 if case["packed"] else case["B"])
        decay = tokens * H * e if case["decay"] == "token" else H * 4
        rows = tokens * (2 * Hk * dk + H * dv) * e + decay  # q, k, v, g
        state = case["B"] * H * dk * dv * 4
        if kind == "lin_decode":
            return {"bytes": rows + tokens * H * dv * e + 2 * state, "flops": 5.0 * tokens * H * dk * dv}
        # two products with the state, and those of a 64-token chunk, the causal ones at half
        C = min(64, case["T"])
        flops = tokens * H * (4.0 * dk * dv + C * (dk + dv))
        bytes_ = rows + tokens * H * dv * e + state * (2 if case["s0"] else 1)
        if kind == "lin_fwd":
            return {"bytes": bytes_, "flops": flops}
        grads = tokens * (2 * Hk * dk + H * dv + (H if case["decay"] == "token" else 0)) * e
        return {"bytes": rows + 2 * tokens * H * dv * e + grads + state * (2 if case["s0"] else 0),
                "flops": flops + tokens * H * (10.0 * dk * dv + C * (3 * dk + 2 * dv))}
    B, T, H, S, dc, dr = (case[n] for n in ("B", "T", "H", "S", "dc", "dr"))
    if kind == "append":
        tokens = T * (1 if case["packed"] else B)
        return {"bytes": 2.0 * tokens * (dc + dr + H * dr) * e, "flops": tokens * (4.0 * dc + 3.0 * dr * (H + 1))}
    # the histories lie between half of S and S
    rows = (0.75 * (B - 1) + 1) * S + B * T
    return {"bytes": rows * (dc + dr) * e + B * T * H * (2 * dc + dr) * e + B * T * H * 4, "flops": 2.0 * rows * T * H * (2 * dc + dr)}
