"""The token path around the attention block: embedding, QK norm + rotation, paged cache, one-token attention.

Each case is one pass through one operator.  With ``own`` false, ``run`` computes it in
elementary torch operations in float32; with ``own`` true it calls the framework.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------- cases


def listed():
    return [
        # The entry of a Llama-70B-width training step: 4096 tokens, eight sequence chunks.
        {"name": "embed-train", "kind": "embed", "dtype": "bf16", "s": 4096, "b": 1, "h": 8192, "vocab": 64000, "tp": 8,
         "scale": 1.0},
        # The entry of a serving step at the 22B width: one new token of each of 64 sequences.
        {"name": "embed-one-token", "kind": "embed", "dtype": "bf16", "s": 1, "b": 64, "h": 6144, "vocab": 51200, "tp": 1,
         "scale": 78.38},
        # The table's gradient added to a float32 main_grad: a micro-batch's last backward step.
        {"name": "embed-main-grad", "kind": "embed_main_grad", "dtype": "bf16", "s": 4096, "b": 1, "h": 8192,
         "vocab": 64000, "tp": 8, "scale": 1.0},
        # The table's gradient written whole in the storage type, four sequences at the 22B width.
        {"name": "embed-grad", "kind": "embed_grad", "dtype": "f16", "s": 2048, "b": 4, "h": 6144, "vocab": 51200, "tp": 8,
         "scale": 78.38},
        # Norm + rotation between the QKV projection and the core: the 22B model's 64 heads of 96.
        {"name": "qk-train", "kind": "qk", "dtype": "bf16", "s": 4096, "b": 1, "heads": 64, "kv_heads": 64, "d": 96,
         "rot": 96, "interleaved": False, "norm": True},
        # Its backward at the Llama-70B-like width, 64 query heads on 8 key/value heads.
        {"name": "qk-train-grad", "kind": "qk_grad", "dtype": "bf16", "s": 4096, "b": 1, "heads": 64, "kv_heads": 8,
         "d": 128, "rot": 128, "interleaved": False, "norm": True},
        # The serving form for one new token of each of 64 sequences: q out, k and v into the cache.
        {"name": "append-one-token", "kind": "append", "dtype": "bf16", "rows": 64, "heads": 64, "kv_heads": 8, "d": 128,
         "rot": 128, "interleaved": False, "norm": True, "page": 64, "pages": 2048},
        # A packed prefill of an odd number of tokens, interleaved pairs, a rotated part of each head.
        {"name": "append-prefill", "kind": "append", "dtype": "f16", "rows": 6151, "heads": 32, "kv_heads": 8, "d": 128,
         "rot": 64, "interleaved": True, "norm": True, "page": 16, "pages": 1024},
        # One long conversation.
        {"name": "decode-long", "kind": "decode", "dtype": "bf16", "n": 1, "heads": 64, "kv_heads": 8, "d": 128,
         "shortest": 131001, "longest": 131001, "page": 64},
        # A serving batch of unequal lengths.
        {"name": "decode-batch", "kind": "decode", "dtype": "bf16", "n": 64, "heads": 64, "kv_heads": 8, "d": 128,
         "shortest": 17, "longest": 8192, "page": 16},
        # Multi-head attention, every head its own keys and values.
        {"name": "decode-mha", "kind": "decode", "dtype": "f16", "n": 16, "heads": 64, "kv_heads": 64, "d": 96,
         "shortest": 1200, "longest": 2900, "page": 32},
        # The first tokens of a few short answers: latency.
        {"name": "decode-short", "kind": "decode", "dtype": "bf16", "n": 4, "heads": 32, "kv_heads": 8, "d": 128,
         "shortest": 1, "longest": 300, "page": 16},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


HEADS = ((64, 8, 128), (64, 64, 96), (32, 8, 128), (40, 8, 128), (12, 4, 96), (8, 1, 128), (28, 4, 128), (16, 16, 64),
         (24, 2, 128), (48, 16, 96), (6, 6, 128))


def draw(rng):
    kind = rng.choice(("embed", "embed_grad", "embed_main_grad", "qk", "qk_grad", "append", "append", "decode", "decode",
                       "decode"))
    dtype = rng.choice(("bf16", "f16"))
    if kind.startswith("embed"):
        tp = rng.choice((1, 2, 4, 8))
        b = rng.choice((1, 1, 2, 3, 8))
        h = 8 * _log(rng, 64, 1024)
        s = max(1, _log(rng, 1, 8192) // (b * tp)) * tp
        return {"kind": kind, "dtype": dtype, "s": s, "b": b, "h": h, "vocab": _log(rng, 100, 64000), "tp": tp,
                "scale": rng.choice((1.0, round(math.sqrt(h), 2)))}
    heads, kv_heads, d = rng.choice(HEADS)
    if kind == "decode":
        n = _log(rng, 1, 128)
        room = max(1, 1_100_000_000 // (4 * kv_heads * d * n))  # bytes of the longest listed case, by the mean length
        longest = _log(rng, 1, min(131072, room))
        return {"kind": kind, "dtype": dtype, "n": n, "heads": heads, "kv_heads": kv_heads, "d": d,
                "shortest": rng.randint(0, longest), "longest": longest, "page": rng.choice((8, 16, 16, 32, 64, 128))}
    rot = rng.choice((d, d, d // 2))
    more = {"heads": heads, "kv_heads": kv_heads, "d": d, "rot": rot, "interleaved": rng.random() < 0.4,
            "norm": rng.random() < 0.8}
    if kind == "append":
        page = rng.choice((16, 32, 64))
        rows = _log(rng, 1, 8192)
        return {"kind": kind, "dtype": dtype, "rows": rows, **more, "page": page, "pages": 2 * rows // page + 3}
    b = rng.choice((1, 1, 2, 3))
    return {"kind": kind, "dtype": dtype, "s": max(1, _log(rng, 1, 4096) // b), "b": b, **more}


# ---------------------------------------------------------------------------- inputs


def _normal(g, *shape, dtype, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _zipf(g, vocab, *shape):
    """Token ids whose frequency falls as one over their rank, as in text."""
    u = torch.rand(*shape, generator=g, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(vocab + 1.0)).floor().long() - 1
    order = torch.randperm(vocab, generator=g, device="cuda")
    return order[rank.clamp_(0, vocab - 1)]


def _tables(rot, count):
    """cos and sin of p·10000^(−2i/rot), computed in 64 bits."""
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    a = torch.arange(count, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * i / rot)
    return a.cos().float(), a.sin().float()


def _gammas(g, c, dtype):
    if not c["norm"]:
        return None, None
    return tuple((1 + 0.1 * torch.randn(c["d"], generator=g, device="cuda")).to(dtype) for _ in range(2))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = case
    dt = DTYPES[c["dtype"]]
    st = {"case": c}
    if c["kind"].startswith("embed"):
        s, b, h, V, tp = c["s"], c["b"], c["h"], c["vocab"], c["tp"]
        st["tokens"] = _zipf(g, V, b, s).t()  # batches come as [b, s]; the trunk is sequence-first
        if c["kind"] == "embed":
            st["table"] = _normal(g, V, h, dtype=dt, std=0.02)
            st["out"] = [torch.zeros(s // tp, b, h, dtype=dt, device="cuda") for _ in range(tp)]
        else:
            st["dx"] = [_normal(g, s // tp, b, h, dtype=dt) for _ in range(tp)]
            if c["kind"] == "embed_main_grad":
                st["grad"] = torch.randn(V, h, generator=g, device="cuda")  # of earlier micro-batches
            else:
                st["grad"] = torch.zeros(V, h, dtype=dt, device="cuda")
        return st
    heads, kv, d = c["heads"], c["kv_heads"], c["d"]
    W = (heads + 2 * kv) * d
    if c["kind"] == "decode":
        n, page = c["n"], c["page"]
        lengths = torch.randint(c["shortest"], c["longest"] + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
        width = -(-max(1, c["longest"]) // page)
        used = (lengths.long() + page - 1) // page
        first = torch.cumsum(used, 0) - used
        pages = n * width
        order = torch.randperm(pages, generator=g, device="cuda").int()
        col = torch.arange(width, device="cuda")
        table = torch.where(col[None] < used[:, None], order[(first[:, None] + col[None]).clamp(max=pages - 1)], -1)
        st["block_table"], st["lengths"] = table.int().contiguous(), lengths
        st["q"] = _normal(g, n, heads, d, dtype=dt)
        st["k"] = torch.empty(pages, page, kv, d, dtype=dt, device="cuda").normal_(generator=g)
        st["v"] = torch.empty(pages, page, kv, d, dtype=dt, device="cuda").normal_(generator=g)
        st["o"] = torch.zeros(n, heads, d, dtype=dt, device="cuda")
        st["lse"] = torch.zeros(n, heads, dtype=torch.float32, device="cuda")
        return st
    st["gq"], st["gk"] = _gammas(g, c, dt)
    if c["kind"] == "append":
        rows, page = c["rows"], c["page"]
        st["qkv"] = _normal(g, rows, W, dtype=dt)
        st["cos"], st["sin"] = _tables(c["rot"], 16384)
        st["positions"] = torch.randint(0, 16384, (rows,), generator=g, device="cuda")
        st["slots"] = torch.randperm(c["pages"] * page, generator=g, device="cuda")[:rows]
        st["k"] = torch.zeros(c["pages"], page, kv, d, dtype=dt, device="cuda")
        st["v"] = torch.zeros(c["pages"], page, kv, d, dtype=dt, device="cuda")
        st["q"] = torch.zeros(rows, heads, d, dtype=dt, device="cuda")
        return st
    rows = c["s"] * c["b"]
    st["qkv"] = _normal(g, rows, W, dtype=dt)
    st["cos"], st["sin"] = _tables(c["rot"], c["s"])
    if c["kind"] == "qk":
        st["out"] = torch.zeros(rows, W, dtype=dt, device="cuda")
    else:
        st["dout"] = _normal(g, rows, W, dtype=dt)
        st["dqkv"] = torch.zeros(rows, W, dtype=dt, device="cuda")
        if c["norm"]:
            st["dgq"], st["dgk"] = torch.zeros(2, d, device="cuda").unbind(0)
    return st


# ---------------------------------------------------------------------------- plain forms (float32)


def _embed(st, c):
    table, tokens = st["table"], st["tokens"]
    x = (table[tokens].float() * c["scale"]).to(table.dtype)
    torch._foreach_copy_(st["out"], list(x.chunk(c["tp"])))
    return st["out"]


def _embed_grad(st, c):
    dx = torch.cat(st["dx"]).reshape(-1, c["h"]).float() * c["scale"]
    tokens = st["tokens"].reshape(-1)
    if c["kind"] == "embed_main_grad":
        return st["grad"].index_add_(0, tokens, dx)
    full = torch.zeros(c["vocab"], c["h"], device="cuda").index_add_(0, tokens, dx)
    return st["grad"].copy_(full)


def _grouped(x, c):
    """[rows, W] as [rows, groups, q heads of the group + k + v, d]."""
    return x.reshape(x.shape[0], c["kv_heads"], c["heads"] // c["kv_heads"] + 2, c["d"])


def _rms(x):
    return 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)


def _rotate(x, cos, sin, c):
    rot = c["rot"]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2 : rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


EPS = 1e-6


def _qk(st, c, cos, sin):
    x = _grouped(st["qkv"].float(), c)
    q, k, v = x[..., :-2, :], x[..., -2:-1, :], x[..., -1:, :]
    if c["norm"]:
        q, k = q * _rms(q) * st["gq"].float(), k * _rms(k) * st["gk"].float()
    return _rotate(q, cos, sin, c), _rotate(k, cos, sin, c), v


def _by_row(table, c):
    """cos or sin of row m = t·b + bi at position t, shaped to stand beside [rows, groups, heads, ·]."""
    return table[: c["s"]].repeat_interleave(c["b"], 0)[:, None, None]


def _qk_train(st, c):
    q, k, v = _qk(st, c, _by_row(st["cos"], c), _by_row(st["sin"], c))
    return st["out"].copy_(torch.cat((q, k, v), 2).flatten(1))


def _norm_grad(x, dn, gamma):
    r = _rms(x)
    n = x * r
    g = dn * gamma.float()
    return r * (g - n * (g * n).mean(-1, keepdim=True)), (dn * n).flatten(0, 2).sum(0)


def _qk_grad(st, c):
    cos, sin = _by_row(st["cos"], c), _by_row(st["sin"], c)
    x, dy = _grouped(st["qkv"].float(), c), _grouped(st["dout"].float(), c)
    dq, dk = _rotate(dy[..., :-2, :], cos, -sin, c), _rotate(dy[..., -2:-1, :], cos, -sin, c)
    if c["norm"]:
        dq, dgq = _norm_grad(x[..., :-2, :], dq, st["gq"])
        dk, dgk = _norm_grad(x[..., -2:-1, :], dk, st["gk"])
        st["dgq"].copy_(dgq)
        st["dgk"].copy_(dgk)
    st["dqkv"].copy_(torch.cat((dq, dk, dy[..., -1:, :]), 2).flatten(1))
    return {k: st[k] for k in ("dqkv", "dgq", "dgk") if k in st}


def _append(st, c):
    pos = st["positions"]
    q, k, v = _qk(st, c, st["cos"][pos][:, None, None], st["sin"][pos][:, None, None])
    st["q"].copy_(q.reshape(st["q"].shape))
    st["k"].flatten(0, 1)[st["slots"]] = k.squeeze(2).to(st["k"].dtype)
    st["v"].flatten(0, 1)[st["slots"]] = v.squeeze(2).to(st["v"].dtype)
    return {"q": st["q"], "k": st["k"], "v": st["v"]}


def _decode(st, c):
    kv, d, n = c["kv_heads"], c["d"], c["n"]
    pages = st["block_table"].clamp(min=0).long()
    k, v = (st[x][pages].flatten(1, 2).float() for x in ("k", "v"))  # [n, keys, kv, d]
    q = st["q"].float().reshape(n, kv, -1, d)
    s = torch.einsum("ngrd,nkgd->ngrk", q, k) * (d**-0.5)
    seen = (torch.arange(k.shape[1], device="cuda")[None] < st["lengths"][:, None])[:, None, None]
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(s - top)
    l = p.sum(-1, keepdim=True)
    o = torch.einsum("ngrk,nkgd->ngrd", p, v) / torch.where(l > 0, l, torch.ones_like(l))
    st["o"].copy_(o.reshape(n, -1, d))
    st["lse"].copy_(((torch.log(l) + top) * math.log2(math.e)).reshape(n, -1))
    return {"o": st["o"], "lse": st["lse"]}


# ---------------------------------------------------------------------------- one pass


def _rope(T, st):
    """The norm weights and rotation tables as a program keeps them."""
    if "rope" not in st:
        st["rope"] = T.QKRope(q_gamma=st["gq"], k_gamma=st["gk"], eps=EPS, cos=st["cos"], sin=st["sin"],
                              interleaved=st["case"]["interleaved"])
    return st["rope"]


def _workspace(st, size):
    if "ws" not in st:
        st["ws"] = torch.empty(max(256, size()), dtype=torch.uint8, device="cuda")
    return st["ws"]


def _cache(T, st):
    if "cache" not in st:
        st["cache"] = T.PagedKVCache(st["k"], st["v"])
    return st["cache"]


def _run_own(st, c):
    import sp_partitioned_transformer_gb300 as T

    kind = c["kind"]
    if kind.startswith("embed"):
        kw = dict(s=c["s"], b=c["b"], h=c["h"], vocab=c["vocab"], tp=c["tp"], scale=c["scale"])
        if kind == "embed":
            T.embed_forward(st["tokens"], st["table"], st["out"], **kw)
            return st["out"]
        ws = _workspace(st, lambda: T.embed_backward_workspace(c["s"], c["b"], c["h"], c["vocab"]))
        call = T.embed_backward_main_grad if kind == "embed_main_grad" else T.embed_backward
        call(st["tokens"], st["dx"], st["grad"], workspace=ws, **kw)
        return st["grad"]
    kw = dict(heads=c["heads"], kv_heads=c["kv_heads"], d=c["d"])
    if kind == "qk":
        T.qk_norm_rope_forward(st["qkv"], st["out"], _rope(T, st), rows=c["s"] * c["b"], b=c["b"], **kw)
        return st["out"]
    if kind == "qk_grad":
        rows = c["s"] * c["b"]
        ws = _workspace(st, lambda: T.qk_norm_rope_backward_workspace(rows, c["heads"], c["kv_heads"], c["d"]))
        T.qk_norm_rope_backward(st["qkv"], st["dout"], st["dqkv"], st.get("dgq"), st.get("dgk"), _rope(T, st), rows=rows,
                                b=c["b"], workspace=ws, **kw)
        return {k: st[k] for k in ("dqkv", "dgq", "dgk") if k in st}
    if kind == "append":
        T.qk_norm_rope_append(st["qkv"], st["q"], _cache(T, st), st["slots"], _rope(T, st), rows=c["rows"],
                              positions=st["positions"], **kw)
        return {"q": st["q"], "k": st["k"], "v": st["v"]}
    ws = _workspace(st, lambda: T.paged_attn_workspace_size(c["n"], c["heads"], c["kv_heads"], c["d"]))
    T.paged_attn_decode(st["q"], _cache(T, st), st["block_table"], st["lengths"], st["o"], st["lse"], n=c["n"],
                        workspace=ws, **kw)
    return {"o": st["o"], "lse": st["lse"]}


PLAIN = {"embed": _embed, "embed_grad": _embed_grad, "embed_main_grad": _embed_grad, "qk": _qk_train,
         "qk_grad": _qk_grad, "append": _append, "decode": _decode}


def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    return PLAIN[c["kind"]](state, c)


# ---------------------------------------------------------------------------- floors


def work(case):
    c = case
    e = 4 if c["dtype"] == "f32" else 2
    if c["kind"].startswith("embed"):
        M, h, V = c["s"] * c["b"], c["h"], c["vocab"]
        # distinct tokens of the draw: rank r has probability log((r+1)/r)/log(V+1)
        r = torch.arange(1, V + 1, dtype=torch.float64)
        distinct = float((1 - (1 - torch.log1p(1 / r) / math.log(V + 1.0)) ** M).sum())
        if c["kind"] == "embed":
            return {"bytes": distinct * h * e + M * (h * e + 8), "flops": M * h}
        if c["kind"] == "embed_main_grad":
            return {"bytes": M * (h * e + 8) + distinct * h * 8, "flops": 2 * M * h}
        return {"bytes": M * (h * e + 8) + V * h * e, "flops": 2 * M * h}
    heads, kv, d = c["heads"], c["kv_heads"], c["d"]
    if c["kind"] == "decode":
        keys = c["n"] * (c["shortest"] + c["longest"]) / 2
        return {"bytes": keys * kv * d * 2 * e + c["n"] * heads * (2 * d * e + 4), "flops": 4 * keys * heads * d}
    rows = c["rows"] if c["kind"] == "append" else c["s"] * c["b"]
    W = (heads + 2 * kv) * d
    tables = min(rows if c["kind"] == "append" else c["s"], 16384) * c["rot"] * 4
    qk = rows * (heads + kv) * d
    if c["kind"] == "qk_grad":
        return {"bytes": 2 * rows * W * e + (qk * e if c["norm"] else 0) + tables, "flops": 20 * qk}
    return {"bytes": 2 * rows * W * e + tables, "flops": 9 * qk}


# ---------------------------------------------------------------------------- 64 bits


def _turn64(x, cos, sin, c, sign):
    """Pairs as complex numbers, multiplied by cos + i·sign·sin."""
    rot = c["rot"]
    z = torch.complex(cos.double(), sign * sin.double())
    part = x[..., :rot]
    if c["interleaved"]:
        w = torch.view_as_complex(part.reshape(*part.shape[:-1], rot // 2, 2).contiguous()) * z
        turned = torch.view_as_real(w).reshape(part.shape)
    else:
        w = torch.complex(part[..., : rot // 2].contiguous(), part[..., rot // 2 :].contiguous()) * z
        turned = torch.cat((w.real, w.imag), -1)
    out = x.clone()
    out[..., :rot] = turned
    return out


def _scaled64(x, gamma):
    """x over its root mean square, times gamma, by the norm of the vector."""
    if gamma is None:
        return x
    d = x.shape[-1]
    size = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
    return x / torch.sqrt(size**2 / d + EPS) * gamma.double()


def _scaled64_grad(x, dn, gamma):
    """The gradient of _scaled64 from its Jacobian's two terms, and of gamma."""
    if gamma is None:
        return dn, None
    d = x.shape[-1]
    ms = x.pow(2).sum(-1, keepdim=True) / d + EPS
    dg = (dn * x * ms.rsqrt()).reshape(-1, d).sum(0)
    t = dn * gamma.double()
    return t * ms.rsqrt() - x * (t * x).sum(-1, keepdim=True) * ms.pow(-1.5) / d, dg


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    kind = c["kind"]
    if kind.startswith("embed"):
        ids = st["tokens"].reshape(-1)
        if kind == "embed":
            x = st["table"].double().index_select(0, ids).mul_(c["scale"])
            return list(x.reshape(c["s"], c["b"], c["h"]).tensor_split(c["tp"]))
        dx = torch.cat([p.reshape(-1, c["h"]) for p in st["dx"]]).double()
        order = torch.argsort(ids, stable=True)
        which, count = torch.unique_consecutive(ids[order], return_counts=True)
        sums = torch.segment_reduce(dx[order], "sum", lengths=count, axis=0) * c["scale"]
        grad = st["grad"].double() if kind == "embed_main_grad" else torch.zeros(c["vocab"], c["h"], dtype=torch.float64,
                                                                                device="cuda")
        grad[which] += sums
        return grad
    heads, kv, d = c["heads"], c["kv_heads"], c["d"]
    r = heads // kv
    if kind == "decode":
        o = torch.zeros(c["n"], heads, d, dtype=torch.float64, device="cuda")
        lse = torch.full((c["n"], heads), -math.inf, dtype=torch.float64, device="cuda")
        for i, length in enumerate(st["lengths"].tolist()):
            if length == 0:
                continue
            own_pages = st["block_table"][i, : -(-length // c["page"])].long()
            k = st["k"][own_pages].reshape(-1, kv, d)[:length].double()
            v = st["v"][own_pages].reshape(-1, kv, d)[:length].double()
            q = st["q"][i].double().reshape(kv, r, d)
            s = torch.matmul(q, k.permute(1, 2, 0)) / math.sqrt(d)
            lse[i] = (torch.logsumexp(s, -1) / math.log(2.0)).reshape(-1)
            o[i] = torch.matmul(torch.softmax(s, -1), v.transpose(0, 1)).reshape(heads, d)
        return {"o": o, "lse": lse}
    rows = st["qkv"].shape[0]
    x = st["qkv"].double().view(rows, kv, r + 2, d)
    if kind == "append":
        at = st["positions"]
    else:
        at = torch.arange(rows, device="cuda") // c["b"]
    cos, sin = st["cos"][at].view(rows, 1, 1, -1), st["sin"][at].view(rows, 1, 1, -1)
    if kind == "qk_grad":
        dy = st["dout"].double().view(rows, kv, r + 2, d)
        out = dy.clone()
        out[:, :, :r], dgq = _scaled64_grad(x[:, :, :r], _turn64(dy[:, :, :r], cos, sin, c, -1.0), st["gq"])
        out[:, :, r : r + 1], dgk = _scaled64_grad(x[:, :, r : r + 1], _turn64(dy[:, :, r : r + 1], cos, sin, c, -1.0),
                                                   st["gk"])
        got = {"dqkv": out.view(rows, -1)}
        return {**got, "dgq": dgq, "dgk": dgk} if c["norm"] else got
    q = _turn64(_scaled64(x[:, :, :r], st["gq"]), cos, sin, c, 1.0)
    k = _turn64(_scaled64(x[:, :, r : r + 1], st["gk"]), cos, sin, c, 1.0)
    if kind == "qk":
        return torch.cat((q, k, x[:, :, r + 1 :]), 2).view(rows, -1)
    kc, vc = st["k"].double(), st["v"].double()
    page, offset = st["slots"] // c["page"], st["slots"] % c["page"]
    kc[page, offset] = k[:, :, 0]
    vc[page, offset] = x[:, :, r + 1]
    return {"q": q.reshape(rows, heads, d), "k": kc, "v": vc}
