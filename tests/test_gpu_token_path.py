"""The operators together, as a program uses them: a training step from token ids
through the attention block with QK norm and rotation and back to the table's
gradient; and a prompt written to a paged cache and continued token by token,
against the training block over the whole sequence.

Training: every tensor within 2e-2 of the fp64 oracle (‖·‖∞ over ‖·‖∞), the
framework's bound for blocks.  Serving: same bound between the two paths, which
round at the same places."""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_common import rel_err, to_np

pytestmark = pytest.mark.gpu
TOL = 2e-2


def _setup(T, s, b, h, heads, kv, dt, norm=True, rot=None, interleaved=False, vocab=50, seed=0):
    g = torch.Generator().manual_seed(seed)
    d = h // heads
    rot = d if rot is None else rot
    W = h + 2 * kv * d
    t = {
        "E": torch.randn(vocab, h, generator=g).mul(0.5).to(dt),
        "Wqkv": torch.randn(W, h, generator=g).mul(0.05).to(dt),
        "Wo": torch.randn(h, h, generator=g).mul(0.05).to(dt),
        "tok": torch.randint(0, vocab, (b, s), generator=g).t(),
        "dZ": torch.randn(s, b, h, generator=g).to(dt),
        "gq": (1 + 0.2 * torch.randn(d, generator=g)).to(dt) if norm else None,
        "gk": (1 + 0.2 * torch.randn(d, generator=g)).to(dt) if norm else None,
    }
    a = torch.arange(s).double()[:, None] * 10000.0 ** (-2.0 * torch.arange(rot // 2).double() / rot)
    t["cos"], t["sin"] = a.cos().float(), a.sin().float()
    dev = {k: (v if v is None else v.cuda()) for k, v in t.items()}
    dev["tok"] = t["tok"].t().contiguous().cuda().t()
    rope = T.QKRope(q_gamma=dev["gq"], k_gamma=dev["gk"], eps=1e-6, cos=dev["cos"], sin=dev["sin"], interleaved=interleaved)
    return t, dev, rope


TRAIN = [
    # s, b, h, heads, kv, tp, sp, dtype, norm, rot, interleaved
    (256, 1, 512, 4, 2, 2, True, torch.bfloat16, True, 128, False),
    (100, 2, 384, 4, 4, 2, True, torch.float16, True, 48, True),  # chunks gathered, heads of 96
    (130, 1, 512, 4, 1, 1, False, torch.bfloat16, False, 128, False),
]


@pytest.mark.parametrize("case", TRAIN, ids=["gqa-sp-in-place", "d96-gathered-partial", "mqa-no-norm"])
def test_training_step(cuda_lib, case):
    s, b, h, heads, kv, tp, sp, dt, norm, rot, inter = case
    T, vocab, scale = cuda_lib, 50, 2.0
    t, dev, rope = _setup(T, s, b, h, heads, kv, dt, norm, rot, inter, vocab)
    nx = tp if sp else 1
    kw = dict(s=s, b=b, h=h, vocab=vocab, tp=nx, scale=scale)
    x = [torch.empty(s // nx, b, h, dtype=dt, device="cuda") for _ in range(nx)]
    T.embed_forward(dev["tok"], dev["E"], x, **kw)
    blk = T.AttnBlock(s, b, h, heads, tp, sp, dt, True, kv_heads=kv, rope=rope)
    arg = x if sp else x[0]
    dz = [c.contiguous() for c in dev["dZ"].chunk(tp)] if sp else dev["dZ"]
    fw = blk.forward(arg, dev["Wqkv"], dev["Wo"])
    bw = blk.backward(arg, dev["Wqkv"], dev["Wo"], fw, dz)
    dE = torch.empty(vocab, h, dtype=dt, device="cuda")
    T.embed_backward(dev["tok"], bw["dx"], dE, **kw)
    torch.cuda.synchronize()
    assert T.device_status() == 0, T.last_error()

    f = lambda v: None if v is None else v.double().numpy()  # noqa: E731
    M, tok = s * b, t["tok"].numpy()
    X = O.embed_forward(f(t["E"]), tok, scale)
    at = np.arange(M) // b
    okw = dict(heads=heads, kv_heads=kv, cos=f(t["cos"])[at], sin=f(t["sin"])[at], gq=f(t["gq"]), gk=f(t["gk"]),
               eps=1e-6 if norm else 0.0, interleaved=inter)
    raw = X @ f(t["Wqkv"]).T
    qkv = O.qk_norm_rope_forward(raw, **okw)
    Q, K, V = O.split_qkv(qkv, heads, kv)
    o = O.attention_core_forward(Q, K, V, s, b, heads, True, kv)
    o = o["O"] if isinstance(o, dict) else o[0]
    dZ = f(t["dZ"]).reshape(M, h)
    dO = dZ @ f(t["Wo"])
    core = O.attention_core_backward(Q, K, V, dO, s, b, heads, True, kv)
    dQ, dK, dV = (core["dQ"], core["dK"], core["dV"]) if isinstance(core, dict) else core[:3]
    dqkv, dgq, dgk = O.qk_norm_rope_backward(raw, O.merge_qkv(dQ, dK, dV, heads, kv), **okw)
    dX = dqkv @ f(t["Wqkv"])
    want = {"z": o @ f(t["Wo"]).T, "qkv": qkv, "dwqkv": dqkv.T @ X, "dwo": dZ.T @ o, "dqkv": dqkv,
            "dE": O.embed_backward(dX, tok, vocab, scale)}
    cat = lambda v: torch.cat(v) if isinstance(v, list) else v  # noqa: E731
    have = {"z": cat(fw["z"]), "qkv": fw["qkv"], "dwqkv": bw["dwqkv"], "dwo": bw["dwo"], "dqkv": bw["dqkv"], "dE": dE}
    if norm:
        want |= {"dgq": dgq, "dgk": dgk}
        have |= {"dgq": bw["dq_gamma"], "dgk": bw["dk_gamma"]}
    errs = {k: rel_err(to_np(have[k]).reshape(w.shape), w) for k, w in want.items()}
    assert all(e <= TOL for e in errs.values()), errs


def test_block_without_rope_is_unchanged(cuda_lib):
    """Angle 0 and no norm: the rope block's bits are the plain block's."""
    T = cuda_lib
    t, dev, _ = _setup(T, 128, 1, 256, 2, 2, torch.bfloat16)
    one = T.QKRope(cos=torch.ones(128, 64, device="cuda"), sin=torch.zeros(128, 64, device="cuda"))
    x, dz = dev["dZ"], dev["dZ"].flip(0).contiguous()
    got = []
    for rope in (None, one):
        blk = T.AttnBlock(128, 1, 256, 2, 1, False, torch.bfloat16, True, rope=rope)
        fw = blk.forward(x, dev["Wqkv"], dev["Wo"])
        bw = blk.backward(x, dev["Wqkv"], dev["Wo"], fw, dz)
        got.append([fw["z"], fw["lse"], bw["dx"], bw["dwqkv"], bw["dwo"]])
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("heads,kv,h,dt,page", [(8, 2, 1024, torch.bfloat16, 16), (4, 4, 384, torch.float16, 5),
                                               (16, 1, 2048, torch.bfloat16, 64)])
def test_prompt_then_tokens_one_by_one(cuda_lib, heads, kv, h, dt, page):
    """Ragged prompts go to the cache in one call, the next tokens one at a time through tpmlp_attn_decode;
    each new token's z is the training block's row of the whole sequence."""
    T, d, n, new = cuda_lib, h // heads, 3, 4
    prompts = [37, 1, 100]
    s = max(prompts) + new
    t, dev, rope = _setup(T, s, n, h, heads, kv, dt, norm=True)
    W = h + 2 * kv * d
    x = torch.empty(s, n, h, dtype=dt, device="cuda")  # every sequence to its end, for the reference
    T.embed_forward(dev["tok"], dev["E"], x, s=s, b=n, h=h, vocab=50, tp=1)
    blk = T.AttnBlock(s, n, h, heads, 1, False, dt, True, kv_heads=kv, rope=rope)
    fw = blk.forward(x, dev["Wqkv"], dev["Wo"])
    want = fw["z"]

    width = -(-s // page)
    order = torch.randperm(n * width + 1, generator=torch.Generator().manual_seed(5)).int()
    table = order[: n * width].view(n, width).cuda()
    k, v = (torch.full((n * width + 1, page, kv, d), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    cache = T.PagedKVCache(k, v)

    def slots(seq, pos):
        return table[seq, pos // page].long() * page + pos % page

    seq = torch.cat([torch.full((p,), i) for i, p in enumerate(prompts)]).cuda()
    pos = torch.cat([torch.arange(p) for p in prompts]).cuda()
    raw = fw["qkv_raw"].view(s, n, W)[pos, seq].contiguous()  # the prompts' tokens, packed
    q = torch.empty(len(seq), heads, d, dtype=dt, device="cuda")
    T.qk_norm_rope_append(raw, q, cache, slots(seq, pos), rope, rows=len(seq), heads=heads, kv_heads=kv, d=d, positions=pos)
    every = torch.arange(n).cuda()
    lengths = torch.tensor(prompts, dtype=torch.int32).cuda()
    ws = torch.empty(T.paged_attn_workspace_size(n, heads, kv, d), dtype=torch.uint8, device="cuda")
    buf = [torch.empty(n, w, dtype=dt, device="cuda") for w in (W, h, h, h)]
    for _ in range(new):
        at = lengths.long()
        lengths += 1  # with the token of this step
        T.attn_decode(x[at, every].contiguous(), dev["Wqkv"], dev["Wo"], rope, cache, at, slots(every, at), table, lengths,
                      *buf, n=n, h=h, heads=heads, kv_heads=kv, workspace=ws)
        assert rel_err(to_np(buf[3]), to_np(want[at, every])) <= TOL
    assert T.device_status() == 0, T.last_error()


def test_tensors_off_the_device_and_of_other_kinds_are_refused(cuda_lib):
    T, d = cuda_lib, 64
    x = torch.zeros(2, 3 * d, dtype=torch.bfloat16)
    g = torch.ones(d, dtype=torch.bfloat16)
    rope, dev_rope = (T.QKRope(q_gamma=t, k_gamma=t) for t in (g, g.cuda()))
    kw = dict(rows=2, b=1, heads=1, kv_heads=1, d=d)
    for a, b, r in ((x, x.cuda(), dev_rope), (x.cuda(), x, dev_rope), (x.cuda(), x.cuda(), rope)):
        with pytest.raises(ValueError, match="current device"):
            T.qk_norm_rope_forward(a, b, r, **kw)
    with pytest.raises(ValueError, match="gamma"):
        T.qk_norm_rope_forward(x.cuda().half(), x.cuda().half(), dev_rope, **kw)
    tok = torch.zeros(2, 1, dtype=torch.int64)
    E = torch.zeros(3, 8, device="cuda")
    with pytest.raises(ValueError, match="current device"):
        T.embed_forward(tok, E, torch.zeros(2, 1, 8, device="cuda"), s=2, b=1, h=8, vocab=3, tp=1)
    with pytest.raises(ValueError, match="current device"):
        T.embed_forward(tok.cuda(), E, torch.zeros(2, 1, 8), s=2, b=1, h=8, vocab=3, tp=1)
    with pytest.raises(ValueError, match="chunks"):
        T.embed_forward(tok.cuda(), E, torch.zeros(2, 1, 8, device="cuda"), s=2, b=1, h=8, vocab=3, tp=2)
    k = torch.zeros(2, 4, 1, d, dtype=torch.bfloat16)
    q = torch.zeros(1, 1, d, dtype=torch.bfloat16, device="cuda")
    one, table = torch.ones(1, dtype=torch.int32, device="cuda"), torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    for cache, lens in ((T.PagedKVCache(k, k), one), (T.PagedKVCache(k.cuda(), k.cuda()), one.cpu())):
        with pytest.raises(ValueError, match="current device"):
            T.paged_attn_decode(q, cache, table, lens, q.clone(), n=1, heads=1, kv_heads=1, d=d)
    with pytest.raises(ValueError, match="cache"):
        T.paged_attn_decode(q.expand(1, 2, d).contiguous(), T.PagedKVCache(k.cuda(), k.cuda()), table, one,
                            q.expand(1, 2, d).contiguous(), n=1, heads=2, kv_heads=2, d=d)


def test_calls_back_to_back_see_each_other(cuda_lib):
    """Launches overlap their predecessors' ends: a chain of calls without a wait, each on the last one's
    output, equals the same chain with a wait after every call."""
    T, d, n = cuda_lib, 128, 40
    g = torch.Generator().manual_seed(2)
    a = torch.rand(64, d // 2, generator=g)
    rope = T.QKRope(cos=a.cos().cuda(), sin=a.sin().cuda())
    x0 = torch.randn(n, 6 * d, generator=g).to(torch.bfloat16).cuda()
    pages = torch.randperm(n, generator=g).int().cuda().view(n, 1)
    slots = pages.view(-1).long() * 16
    pos = torch.randint(0, 64, (n,), generator=g).cuda()
    lens = torch.ones(n, dtype=torch.int32, device="cuda")
    ws = torch.empty(T.paged_attn_workspace_size(n, 4, 1, d), dtype=torch.uint8, device="cuda")

    def chain(wait):
        k, v = (torch.zeros(n, 16, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        cache, x = T.PagedKVCache(k, v), x0.clone()
        q, o = (torch.empty(n, 4, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        for i in range(16):
            for step in (lambda: T.qk_norm_rope_forward(x, x, rope, rows=n, b=1, heads=4, kv_heads=1, d=d, positions=pos),
                         lambda: T.qk_norm_rope_append(x, q, cache, slots + i, rope, rows=n, heads=4, kv_heads=1, d=d,
                                                       positions=pos),
                         lambda: T.paged_attn_decode(q, cache, pages, lens + i, o, n=n, heads=4, kv_heads=1, d=d,
                                                     workspace=ws),
                         lambda: T.qk_norm_rope_forward(o.view(n, 4 * d), x[:, : 4 * d], rope, rows=n, b=1, heads=2,
                                                        kv_heads=1, d=d, positions=pos)):
                step()
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return x, o, k, v

    assert all(torch.equal(a, b) for a, b in zip(chain(False), chain(True)))


@pytest.mark.parametrize("as_int", [False, True])
def test_temporary_workspaces_outlive_calls_on_other_streams(cuda_lib, as_int):
    """Without a workspace of the caller's, one is made for the call: on a stream of its own it must not be
    given out again before that stream has used it."""
    T, d, n = cuda_lib, 128, 6
    g = torch.Generator().manual_seed(8)
    k, v = (torch.randn(600, 16, 1, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(n, 8, d, generator=g).to(torch.bfloat16).cuda()
    table = torch.arange(600).int().view(n, 100).cuda()
    lens = torch.tensor([1600, 3, 900, 0, 1599, 64], dtype=torch.int32).cuda()
    want, got = torch.empty_like(q), torch.empty_like(q)
    kw = dict(n=n, heads=8, kv_heads=1, d=d)
    T.paged_attn_decode(q, T.PagedKVCache(k, v), table, lens, want, **kw)
    size = T.paged_attn_workspace_size(n, 8, 1, d)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        T.paged_attn_decode(q, T.PagedKVCache(k, v), table, lens, got, stream=st.cuda_stream if as_int else st, **kw)
        torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xFF)  # what takes the freed block's place
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_empty_batches(cuda_lib):
    """No tokens, rows or sequences (tensors of no elements): gradients become zero, sums and the cache stay."""
    T, dt, h, vocab = cuda_lib, torch.bfloat16, 256, 5
    E = lambda *shape, dtype=dt: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    kw = dict(s=0, b=2, h=h, vocab=vocab, tp=2)
    tok, x = E(0, 2, dtype=torch.int64), [E(0, 2, h), E(0, 2, h)]
    T.embed_forward(tok, E(vocab, h), x, **kw)
    grad, main = torch.ones(vocab, h, dtype=dt, device="cuda"), torch.ones(vocab, h, device="cuda")
    T.embed_backward(tok, x, grad, **kw)
    T.embed_backward_main_grad(tok, x, main, **kw)
    assert (grad == 0).all() and (main == 1).all()
    one, tab = torch.ones(64, dtype=dt, device="cuda"), torch.ones(4, 32, device="cuda")
    rope = T.QKRope(q_gamma=one, k_gamma=one, cos=tab, sin=tab)
    kw = dict(rows=0, heads=4, kv_heads=2, d=64)
    T.qk_norm_rope_forward(E(0, 512), E(0, 512), rope, b=1, **kw)
    dq, dk = torch.ones(2, 64, device="cuda").unbind(0)
    T.qk_norm_rope_backward(E(0, 512), E(0, 512), E(0, 512), dq, dk, rope, b=1, **kw)
    assert (dq == 0).all() and (dk == 0).all()
    k, v = (torch.ones(2, 4, 2, 64, dtype=dt, device="cuda") for _ in range(2))
    cache, i32 = T.PagedKVCache(k, v), dict(dtype=torch.int32)
    none = E(0, dtype=torch.int64)
    T.qk_norm_rope_append(E(0, 512), E(0, 4, 64), cache, none, rope, positions=none, **kw)
    T.paged_attn_decode(E(0, 4, 64), cache, E(0, 2, **i32), E(0, **i32), E(0, 4, 64), E(0, 4, dtype=torch.float32), n=0,
                        heads=4, kv_heads=2, d=64)
    T.attn_decode(E(0, h), E(512, h), E(h, h), rope, cache, none, none, E(0, 2, **i32), E(0, **i32), E(0, 512), E(0, h),
                  E(0, h), E(0, h), n=0, h=h, heads=4, kv_heads=2)
    assert (k == 1).all() and (v == 1).all() and T.device_status() == 0
