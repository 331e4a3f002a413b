"""Calls at the edges of what the token path's documentation allows: streams that
run side by side without workspaces of the caller's, norms without eps, weights written just before, rows
beside and in place of each other."""
import pytest
import torch

import test_gpu_qk_rope as qk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("as_int", [False, True])
def test_calls_without_workspaces_on_two_running_streams(cuda_lib, as_int):
    """Calls on the current stream and on another, none waiting for the other: the results of each by itself."""
    T, d, n, heads, kv, keys, page = cuda_lib, 128, 2, 16, 4, 30000, 16
    g = torch.Generator(device="cuda").manual_seed(8)
    normal = lambda *shape, dtype=torch.bfloat16: torch.randn(*shape, generator=g, device="cuda").to(dtype)  # noqa: E731
    pages = n * (keys // page)
    table = torch.arange(pages, device="cuda").int().view(n, -1)
    lens = torch.tensor([keys, keys - 777], dtype=torch.int32, device="cuda")
    s, h, vocab = 3000, 512, 91
    tok = torch.randint(0, vocab, (s, 1), generator=g, device="cuda")
    akw, ekw = dict(n=n, heads=heads, kv_heads=kv, d=d), dict(s=s, b=1, h=h, vocab=vocab, tp=1)
    sides = []
    for _ in range(2):
        cache = T.PagedKVCache(normal(pages, page, kv, d), normal(pages, page, kv, d))
        sides.append((normal(n, heads, d), cache, normal(s, 1, h), normal(n, heads, d),
                      torch.empty(vocab, h, dtype=torch.bfloat16, device="cuda")))

    def run(side, stream=None, **own):
        q, cache, dx, o, grad = side
        T.paged_attn_decode(q, cache, table, lens, o, stream=stream, workspace=own.get("attn"), **akw)
        T.embed_backward(tok, dx, grad, stream=stream, workspace=own.get("embed"), **ekw)

    size = {"attn": T.paged_attn_workspace_size(n, heads, kv, d), "embed": T.embed_backward_workspace(s, 1, h, vocab)}
    want = []
    for side in sides:
        run(side, **{k: torch.empty(v, dtype=torch.uint8, device="cuda") for k, v in size.items()})
        torch.cuda.synchronize()
        want.append([t.clone() for t in side[3:]])
    st = torch.cuda.Stream()
    for _ in range(20):
        for side in sides:
            for t in side[3:]:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        run(sides[0])
        run(sides[1], st.cuda_stream if as_int else st)
        torch.cuda.synchronize()
        assert all(torch.equal(t, w) for side, ws in zip(sides, want) for t, w in zip(side[3:], ws))


NO_EPS = [
    # rows, b, heads, kv, d, rot, interleaved, norm, dtype, positions: heads that leave places of an item empty
    (5, 1, 4, 1, 128, 128, False, True, torch.bfloat16, False),
    (9, 1, 64, 64, 96, 96, False, True, torch.bfloat16, False),
    (40, 2, 6, 2, 64, 32, True, True, torch.float16, True),
    (3, 1, 3, 3, 80, 80, False, True, torch.float32, False),
    (7, 1, 2, 1, 256, 0, False, True, torch.bfloat16, False),
    (12, 1, 16, 16, 64, 64, False, True, torch.bfloat16, False),  # and none
]


@pytest.mark.parametrize("case", NO_EPS, ids=lambda c: f"{c[2]}x{c[3]}x{c[4]}")
def test_norms_without_eps(cuda_lib, monkeypatch, case):
    monkeypatch.setattr(qk, "EPS", 0.0)
    qk.test_forward(cuda_lib, case)
    qk.test_backward(cuda_lib, case)


def test_weights_and_tables_written_by_the_call_before(cuda_lib):
    """γ, cos and sin are rows of a table that a lookup writes just before: a chain without a wait equals the chain
    with a wait after every call."""
    T, d, rows, n = cuda_lib, 128, 600, 40
    g = torch.Generator().manual_seed(3)
    gammas = torch.rand(n, d, generator=g).to(torch.bfloat16).cuda()
    tables = torch.rand(n, 8 * d // 2, generator=g).cuda()
    x = torch.randn(rows, 6 * d, generator=g).to(torch.bfloat16).cuda()
    dy = torch.randn(rows, 6 * d, generator=g).to(torch.bfloat16).cuda()
    tok = torch.randint(0, n, (16, 4, 1), generator=g).cuda()
    pos = torch.randint(0, 8, (rows,), generator=g).cuda()
    ws = torch.empty(T.qk_norm_rope_backward_workspace(rows, 4, 1, d), dtype=torch.uint8, device="cuda")

    def chain(wait):
        gq, gk = torch.zeros(2, d, dtype=torch.bfloat16, device="cuda").unbind(0)
        cos, sin = torch.zeros(2, 8, d // 2, device="cuda").unbind(0)
        rope = T.QKRope(q_gamma=gq, k_gamma=gk, cos=cos, sin=sin)
        kw = dict(rows=rows, b=1, heads=4, kv_heads=1, d=d, positions=pos)
        outs = []
        for i in range(16):
            y, dx, dg = torch.empty_like(x), torch.empty_like(x), torch.empty(2, d, device="cuda")
            steps = [lambda j=j, t=t, src=src: T.embed_forward(tok[i, j : j + 1], src, t.view(1, 1, -1), s=1, b=1,
                                                               h=t.numel(), vocab=n, tp=1)
                     for j, (t, src) in enumerate(((gq, gammas), (gk, gammas), (cos, tables), (sin, tables)))]
            steps += [lambda: T.qk_norm_rope_forward(x, y, rope, **kw),
                      lambda: T.qk_norm_rope_backward(x, dy, dx, dg[0], dg[1], rope, workspace=ws, **kw)]
            # the last writer of γ, and of the tables, directly before the reader in turn
            for step in steps[:4][i % 4 :] + steps[:4][: i % 4] + steps[4:]:
                step()
                if wait:
                    torch.cuda.synchronize()
            outs += [y, dx, dg]
        torch.cuda.synchronize()
        return outs

    assert all(torch.equal(a, b) for a, b in zip(chain(False), chain(True)))


def test_rows_beside_each_other_and_in_place(cuda_lib):
    """Queries in the gaps between qkv's rows, at the same and at another stride; a gradient in its input's place."""
    T, rows, heads, kv, d = cuda_lib, 37, 4, 2, 64
    W, kw = (heads + 2 * kv) * d, dict(rows=rows, heads=heads, kv_heads=kv, d=d)
    g = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(rows, W, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    a, gamma = torch.rand(rows, d // 2, generator=g).cuda(), (1 + torch.rand(d, generator=g)).to(torch.bfloat16).cuda()
    rope = T.QKRope(q_gamma=gamma, k_gamma=gamma, cos=a.cos(), sin=a.sin())
    at = torch.arange(rows, device="cuda")
    cache = lambda: T.PagedKVCache(*(torch.zeros(5, 8, kv, d, dtype=x.dtype, device="cuda") for _ in range(2)))  # noqa: E731
    want, kept = torch.empty(rows, heads * d, dtype=x.dtype, device="cuda"), cache()
    T.qk_norm_rope_append(x, want, kept, at, rope, positions=at, **kw)
    for first, stride in ((W, 2 * W), (2 * W - heads * d, 2 * W), (W, 4 * W)):
        buf = torch.full((rows * 4 * W + 2 * W,), 3.5, dtype=x.dtype, device="cuda")
        qkv = buf.as_strided((rows, W), (2 * W, 1)).copy_(x)
        q, c = buf.as_strided((rows, heads * d), (stride, 1), first), cache()
        T.qk_norm_rope_append(qkv, q, c, at, rope, positions=at, **kw)
        assert torch.equal(q, want) and torch.equal(c.k, kept.k) and torch.equal(c.v, kept.v) and torch.equal(qkv, x)
    dx, dg, dg2 = torch.empty_like(x), torch.empty(2, d, device="cuda"), torch.empty(2, d, device="cuda")
    T.qk_norm_rope_backward(x, dy, dx, dg[0], dg[1], rope, b=1, **kw)
    T.qk_norm_rope_backward(x, dy, x, dg2[0], dg2[1], rope, b=1, **kw)
    assert torch.equal(x, dx) and torch.equal(dg, dg2)
