"""Calls at the edges of what the token path's documentation allows: streams that
run side by side without workspaces of the caller's, norms without eps."""
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
