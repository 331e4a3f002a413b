"""Embedding lookup and its gradient by sorted tokens on the GPU against the fp64
oracle.  The lookup is one float32 product rounded once: equal bits.  The
gradient is a float32 sum rounded once, so per element
|error| ≤ eps/2·|ref| + (n + 2)·2^-24·scale·Σ|dx| over the token's n rows."""
import ctypes

import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu



def _half(dt):
    return torch.finfo(dt).eps / 2


def _tokens(s, b, vocab, how, seed, wide):
    g = torch.Generator().manual_seed(seed)
    if how == "same":
        t = torch.full((s, b), vocab - 1)
    elif how == "few":
        t = torch.randint(0, min(vocab, 3), (s, b), generator=g)
    elif how == "out":
        t = torch.randint(-2, vocab + 2, (s, b), generator=g)
    elif how == "none":
        t = torch.full((s, b), -1)
    else:
        t = torch.randint(0, vocab, (s, b), generator=g)
    return t.to(torch.int64 if wide else torch.int32)


CASES = [
    # s, b, h, vocab, tp, dtype, tokens, int64, scale
    (1, 1, 8, 1, 1, torch.bfloat16, "any", True, 1.0),
    (16, 2, 64, 50, 2, torch.float32, "any", False, 3.0),
    (33, 1, 1024, 7, 1, torch.float16, "few", True, 0.5),
    (31, 3, 13, 100, 1, torch.bfloat16, "out", True, 1.7),  # rows that 16 bytes do not divide
    (100, 1, 36, 1000, 4, torch.float32, "out", False, 1.0),
    (513, 2, 136, 600, 1, torch.bfloat16, "any", False, 11.66),
    (96, 1, 2056, 513, 8, torch.float16, "same", True, 1.0),  # one run over three pieces, a ragged column tile
    (64, 1, 40, 1 << 18, 2, torch.bfloat16, "any", True, 1.0),  # three digits to sort
    (1500, 3, 64, 40, 4, torch.bfloat16, "any", True, 1.0),  # long runs, a cluster sorts
    (2049, 1, 24, 5000, 1, torch.float16, "out", False, 1.0),
    (4096, 1, 16, 9, 8, torch.float32, "same", True, 1.0),
    (40000, 1, 8, 300, 1, torch.bfloat16, "any", True, 1.0),  # several rounds a warp
    (50, 1, 32, 20, 1, torch.bfloat16, "none", True, 1.0),
    (32768, 1, 8, 700, 1, torch.bfloat16, "out", True, 1.0),  # two digits, handed on in shared memory: the most
    (33000, 1, 8, 70000, 1, torch.float16, "any", False, 1.0),  # and more than that
    (1000, 1, 16, 1 << 18, 1, torch.float32, "out", True, 1.0),  # three digits, a cluster sorts
]


def _ids(c):
    return f"s{c[0]}b{c[1]}h{c[2]}v{c[3]}tp{c[4]}-{str(c[5])[6:]}-{c[6]}"


def _inputs(case, seed=0):
    s, b, h, vocab, tp, dt, how, wide, scale = case
    g = torch.Generator().manual_seed(seed)
    tok = _tokens(s, b, vocab, how, seed + 1, wide)
    table = torch.randn(vocab, h, generator=g).to(dt)
    dx = torch.randn(s, b, h, generator=g).to(dt)
    return tok, table, dx


@pytest.mark.parametrize("case", CASES, ids=_ids)
def test_forward_is_the_rounded_product(cuda_lib, case):
    s, b, h, vocab, tp, dt, how, wide, scale = case
    tok, table, _ = _inputs(case)
    # a [b, s] batch read in place, between sentinels
    dev_tok = tok.t().contiguous().cuda().t()
    out = [torch.full((s // tp, b, h), float("nan"), dtype=dt, device="cuda") for _ in range(tp)]
    cuda_lib.embed_forward(dev_tok, table.cuda(), out, s=s, b=b, h=h, vocab=vocab, tp=tp, scale=scale)
    ok = (tok >= 0) & (tok < vocab)
    want = table[tok.long().clamp(0, vocab - 1)].float() * torch.tensor(scale, dtype=torch.float32)
    want = torch.where(ok[..., None], want, torch.zeros(())).to(dt)
    assert torch.equal(torch.cat(out).cpu(), want)


@pytest.mark.parametrize("main_grad", [False, True], ids=["table", "main_grad"])
@pytest.mark.parametrize("case", CASES, ids=_ids)
def test_gradient_against_the_oracle(cuda_lib, case, main_grad):
    s, b, h, vocab, tp, dt, how, wide, scale = case
    tok, _, dx = _inputs(case, 5)
    flat = dx.double().reshape(s * b, h).numpy()
    ref = O.embed_backward(flat, tok.numpy(), vocab, scale)
    size = O.embed_backward(np.abs(flat), tok.numpy(), vocab, abs(scale))
    count = O.embed_backward(np.ones((s * b, 1)), tok.numpy(), vocab)
    chunks = [c.contiguous().cuda() for c in dx.chunk(tp)]
    kw = dict(s=s, b=b, h=h, vocab=vocab, tp=tp, scale=scale)
    guard = 64
    if main_grad:
        base = torch.randn(vocab, h, generator=torch.Generator().manual_seed(9))
        ref = base.double().numpy() + ref
        buf = torch.full((vocab * h + guard,), 7.5, device="cuda")
        got = buf[: vocab * h].view(vocab, h).copy_(base)
        cuda_lib.embed_backward_main_grad(tok.cuda(), chunks, got, **kw)
        half, size = _half(torch.float32), size + np.abs(base.numpy())
    else:
        buf = torch.full((vocab * h + guard,), 7.5, device="cuda", dtype=dt)
        got = buf[: vocab * h].view(vocab, h)
        cuda_lib.embed_backward(tok.cuda(), chunks, got, **kw)
        half = _half(dt)
    out = got.double().cpu().numpy()
    assert np.all(np.abs(out - ref) <= half * np.abs(ref) + (count + 2) * 2.0**-24 * size + 2.0**-25 * (dt == torch.float16))
    assert (buf[vocab * h :] == 7.5).all()  # what lies behind the table stays
    if main_grad:
        untouched = torch.from_numpy(count[:, 0] == 0)
        assert torch.equal(got.cpu()[untouched], base[untouched])


def test_gradient_is_the_same_bits_on_every_call_and_any_workspace(cuda_lib):
    case = (3000, 1, 512, 77, 4, torch.bfloat16, "any", True, 1.0)
    s, b, h, vocab, tp, dt = case[:6]
    tok, _, dx = _inputs(case)
    chunks = [c.contiguous().cuda() for c in dx.chunk(tp)]
    tok = tok.cuda()
    n = cuda_lib.embed_backward_workspace(s, b, h, vocab)
    got = []
    for fill in (0, 0xFF, 0x5A):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        g = torch.zeros(vocab, h, device="cuda")
        cuda_lib.embed_backward_main_grad(tok, chunks, g, s=s, b=b, h=h, vocab=vocab, tp=tp, workspace=ws)
        got.append(g)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_gradient_matches_differences_of_the_forward(cuda_lib):
    """Σ w·(x(E + t·D) − x(E)) is linear in t: equal to t·⟨dE, D⟩ in exact integers."""
    s, b, h, vocab, tp = 24, 2, 48, 10, 2
    g = torch.Generator().manual_seed(3)
    tok = torch.randint(0, vocab, (s, b), generator=g).cuda()
    E, D = (torch.randint(-4, 5, (vocab, h), generator=g).float().cuda() for _ in range(2))
    w = torch.randint(-4, 5, (s, b, h), generator=g).float().cuda()
    wc = [c.contiguous() for c in w.chunk(tp)]
    x = [[torch.empty(s // tp, b, h, device="cuda") for _ in range(tp)] for _ in range(2)]
    kw = dict(s=s, b=b, h=h, vocab=vocab, tp=tp, scale=2.0)
    cuda_lib.embed_forward(tok, E, x[0], **kw)
    cuda_lib.embed_forward(tok, E + D, x[1], **kw)
    dE = torch.empty(vocab, h, device="cuda")
    cuda_lib.embed_backward(tok, wc, dE, **kw)
    assert ((torch.cat(x[1]) - torch.cat(x[0])) * w).sum().item() == (dE * D).sum().item()


def test_element_aligned_views_and_streams(cuda_lib):
    """Tables and chunks at addresses that 16 bytes do not divide, on a stream of their own."""
    s, b, h, vocab = 20, 1, 64, 30
    g = torch.Generator().manual_seed(4)
    tok = torch.randint(0, vocab, (s, b), generator=g).cuda()
    table = torch.randn(vocab * h + 1, generator=g).to(torch.bfloat16).cuda()[1:].view(vocab, h)
    out = torch.empty(s * b * h + 1, dtype=torch.bfloat16, device="cuda")[1:].view(s, b, h)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        cuda_lib.embed_forward(tok, table, out, s=s, b=b, h=h, vocab=vocab, tp=1)
        dE = torch.empty(vocab, h, dtype=torch.bfloat16, device="cuda")
        cuda_lib.embed_backward(tok, out, dE, s=s, b=b, h=h, vocab=vocab, tp=1)
    st.synchronize()
    assert torch.equal(out, table[tok])
    want = torch.zeros(vocab, h, dtype=torch.float64, device="cuda").index_add_(0, tok.view(-1), out.double().view(-1, h))
    assert ((dE.double() - want).abs() <= want.abs() * _half(torch.bfloat16) + 2.0**-20 * want.abs().max()).all()


def test_no_tokens(cuda_lib):
    """No rows: an empty sum for the whole table, nothing added to main_grad (through the C ABI: empty
    torch tensors have no address)."""
    keep = torch.zeros(1, dtype=torch.int64, device="cuda")
    dx, g = torch.empty(16, device="cuda"), torch.full((5, 16), 3.0, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    arr = (ctypes.c_void_p * 1)(dx.data_ptr())
    lib, st = cuda_lib.load(), torch.cuda.current_stream().cuda_stream
    args = (keep.data_ptr(), 1, 1, 1, arr, g.data_ptr(), 1.0, ws.data_ptr(), 256, 0, 1, 16, 5, 1, 0, st)
    assert lib.tpmlp_embed_backward_main_grad(*args) == 0
    assert (g == 3.0).all()
    assert lib.tpmlp_embed_backward(*args) == 0
    assert (g == 0.0).all()


def test_captured_and_replayed(cuda_lib):
    s, b, h, vocab = 2500, 1, 128, 90
    g = torch.Generator().manual_seed(6)
    tok = torch.randint(0, vocab, (s, b), generator=g).cuda()
    dx = torch.randn(s, b, h, generator=g).cuda()
    grad = torch.zeros(vocab, h, device="cuda")
    kw = dict(s=s, b=b, h=h, vocab=vocab, tp=1)
    ws = torch.empty(cuda_lib.embed_backward_workspace(s, b, h, vocab), dtype=torch.uint8, device="cuda")
    cuda_lib.embed_backward(tok, dx, grad, workspace=ws, **kw)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        cuda_lib.embed_backward(tok, dx, grad, workspace=ws, **kw)
    for seed in (7, 8):
        tok.copy_(torch.randint(0, vocab, (s, b), generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        want = torch.empty_like(grad)
        cuda_lib.embed_backward(tok, dx, want, **kw)
        assert torch.equal(grad, want)
