"""Norms of queries and keys with the rotation, forward, backward and the cache
form, on the GPU against the fp64 oracle.

Float32 inside, one rounding out.  With N = the largest |x̂·γ| (or |x| without
norm) of a head: a sum of d squares is off by at most d/2 + 2 steps of 2^-24
after the square root, each further product or sum by one, so an output is off by
at most eps/2·|ref| + (d/2 + 16)·2^-24·2N.  The backward's subtraction adds the
two terms' sizes, and each is a sum of d products over d."""
import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu
F32 = 2.0**-24


def _half(dt):
    return torch.finfo(dt).eps / 2


CASES = [
    # rows, b, heads, kv, d, rot, interleaved, norm, dtype, positions
    (1, 1, 1, 1, 16, 16, False, True, torch.float32, False),
    (7, 1, 4, 2, 64, 64, False, True, torch.bfloat16, False),
    (7, 3, 4, 2, 64, 32, True, True, torch.float16, False),
    (33, 1, 8, 1, 128, 128, False, True, torch.bfloat16, True),
    (33, 2, 8, 8, 128, 64, False, False, torch.float16, True),
    (10, 1, 5, 5, 96, 96, True, True, torch.bfloat16, False),
    (300, 1, 6, 2, 96, 48, False, True, torch.float32, True),
    (65, 1, 3, 3, 80, 80, False, True, torch.float16, False),
    (40, 2, 2, 1, 256, 256, True, True, torch.bfloat16, True),
    (12, 1, 16, 2, 256, 16, False, True, torch.float32, False),
    (29, 1, 12, 4, 112, 0, False, True, torch.bfloat16, False),  # norm alone
    (700, 1, 32, 8, 128, 128, False, True, torch.bfloat16, True),  # four heads a lane group
    (1000, 4, 20, 4, 64, 64, True, False, torch.float16, False),
]
IDS = [f"m{c[0]}b{c[1]}-{c[2]}x{c[3]}x{c[4]}-rot{c[5]}{'i' if c[6] else ''}{'n' if c[7] else ''}-{str(c[8])[6:]}" for c in CASES]
EPS = 1e-5


class Case:
    def __init__(self, T, c, seed=0):
        self.rows, self.b, self.heads, self.kv, self.d, self.rot, self.inter, self.norm, self.dt, pos = c
        g = torch.Generator().manual_seed(seed)
        self.W = (self.heads + 2 * self.kv) * self.d
        self.x = torch.randn(self.rows, self.W, generator=g).to(self.dt)
        self.dy = torch.randn(self.rows, self.W, generator=g).to(self.dt)
        n = max(1, -(-self.rows // self.b))
        self.pos = torch.randint(0, n, (self.rows,), generator=g) if pos else None
        at = (self.pos if pos else torch.arange(self.rows) // self.b).numpy()
        self.gq, self.gk = (((1 + 0.2 * torch.randn(self.d, generator=g)).to(self.dt) for _ in range(2))
                            if self.norm else (None, None))
        a = torch.arange(n).double()[:, None] * 10000.0 ** (-2.0 * torch.arange(self.rot // 2).double() / max(self.rot, 1))
        cos, sin = a.cos().float(), a.sin().float()
        self.cos, self.sin = cos.double().numpy()[at], sin.double().numpy()[at]
        dev = lambda t: None if t is None else t.cuda()  # noqa: E731
        tables = dict(cos=dev(cos), sin=dev(sin)) if self.rot else {}
        self.rope = T.QKRope(q_gamma=dev(self.gq), k_gamma=dev(self.gk), eps=EPS, interleaved=self.inter, **tables)
        f = lambda t: None if t is None else t.double().numpy()  # noqa: E731
        self.okw = dict(heads=self.heads, kv_heads=self.kv, cos=self.cos, sin=self.sin, gq=f(self.gq), gk=f(self.gk),
                        eps=EPS if self.norm else 0.0, interleaved=self.inter)
        self.kw = dict(heads=self.heads, kv_heads=self.kv, d=self.d)
        self.dpos = None if self.pos is None else self.pos.cuda()

    def ref(self):
        return O.qk_norm_rope_forward(self.x.double().numpy(), **self.okw)

    def size(self):
        """2N per element: the rotation mixes two elements of the head."""
        y = np.abs(O.qk_norm_rope_forward(self.x.double().numpy(), **{**self.okw, "cos": self.cos[:, :0], "sin": self.sin[:, :0]}))
        h = y.reshape(self.rows, -1, self.d).max(-1, keepdims=True)
        return 2 * np.broadcast_to(h, (self.rows, h.shape[1], self.d)).reshape(self.rows, -1)

    def tol(self, ref):
        tiny = 2.0**-25 if self.dt == torch.float16 else 0.0  # half a step of fp16's subnormals
        return _half(self.dt) * np.abs(ref) + (self.d / 2 + 16) * F32 * self.size() + tiny


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(cuda_lib, case):
    c = Case(cuda_lib, case)
    ref = c.ref()
    x = c.x.cuda()
    buf = torch.full((c.rows, c.W + 16), 5.5, dtype=c.dt, device="cuda")  # a row stride of its own
    out = buf[:, : c.W]
    cuda_lib.qk_norm_rope_forward(x, out, c.rope, rows=c.rows, b=c.b, positions=c.dpos, **c.kw)
    got = out.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= c.tol(ref))
    assert (buf[:, c.W :] == 5.5).all()
    v = [i for i, lab in enumerate(O.qkv_row_labels(c.heads, c.kv)) if lab[0] == "v"]
    assert np.array_equal(got.reshape(c.rows, -1, c.d)[:, v], c.x.double().numpy().reshape(c.rows, -1, c.d)[:, v])
    cuda_lib.qk_norm_rope_forward(x, x, c.rope, rows=c.rows, b=c.b, positions=c.dpos, **c.kw)  # in place
    assert torch.equal(x, out)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(cuda_lib, case):
    c = Case(cuda_lib, case, 1)
    x64, dy64 = c.x.double().numpy(), c.dy.double().numpy()
    ref, rq, rk = O.qk_norm_rope_backward(x64, dy64, **c.okw)
    dqkv = torch.empty(c.rows, c.W, dtype=c.dt, device="cuda")
    dg = [torch.full((c.d,), float("nan"), device="cuda") for _ in range(2)] if c.norm else [None, None]
    run = lambda dy, out: cuda_lib.qk_norm_rope_backward(c.x.cuda(), dy, out, *dg, c.rope, rows=c.rows, b=c.b,  # noqa: E731
                                                         positions=c.dpos, **c.kw)
    dy = c.dy.cuda()
    run(dy, dqkv)
    # per head: |t| ≤ 2·max|dy|·max|γ|, times rstd; and x̂ times the mean of |t·x̂|
    dyh = 2 * np.abs(dy64).reshape(c.rows, -1, c.d).max(-1, keepdims=True)
    if c.norm:
        xh = x64.reshape(c.rows, -1, c.d)
        r = 1 / np.sqrt((xh * xh).mean(-1, keepdims=True) + EPS)
        g = max(np.abs(c.okw["gq"]).max(), np.abs(c.okw["gk"]).max())
        size = dyh * g * r * (1 + np.abs(xh * r) * np.abs(xh * r).mean(-1, keepdims=True))
    else:
        size = np.broadcast_to(dyh, (c.rows, dyh.shape[1], c.d))
    tiny = 2.0**-25 if c.dt == torch.float16 else 0.0
    got = dqkv.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= _half(c.dt) * np.abs(ref) + (2 * c.d + 32) * F32 * size.reshape(c.rows, -1) + tiny)
    if c.norm:
        kinds = np.array([lab[0] for lab in O.qkv_row_labels(c.heads, c.kv)])
        for kind, want, have in (("q", rq, dg[0]), ("k", rk, dg[1])):
            terms = np.abs(xh * r) * dyh  # each term of the sum over rows and heads
            s = terms[:, kinds == kind].sum((0, 1))
            n = c.rows * (kinds == kind).sum()
            assert np.all(np.abs(have.double().cpu().numpy() - want) <= (n + c.d / 2 + 16) * F32 * s)
    again = dy.clone()
    keep = None if not c.norm else [t.clone() for t in dg]
    run(again, again)  # in place, and the same bits
    assert torch.equal(again, dqkv)
    assert keep is None or all(torch.equal(a, b) for a, b in zip(keep, dg))


@pytest.mark.parametrize("layout", ["page-token-head", "page-head-token"])
@pytest.mark.parametrize("case", [c for c in CASES if c[8] != torch.float32 or c[4] == 96],
                         ids=[i for i, c in zip(IDS, CASES) if c[8] != torch.float32 or c[4] == 96])
def test_append(cuda_lib, case, layout):
    c = Case(cuda_lib, case, 2)
    page, pages = 5, -(-c.rows // 5) + 2
    shape = (pages, page, c.kv, c.d) if layout == "page-token-head" else (pages, c.kv, page, c.d)
    kv = [torch.full(shape, -3.25, dtype=c.dt, device="cuda") for _ in range(2)]
    k, v = (t if layout == "page-token-head" else t.transpose(1, 2) for t in kv)
    g = torch.Generator().manual_seed(3)
    slots = torch.randperm(pages * page, generator=g)[: c.rows]
    slots[c.rows // 2] = -1  # not cached
    pos = torch.arange(c.rows) // c.b if c.pos is None else c.pos
    q = torch.empty(c.rows, c.heads, c.d, dtype=c.dt, device="cuda")
    cuda_lib.qk_norm_rope_append(c.x.cuda(), q, cuda_lib.PagedKVCache(k, v), slots.cuda(), c.rope, rows=c.rows,
                                 positions=pos.int().cuda(), **c.kw)
    whole = torch.empty(c.rows, c.W, dtype=c.dt, device="cuda")
    cuda_lib.qk_norm_rope_forward(c.x.cuda(), whole, c.rope, rows=c.rows, b=c.b, positions=c.dpos, **c.kw)
    parts = whole.view(c.rows, c.kv, -1, c.d).cpu()  # the training form's bits
    assert torch.equal(q.cpu(), parts[:, :, :-2].reshape(c.rows, c.heads, c.d))
    for t, j in ((k, -2), (v, -1)):
        want = torch.full((pages * page, c.kv, c.d), -3.25, dtype=c.dt)
        want[slots[slots >= 0]] = parts[:, :, j][slots >= 0]
        assert torch.equal(t.cpu().reshape(-1, c.kv, c.d), want)
    assert cuda_lib.device_status() == 0


def test_infinities_stay_in_their_columns(cuda_lib):
    """Columns behind the rotated part meet no sine, and v no norm."""
    d, rot = 64, 32
    x = torch.randn(3, 3 * d, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    x[:, rot + 1], x[:, d + rot + 2], x[:, 2 * d] = float("inf"), float("-inf"), float("nan")
    a = torch.rand(3, rot // 2)
    rope = cuda_lib.QKRope(cos=a.cos().cuda(), sin=a.sin().cuda())
    y = x.cuda()
    cuda_lib.qk_norm_rope_forward(y, y, rope, rows=3, b=1, heads=1, kv_heads=1, d=d)
    y = y.cpu()
    assert torch.equal(torch.isfinite(y), torch.isfinite(x))
    assert torch.equal(y[:, rot:d], x[:, rot:d])


def test_positions_and_slots_out_of_range_are_reported(cuda_lib):
    T, d = cuda_lib, 64
    a = torch.rand(4, d // 2)
    rope = T.QKRope(cos=a.cos().cuda(), sin=a.sin().cuda())
    x = torch.randn(4, 3 * d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    assert T.device_status(reset=True) in (0, -1)
    k, v = (torch.zeros(2, 2, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.empty(4, 1, d, dtype=torch.bfloat16, device="cuda")
    cache = T.PagedKVCache(k, v)
    kw = dict(rows=4, heads=1, kv_heads=1, d=d)
    good = torch.tensor([0, 1, 2, 3]).cuda()
    T.qk_norm_rope_append(x, q, cache, good, rope, positions=torch.tensor([0, 3, -1, 4]).cuda(), **kw)
    assert T.device_status(reset=True) == -1 and "outside" in T.last_error()
    want = torch.empty_like(q)
    T.qk_norm_rope_append(x, want, cache, good, rope, positions=torch.tensor([0, 3, 0, 3]).cuda(), **kw)
    assert T.device_status() == 0 and torch.equal(q, want)
    k.zero_()
    T.qk_norm_rope_append(x, q, cache, torch.tensor([3, 4, 1 << 40, -7]).cuda(), rope, positions=good, **kw)
    assert T.device_status(reset=True) == -1
    assert not k.reshape(4, -1)[:3].any() and k.reshape(4, -1)[3].any()


def test_no_rows_leave_zero_gammas(cuda_lib):
    import ctypes

    d = 32
    g = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    rope = cuda_lib.QKRope(q_gamma=g, k_gamma=g)
    buf = torch.zeros(1, 96, dtype=torch.bfloat16, device="cuda")
    dg = torch.full((2, d), 4.0, device="cuda")
    lib, st = cuda_lib.load(), torch.cuda.current_stream().cuda_stream
    p = buf.data_ptr()
    assert lib.tpmlp_qk_norm_rope_backward(p, 96, p, 96, p, 96, dg[0].data_ptr(), dg[1].data_ptr(), ctypes.byref(rope.c),
                                           None, 0, 0, 1, 1, 1, d, 2, None, 0, st) == 0
    assert not dg.any()
