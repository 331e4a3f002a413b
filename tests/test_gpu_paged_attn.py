"""Attention of one new token over the paged cache on the GPU against the fp64
oracle.  Per element, with A = Σ p·|v| and δ = (d + 4)·2^-24·scale·max_u Σ|q·k_u|
the error of a float32 score: the probabilities are rounded to the storage type
(eps/2 each), so |o − ref| ≤ eps/2·|ref| + A·(eps/2 + 2δ + (n + 16)·2^-23), and
|lse − ref| ≤ (δ + (n + 16)·2^-23)·log2 e + 2^-23·|ref|."""
import math

import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu


def _half(dt):
    return torch.finfo(dt).eps / 2


class Batch:
    def __init__(self, lengths, heads, kv, d, page, dt, seed=0, layout="page-token-head", poison=True, std=1.0, pad=0):
        g = torch.Generator().manual_seed(seed)
        self.heads, self.kv, self.d, self.page, self.dt, self.n = heads, kv, d, page, dt, len(lengths)
        self.lengths = torch.tensor(lengths, dtype=torch.int32)
        used = [-(-max(0, x) // page) for x in lengths]
        width = max(1, max(used)) + 1
        pages = sum(used) + 2
        order = torch.randperm(pages, generator=g).int()
        self.table = torch.full((self.n, width + pad), -9, dtype=torch.int32)[:, :width]
        self.k, self.v = (std * torch.randn(pages, page, kv, d, generator=g).to(dt) for _ in range(2))
        at = 0
        seen = torch.zeros(pages, page, dtype=torch.bool)
        for i, (x, u) in enumerate(zip(lengths, used)):
            self.table[i, :u] = order[at : at + u]
            at += u
            for j in range(u):
                seen[self.table[i, j], : min(page, x - j * page)] = True
        if poison:  # what nobody may look at
            bad = torch.tensor([float("nan"), float("inf"), float("-inf")]).to(dt)
            self.k[~seen] = bad[torch.randint(0, 3, self.k[~seen].shape, generator=g)]
            self.v[~seen] = bad[torch.randint(0, 3, self.v[~seen].shape, generator=g)]
        self.q = torch.randn(self.n, heads, d, generator=g).to(dt)
        self.layout = layout

    def keys(self, t, i):
        u = -(-max(0, int(self.lengths[i])) // self.page)
        return t[self.table[i, :u].long()].reshape(-1, self.kv, self.d)[: max(0, int(self.lengths[i]))].double().numpy()

    def cache(self, T):
        place = lambda t: (t.transpose(1, 2).contiguous().cuda().transpose(1, 2)  # noqa: E731
                           if self.layout == "page-head-token" else t.cuda())
        return T.PagedKVCache(place(self.k), place(self.v))

    def run(self, T, scale=None, ws=None, lse=True):
        o = torch.full((self.n, self.heads, self.d), float("nan"), dtype=self.dt, device="cuda")
        l = torch.full((self.n, self.heads), float("nan"), device="cuda") if lse else None
        table = self.table
        dev = torch.empty_strided(table.shape, table.stride(), dtype=torch.int32, device="cuda").copy_(table)
        T.paged_attn_decode(self.q.cuda(), self.cache(T), dev, self.lengths.cuda(), o, l, n=self.n, heads=self.heads,
                            kv_heads=self.kv, d=self.d, scale=scale, workspace=ws)
        return o, l

    def check(self, o, lse, scale=None):
        scale = self.d**-0.5 if scale is None else scale
        r = self.heads // self.kv
        for i in range(self.n):
            K, V, q = self.keys(self.k, i), self.keys(self.v, i), self.q[i].double().numpy()
            ref, rl = O.decode_one_token(q, K, V, scale)
            got, gl = o[i].double().cpu().numpy(), lse[i].double().cpu().numpy()
            if K.shape[0] == 0:
                assert not got.any() and np.all(gl == -np.inf)
                continue
            A, _ = O.decode_one_token(q, K, np.abs(V), scale)
            for j in range(self.heads):
                delta = (self.d + 4) * 2.0**-24 * abs(scale) * (np.abs(K[:, j // r]) @ np.abs(q[j])).max()
                run = (K.shape[0] + 16) * 2.0**-23
                tiny = 2.0**-24 if self.dt == torch.float16 else 0.0
                tol = _half(self.dt) * np.abs(ref[j]) + A[j] * (_half(self.dt) + 2 * delta + run) + tiny
                assert np.all(np.abs(got[j] - ref[j]) <= tol), (i, j, np.abs(got[j] - ref[j]).max())
                assert abs(gl[j] - rl[j]) <= (delta + run) * math.log2(math.e) + 2.0**-23 * abs(rl[j])


CASES = [
    # lengths, heads, kv heads, d, page, dtype, layout
    ([1], 1, 1, 128, 16, torch.bfloat16, "page-token-head"),
    ([0], 8, 2, 64, 16, torch.float16, "page-token-head"),
    ([5, 0, 64, 65, 127, 128, 129, 1], 8, 1, 128, 16, torch.bfloat16, "page-token-head"),
    ([300, 17, 0, 1], 4, 4, 96, 7, torch.float16, "page-head-token"),  # pages that end inside a tile
    ([63, 1000, 2], 6, 2, 64, 1, torch.bfloat16, "page-token-head"),  # one key a page
    ([2000, 3, 511], 32, 8, 128, 64, torch.bfloat16, "page-head-token"),
    ([777], 16, 1, 128, 256, torch.float16, "page-token-head"),  # 16 heads a group
    ([130, 90], 40, 2, 96, 16, torch.bfloat16, "page-token-head"),  # 20 heads a group: two blocks
    ([257, 16, 0, 33], 9, 1, 64, 3, torch.float16, "page-token-head"),
    ([70, 1], 71, 1, 128, 16, torch.bfloat16, "page-head-token"),
    ([20000], 8, 1, 128, 32, torch.bfloat16, "page-token-head"),  # one unit over every CTA
    ([9000, 1, 1, 7000], 12, 4, 96, 16, torch.float16, "page-head-token"),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{len(c[0])}x{max(c[0])}-{c[1]}x{c[2]}x{c[3]}-p{c[4]}-{str(c[5])[6:]}" for c in CASES])
def test_against_the_oracle(cuda_lib, case):
    lengths, heads, kv, d, page, dt, layout = case
    x = Batch(lengths, heads, kv, d, page, dt, layout=layout, pad=3)
    o, lse = x.run(cuda_lib)
    assert cuda_lib.device_status() == 0, cuda_lib.last_error()
    x.check(o, lse)


def test_many_sequences(cuda_lib):
    """More sequences than one launch takes, most of them short, some empty."""
    g = torch.Generator().manual_seed(1)
    lengths = torch.randint(0, 40, (2100,), generator=g).tolist()
    x = Batch(lengths, 2, 1, 64, 16, torch.bfloat16)
    x.check(*x.run(cuda_lib))


@pytest.mark.parametrize("std", [0.0, 30.0])
def test_flat_and_peaked_scores(cuda_lib, std):
    """Equal scores, and ones so far apart that one key takes all; also a negative scale."""
    x = Batch([1025, 200], 8, 1, 128, 16, torch.bfloat16, std=std)
    x.check(*x.run(cuda_lib))
    x.check(*x.run(cuda_lib, scale=-0.3), scale=-0.3)


def test_rising_maximum(cuda_lib):
    """The running maximum is raised by every tile: old sums are rescaled each time."""
    x = Batch([3000], 8, 1, 64, 16, torch.float16)
    ramp = torch.linspace(0, 6, 3000 + 8)[:3008]
    pages = x.table[0, :188].long()
    x.k[pages] = (x.q[0, 0][None] * ramp[:, None]).view(188, 16, 1, 64).to(torch.float16)
    x.check(*x.run(cuda_lib))


def test_nan_among_the_keys_reaches_the_output(cuda_lib):
    x = Batch([40, 40], 2, 1, 64, 16, torch.bfloat16)
    x.k[x.table[0, 1].long(), 3] = float("nan")
    o, lse = x.run(cuda_lib)
    assert torch.isnan(o[0]).all() and torch.isnan(lse[0]).all() and torch.isfinite(o[1]).all()


def test_bad_pages_and_lengths_are_left_out_and_reported(cuda_lib):
    x = Batch([50, 30], 4, 2, 64, 16, torch.bfloat16)
    cuda_lib.device_status(reset=True)
    for bad in (-1, x.k.shape[0], 2**31 - 1):
        y = Batch([50, 30], 4, 2, 64, 16, torch.bfloat16)
        good = y.table[0, 1].item()
        y.table[0, 1] = bad
        o, lse = y.run(cuda_lib)
        assert cuda_lib.device_status(reset=True) == -1
        y.table[0, 1] = good  # the same without keys 16 … 31
        y.k[good] = 0
        keys = lambda t: np.delete(y.keys(t, 0), slice(16, 32), 0)  # noqa: E731
        ref, rl = O.decode_one_token(y.q[0].double().numpy(), keys(y.k), keys(y.v), 64**-0.5)
        assert np.allclose(o[0].double().cpu().numpy(), ref, atol=2e-2) and np.allclose(lse[0].cpu().numpy(), rl, atol=1e-4)
        want, _ = x.run(cuda_lib)
        assert torch.equal(o[1], want[1])
    y = Batch([64, 30], 4, 2, 64, 16, torch.bfloat16)
    y.table = y.table[:, :4].contiguous()
    want = y.run(cuda_lib)
    assert cuda_lib.device_status() == 0
    y.lengths[0] = 2**31 - 1  # beyond the row: as many keys as the row has
    got = y.run(cuda_lib)
    assert cuda_lib.device_status(reset=True) == -1
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    y.lengths[0] = -5
    assert not y.run(cuda_lib)[0][0].any() and cuda_lib.device_status() == 0


def test_same_bits_on_every_call_and_any_workspace(cuda_lib):
    x = Batch([5000, 1, 333, 0, 2600], 16, 2, 128, 16, torch.bfloat16)
    n = cuda_lib.paged_attn_workspace_size(5, 16, 2, 128)
    runs = [x.run(cuda_lib, ws=torch.full((n,), f, dtype=torch.uint8, device="cuda")) for f in (0, 0xFF, 0x5A)]
    assert all(torch.equal(r[0], runs[0][0]) and torch.equal(r[1], runs[0][1]) for r in runs)
    assert torch.equal(x.run(cuda_lib, lse=False)[0], runs[0][0])


def test_offsets_beyond_32_bits(cuda_lib):
    """A cache of more than 2^32 elements: pages at both of its ends."""
    page, kv, d, dt = 64, 8, 128, torch.bfloat16
    pages = (1 << 32) // (page * kv * d) + 3
    k, v = (torch.zeros(pages, page, kv, d, dtype=dt, device="cuda") for _ in range(2))
    small = Batch([100, 70], 16, kv, d, page, dt, poison=False)
    ends = torch.tensor([[0, pages - 1], [pages - 2, 1]], dtype=torch.int32)
    for i in range(2):
        for j in range(2):
            k[ends[i, j].long()] = small.k[small.table[i, j].long()].cuda()
            v[ends[i, j].long()] = small.v[small.table[i, j].long()].cuda()
    o, lse = torch.empty(2, 16, d, dtype=dt, device="cuda"), torch.empty(2, 16, device="cuda")
    cuda_lib.paged_attn_decode(small.q.cuda(), cuda_lib.PagedKVCache(k, v), ends.cuda(), small.lengths.cuda(), o, lse,
                               n=2, heads=16, kv_heads=kv, d=d)
    small.check(o, lse)
    x = torch.randn(2, 32 * d, generator=torch.Generator().manual_seed(0)).to(dt)
    slots = torch.tensor([pages * page - 1, 5])
    q = torch.empty(2, 16, d, dtype=dt, device="cuda")
    one = cuda_lib.QKRope(cos=torch.ones(1, 64, device="cuda"), sin=torch.zeros(1, 64, device="cuda"))
    cuda_lib.qk_norm_rope_append(x.cuda(), q, cuda_lib.PagedKVCache(k, v), slots.cuda(), one, rows=2, heads=16,
                                 kv_heads=kv, d=d, positions=torch.zeros(2, dtype=torch.int64, device="cuda"))
    parts = x.view(2, kv, 4, d)
    assert torch.equal(k[-1, -1].cpu(), parts[0, :, 2]) and torch.equal(v[0, 5].cpu(), parts[1, :, 3])


def test_captured_replayed_and_two_streams(cuda_lib):
    """A captured call sees new lengths; two calls side by side have two workspaces."""
    T = cuda_lib
    x, y = (Batch([900, 40, 3000], 8, 2, 128, 16, torch.bfloat16, seed=s, poison=False) for s in (1, 2))
    want = [b.run(T) for b in (x, y)]
    n = T.paged_attn_workspace_size(3, 8, 2, 128)
    calls = []
    for b in (x, y):
        o, lse = torch.zeros(3, 8, 128, dtype=b.dt, device="cuda"), torch.zeros(3, 8, device="cuda")
        c, lens, ws = b.cache(T), b.lengths.cuda(), torch.empty(n, dtype=torch.uint8, device="cuda")
        args = (b.q.cuda(), c, b.table.contiguous().cuda(), lens, o, lse)
        calls.append((args, dict(n=3, heads=8, kv_heads=2, d=128, workspace=ws)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(20):
        for st, (args, kw) in zip(streams, calls):
            T.paged_attn_decode(*args, stream=st, **kw)
    torch.cuda.synchronize()
    for (args, _), w in zip(calls, want):
        assert torch.equal(args[4], w[0]) and torch.equal(args[5], w[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        T.paged_attn_decode(*calls[0][0], **calls[0][1])
    calls[0][0][3].copy_(torch.tensor([17, 0, 2999]))
    graph.replay()
    x.lengths = torch.tensor([17, 0, 2999], dtype=torch.int32)
    x.check(calls[0][0][4], calls[0][0][5])
