"""The decode block on the GPU over the calls that its documentation allows: every
head width, batches around the GEMM's row tile, padded sequences, captured with
copies and on forked streams; and queries and outputs inside wider rows.

Blocks: every tensor within 2e-2 of the fp64 oracle (‖·‖∞ over ‖·‖∞), the
framework's bound.

The attention by itself, with A = Σ p·|v|, δ the error of a float32 score (d + 4
roundings of Σ|q·k|·scale) and n keys: a probability enters the second product as
a value of the storage type within three half steps of it and the rounding of what
that leaves, so it is off by 3·(eps/2)² of itself (fp16: or half a step of the
subnormals, 2^-25, where the largest probability is 2^15), and
|o − ref| ≤ eps/2·|ref| + A·(3·(eps/2)² + 2δ + (n + 16)·2^-23) + fp16's 2^-25 + 2^-39·Σ|v|."""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_common import rel_err, to_np
from test_gpu_paged_attn import Batch

pytestmark = pytest.mark.gpu
TOL = 2e-2


class Block:
    """n sequences in a paged cache, each about to take one more token; sequences `padded` have none."""

    def __init__(self, T, n, heads, kv, d, dt, page=16, longest=70, padded=(), seed=0):
        g = torch.Generator().manual_seed(seed)
        self.T, self.n, self.heads, self.kv, self.d, self.dt, self.h = T, n, heads, kv, d, dt, heads * d
        self.W = (heads + 2 * kv) * d
        self.x = torch.randn(n, self.h, generator=g).to(dt)
        self.wqkv = torch.randn(self.W, self.h, generator=g).mul(self.h**-0.5).to(dt)
        self.wo = torch.randn(self.h, self.h, generator=g).mul(self.h**-0.5).to(dt)
        self.gq, self.gk = ((1 + 0.2 * torch.randn(d, generator=g)).to(dt) for _ in range(2))
        a = torch.rand(longest + 1, d // 2, generator=g)
        self.cos, self.sin = a.cos(), a.sin()
        self.old = torch.randint(0, longest, (n,), generator=g)  # keys in the cache before this token
        width = longest // page + 1
        self.table = torch.randperm(n * width, generator=g).int().view(n, width)
        self.k, self.v = (torch.randn(n * width, page, kv, d, generator=g).to(dt) for _ in range(2))
        self.slots = self.table[torch.arange(n), self.old // page].long() * page + self.old % page
        self.lengths = (self.old + 1).int()
        self.padded = list(padded)
        self.slots[self.padded], self.lengths[self.padded] = -1, 0
        self.page = page

    def device(self):
        c = lambda t: t.cuda()  # noqa: E731
        T, E = self.T, lambda w: torch.full((self.n, w), float("nan"), dtype=self.dt, device="cuda")  # noqa: E731
        rope = T.QKRope(q_gamma=c(self.gq), k_gamma=c(self.gk), eps=1e-6, cos=c(self.cos), sin=c(self.sin))
        self.cache = T.PagedKVCache(c(self.k), c(self.v))
        self.out = [E(self.W), E(self.h), E(self.h), E(self.h)]
        self.args = (c(self.x), c(self.wqkv), c(self.wo), rope, self.cache, c(self.old), c(self.slots), c(self.table),
                     c(self.lengths), *self.out)
        self.kw = dict(n=self.n, h=self.h, heads=self.heads, kv_heads=self.kv)
        return self

    def check(self):
        f = lambda t: t.double().numpy()  # noqa: E731
        qkv = O.qk_norm_rope_forward(f(self.x) @ f(self.wqkv).T, self.heads, self.kv, f(self.cos)[self.old.numpy()],
                                     f(self.sin)[self.old.numpy()], f(self.gq), f(self.gk), 1e-6)
        Q, K, V = O.split_qkv(qkv, self.heads, self.kv)
        o = np.zeros((self.n, self.heads, self.d))
        for i in range(self.n):
            if i in self.padded:
                continue
            u = int(self.old[i])
            pages = self.table[i, : u // self.page + 1].long()
            old = [f(t[pages]).reshape(-1, self.kv, self.d)[:u] for t in (self.k, self.v)]
            new = [t[i].reshape(1, self.kv, self.d) for t in (K, V)]
            kk, vv = (np.concatenate(p) for p in zip(old, new))
            o[i] = O.decode_one_token(Q[i].reshape(self.heads, self.d), kk, vv, self.d**-0.5)[0]
        o = o.reshape(self.n, -1)
        assert rel_err(to_np(self.out[2]), o) <= TOL and rel_err(to_np(self.out[3]), o @ f(self.wo).T) <= TOL
        assert self.T.device_status() == 0, self.T.last_error()
        assert not to_np(self.out[3])[self.padded].any()
        # the cache: the new keys and values in their slots, everything else as it was
        for t, was, new in ((self.cache.k, self.k, K), (self.cache.v, self.v, V)):
            t, was = t.cpu().reshape(-1, self.kv, self.d), was.reshape(-1, self.kv, self.d)
            live = self.slots >= 0
            assert rel_err(t[self.slots[live]].double().numpy().reshape(int(live.sum()), -1),
                           new[live.numpy()].reshape(int(live.sum()), -1)) <= TOL
            rest = torch.ones(len(was), dtype=torch.bool)
            rest[self.slots[live]] = False
            assert torch.equal(t[rest], was[rest])


BLOCKS = [
    # n, heads, kv, d, dtype, page
    (1, 1, 1, 64, torch.bfloat16, 16),
    (3, 4, 2, 64, torch.float16, 7),
    (129, 8, 1, 64, torch.bfloat16, 32),
    (64, 12, 4, 96, torch.bfloat16, 16),
    (128, 4, 2, 128, torch.float16, 64),
    (257, 2, 2, 128, torch.bfloat16, 1),
]


@pytest.mark.parametrize("case", BLOCKS, ids=lambda c: f"n{c[0]}-{c[1]}x{c[2]}x{c[3]}-p{c[5]}-{str(c[4])[6:]}")
def test_against_the_oracle(cuda_lib, case):
    n, heads, kv, d, dt, page = case
    b = Block(cuda_lib, n, heads, kv, d, dt, page).device()
    cuda_lib.attn_decode(*b.args, **b.kw)
    b.check()


def test_padded_sequences(cuda_lib):
    """No slot and no keys: rows that fill a batch up; their output is zero and the cache stays."""
    b = Block(cuda_lib, 9, 8, 2, 128, torch.bfloat16, padded=(0, 4, 8)).device()
    cuda_lib.attn_decode(*b.args, **b.kw)
    b.check()


def test_captured_behind_copies_and_beside_another_stream(cuda_lib):
    """One graph: inputs copied and buffers cleared directly before the calls, a second block on a stream forked
    inside the capture, joined again; replayed on new inputs."""
    T = cuda_lib
    blocks = [Block(T, n, 8, 2, 128, torch.bfloat16, seed=i).device() for i, n in enumerate((5, 40))]
    ws = [torch.empty(T.paged_attn_workspace_size(b.n, 8, 2, 128), dtype=torch.uint8, device="cuda") for b in blocks]
    staged = [b.args[0].clone() for b in blocks]
    side = torch.cuda.Stream()

    def step(b, w, src):
        b.args[0].copy_(src)
        T.attn_decode(*b.args, workspace=w, **b.kw)
        b.out[0].zero_()

    for b, w, src in zip(blocks, ws, staged):  # once outside the capture
        step(b, w, src)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        step(blocks[0], ws[0], staged[0])
        with torch.cuda.stream(side):
            T.paged_attn_decode(blocks[1].args[0], blocks[1].cache, *blocks[1].args[7:9], blocks[1].out[2], workspace=ws[1],
                                n=40, heads=8, kv_heads=2, d=128)  # the first node of the forked stream
            step(blocks[1], ws[1], staged[1])
        here.wait_stream(side)
        T.attn_decode(*blocks[0].args, workspace=ws[0], **blocks[0].kw)  # behind two streams' ends
    for seed in (3, 4):
        for b, src in zip(blocks, staged):
            b.x = torch.randn(b.x.shape, generator=torch.Generator().manual_seed(seed)).to(b.dt)
            src.copy_(b.x)
        for b in blocks:
            for o in b.out:
                o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for b in blocks:
            b.check()
        assert not blocks[1].out[0].any()


@pytest.mark.parametrize("d,dt", [(128, torch.bfloat16), (96, torch.float16), (64, torch.bfloat16)])
def test_queries_and_outputs_inside_wider_rows(cuda_lib, d, dt):
    """q in the columns of a fused projection, o in those of another buffer: their neighbours stay as they were."""
    T, heads, kv = cuda_lib, 8, 2
    x = Batch([900, 0, 17, 4000], heads, kv, d, 16, dt, seed=4)
    want, want_lse = x.run(T)
    wide = torch.full((4, (heads + 3) * d), float("nan"), dtype=dt, device="cuda")
    wide[:, d : (heads + 1) * d] = x.q.cuda().view(4, -1)
    out = torch.full((4, (heads + 1) * d + 8), 3.0, dtype=dt, device="cuda")
    lse = torch.full((4, heads), float("nan"), device="cuda")
    T.paged_attn_decode(wide[:, d : (heads + 1) * d], x.cache(T), x.table.contiguous().cuda(), x.lengths.cuda(),
                        out[:, 8 : heads * d + 8], lse, n=4, heads=heads, kv_heads=kv, d=d)
    assert torch.equal(out[:, 8 : heads * d + 8].reshape(4, heads, d), want) and torch.equal(lse, want_lse)
    assert (out[:, :8] == 3.0).all() and (out[:, heads * d + 8 :] == 3.0).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads,kv,d", [(8, 1, 64), (8, 2, 128), (12, 12, 96), (6, 3, 96), (32, 2, 128)])
def test_probabilities_are_not_rounded_to_the_storage_type(cuda_lib, heads, kv, d, dt):
    """Flat and ordinary scores over few keys, where nothing else hides the probabilities' own error."""
    half = torch.finfo(dt).eps / 2
    x = Batch([20, 33, 64, 1, 100, 47], heads, kv, d, 16, dt, seed=6)
    for scale in (0.01, d**-0.5):
        o, _ = x.run(cuda_lib, scale=scale)
        for i in range(x.n):
            K, V, q = x.keys(x.k, i), x.keys(x.v, i), x.q[i].double().numpy()
            ref, A = (O.decode_one_token(q, K, v, scale)[0] for v in (V, np.abs(V)))
            for j in range(heads):
                g = j // (heads // kv)
                delta = (d + 4) * 2.0**-24 * scale * (np.abs(K[:, g]) @ np.abs(q[j])).max()
                tol = half * np.abs(ref[j]) + A[j] * (3 * half**2 + 2 * delta + (len(K) + 16) * 2.0**-23)
                if dt == torch.float16:
                    tol = tol + 2.0**-25 + 2.0**-39 * np.abs(V[:, g]).sum(0)
                assert np.all(np.abs(o[i, j].double().cpu().numpy() - ref[j]) <= tol), (i, j)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads,kv,d", [(8, 1, 64), (12, 12, 96), (32, 2, 128)])
def test_infinite_values_reach_their_column(cuda_lib, heads, kv, d, dt):
    """p·∞ = ∞ for every probability above zero, likely or not; ∞ − ∞ is NaN; other columns and heads know nothing."""
    x = Batch([100, 700, 3000], heads, kv, d, 16, dt, seed=7)
    inf = float("inf")
    for key, column, value in ((0, 0, inf), (57, 9, -inf), (99, 17, inf), (3, 30, inf), (4, 30, -inf), (5, 31, float("nan"))):
        for i in range(3):
            x.v[x.table[i, key // 16].long(), key % 16, 0, column] = value
    o, lse = x.run(cuda_lib)
    r = heads // kv
    for i in range(3):
        for j in range(heads):
            got = o[i, j].double().cpu().numpy()
            want = np.zeros(d)
            if j < r:
                want[[0, 17]], want[9], want[[30, 31]] = inf, -inf, np.nan
            assert np.array_equal(got[~np.isfinite(want)], want[~np.isfinite(want)], equal_nan=True)
            assert np.isfinite(got[np.isfinite(want)]).all()
    assert torch.isfinite(lse).all() and cuda_lib.device_status() == 0
