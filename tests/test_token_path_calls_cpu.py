"""How the binding of the token path makes its calls: temporary workspaces, streams,
the tensors that its handles keep, and further refusals (no GPU needed)."""
import contextlib
import ctypes
import os
import re

import pytest
import torch


@pytest.fixture(scope="module")
def T():
    from sp_partitioned_transformer_gb300 import build

    build.build()
    import sp_partitioned_transformer_gb300 as tpmlp

    tpmlp.load()
    return tpmlp


@pytest.mark.parametrize("stream,on", [(None, None), ("side", "side"), (77, ("external", 77, "cpu"))])
def test_a_temporary_workspace_is_allocated_on_the_stream_that_uses_it(T, monkeypatch, stream, on):
    """A block of another stream's pool may still be in use there when the call starts."""
    current, seen, empty = [None], [], torch.empty

    @contextlib.contextmanager
    def use(s):
        current.append(s)
        yield
        current.pop()

    def allocate(*shape, **kw):
        seen.append(current[-1])
        return empty(*shape, **kw)

    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle, device))
    monkeypatch.setattr(torch, "empty", allocate)
    ws = T._temporary(1000, "cpu", stream)
    assert seen == [on] and ws.numel() == 1000 and ws.dtype is torch.uint8
    assert T._temporary(0, "cpu", stream).numel() == 256


class _Library:
    """Stands in for the loaded library: records the calls that the binding lets through."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def on_host(T, monkeypatch):
    """The binding with host tensors for device tensors, and no library behind it."""
    lib = _Library()
    monkeypatch.setattr(T, "_lib", lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(T, "_stream", lambda stream, device=None: 0)
    return lib


class _Elsewhere(torch.Tensor):
    def get_device(self):
        return 3


def _block_tensors(T, norm=True, s=4, b=2, heads=4, kv=2, d=128, tp=2, sp=True, dt=torch.bfloat16):
    h, n = heads * d, tp if sp else 1
    W = h + 2 * kv * d
    z = lambda *shape, dtype=dt: torch.zeros(*shape, dtype=dtype)  # noqa: E731
    chunks = lambda: [z(s // n, b, h) for _ in range(n)]  # noqa: E731
    rope = T.QKRope(**(dict(q_gamma=z(d), k_gamma=z(d)) if norm else {}), cos=torch.zeros(s, d // 2),
                    sin=torch.zeros(s, d // 2))
    t = dict(x=chunks(), wqkv=z(W, h), wo=z(h, h), rope=rope, qkv_raw=z(s * b, W), qkv=z(s * b, W), o=z(s * b, h),
             lse=z(b, heads, 128, dtype=torch.float32))
    fwd = dict(t, z=chunks())
    bwd = dict(t, dz=chunks(), dx=chunks(), dwqkv=z(W, h), dwo=z(h, h), dq_gamma=z(d, dtype=torch.float32),
               dk_gamma=z(d, dtype=torch.float32), dqkv=z(s * b, W), dout=z(s * b, h),
               workspace=z(256, dtype=torch.uint8))
    kw = dict(s=s, b=b, h=h, heads=heads, kv_heads=kv, tp=tp, sp=sp, causal=True)
    return fwd, bwd, kw


def test_rope_block_takes_what_it_documents(T, on_host):
    for norm in (True, False):
        for sp in (True, False):
            fwd, bwd, kw = _block_tensors(T, norm, sp=sp)
            T.attn_rope_forward(**fwd, **kw)
            T.attn_rope_backward(**bwd, **kw)
            if not norm:  # neither read nor written then
                T.attn_rope_backward(**{**bwd, "qkv_raw": None, "dq_gamma": None, "dk_gamma": None}, **kw)
    fwd, bwd, kw = _block_tensors(T, sp=False, tp=1)
    T.attn_rope_forward(**{**fwd, "x": fwd["x"][0], "z": fwd["z"][0]}, **kw, dtype="bf16")
    name, args = on_host.calls[-1]
    assert name == "tpmlp_attn_rope_forward" and len(args) == 21
    assert len(on_host.calls) == 4 * 2 + 2 + 1


@pytest.mark.parametrize("norm", [True, False])
def test_rope_block_checks_its_tensors(T, on_host, norm):
    fwd, bwd, kw = _block_tensors(T, norm)
    for call, args in ((T.attn_rope_forward, fwd), (T.attn_rope_backward, bwd)):
        for name, good in args.items():
            if name in ("rope", "workspace") or (not norm and call is T.attn_rope_backward
                                                 and name in ("qkv_raw", "dq_gamma", "dk_gamma")):
                continue
            if isinstance(good, list):
                change = lambda f, good=good: [good[0], f(good[1])]  # noqa: E731
                bad = [good[:1], good + good]
            else:
                change, bad = lambda f, good=good: f(good), []
            bad += [change(lambda t: t[:-1]), change(lambda t: t.half()), change(lambda t: t.as_subclass(_Elsewhere)),
                    change(lambda t: torch.stack((t, t), -1)[..., 0])]  # short, another type, off the device, strided
            for b in bad:
                with pytest.raises(ValueError):
                    call(**{**args, name: b}, **kw)
    for name in ("dq_gamma", "dk_gamma") if norm else ():  # as empty_like(gamma) makes them: half the bytes
        with pytest.raises(ValueError, match=name):
            T.attn_rope_backward(**{**bwd, name: torch.zeros(128, dtype=torch.bfloat16)}, **kw)
    with pytest.raises(ValueError, match="not f16"):
        T.attn_rope_forward(**fwd, **kw, dtype="f16")
    with pytest.raises(ValueError, match="current device"):
        T.attn_rope_backward(**{**bwd, "workspace": bwd["workspace"].as_subclass(_Elsewhere)}, **kw)
    assert not on_host.calls


def test_dependent_launches_read_coherently(T):
    """A kernel that may start beside its predecessor must not read through the non-coherent path."""
    from sp_partitioned_transformer_gb300 import build

    found = []
    for name in build.SOURCES:
        with open(os.path.join(build.CSRC, name), encoding="utf-8") as f:
            code = re.sub(r"//.*|/\*(?s:.*?)\*/", "", f.read())
        if "pdl_wait()" in code:
            found.append(name)
            assert not re.search(r"__ldg\b|ldg_nc|\.nc\.|__restrict__", code), name
    assert found == ["decode.cu", "embed.cu", "qk_rope.cu"]


INVALID = -1
A = 0x100000  # never dereferenced


def test_overlapping_rows_are_refused(T):
    """Ten rows of 512 elements of 2 bytes (queries: 256), overlapping in part."""
    lib, rope = T.load(), T._QKRope(A, A, A, A, 100, 1e-6, 64, 0)
    cache = T._KVCache(2 * A, 2 * A, 4, 16, 16 * 128, 128, 64)
    shape = (10, 4, 2, 64, 2)

    def append(q, ld=512, ldq=256):
        return lib.tpmlp_qk_norm_rope_append(A, ld, q, ldq, ctypes.byref(cache), 3 * A, ctypes.byref(rope), 3 * A, 0, *shape,
                                             None)

    def forward(out, ld=512, ldo=512):
        return lib.tpmlp_qk_norm_rope_forward(A, ld, out, ldo, ctypes.byref(rope), None, 0, 10, 1, *shape[1:], None)

    def backward(x, dy, dx, ld=512, ldx=512):
        return lib.tpmlp_qk_norm_rope_backward(x, ld, dy, 512, dx, ldx, A, A, ctypes.byref(rope), None, 0, 10, 1, *shape[1:],
                                               3 * A, 1 << 40, None)

    row = 1024
    for q in (A, A + 16, A + 9 * row + row - 16, A - 10 * 512 + 16):  # inside, the last bytes, from before
        assert append(q) == INVALID and "qkv and q must not overlap" in T.last_error(), q
    for q, ld, ldq in ((A + row - 16, 1024, 1024), (A + 2 * row - 512 + 16, 1024, 1024),  # rows in the gaps, 16 bytes too far
                       (A - 512 + 16, 1024, 1024), (A + row, 1024, 264),  # another stride: into the next row
                       (A + 2 * row * 9 - 264 * 2 * 9, 1024, 264)):
        assert append(q, ld, ldq) == INVALID and "overlap" in T.last_error(), (q, ld, ldq)
    for out, ld, ldo in ((A + 16, 512, 512), (A - 16, 512, 512), (A + 9 * row + 1008, 512, 512), (A + row, 1024, 520)):
        assert forward(out, ld, ldo) == INVALID and "qkv and out" in T.last_error(), (out, ld, ldo)
    assert backward(4 * A, A, A + 16) == INVALID and "dout and dqkv" in T.last_error()
    assert backward(A, 4 * A, A + 16) == INVALID and "qkv and dqkv" in T.last_error()
    assert backward(A, 4 * A, A, 512, 520) == INVALID and "qkv and dqkv" in T.last_error()


def test_rope_block_refuses_overlaps_before_its_first_step(T):
    lib, rope = T.load(), T._QKRope(A, A, A, A, 256, 1e-6, 64, 0)
    one, far = (ctypes.c_void_p * 1)(A), 1 << 40
    size = 256 * (512 + 2 * 2 * 128) * 2
    for raw in (far - size + 16, far + size - 16):
        assert lib.tpmlp_attn_rope_forward(256, 1, 512, 4, 2, 2, 0, 2, 1, one, A, A, ctypes.byref(rope), raw, far, A, A, one,
                                           None, 0, None) == INVALID and "qkv_raw and qkv" in T.last_error()
    for raw in (far - size + 16, far, far + size - 16):
        assert lib.tpmlp_attn_rope_backward(256, 1, 512, 4, 2, 2, 0, 2, 1, one, A, A, ctypes.byref(rope), raw, A, A, A, one,
                                            one, A, A, A, A, far, A, A, 1 << 50, None) == INVALID
        assert "qkv_raw and dqkv" in T.last_error()


@pytest.mark.parametrize("private", [True, False])
def test_current_stream_with_and_without_the_private_call(T, monkeypatch, private):
    class Stream:
        def __init__(self, device):
            self.cuda_stream = 40 + device

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 40 + device, raising=False)
    if not private:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    assert T._stream(None) == 41 and T._stream(None, 2) == 42
    assert T._stream(7) == 7 and T._stream(Stream(3)) == 43


def test_handles_keep_the_memory_that_they_pass_on(T):
    """A parameter that is given other memory later frees its old one."""
    given = [torch.nn.Parameter(torch.full((16,), float(i))) for i in range(2)]
    given += [torch.nn.Parameter(torch.full((4, 8), float(i)), requires_grad=False) for i in (2, 3)]
    rope = T.QKRope(q_gamma=given[0], k_gamma=given[1], cos=given[2], sin=given[3])
    kv = [torch.nn.Parameter(torch.full((2, 4, 1, 64), float(i))) for i in (4, 5)]
    cache = T.PagedKVCache(*kv)
    with torch.no_grad():
        given[0][3] = -1.0  # in place: seen
    for t in given + kv:
        t.data = torch.zeros_like(t)
    held = [(rope.c.q_gamma, rope.q_gamma), (rope.c.k_gamma, rope.k_gamma), (rope.c.cos, rope.cos), (rope.c.sin, rope.sin),
            (cache.c.k, cache.k), (cache.c.v, cache.v)]
    for i, (address, t) in enumerate(held):
        assert t.data_ptr() == address and (t.reshape(-1)[-1] == i)
    assert rope.q_gamma[3] == -1.0


def test_expanded_workspaces_are_refused(T, on_host):
    """One byte that pretends to be many."""
    z, bf = torch.zeros, torch.bfloat16
    ws = z(1, dtype=torch.uint8).expand(1 << 40)
    one, i32 = z(1, dtype=torch.int64), z(1, dtype=torch.int32)
    cache = T.PagedKVCache(z(2, 4, 1, 64, dtype=bf), z(2, 4, 1, 64, dtype=bf))
    rope = T.QKRope(q_gamma=z(64, dtype=bf), k_gamma=z(64, dtype=bf))
    heads, ekw = dict(heads=1, kv_heads=1), dict(s=1, b=1, h=8, vocab=4, tp=1)
    q, row, g = z(1, 64, dtype=bf), z(1, 192, dtype=bf), z(64)
    _, bwd, kw = _block_tensors(T)
    fwd = {k: bwd[k] for k in ("x", "wqkv", "wo", "rope", "qkv_raw", "qkv", "o", "lse")}
    for call in (lambda ws: T.embed_backward(one.view(1, 1), z(1, 1, 8), z(4, 8), workspace=ws, **ekw),
                 lambda ws: T.embed_backward_main_grad(one.view(1, 1), z(1, 1, 8), z(4, 8), workspace=ws, **ekw),
                 lambda ws: T.qk_norm_rope_backward(row, row, row, g, g, rope, rows=1, b=1, d=64, workspace=ws, **heads),
                 lambda ws: T.paged_attn_decode(q, cache, i32.view(1, 1), i32, q, n=1, d=64, workspace=ws, **heads),
                 lambda ws: T.attn_decode(q, row.expand(64, 192).reshape(192, 64), q.expand(64, 64).contiguous(), rope, cache,
                                          one, one, i32.view(1, 1), i32, row, q, q, q, n=1, h=64, workspace=ws, **heads),
                 lambda ws: T.attn_rope_forward(**fwd, z=bwd["dz"], workspace=ws, **kw),
                 lambda ws: T.attn_rope_backward(**{**bwd, "workspace": ws}, **kw)):
        call(z(1 << 20, dtype=torch.uint8))
        n = len(on_host.calls)
        with pytest.raises(ValueError, match="contiguous"):
            call(ws)
        assert len(on_host.calls) == n
