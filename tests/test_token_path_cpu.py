"""Refusals of the embedding, QK norm + rotation and paged attention entry points:
every case fails on the host before anything is launched (no GPU needed), and the
binding's own checks of tensors."""
import ctypes

import pytest
import torch

INVALID, NOT_DIV, UNSUP, WORKSPACE = -1, -2, -3, -4
A = 0x10000  # never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def T():
    from sp_partitioned_transformer_gb300 import build

    build.build()
    import sp_partitioned_transformer_gb300 as tpmlp

    tpmlp.load()
    return tpmlp


def _vp(*vals):
    return (ctypes.c_void_p * len(vals))(*vals)


def _embed(T, fn="tpmlp_embed_forward", tok=A, tok_type=1, table=A, chunks=None, ws=A, ws_bytes=BIG, s=8, b=2, h=64,
           vocab=10, tp=2, dt=2):
    chunks = _vp(*([A] * tp)) if chunks is None else chunks
    lib = T.load()
    if fn == "tpmlp_embed_forward":
        return lib.tpmlp_embed_forward(tok, tok_type, 1, s, table, 1.0, chunks, s, b, h, vocab, tp, dt, None)
    return getattr(lib, fn)(tok, tok_type, 1, s, chunks, table, 1.0, ws, ws_bytes, s, b, h, vocab, tp, dt, None)


@pytest.mark.parametrize("fn", ["tpmlp_embed_forward", "tpmlp_embed_backward", "tpmlp_embed_backward_main_grad"])
def test_embedding_refusals(T, fn):
    f = lambda **k: _embed(T, fn, **k)  # noqa: E731
    for bad in (dict(s=-1), dict(b=-1), dict(h=0), dict(vocab=0), dict(tp=0, chunks=_vp(A)), dict(dt=3), dict(tok_type=2),
                dict(tok=None), dict(table=None), dict(chunks=_vp(A, None)), dict(tok=A + 4), dict(table=A + 1),
                dict(chunks=_vp(A, A + 1)), dict(tp=65)):
        assert f(**bad) == INVALID, bad
        assert T.last_error()
    assert f(s=7) == NOT_DIV and "First dimension" in T.last_error()
    for big in (dict(s=1 << 31, b=2), dict(vocab=1 << 31), dict(h=1 << 31), dict(s=1 << 33, b=1 << 33)):
        assert f(**big) == UNSUP, big
    if fn != "tpmlp_embed_forward":
        need = T.embed_backward_workspace(8, 2, 64, 10)
        assert f(ws_bytes=need - 1) == WORKSPACE and str(need) in T.last_error()
        assert f(ws=None) == WORKSPACE
        assert f(ws=A + 16) == UNSUP


def test_embedding_workspace(T):
    # two arrays of (token, row), a mark for each row of the table, then for each piece of 8 sorted tokens (64
    # where there are enough; none for a single piece) a counter per 128 columns and two float32 rows
    assert T.embed_backward_workspace(8, 1, 100, 5) == 2 * 256 + 256
    assert T.embed_backward_workspace(16, 1, 128, 500) == 2 * 256 + 512 + 256 + 2 * 2 * 128 * 4
    assert T.embed_backward_workspace(1 << 17, 1, 128, 500) == 2 * 8 * (1 << 17) + 512 + 2048 * (4 + 2 * 128 * 4)
    assert T.embed_backward_workspace(0, 1, 128, 5) == 0 and T.embed_backward_workspace(-1, 1, 128, 5) == 0


def _rope(T, q=A, k=A, eps=1e-6, cos=A, sin=A, max_pos=100, rot=64, inter=0):
    return T._QKRope(q, k, cos, sin, max_pos, eps, rot, inter)


def _cache(T, k=A, v=A, pages=4, page=16, ps=16 * 2 * 64, ts=2 * 64, hs=64):
    return T._KVCache(k, v, pages, page, ps, ts, hs)


def _qk(T, which="forward", x=A, ld=512, out=A + 64, ldo=512, rope=None, pos=None, pos_type=0, rows=10, b=1, heads=4, kv=2,
        d=64, dt=2, cache=None, slots=A, dg=A, ws=A, ws_bytes=BIG):
    lib = T.load()
    rope = _rope(T) if rope is None else rope
    r = None if rope == "none" else ctypes.byref(rope)
    if which == "forward":
        return lib.tpmlp_qk_norm_rope_forward(x, ld, out, ldo, r, pos, pos_type, rows, b, heads, kv, d, dt, None)
    if which == "backward":
        return lib.tpmlp_qk_norm_rope_backward(x, ld, x, ld, out, ldo, dg, dg, r, pos, pos_type, rows, b, heads, kv, d, dt,
                                               ws, ws_bytes, None)
    cache = _cache(T) if cache is None else cache
    c = None if cache == "none" else ctypes.byref(cache)
    return lib.tpmlp_qk_norm_rope_append(x, ld, out, ldo, c, slots, r, A if pos is None else pos, pos_type, rows, heads, kv,
                                         d, dt, None)


@pytest.mark.parametrize("which", ["forward", "backward", "append"])
def test_qk_refusals(T, which):
    f = lambda **k: _qk(T, which, **k)  # noqa: E731
    for bad in (dict(rows=-1), dict(dt=9), dict(heads=0), dict(kv=0), dict(kv=8), dict(x=None), dict(out=None), dict(ld=511),
                dict(rope="none"), dict(rope=_rope(T, k=None)), dict(rope=_rope(T, q=None)), dict(rope=_rope(T, eps=-1.0)),
                dict(rope=_rope(T, eps=float("nan"))), dict(rope=_rope(T, inter=2)), dict(rope=_rope(T, rot=-16)),
                dict(rope=_rope(T, rot=80)), dict(rope=_rope(T, cos=None)), dict(rope=_rope(T, max_pos=0)),
                dict(pos_type=7), dict(pos=A + 2)):
        assert f(**bad) == INVALID, bad
        assert T.last_error()
    assert f(heads=5) == NOT_DIV
    for bad in (dict(d=72), dict(d=272, ld=1 << 20), dict(rope=_rope(T, rot=24)), dict(x=A + 8), dict(out=A + 8),
                dict(ld=516), dict(rope=_rope(T, q=A + 8)), dict(rope=_rope(T, sin=A + 4)), dict(rows=1 << 31)):
        assert f(**bad) == UNSUP, bad
    if which != "append":
        assert f(b=0) == INVALID
        assert f(rope=_rope(T, max_pos=9)) == INVALID and "shorter" in T.last_error()
        assert f(rope=_rope(T, max_pos=4), b=2) == INVALID
        assert f(out=A, ldo=520) == INVALID  # in place with another row stride
    if which == "backward":
        need = T.qk_norm_rope_backward_workspace(10, 4, 2, 64)
        assert need == 1024 * 2 * 64 * 4
        assert f(ws_bytes=need - 1) == WORKSPACE and f(ws=None) == WORKSPACE and f(ws=A + 8) == UNSUP
        assert f(dg=None) == INVALID
    if which == "append":
        for bad in (dict(slots=None), dict(slots=A + 4), dict(cache="none"), dict(cache=_cache(T, k=None)),
                    dict(cache=_cache(T, pages=0)), dict(cache=_cache(T, page=0)), dict(cache=_cache(T, hs=63)),
                    dict(cache=_cache(T, ts=8))):
            assert f(**bad) == INVALID, bad
        for bad in (dict(cache=_cache(T, v=A + 8)), dict(cache=_cache(T, hs=68)), dict(cache=_cache(T, pages=1 << 31))):
            assert f(**bad) == UNSUP, bad


def _decode(T, q=A, ldq=256, cache=None, table=A, ldt=8, width=8, lengths=A, scale=0.1, o=A, ldo=256, lse=None, n=3, heads=4,
            kv=2, d=64, dt=2, ws=A, ws_bytes=BIG):
    c = ctypes.byref(_cache(T) if cache is None else cache)
    return T.load().tpmlp_paged_attn_decode(q, ldq, c, table, ldt, width, lengths, scale, o, ldo, lse, n, heads, kv, d, dt,
                                            ws, ws_bytes, None)


def test_paged_attention_refusals(T):
    f = lambda **k: _decode(T, **k)  # noqa: E731
    for bad in (dict(n=-1), dict(heads=0), dict(kv=0), dict(kv=8), dict(q=None), dict(o=None), dict(table=None),
                dict(lengths=None), dict(lengths=A + 2), dict(ldq=255), dict(ldo=248), dict(width=0), dict(ldt=7),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(lse=A + 2), dict(cache=_cache(T, page=0))):
        assert f(**bad) == INVALID, bad
        assert T.last_error()
    assert f(heads=5) == NOT_DIV
    for bad in (dict(dt=0), dict(d=80), dict(d=256), dict(q=A + 8), dict(o=A + 8), dict(ldq=260), dict(ws=A + 16),
                dict(cache=_cache(T, ts=132)), dict(n=1 << 24)):
        assert f(**bad) == UNSUP, bad
    need = T.paged_attn_workspace_size(3, 4, 2, 64)
    assert need > 0 and T.paged_attn_workspace_size(1000, 4, 2, 64) == need  # the same for every batch
    assert f(ws_bytes=need - 1) == WORKSPACE and f(ws=None) == WORKSPACE
    assert T.paged_attn_workspace_size(3, 4, 3, 64) == 0 and T.paged_attn_workspace_size(3, 4, 2, 48) == 0


def _block(T, n=2, h=256, heads=4, kv=2, dt=2, x=A, rope=None, cache=None, slots=A, table=A, lengths=A, pos=A, z=A,
           ws_bytes=BIG):
    rope, cache = rope or _rope(T), cache or _cache(T)
    return T.load().tpmlp_attn_decode(n, h, heads, kv, dt, x, A, A, ctypes.byref(rope), pos, 1, ctypes.byref(cache), slots,
                                      table, 8, 8, lengths, A, A, A, z, A, ws_bytes, None)


def test_decode_block_refuses_before_its_first_step(T):
    f = lambda **k: _block(T, **k)  # noqa: E731
    for bad in (dict(n=-1), dict(heads=0), dict(x=None), dict(z=None), dict(slots=None), dict(table=None), dict(lengths=None),
                dict(pos=None), dict(rope=_rope(T, k=None)), dict(cache=_cache(T, k=None))):
        assert f(**bad) == INVALID, bad
    assert f(heads=3) == UNSUP and f(h=320) == UNSUP and f(dt=0) == UNSUP and f(x=A + 8) == UNSUP
    assert f(kv=3) == NOT_DIV
    assert f(ws_bytes=100) == WORKSPACE


def test_rope_block_refusals(T):
    lib = T.load()

    def fwd(rope=_rope(T), raw=A, qkv=A + 64, s=256, tables=None, dt=2, d=128):
        r = None if rope is None else ctypes.byref(rope)
        return lib.tpmlp_attn_rope_forward(s, 1, 4 * d, 4, 2, 2, 0, dt, 1, _vp(A), A, A, r, raw, qkv, A, A, _vp(A), None, 0,
                                           None)

    assert fwd(rope=None) == INVALID and fwd(raw=None) == INVALID
    assert fwd(rope=_rope(T, max_pos=255)) == INVALID and "shorter" in T.last_error()
    assert fwd(rope=_rope(T, max_pos=256), raw=A, qkv=A) == INVALID and "qkv_raw" in T.last_error()
    assert fwd(rope=_rope(T, max_pos=256), dt=0) == UNSUP and fwd(rope=_rope(T, max_pos=256, rot=8)) == UNSUP
    assert fwd(rope=_rope(T, max_pos=256, rot=144)) == INVALID

    def bwd(dg=A, raw=A, ws_bytes=BIG, rope=_rope(T, max_pos=256)):
        return lib.tpmlp_attn_rope_backward(256, 1, 512, 4, 2, 2, 0, 2, 1, _vp(A), A, A, ctypes.byref(rope), raw, A, A, A,
                                            _vp(A), _vp(A), A, A, dg, dg, A, A, A, ws_bytes, None)

    plain = T.attn_workspace_size(256, 1, 512, 4, 2, False, "bf16", True, 2)
    need = T.attn_rope_workspace_size(256, 1, 512, 4, 2, False, "bf16", True, 2)
    assert need >= plain + T.qk_norm_rope_backward_workspace(256, 4, 2, 128)
    assert bwd(dg=None) == INVALID and bwd(raw=None) == INVALID and bwd(ws_bytes=need - 1) == WORKSPACE


def test_empty_calls_take_null_arrays(T):
    assert _embed(T, s=0, tok=None, chunks=_vp(None, None)) == 0 and _embed(T, b=0, tok=None, chunks=_vp(None, None)) == 0
    assert _qk(T, rows=0, x=None, out=None) == 0
    assert _qk(T, "append", rows=0, x=None, out=None, slots=None) == 0
    assert _decode(T, n=0, q=None, o=None, table=None, lengths=None) == 0
    assert _block(T, n=0, x=None, z=None, slots=None, table=None, lengths=None, pos=None) == 0
    # what does not depend on the rows is still checked
    assert _embed(T, s=0, table=None) == INVALID and _qk(T, rows=0, rope=_rope(T, k=None)) == INVALID
    assert _decode(T, n=0, cache=_cache(T, k=None)) == INVALID and _decode(T, n=0, ws=None) == WORKSPACE
    assert _block(T, n=0, rope=_rope(T, rot=24)) == UNSUP


def test_binding_checks_tensors(T):
    z = torch.zeros
    kw = dict(s=3, b=4, h=8, vocab=5, tp=1)
    tok = z(3, 4, dtype=torch.int64)
    for bad, what in ((lambda: T.embed_forward(z(4, 3, dtype=torch.int64), z(5, 8), z(3, 4, 8), **kw), "tokens"),
                      (lambda: T.embed_forward(tok, z(6, 8), z(3, 4, 8), **kw), "table"),
                      (lambda: T.embed_forward(tok, z(8, 5).t(), z(3, 4, 8), **kw), "table"),
                      (lambda: T.embed_backward(tok, z(3, 4, 8).half(), z(5, 8), **kw), "gradient"),
                      (lambda: T.embed_backward_main_grad(tok, z(3, 4, 8).half(), z(5, 8).half(), **kw), "gradient")):
        with pytest.raises(ValueError, match=what):
            bad()
    with pytest.raises(TypeError, match="tokens"):
        T.embed_forward(z(3, 4), z(5, 8), z(3, 4, 8), **kw)
    with pytest.raises(ValueError):
        T.QKRope(cos=z(4, 8))
    with pytest.raises(ValueError, match="gamma"):
        T.QKRope(q_gamma=z(8), k_gamma=z(8).half())
    with pytest.raises(TypeError):
        T.QKRope(cos=z(4, 8).half(), sin=z(4, 8).half())
    with pytest.raises(ValueError):
        T.PagedKVCache(z(2, 4, 1, 64), z(2, 4, 1, 32))
    with pytest.raises(ValueError):
        T.PagedKVCache(z(2, 4, 64, 2).transpose(2, 3), z(2, 4, 64, 2).transpose(2, 3))
    rope = T.QKRope(cos=z(4, 32), sin=z(4, 32), q_gamma=z(64), k_gamma=z(64))
    kw = dict(rows=2, b=1, heads=1, kv_heads=1, d=64)
    with pytest.raises(ValueError, match="out"):
        T.qk_norm_rope_forward(z(2, 192), z(2, 192).half(), rope, **kw)
    with pytest.raises(ValueError, match="qkv"):
        T.qk_norm_rope_forward(z(2, 190), z(2, 192), rope, **kw)
    with pytest.raises(ValueError, match="rows of out"):
        T.qk_norm_rope_forward(z(2, 192), z(192, 2).t(), rope, **kw)
    with pytest.raises(TypeError, match="positions"):
        T.qk_norm_rope_forward(z(2, 192), z(2, 192), rope, positions=z(2), **kw)
    with pytest.raises(ValueError, match="dk_gamma"):
        T.qk_norm_rope_backward(z(2, 192), z(2, 192), z(2, 192), z(64), z(64).half(), rope, **kw)
    cache = T.PagedKVCache(z(2, 4, 1, 64).half(), z(2, 4, 1, 64).half())
    q = z(1, 1, 64).half()
    one, table = z(1, dtype=torch.int32), z(1, 2, dtype=torch.int32)
    kw = dict(n=1, heads=1, kv_heads=1, d=64, workspace=z(1))
    with pytest.raises(TypeError, match="block_table"):
        T.paged_attn_decode(q, cache, table.long(), one, q, **kw)
    with pytest.raises(TypeError, match="lengths"):
        T.paged_attn_decode(q, cache, table, one.long(), q, **kw)
    with pytest.raises(ValueError, match="lse"):
        T.paged_attn_decode(q, cache, table, one, q, z(1, 2), **kw)
    with pytest.raises(TypeError, match="slots"):
        T.qk_norm_rope_append(z(1, 192).half(), q, cache, one, rope, rows=1, heads=1, kv_heads=1, d=64, positions=one)
