"""Pins of the token-path oracle (oracle/token_path_fp64.py): finite differences,
closed forms and the attention oracle's own last row."""
import numpy as np
import pytest

import oracle as O


def _angles(rows, rot, seed=0):
    p = np.random.default_rng(seed).integers(0, 50, rows)
    a = p[:, None] * 100.0 ** (-2.0 * np.arange(rot // 2) / max(rot, 1))
    return np.cos(a), np.sin(a)


def test_embedding_rows_order_and_mask():
    E = np.arange(12.0).reshape(4, 3)
    tokens = np.array([[0, 3], [-1, 4], [3, 1]])  # [s, b]: row m = t·b + bi
    assert O.embed_forward(E, tokens, 2.0).tolist() == [[0, 2, 4], [18, 20, 22], [0, 0, 0], [0, 0, 0], [18, 20, 22], [6, 8, 10]]
    dX = np.arange(18.0).reshape(6, 3)
    dE = O.embed_backward(dX, tokens, 4, 0.5)
    assert dE.tolist() == [[0, 0.5, 1], [7.5, 8, 8.5], [0, 0, 0], [(3 + 12) / 2, (4 + 13) / 2, (5 + 14) / 2]]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 8])
def test_qk_backward_is_the_derivative(interleaved, norm, rot):
    rng = np.random.default_rng(1)
    heads, kv, d, rows = 4, 2, 8, 3
    W = (heads + 2 * kv) * d
    x, w = rng.normal(size=(rows, W)), rng.normal(size=(rows, W))
    g = [1 + 0.3 * rng.normal(size=d) for _ in range(2)] if norm else [None, None]
    cos, sin = _angles(rows, rot)
    f = lambda x, gq, gk: (O.qk_norm_rope_forward(x, heads, kv, cos, sin, gq, gk, 1e-3, interleaved) * w).sum()  # noqa: E731
    dx, dgq, dgk = O.qk_norm_rope_backward(x, w, heads, kv, cos, sin, *g, 1e-3, interleaved)
    h = 1e-6
    for _ in range(60):
        i, j = rng.integers(rows), rng.integers(W)
        e = np.zeros_like(x)
        e[i, j] = h
        assert abs((f(x + e, *g) - f(x - e, *g)) / (2 * h) - dx[i, j]) < 1e-7
    if norm:
        for j in range(d):
            e = np.zeros(d)
            e[j] = h
            assert abs((f(x, g[0] + e, g[1]) - f(x, g[0] - e, g[1])) / (2 * h) - dgq[j]) < 1e-6
            assert abs((f(x, g[0], g[1] + e) - f(x, g[0], g[1] - e)) / (2 * h) - dgk[j]) < 1e-6


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotated_products_depend_on_the_distance_alone(interleaved):
    rng = np.random.default_rng(2)
    d = 16
    qkv = rng.normal(size=(1, 3 * d))
    freq = 10.0 ** -np.arange(d // 2)

    def at(p):
        a = p * freq[None]
        y = O.qk_norm_rope_forward(qkv, 1, 1, np.cos(a), np.sin(a), interleaved=interleaved)[0]
        assert np.array_equal(y[2 * d :], qkv[0, 2 * d :])  # v passes
        return y[:d], y[d : 2 * d]

    assert np.isclose(at(7)[0] @ at(3)[1], at(104)[0] @ at(100)[1])
    assert not np.isclose(at(7)[0] @ at(3)[1], at(7)[0] @ at(4)[1])


def test_norm_makes_the_mean_square_gamma_squared():
    x = np.random.default_rng(3).normal(size=(5, 3 * 16)) * 7
    g = np.full(16, 1.5)
    z = np.zeros((5, 0))
    y = O.qk_norm_rope_forward(x, 1, 1, z, z, g, 2 * g, 0.0)
    assert np.allclose((y[:, :16] ** 2).mean(1), 2.25) and np.allclose((y[:, 16:32] ** 2).mean(1), 9.0)


def test_one_token_is_the_last_row_of_causal_attention():
    rng = np.random.default_rng(4)
    s, heads, kv, d = 9, 4, 2, 8
    Q, K, V = (rng.normal(size=(s, n * d)) for n in (heads, kv, kv))
    core = O.attention_core_forward(Q, K, V, s, 1, heads, True, kv)
    want_o, want_l = (core["O"], core["lse2"]) if isinstance(core, dict) else core[:2]
    o, lse = O.decode_one_token(Q[-1].reshape(heads, d), K.reshape(s, kv, d), V.reshape(s, kv, d), d**-0.5)
    assert np.allclose(o.reshape(-1), np.asarray(want_o).reshape(s, -1)[-1])
    assert np.allclose(lse, np.asarray(want_l).reshape(heads, -1)[:, s - 1])
    o, lse = O.decode_one_token(Q[-1].reshape(heads, d), np.zeros((0, kv, d)), np.zeros((0, kv, d)), 1.0)
    assert not o.any() and np.all(lse == -np.inf)
