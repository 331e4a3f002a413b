"""fp64 CPU oracle of the token path around the attention block: embedding lookup
and its gradient, norms of queries and keys with the position rotation, and the
attention of one new token over cached keys and values.

TEST INFRASTRUCTURE ONLY — never imported by the product path.

* Embedding: ``x[m] = scale·E[tok_m]``; a token outside the table gives zeros (the
  mask of the vocab-parallel embedding, "Tensor Parallelism（TP）与 Sequence
  Parallelism（SP）", §5 table).  Rows are sequence-first, m = t·b + bi.
* Per head: ``x̂ = x/√(mean x² + eps)``, ``n = x̂·γ``, and the rotation of the first
  ``2·cos.shape[1]`` columns by the row's angles, pairs (i, i + rot/2) or (2i, 2i+1).
* One token: ``softmax(q·Kᵀ·scale)·V`` per head over its group's keys, and the base-2
  log-sum-exp of the scaled scores; no keys give zeros and −∞.
"""
from __future__ import annotations

import math

import numpy as np

from .attn_fp64 import qkv_row_labels

__all__ = ["embed_forward", "embed_backward", "qk_norm_rope_forward", "qk_norm_rope_backward", "decode_one_token"]


def embed_forward(E, tokens, scale=1.0):
    """E [V, h], tokens [s, b] -> [s·b, h]."""
    t = np.asarray(tokens).reshape(-1)
    ok = (t >= 0) & (t < E.shape[0])
    return np.where(ok[:, None], scale * E[np.where(ok, t, 0)], 0.0)


def embed_backward(dX, tokens, vocab, scale=1.0):
    """dX [s·b, h], tokens [s, b] -> dE [V, h]."""
    dE = np.zeros((vocab, dX.shape[1]))
    for m, v in enumerate(np.asarray(tokens).reshape(-1)):
        if 0 <= v < vocab:
            dE[v] += scale * dX[m]
    return dE


def _pairs(d, rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def _turn(x, cos, sin, interleaved):
    """x [rows, d] by angles [rows, rot/2]."""
    a, b = _pairs(x.shape[1], 2 * cos.shape[1], interleaved)
    y = x.copy()
    y[:, a] = x[:, a] * cos - x[:, b] * sin
    y[:, b] = x[:, b] * cos + x[:, a] * sin
    return y


def _head_columns(heads, kv_heads, d):
    """(kind, first column) of every head of the fused projection, in memory order."""
    return [(lab[0], i * d) for i, lab in enumerate(qkv_row_labels(heads, kv_heads))]


def qk_norm_rope_forward(QKV, heads, kv_heads, cos, sin, gq=None, gk=None, eps=0.0, interleaved=False):
    """QKV [rows, W]; cos, sin [rows, rot/2] already taken at each row's position."""
    out = QKV.copy()
    d = QKV.shape[1] // (heads + 2 * kv_heads)
    for kind, c in _head_columns(heads, kv_heads, d):
        if kind == "v":
            continue
        x = QKV[:, c : c + d]
        if gq is not None:
            x = x / np.sqrt((x * x).mean(1, keepdims=True) + eps) * (gq if kind == "q" else gk)
        out[:, c : c + d] = _turn(x, cos, sin, interleaved)
    return out


def qk_norm_rope_backward(QKV, dOut, heads, kv_heads, cos, sin, gq=None, gk=None, eps=0.0, interleaved=False):
    """(dQKV, dγ_q, dγ_k); the γ gradients are None without norms."""
    dQKV = dOut.copy()
    d = QKV.shape[1] // (heads + 2 * kv_heads)
    dg = {"q": np.zeros(d), "k": np.zeros(d)}
    for kind, c in _head_columns(heads, kv_heads, d):
        if kind == "v":
            continue
        dn = _turn(dOut[:, c : c + d], cos, -sin, interleaved)
        if gq is not None:
            x = QKV[:, c : c + d]
            r = 1.0 / np.sqrt((x * x).mean(1, keepdims=True) + eps)
            n = x * r
            dg[kind] += (dn * n).sum(0)
            t = dn * (gq if kind == "q" else gk)
            dn = r * (t - n * (t * n).mean(1, keepdims=True))
        dQKV[:, c : c + d] = dn
    return (dQKV, dg["q"], dg["k"]) if gq is not None else (dQKV, None, None)


def decode_one_token(q, K, V, scale):
    """q [heads, d], K and V [keys, kv_heads, d] -> (o [heads, d], lse2 [heads])."""
    heads = q.shape[0]
    r = heads // K.shape[1]
    o, lse = np.zeros(q.shape), np.full(heads, -math.inf)
    if K.shape[0] == 0:
        return o, lse
    for j in range(heads):
        x = K[:, j // r] @ q[j] * scale
        top = x.max()
        p = np.exp(x - top)
        o[j] = p @ V[:, j // r] / p.sum()
        lse[j] = (top + math.log(p.sum())) / math.log(2.0)
    return o, lse
