"""Checkpoints at the ends of their range: values that round up past the storage type's largest are restored as that,
also where the norms' backward and the block's read them; infinities are NaN, which has to show in the gradients."""
import numpy as np
import pytest
import test_gpu_checkpoint as C
import test_gpu_norm_residual as N
import torch

import oracle as O

pytestmark = pytest.mark.gpu
F32 = 2.0**-24
B16, H16, F = torch.bfloat16, torch.float16, torch.float32


def _restored(held, dt):
    """The checkpoint's values, those past dt's largest as that."""
    top = torch.finfo(dt).max
    return np.clip(O.checkpoint_decode(held.codes.cpu().numpy(), held.scales.cpu().numpy()), -top, top)


@pytest.mark.parametrize("h", [264, 1001, 700, 5002, 6144, 8203, 12288])
@pytest.mark.parametrize("dt,post", [(H16, True), (H16, False), (B16, False), (F, False)], ids=str)
def test_norms_from_a_checkpoint_at_the_end_of_the_range(cuda_lib, h, dt, post):
    """Row 1 holds the type's largest values of both signs, row 3 too, without a gradient: it adds zero to the gate's.
    Bounds as in test_gpu_norm_residual (pre is on with a norm behind the block: dr has an error then)."""
    c = N.Case(cuda_lib, (5, 1, h, 1, dt, post, post, "column", 0.5, True), 11)
    top, a = torch.finfo(dt).max, np.abs
    for m in (1, 3):
        c.Z[m, 3::7], c.Z[m, 5::11] = top, -top
    c.dX[1] *= 2.0**-12
    c.dY[1] *= 2.0**-12
    c.dX[3], c.dY[3] = 0.0, 0.0
    (rz, rx), got = N._backward(c, cuda_lib)
    Z = _restored(c.held, dt)
    assert a(Z).max() == top
    f = lambda t: None if t is None else t.double().numpy()[:, None]  # noqa: E731
    rz, rx = f(rz), f(rx)
    R, dX, dY = (t.double().numpy() for t in (c.R, c.dX, c.dY))
    ref = O.rms_residual_backward(dX, dY if post else None, R, Z, **c.o, scale=c.scalar, rz=rz, rx=rx)
    half, n, rows = torch.finfo(dt).eps / 2, (h + 16) * F32, (c.M + 16) * F32
    e_dr = 0.0 * dX
    if post:
        xh, t = R * rx, dY * c.o["pre"]
        e_dr = 4 * F32 * a(dX) + n * rx * (a(t) + a(xh) * a(t * xh).mean(1, keepdims=True))
    cg = a(c.scalar * c.o["gate"] * (c.o["post"] if post else 1.0))
    zh, dr = a(Z * rz) if post else a(Z), a(ref["dr"])
    t = cg * dr
    e_dz = e_t = cg * e_dr + 4 * F32 * t
    if post:
        e_dz = rz * (e_t + zh * (e_t * zh).mean(1, keepdims=True) + n * (t + zh * (t * zh).mean(1, keepdims=True)))
    assert np.all(a(c.join(got["dz"]) - ref["dz"]) <= half * a(ref["dz"]) + e_dz + N._tiny(dt))
    w = c.scalar * zh * (a(c.o["post"]) if post else 1.0)
    have = got["dgate"].double().cpu().numpy()
    assert np.all(a(have - ref["dgate"]) <= rows * (w * dr).sum(0) + (1 + rows) * (w * (e_dr + 4 * F32 * dr)).sum(0))


def _block(T, act, dt, M, seed=0):
    """A block whose token 3 has a value of its own in column 0, which no other token has, and whose W1 takes it to
    column 5 (and 9, negated) of U only."""
    c = C.Block(T, (M, 1, 64, 96, 1, False, act, "fused", dt), seed)
    c.X[:, :, 0], c.W1[:, 0] = 0.0, 0.0
    c.X[3] = 0.0
    return c


def _set(c, x, w):
    c.X[3, 0, 0], c.W1[5, 0], c.W1[9, 0] = x, w, -w
    c.x, c.w1 = c.cut(c.X), c.W1.cuda()


ENDS = [(H16, 1000.0, 64.0), (B16, 254 / 128 * 2.0**64, 2.0**63), (F, 254 / 128 * 2.0**64, 2.0**63)]


@pytest.mark.parametrize("M", [40, 300])
@pytest.mark.parametrize("act", ["identity", "relu", "gelu", "swiglu"])
@pytest.mark.parametrize("dt,x,w", ENDS, ids=["f16", "bf16", "f32"])
def test_block_with_values_at_the_end_of_the_range(cuda_lib, M, act, dt, x, w):
    """U[3, 5] = x·w lies in the type's range and rounds up past it: Y and the gradients are of the type's largest."""
    if dt is not H16 and act in ("gelu", "swiglu"):
        pytest.skip("u² has left float32 long before")
    c = _block(cuda_lib, act, dt, M)
    if act == "swiglu":
        c.W1[c.f + 5, 0], c.W1[c.f + 9, 0] = 2.0**-12, 2.0**-12
        c.W1[c.f + 20, 0], c.W1[20, 0] = 64.0, 2.0**-12  # an up half at the end
    _set(c, x, w)
    c.dZ[3] *= 2.0**-12
    c.dz = c.cut(c.dZ)
    fw = c.blk.forward(c.x, c.w1, c.w2)
    g1, g2 = torch.zeros(c.n1, c.h, device="cuda"), torch.zeros(c.h, c.f, device="cuda")
    bw = c.blk.backward_main_grad(c.x, c.w1, c.w2, fw, c.dz, g1, g2)
    torch.cuda.synchronize()
    X, W1, W2, dZ = c.f64()
    top, a = torch.finfo(dt).max, np.abs
    raw = c.u_values(fw["u"])
    assert a(X @ W1.T).max() <= top < a(raw).max()
    U = np.clip(raw, -top, top)
    Y, dU, e_y, e_du = C._bounds(c, X, W1, W2, dZ, U)
    for name, got, ref, err, terms, n, r in (
        ("dx", c.joined(bw["dx"]), dU @ W1, e_du @ a(W1), a(dU) @ a(W1), c.n1, torch.finfo(dt).eps / 2),
        ("dw1", g1.double().cpu().numpy(), dU.T @ X, e_du.T @ a(X), a(dU).T @ a(X), M, F32),
        ("dw2", g2.double().cpu().numpy(), dZ.T @ Y, a(dZ).T @ e_y, a(dZ).T @ a(Y), M, F32),
    ):
        assert np.isfinite(got).all(), name
        bound = err + n * F32 * (terms + err) + r * (a(ref) + err) + (2.0**-25 if dt is H16 else 0.0)
        assert np.all(a(got - ref) <= bound), name


@pytest.mark.parametrize("M", [40, 300])
@pytest.mark.parametrize("act", ["relu", "identity", "gelu", "swiglu"])
@pytest.mark.parametrize("dt", [B16, F], ids=["bf16", "f32"])
def test_block_shows_infinite_values_of_u(cuda_lib, M, act, dt):
    """U[3, 5] = +inf and U[3, 9] = −inf, NaN in the checkpoint: the gradients of W1's and W2's columns 5 and 9 and of
    token 3 are NaN, all others finite.  (An identity's derivative is 1 whatever U is: W2's columns only.)"""
    c = _block(cuda_lib, act, dt, M, 1)
    _set(c, 2.0**100, 2.0**100)
    fw = c.blk.forward(c.x, c.w1, c.w2)
    bw = c.blk.backward(c.x, c.w1, c.w2, fw, c.dz)
    torch.cuda.synchronize()
    nan = np.isnan(c.u_values(fw["u"]))
    assert nan[3, 5] and nan[3, 9] and nan.sum() == 2
    cols = torch.zeros(c.f, dtype=torch.bool)
    cols[[5, 9]] = True
    rows = torch.cat([cols, cols]) if act == "swiglu" else cols
    token = torch.zeros(M, dtype=torch.bool)
    token[3] = True
    for got, where in ((bw["dw2"].cpu().T, cols), (bw["dw1"].cpu(), rows), (bw["dx"].cpu().view(M, -1), token)):
        assert torch.isnan(got[where]).all() and torch.isfinite(got[~where]).all()
        if act == "identity":
            assert torch.isfinite(bw["dw1"]).all() and torch.isfinite(bw["dx"]).all()
            break
