"""Outputs of the layer's calls that meet another of the call's arrays are refused (no GPU: a call that were let through
would meet addresses that are nobody's, so these stay off where there is one)."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="its addresses are not memory")
INVALID, AT = -1, 0x100000


@pytest.fixture(scope="module")
def lib():
    from sp_partitioned_transformer_gb300 import build

    build.build()
    import sp_partitioned_transformer_gb300 as tpmlp

    return tpmlp.load()


# s 8, b 2, h 64, tp 2 in bf16: two chunks of 1024 bytes, 16 rows of 64 columns, a gate for each of two batch entries
NAMES = ("r", "z", "x", "y", "dx", "dy", "dr", "dz", "codes", "scales", "rz", "rx", "post", "pre", "gate", "dpost", "dpre",
         "dgate", "ws")
SIZE = dict(codes=16 * 64, scales=16 * 2, rz=64, rx=64, post=128, pre=128, gate=256, dpost=256, dpre=256, dgate=512)
CHUNKS = NAMES[:8]
FORWARD = ("x", "y", "codes", "scales", "rz", "rx"), ("r", "z", "post", "pre", "gate")
BACKWARD = ("dr", "dz", "dpost", "dpre", "dgate", "ws"), ("dx", "dy", "x", "codes", "scales", "rz", "rx", "post", "pre", "gate")


def _size(lib, name):
    if name in CHUNKS:
        return 1024
    return SIZE[name] if name in SIZE else lib.tpmlp_sp_rms_residual_backward_workspace(8, 2, 64, 2)


def _call(lib, forward, place):
    import sp_partitioned_transformer_gb300 as T

    at = {n: AT * (1 + i) for i, n in enumerate(NAMES)}
    second = {n: at[n] + AT // 2 for n in CHUNKS}
    at.update(place)
    v = {n: (ctypes.c_void_p * 2)(at[n], second[n]) if n in CHUNKS else at[n] for n in NAMES}
    norms = ctypes.byref(T._RMSResidual(v["post"], v["pre"], v["gate"], 2, 1.0, 1e-6))
    if forward:
        return lib.tpmlp_sp_rms_residual_forward(v["r"], v["z"], norms, v["x"], v["y"], v["codes"], v["scales"], v["rz"], v["rx"],
                                                 8, 2, 64, 2, 2, None)
    return lib.tpmlp_sp_rms_residual_backward(v["dx"], v["dy"], v["x"], None, v["codes"], v["scales"], norms, v["rz"], v["rx"],
                                              v["dr"], v["dz"], v["dpost"], v["dpre"], v["dgate"], v["ws"], 1 << 30, 8, 2, 64,
                                              2, 2, None)


@pytest.mark.parametrize("forward", [True, False], ids=["forward", "backward"])
def test_norms_refuse_outputs_that_meet_any_array(lib, forward):
    outputs, inputs = FORWARD if forward else BACKWARD
    base = {n: AT * (1 + i) for i, n in enumerate(NAMES)}
    for out in outputs:
        for other in outputs + inputs:
            if other == out or (out, other) in (("x", "r"), ("dr", "dx")):
                continue
            for moved, still in ((out, other), (other, out)):
                # on its first bytes, from before it, and on its last ones (what each name's alignment allows)
                step = 256 if moved == "ws" else 4
                for at in (base[still], base[still] - _size(lib, moved) + step, base[still] + (_size(lib, still) - 1) // step * step):
                    if at % step == 0:
                        assert _call(lib, forward, {moved: at}) == INVALID, (moved, still, at)
                        assert b"overlap" in lib.tpmlp_last_error(), (moved, still, at)


@pytest.mark.parametrize("scales", [AT, AT - 7, AT + 4 * 64 - 1], ids=["first", "before", "last"])
def test_pack_refuses_codes_that_meet_their_scales(lib, scales):
    """Codes of [4, 64] at AT, eight scale bytes."""
    assert lib.tpmlp_checkpoint_pack(3 * AT, 64, AT, scales, 4, 64, 2, None) == INVALID
    assert b"codes and scales" in lib.tpmlp_last_error()


@pytest.mark.parametrize("act,scales", [(0, AT), (0, AT - 240), (0, AT + 32 * 256 - 16), (1, AT + 32 * 512 - 16), (1, AT - 496)])
@pytest.mark.parametrize("dt", [0, 2], ids=["f32", "bf16"])
def test_block_refuses_codes_that_meet_their_scales(lib, dt, act, scales):
    """32 tokens, f 256: codes [32, 256] (SwiGLU [32, 512]) at AT, 8 (16) scale bytes a token."""
    io = (ctypes.c_void_p * 1)(2 * AT)
    assert lib.tpmlp_forward_checkpoint(16, 2, 64, 256, 1, 0, dt, act, 1, io, 3 * AT, 4 * AT, AT, scales, io, 16 * AT, 1 << 40,
                                        None) == INVALID
    assert b"codes and scales" in lib.tpmlp_last_error()
