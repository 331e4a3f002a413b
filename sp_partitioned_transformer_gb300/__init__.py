"""Python binding of ``libtpmlp.so`` — the GB300 tensor/sequence-parallel MLP block.

Argument marshalling only: every step of the block runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current CUDA stream.  If the
library has not been built, ``load()`` raises; there is no fallback path.

Entry points mirror the C ABI in ``include/tpmlp.h``:

* ``workspace_size``, ``forward_workspace_size``, ``forward``, ``backward``
* ``split_dim0``, ``gather_dim0``, ``reduce_scatter_dim0``
* ``last_error``, ``device_status``, ``set_wait_timeout_ns``, ``wait_timeout_selftest``
* ``embed_forward``, ``embed_backward``, ``embed_backward_main_grad``
* ``qk_norm_rope_forward``, ``qk_norm_rope_backward``, ``qk_norm_rope_append`` (``QKRope``)
* ``paged_attn_decode``, ``attn_decode`` (``PagedKVCache``), ``attn_rope_forward``, ``attn_rope_backward``
* ``sp_rms_residual_forward``, ``sp_rms_residual_backward`` (``RMSResidual``)
* ``checkpoint_pack``, ``checkpoint_unpack``, ``forward_checkpoint``, ``backward_checkpoint`` (``Checkpoint8``)

``MLPBlock`` is a convenience holder that allocates outputs and the workspace
with ``torch.empty`` for one configuration and calls the entry points.
"""
from __future__ import annotations

import ctypes
import os
from array import array
from dataclasses import dataclass, field

import torch

__all__ = [
    "TpmlpError",
    "load",
    "lib_path",
    "STATUS",
    "DTYPE",
    "ACT",
    "MODE",
    "workspace_size",
    "forward_workspace_size",
    "forward",
    "forward_noalloc",
    "NOALLOC_SCRATCH_BYTES",
    "backward",
    "backward_main_grad",
    "split_dim0",
    "gather_dim0",
    "reduce_scatter_dim0",
    "last_error",
    "device_status",
    "set_wait_timeout_ns",
    "wait_timeout_selftest",
    "abi_version",
    "sp_layernorm_forward",
    "sp_layernorm_backward",
    "sp_layernorm_backward_workspace",
    "sp_residual_dropout_forward",
    "sp_residual_dropout_backward",
    "profile_start",
    "profile_stop",
    "PROFILE_KINDS",
    "MLPBlock",
    "attn_workspace_size",
    "attn_forward",
    "attn_backward",
    "AttnBlock",
    "embed_forward",
    "embed_backward",
    "embed_backward_main_grad",
    "embed_backward_workspace",
    "QKRope",
    "PagedKVCache",
    "qk_norm_rope_forward",
    "qk_norm_rope_backward",
    "qk_norm_rope_backward_workspace",
    "qk_norm_rope_append",
    "paged_attn_decode",
    "paged_attn_workspace_size",
    "attn_decode",
    "attn_rope_forward",
    "attn_rope_backward",
    "attn_rope_workspace_size",
    "RMSResidual",
    "sp_rms_residual_forward",
    "sp_rms_residual_backward",
    "sp_rms_residual_backward_workspace",
    "Checkpoint8",
    "checkpoint_pack",
    "checkpoint_unpack",
    "checkpoint_workspace_size",
    "forward_checkpoint",
    "backward_checkpoint",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "_lib", "libtpmlp.so")

STATUS = {
    0: "TPMLP_OK",
    -1: "TPMLP_ERR_INVALID_ARG",
    -2: "TPMLP_ERR_NOT_DIVISIBLE",
    -3: "TPMLP_ERR_UNSUPPORTED",
    -4: "TPMLP_ERR_WORKSPACE",
    -5: "TPMLP_ERR_CUDA",
    -6: "TPMLP_ERR_TIMEOUT",
}
DTYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
DTYPE_NAMES = {"f32": 0, "f16": 1, "bf16": 2}
ACT = {"gelu": 0, "swiglu": 1, "identity": 2, "relu": 3}
MODE = {"partials": 0, "fused": 1}

PROFILE_KINDS = ("gemm_tc", "gemm_f32", "copy_dim0", "shard_sum", "sp_region", "attn_core")

INDEX = {torch.int32: 0, torch.int64: 1}

_lib = None


class _QKRope(ctypes.Structure):
    _fields_ = [("q_gamma", ctypes.c_void_p), ("k_gamma", ctypes.c_void_p), ("cos", ctypes.c_void_p),
                ("sin", ctypes.c_void_p), ("max_pos", ctypes.c_int64), ("eps", ctypes.c_float), ("rot", ctypes.c_int),
                ("interleaved", ctypes.c_int)]


class _KVCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class _RMSResidual(ctypes.Structure):
    _fields_ = [("post_gamma", ctypes.c_void_p), ("pre_gamma", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("gate_rows", ctypes.c_int64), ("scale", ctypes.c_float), ("eps", ctypes.c_float)]


class _Profile(ctypes.Structure):
    _fields_ = [("launches", ctypes.c_int * 6), ("ms", ctypes.c_double * 6), ("work", ctypes.c_double * 6)]


class TpmlpError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code
        self.status = STATUS.get(code, str(code))


def lib_path() -> str:
    return _LIB_PATH


def load(path: str | None = None):
    """Load libtpmlp.so (raises ImportError if it is missing — no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or _LIB_PATH
    if not os.path.exists(p):
        raise ImportError(
            f"{p} is not built; run `python -m sp_partitioned_transformer_gb300.build` "
            "(nvcc, sm_103a) first"
        )
    lib = ctypes.CDLL(p)
    i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    vpp = ctypes.POINTER(ctypes.c_void_p)
    lib.tpmlp_abi_version.restype = i32
    lib.tpmlp_abi_version.argtypes = []
    lib.tpmlp_last_error.restype = ctypes.c_char_p
    lib.tpmlp_last_error.argtypes = []
    lib.tpmlp_workspace_size.restype = sz
    lib.tpmlp_workspace_size.argtypes = [i64, i64, i64, i64, i32, i32, i32, i32, i32]
    lib.tpmlp_forward_workspace_size.restype = sz
    lib.tpmlp_forward_workspace_size.argtypes = [i64, i64, i64, i64, i32, i32, i32, i32, i32]
    lib.tpmlp_forward.restype = i32
    lib.tpmlp_forward.argtypes = [i64, i64, i64, i64, i32, i32, i32, i32, i32,
                                  vpp, vp, vp, vp, vp, vpp, vp, sz, vp]
    lib.tpmlp_backward.restype = i32
    lib.tpmlp_backward.argtypes = [i64, i64, i64, i64, i32, i32, i32, i32, i32,
                                   vpp, vp, vp, vp, vp, vpp, vpp, vp, vp, vp, vp, sz, vp]
    lib.tpmlp_backward_main_grad.restype = i32
    lib.tpmlp_backward_main_grad.argtypes = [i64, i64, i64, i64, i32, i32, i32, i32, i32,
                                             vpp, vp, vp, vp, vp, vpp, vpp, vp, vp, vp, vp, sz, vp]
    lib.tpmlp_split_dim0.restype = i32
    lib.tpmlp_split_dim0.argtypes = [vp, vpp, i64, i64, i64, i32, i32, vp]
    lib.tpmlp_gather_dim0.restype = i32
    lib.tpmlp_gather_dim0.argtypes = [vpp, vp, i64, i64, i64, i32, i32, vp]
    lib.tpmlp_reduce_scatter_dim0.restype = i32
    lib.tpmlp_reduce_scatter_dim0.argtypes = [vp, vpp, i64, i64, i64, i32, i32, i32, vp]
    lib.tpmlp_device_status.restype = i32
    lib.tpmlp_device_status.argtypes = [vp, i32]
    lib.tpmlp_set_wait_timeout_ns.restype = None
    lib.tpmlp_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
    lib.tpmlp_wait_timeout_selftest.restype = i32
    lib.tpmlp_wait_timeout_selftest.argtypes = [ctypes.c_uint64, vp]
    lib.tpmlp_forward_noalloc.restype = i32
    lib.tpmlp_forward_noalloc.argtypes = [i64, i64, i64, i64, i32, i32, i32, i32, i32,
                                          vpp, vp, vp, vp, vp, vpp, vp]
    f32 = ctypes.c_float
    lib.tpmlp_sp_layernorm_forward.restype = i32
    lib.tpmlp_sp_layernorm_forward.argtypes = [vpp, vp, vp, f32, vpp, vp, vp, i64, i64, i64, i32, i32, vp]
    lib.tpmlp_sp_layernorm_backward_workspace.restype = sz
    lib.tpmlp_sp_layernorm_backward_workspace.argtypes = [i64, i64, i64]
    lib.tpmlp_sp_layernorm_backward.restype = i32
    lib.tpmlp_sp_layernorm_backward.argtypes = [vpp, vp, vp, vp, vpp, vpp, i32, vp, vp, vp, sz, i64, i64, i64, i32,
                                                i32, vp]
    lib.tpmlp_sp_residual_dropout_forward.restype = i32
    lib.tpmlp_sp_residual_dropout_forward.argtypes = [vpp, vpp, vpp, f32, vpp, i64, i64, i64, i32, i32, vp]
    lib.tpmlp_sp_residual_dropout_backward.restype = i32
    lib.tpmlp_sp_residual_dropout_backward.argtypes = [vpp, vpp, f32, vpp, i64, i64, i64, i32, i32, vp]
    lib.tpmlp_attn_workspace_size.restype = sz
    lib.tpmlp_attn_workspace_size.argtypes = [i64, i64, i64, i32, i32, i32, i32, i32, i32]
    lib.tpmlp_attn_forward.restype = i32
    lib.tpmlp_attn_forward.argtypes = [i64, i64, i64, i32, i32, i32, i32, i32, i32,
                                       vpp, vp, vp, vp, vp, vp, vpp, vp, sz, vp]
    lib.tpmlp_attn_backward.restype = i32
    lib.tpmlp_attn_backward.argtypes = [i64, i64, i64, i32, i32, i32, i32, i32, i32,
                                        vpp, vp, vp, vp, vp, vp, vpp, vpp, vp, vp, vp, vp, vp, sz, vp]
    lib.tpmlp_embed_forward.restype = i32
    lib.tpmlp_embed_forward.argtypes = [vp, i32, i64, i64, vp, f32, vpp, i64, i64, i64, i64, i32, i32, vp]
    lib.tpmlp_embed_backward_workspace.restype = sz
    lib.tpmlp_embed_backward_workspace.argtypes = [i64, i64, i64, i64]
    for fn in (lib.tpmlp_embed_backward, lib.tpmlp_embed_backward_main_grad):
        fn.restype = i32
        fn.argtypes = [vp, i32, i64, i64, vpp, vp, f32, vp, sz, i64, i64, i64, i64, i32, i32, vp]
    rope, cache = ctypes.POINTER(_QKRope), ctypes.POINTER(_KVCache)
    lib.tpmlp_qk_norm_rope_forward.restype = i32
    lib.tpmlp_qk_norm_rope_forward.argtypes = [vp, i64, vp, i64, rope, vp, i32, i64, i64, i32, i32, i32, i32, vp]
    lib.tpmlp_qk_norm_rope_backward_workspace.restype = sz
    lib.tpmlp_qk_norm_rope_backward_workspace.argtypes = [i64, i32, i32, i32]
    lib.tpmlp_qk_norm_rope_backward.restype = i32
    lib.tpmlp_qk_norm_rope_backward.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, rope, vp, i32, i64, i64, i32, i32,
                                                i32, i32, vp, sz, vp]
    lib.tpmlp_qk_norm_rope_append.restype = i32
    lib.tpmlp_qk_norm_rope_append.argtypes = [vp, i64, vp, i64, cache, vp, rope, vp, i32, i64, i32, i32, i32, i32, vp]
    lib.tpmlp_paged_attn_workspace_size.restype = sz
    lib.tpmlp_paged_attn_workspace_size.argtypes = [i64, i32, i32, i32]
    lib.tpmlp_paged_attn_decode.restype = i32
    lib.tpmlp_paged_attn_decode.argtypes = [vp, i64, cache, vp, i64, i64, vp, f32, vp, i64, vp, i64, i32, i32, i32, i32,
                                            vp, sz, vp]
    lib.tpmlp_attn_decode.restype = i32
    lib.tpmlp_attn_decode.argtypes = [i64, i64, i32, i32, i32, vp, vp, vp, rope, vp, i32, cache, vp, vp, i64, i64, vp,
                                      vp, vp, vp, vp, vp, sz, vp]
    lib.tpmlp_attn_rope_workspace_size.restype = sz
    lib.tpmlp_attn_rope_workspace_size.argtypes = [i64, i64, i64, i32, i32, i32, i32, i32, i32]
    lib.tpmlp_attn_rope_forward.restype = i32
    lib.tpmlp_attn_rope_forward.argtypes = [i64, i64, i64, i32, i32, i32, i32, i32, i32,
                                            vpp, vp, vp, rope, vp, vp, vp, vp, vpp, vp, sz, vp]
    lib.tpmlp_attn_rope_backward.restype = i32
    lib.tpmlp_attn_rope_backward.argtypes = [i64, i64, i64, i32, i32, i32, i32, i32, i32,
                                             vpp, vp, vp, rope, vp, vp, vp, vp, vpp, vpp, vp, vp, vp, vp, vp, vp, vp,
                                             sz, vp]
    norms = ctypes.POINTER(_RMSResidual)
    lib.tpmlp_sp_rms_residual_forward.restype = i32
    # the chunk arrays as addresses of host arrays
    lib.tpmlp_sp_rms_residual_forward.argtypes = [vp, vp, norms, vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, i32, vp]
    lib.tpmlp_sp_rms_residual_backward_workspace.restype = sz
    lib.tpmlp_sp_rms_residual_backward_workspace.argtypes = [i64, i64, i64, i64]
    lib.tpmlp_sp_rms_residual_backward.restype = i32
    lib.tpmlp_sp_rms_residual_backward.argtypes = [vp, vp, vp, vp, vp, vp, norms, vp, vp, vp, vp, vp, vp, vp, vp, sz,
                                                   i64, i64, i64, i32, i32, vp]
    lib.tpmlp_checkpoint_pack.restype = i32
    lib.tpmlp_checkpoint_pack.argtypes = [vp, i64, vp, vp, i64, i64, i32, vp]
    lib.tpmlp_checkpoint_unpack.restype = i32
    lib.tpmlp_checkpoint_unpack.argtypes = [vp, vp, vp, i64, i64, i64, i32, vp]
    lib.tpmlp_checkpoint_workspace_size.restype = sz
    lib.tpmlp_checkpoint_workspace_size.argtypes = [i64, i64, i64, i64, i32, i32, i32, i32, i32]
    lib.tpmlp_forward_checkpoint.restype = i32
    lib.tpmlp_forward_checkpoint.argtypes = [i64, i64, i64, i64, i32, i32, i32, i32, i32, vpp, vp, vp, vp, vp, vpp, vp, sz,
                                             vp]
    lib.tpmlp_backward_checkpoint.restype = i32
    lib.tpmlp_backward_checkpoint.argtypes = [i64, i64, i64, i64, i32, i32, i32, i32, i32, vpp, vp, vp, vp, vp, vpp, vpp, vp,
                                              vp, i32, vp, sz, vp]
    lib.tpmlp_profile_start.restype = i32
    lib.tpmlp_profile_start.argtypes = []
    lib.tpmlp_profile_stop.restype = i32
    lib.tpmlp_profile_stop.argtypes = [ctypes.POINTER(_Profile)]
    _lib = lib
    return lib


# ---------------------------------------------------------------- marshalling


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _ptrs(ts):
    """Host array of device pointers (a list/tuple of tensors, or one tensor)."""
    if ts is None:
        return None
    if isinstance(ts, (list, tuple)):
        vals = [_ptr(t) for t in ts]
    else:
        vals = [_ptr(ts)]
    return (ctypes.c_void_p * len(vals))(*vals)


def _stream(stream, device=None) -> int:
    if stream is None:
        # the current stream's handle without building a Stream object (2.6 of a small call's 12 µs), where torch
        # has the call
        device = torch.cuda.current_device() if device is None else device
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return torch.cuda.current_stream(device).cuda_stream if raw is None else raw(device)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype_code(dtype) -> int:
    if isinstance(dtype, str):
        return DTYPE_NAMES[dtype]
    if isinstance(dtype, int):
        return dtype
    return DTYPE[dtype]


def _check(rc: int) -> None:
    if rc != 0:
        raise TpmlpError(rc, last_error())


def abi_version() -> int:
    return load().tpmlp_abi_version()


def last_error() -> str:
    return load().tpmlp_last_error().decode(errors="replace")


def workspace_size(s, b, h, f, tp, sp, dtype, act="gelu", mode="fused") -> int:
    return int(load().tpmlp_workspace_size(s, b, h, f, tp, int(sp), _dtype_code(dtype), ACT[act], MODE[mode]))


def forward_workspace_size(s, b, h, f, tp, sp, dtype, act="gelu", mode="fused") -> int:
    return int(load().tpmlp_forward_workspace_size(s, b, h, f, tp, int(sp), _dtype_code(dtype), ACT[act],
                                                   MODE[mode]))


def forward(x, w1, w2, u, y, z, *, s, b, h, f, tp, sp, act="gelu", mode="fused", workspace=None,
            workspace_bytes=None, dtype=None, stream=None) -> None:
    """Enqueue the block's forward.  x, z: a tensor, or a list of tp SP chunks."""
    dt = _dtype_code(dtype if dtype is not None else w1.dtype)
    ws_bytes = workspace_bytes if workspace_bytes is not None else (
        0 if workspace is None or isinstance(workspace, int) else workspace.numel() * workspace.element_size())
    rc = load().tpmlp_forward(s, b, h, f, tp, int(sp), dt, ACT[act], MODE[mode], _ptrs(x), _ptr(w1), _ptr(w2),
                              _ptr(u), _ptr(y), _ptrs(z), _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc)


NOALLOC_SCRATCH_BYTES = 64 << 20


def forward_noalloc(x, w1, w2, u, y, z, *, s, b, h, f, tp, sp, act="gelu", mode="fused", dtype=None,
                    stream=None) -> None:
    """The forward without a caller workspace: the library's built-in 64 MiB
    scratch is used instead (for callers that cannot allocate device memory where
    they call the block).  Calls share that scratch: do not overlap them on the GPU."""
    dt = _dtype_code(dtype if dtype is not None else w1.dtype)
    rc = load().tpmlp_forward_noalloc(s, b, h, f, tp, int(sp), dt, ACT[act], MODE[mode], _ptrs(x), _ptr(w1),
                                      _ptr(w2), _ptr(u), _ptr(y), _ptrs(z), _stream(stream))
    _check(rc)


def backward(x, w1, w2, u, y, dz, dx, dw1, dw2, du, *, s, b, h, f, tp, sp, act="gelu", mode="fused",
             workspace=None, workspace_bytes=None, dtype=None, stream=None) -> None:
    """Enqueue the block's backward.  x, dz, dx: a tensor, or a list of tp SP chunks."""
    dt = _dtype_code(dtype if dtype is not None else w1.dtype)
    ws_bytes = workspace_bytes if workspace_bytes is not None else (
        0 if workspace is None or isinstance(workspace, int) else workspace.numel() * workspace.element_size())
    rc = load().tpmlp_backward(s, b, h, f, tp, int(sp), dt, ACT[act], MODE[mode], _ptrs(x), _ptr(w1), _ptr(w2),
                               _ptr(u), _ptr(y), _ptrs(dz), _ptrs(dx), _ptr(dw1), _ptr(dw2), _ptr(du),
                               _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc)


def backward_main_grad(x, w1, w2, u, y, dz, dx, main_grad_w1, main_grad_w2, du, *, s, b, h, f, tp, sp,
                       act="gelu", mode="fused", workspace=None, workspace_bytes=None, dtype=None,
                       stream=None) -> None:
    """tpmlp_backward with the weight gradients added into float32 main_grad buffers."""
    dt = _dtype_code(dtype if dtype is not None else w1.dtype)
    ws_bytes = workspace_bytes if workspace_bytes is not None else (
        0 if workspace is None or isinstance(workspace, int) else workspace.numel() * workspace.element_size())
    rc = load().tpmlp_backward_main_grad(s, b, h, f, tp, int(sp), dt, ACT[act], MODE[mode], _ptrs(x), _ptr(w1),
                                         _ptr(w2), _ptr(u), _ptr(y), _ptrs(dz), _ptrs(dx), _ptr(main_grad_w1),
                                         _ptr(main_grad_w2), _ptr(du), _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc)


def split_dim0(full, shards, *, s, b, h, tp, dtype=None, stream=None) -> None:
    dt = _dtype_code(dtype if dtype is not None else full.dtype)
    _check(load().tpmlp_split_dim0(_ptr(full), _ptrs(shards), s, b, h, tp, dt, _stream(stream)))


def gather_dim0(shards, full, *, s, b, h, tp, dtype=None, stream=None) -> None:
    dt = _dtype_code(dtype if dtype is not None else full.dtype)
    _check(load().tpmlp_gather_dim0(_ptrs(shards), _ptr(full), s, b, h, tp, dt, _stream(stream)))


def reduce_scatter_dim0(partials, out, *, s, b, h, tp, scatter, dtype=None, stream=None) -> None:
    outs = out if isinstance(out, (list, tuple)) else [out]
    dt = _dtype_code(dtype if dtype is not None else outs[0].dtype)
    _check(load().tpmlp_reduce_scatter_dim0(_ptr(partials), _ptrs(outs), s, b, h, tp, int(scatter), dt,
                                            _stream(stream)))


def device_status(reset: bool = False, stream=None) -> int:
    """Synchronise the stream and return the device status (0 = OK, -6 = a wait timed out, -1 = a kernel met a
    position, cache slot, page or length outside its table)."""
    return int(load().tpmlp_device_status(_stream(stream), int(reset)))


def set_wait_timeout_ns(ns: int) -> None:
    load().tpmlp_set_wait_timeout_ns(int(ns))


def wait_timeout_selftest(timeout_ns: int, stream=None) -> None:
    _check(load().tpmlp_wait_timeout_selftest(int(timeout_ns), _stream(stream)))


def _as_list(t):
    return list(t) if isinstance(t, (list, tuple)) else [t]


def sp_layernorm_forward(x, gamma, beta, eps, y, mean, rstd, *, s, b, h, tp, dtype=None, stream=None) -> None:
    """LayerNorm over h on the SP chunks (lists of tp [s/tp,b,h] tensors, or one tensor with tp=1)."""
    xs, ys = _as_list(x), _as_list(y)
    dt = _dtype_code(dtype if dtype is not None else xs[0].dtype)
    _check(load().tpmlp_sp_layernorm_forward(_ptrs(xs), _ptr(gamma), _ptr(beta), float(eps), _ptrs(ys), _ptr(mean),
                                             _ptr(rstd), s, b, h, tp, dt, _stream(stream)))


def sp_layernorm_backward_workspace(s, b, h) -> int:
    return int(load().tpmlp_sp_layernorm_backward_workspace(s, b, h))


def sp_layernorm_backward(x, gamma, mean, rstd, dy, dx, dgamma, dbeta, *, s, b, h, tp, accumulate=False,
                          workspace=None, dtype=None, stream=None) -> None:
    xs, dys, dxs = _as_list(x), _as_list(dy), _as_list(dx)
    dt = _dtype_code(dtype if dtype is not None else xs[0].dtype)
    need = sp_layernorm_backward_workspace(s, b, h)
    if workspace is None:
        workspace = _temporary(need, xs[0].device, stream)
    _check(load().tpmlp_sp_layernorm_backward(_ptrs(xs), _ptr(gamma), _ptr(mean), _ptr(rstd), _ptrs(dys),
                                              _ptrs(dxs), int(accumulate), _ptr(dgamma), _ptr(dbeta),
                                              _ptr(workspace), workspace.numel() * workspace.element_size(), s, b, h,
                                              tp, dt, _stream(stream)))


def sp_residual_dropout_forward(r, z, keep, p, out, *, s, b, h, tp, dtype=None, stream=None) -> None:
    rs = _as_list(r)
    dt = _dtype_code(dtype if dtype is not None else rs[0].dtype)
    _check(load().tpmlp_sp_residual_dropout_forward(_ptrs(rs), _ptrs(_as_list(z)), _ptrs(_as_list(keep)), float(p),
                                                    _ptrs(_as_list(out)), s, b, h, tp, dt, _stream(stream)))


def sp_residual_dropout_backward(dout, keep, p, dz, *, s, b, h, tp, dtype=None, stream=None) -> None:
    ds = _as_list(dout)
    dt = _dtype_code(dtype if dtype is not None else ds[0].dtype)
    _check(load().tpmlp_sp_residual_dropout_backward(_ptrs(ds), _ptrs(_as_list(keep)), float(p), _ptrs(_as_list(dz)),
                                                     s, b, h, tp, dt, _stream(stream)))


def profile_start() -> None:
    """Start launch accounting on this thread (CUDA events around every launch)."""
    _check(load().tpmlp_profile_start())


def profile_stop() -> dict:
    """Stop accounting; per kernel kind: launches, summed ms, algorithmic work
    (FLOPs for the GEMMs, bytes for the copy and shard-sum kernels)."""
    pr = _Profile()
    _check(load().tpmlp_profile_stop(ctypes.byref(pr)))
    return {k: {"launches": pr.launches[i], "ms": pr.ms[i], "work": pr.work[i]} for i, k in enumerate(PROFILE_KINDS)}


# ---------------------------------------------------------------- convenience


@dataclass
class MLPBlock:
    """One block configuration; allocates outputs and workspace with torch.empty.

    f is the ffn width (F for SwiGLU).  With sp, activations are lists of tp
    chunks [s/tp, b, h]; otherwise single [s, b, h] tensors.  With checkpoint, the
    forward keeps U as a Checkpoint8 (no "y", and no "du" of the backward); z is that of
    the block without one, but for a SwiGLU's in 16 bits, whose Y takes an approximate
    divide.  Blocks that run one after the other on one stream may share a `workspace`.
    """

    s: int
    b: int
    h: int
    f: int
    tp: int
    sp: bool
    dtype: torch.dtype
    act: str = "gelu"
    mode: str = "fused"
    device: str = "cuda"
    checkpoint: bool = False
    workspace: torch.Tensor | None = field(default=None, repr=False, compare=False)

    def __post_init__(self):
        self.M = self.s * self.b
        self.n1 = 2 * self.f if self.act == "swiglu" else self.f
        size = checkpoint_workspace_size if self.checkpoint else workspace_size
        self.ws_bytes = size(self.s, self.b, self.h, self.f, self.tp, self.sp, self.dtype, self.act, self.mode)
        if self.workspace is None:
            self.workspace = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=self.device)
        elif _size(self.workspace) < self.ws_bytes:
            raise ValueError(f"the workspace must have {self.ws_bytes} bytes")

    def act_tensor(self):
        if self.sp:
            return [torch.empty(self.s // self.tp, self.b, self.h, dtype=self.dtype, device=self.device)
                    for _ in range(self.tp)]
        return torch.empty(self.s, self.b, self.h, dtype=self.dtype, device=self.device)

    def alloc_forward(self):
        if self.checkpoint:
            return {"u": Checkpoint8.empty(self.M * (self.n1 // self.f), self.f, self.device), "z": self.act_tensor()}
        return {
            "u": torch.empty(self.M, self.n1, dtype=self.dtype, device=self.device),
            "y": torch.empty(self.M, self.f, dtype=self.dtype, device=self.device),
            "z": self.act_tensor(),
        }

    def alloc_backward(self):
        out = {
            "dx": self.act_tensor(),
            "dw1": torch.empty(self.n1, self.h, dtype=self.dtype, device=self.device),
            "dw2": torch.empty(self.h, self.f, dtype=self.dtype, device=self.device),
        }
        if not self.checkpoint:
            out["du"] = torch.empty(self.M, self.n1, dtype=self.dtype, device=self.device)
        return out

    def _kw(self):
        kw = dict(s=self.s, b=self.b, h=self.h, f=self.f, tp=self.tp, sp=self.sp, act=self.act, mode=self.mode,
                  workspace=self.workspace)
        return kw if self.checkpoint else dict(kw, workspace_bytes=_size(self.workspace), dtype=self.dtype)

    def forward(self, x, w1, w2, out=None, stream=None):
        out = out or self.alloc_forward()
        if self.checkpoint:
            forward_checkpoint(x, w1, w2, out["u"], out["z"], stream=stream, **self._kw())
            return out
        forward(x, w1, w2, out["u"], out["y"], out["z"], stream=stream, **self._kw())
        return out

    def backward_main_grad(self, x, w1, w2, fwd, dz, main_grad_w1, main_grad_w2, out=None, stream=None):
        """Backward whose weight gradients are added into float32 main_grad buffers."""
        out = out or self.alloc_backward()
        if self.checkpoint:
            backward_checkpoint(x, w1, w2, fwd["u"], dz, out["dx"], main_grad_w1, main_grad_w2, main_grad=True,
                                stream=stream, **self._kw())
            return out
        backward_main_grad(x, w1, w2, fwd["u"], fwd["y"], dz, out["dx"], main_grad_w1, main_grad_w2, out["du"],
                           stream=stream, **self._kw())
        return out

    def backward(self, x, w1, w2, fwd, dz, out=None, stream=None):
        out = out or self.alloc_backward()
        if self.checkpoint:
            backward_checkpoint(x, w1, w2, fwd["u"], dz, out["dx"], out["dw1"], out["dw2"], stream=stream, **self._kw())
            return out
        backward(x, w1, w2, fwd["u"], fwd["y"], dz, out["dx"], out["dw1"], out["dw2"], out["du"], stream=stream,
                 **self._kw())
        return out


# ---------------------------------------------------------------- attention block


def attn_workspace_size(s, b, h, heads, tp, sp, dtype, causal, kv_heads=None) -> int:
    kv = heads if kv_heads is None else kv_heads
    return int(load().tpmlp_attn_workspace_size(s, b, h, heads, kv, tp, int(bool(sp)), _dtype_code(dtype),
                                                 int(bool(causal))))


def attn_forward(x, wqkv, wo, qkv, o, lse, z, *, s, b, h, heads, tp, sp, causal, kv_heads=None, workspace=None,
                 dtype=None, stream=None) -> None:
    """tpmlp_attn_forward.  x, z: lists of tp chunks under sp, else single tensors;
    kv_heads None = one key/value head per query head."""
    dt = _dtype_code(dtype if dtype is not None else wqkv.dtype)
    kv = heads if kv_heads is None else kv_heads
    _check(load().tpmlp_attn_forward(s, b, h, heads, kv, tp, int(bool(sp)), dt, int(bool(causal)), _ptrs(x),
                                     _ptr(wqkv), _ptr(wo), _ptr(qkv), _ptr(o), _ptr(lse), _ptrs(z), _ptr(workspace),
                                     0 if workspace is None else workspace.numel() * workspace.element_size(),
                                     _stream(stream)))


def attn_backward(x, wqkv, wo, qkv, o, lse, dz, dx, dwqkv, dwo, dqkv, dout, *, s, b, h, heads, tp, sp, causal,
                  workspace, kv_heads=None, dtype=None, stream=None) -> None:
    """tpmlp_attn_backward.  x, dz, dx: lists of tp chunks under sp, else single tensors."""
    dt = _dtype_code(dtype if dtype is not None else wqkv.dtype)
    kv = heads if kv_heads is None else kv_heads
    _check(load().tpmlp_attn_backward(s, b, h, heads, kv, tp, int(bool(sp)), dt, int(bool(causal)), _ptrs(x),
                                      _ptr(wqkv), _ptr(wo), _ptr(qkv), _ptr(o), _ptr(lse), _ptrs(dz), _ptrs(dx),
                                      _ptr(dwqkv), _ptr(dwo), _ptr(dqkv), _ptr(dout), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _stream(stream)))


class AttnBlock:
    """One attention-block configuration; allocates outputs, saved activations and
    workspace with torch.empty (the library itself allocates nothing).  With a
    QKRope, queries and keys are normalised and rotated before the core; the
    forward's "qkv_raw" is then the projection, and the backward gives
    "dq_gamma" and "dk_gamma" (None without norms).  Outputs and workspace belong
    to the current stream: a `stream` of another waits for it before the call, and
    the current one for that stream afterwards, as with any tensor of torch's."""

    def __init__(self, s, b, h, heads, tp, sp, dtype, causal, device="cuda", kv_heads=None, rope=None):
        self.s, self.b, self.h, self.heads, self.tp, self.sp = s, b, h, heads, tp, bool(sp)
        self.kv_heads = heads if kv_heads is None else kv_heads
        self.dtype, self.causal, self.device = dtype, bool(causal), device
        self.M = s * b
        self.s_pad = (s + 127) // 128 * 128
        self.qkv_w = h + 2 * self.kv_heads * (h // heads)  # fused projection width h + 2·h_kv
        self.rope = rope
        size = attn_workspace_size if rope is None else attn_rope_workspace_size
        n = size(s, b, h, heads, tp, sp, dtype, causal, self.kv_heads)
        self.ws = torch.empty(max(n, 256), dtype=torch.uint8, device=device)

    def _act(self):
        if self.sp:
            return [torch.empty(self.s // self.tp, self.b, self.h, dtype=self.dtype, device=self.device)
                    for _ in range(self.tp)]
        return torch.empty(self.s, self.b, self.h, dtype=self.dtype, device=self.device)

    def _kw(self):
        return dict(s=self.s, b=self.b, h=self.h, heads=self.heads, tp=self.tp, sp=self.sp, causal=self.causal,
                    kv_heads=self.kv_heads)

    def forward(self, x, wqkv, wo, stream=None):
        qkv = torch.empty(self.M, self.qkv_w, dtype=self.dtype, device=self.device)
        o = torch.empty(self.M, self.h, dtype=self.dtype, device=self.device)
        lse = torch.empty(self.b, self.heads, self.s_pad, dtype=torch.float32, device=self.device)
        z = self._act()
        if self.rope is not None:
            raw = qkv if self.rope.q_gamma is None else torch.empty_like(qkv)
            attn_rope_forward(x, wqkv, wo, self.rope, raw, qkv, o, lse, z, workspace=self.ws, stream=stream,
                              **self._kw())
            return {"qkv_raw": raw, "qkv": qkv, "o": o, "lse": lse, "z": z}
        attn_forward(x, wqkv, wo, qkv, o, lse, z, workspace=self.ws, stream=stream, **self._kw())
        return {"qkv": qkv, "o": o, "lse": lse, "z": z}

    def backward(self, x, wqkv, wo, fw, dz, stream=None):
        dx = self._act()
        dwqkv = torch.empty(self.qkv_w, self.h, dtype=self.dtype, device=self.device)
        dwo = torch.empty(self.h, self.h, dtype=self.dtype, device=self.device)
        dqkv = torch.empty(self.M, self.qkv_w, dtype=self.dtype, device=self.device)
        dout = torch.empty(self.M, self.h, dtype=self.dtype, device=self.device)
        if self.rope is not None:
            dgq = dgk = None
            if self.rope.q_gamma is not None:
                dgq, dgk = torch.empty(2, self.h // self.heads, dtype=torch.float32, device=self.device).unbind(0)
            attn_rope_backward(x, wqkv, wo, self.rope, fw["qkv_raw"], fw["qkv"], fw["o"], fw["lse"], dz, dx, dwqkv, dwo,
                               dgq, dgk, dqkv, dout, workspace=self.ws, stream=stream, **self._kw())
            return {"dx": dx, "dwqkv": dwqkv, "dwo": dwo, "dqkv": dqkv, "dout": dout, "dq_gamma": dgq, "dk_gamma": dgk}
        attn_backward(x, wqkv, wo, fw["qkv"], fw["o"], fw["lse"], dz, dx, dwqkv, dwo, dqkv, dout,
                      workspace=self.ws, stream=stream, **self._kw())
        return {"dx": dx, "dwqkv": dwqkv, "dwo": dwo, "dqkv": dqkv, "dout": dout}


# ---------------------------------------------------------------- embedding


def _on_device(*tensors) -> int:
    """The current device, on which the tensors lie (None: not given)."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{dev}")
    return dev


def _temporary(nbytes, device, stream):
    """Workspace for one call, allocated on the stream that uses it: what held the block before, and what gets
    it afterwards, is ordered with the call by that stream."""
    if stream is None:
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream):
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _size(workspace) -> int:
    if workspace is None:
        return 0
    if not workspace.is_contiguous():  # an expanded tensor has fewer bytes than its elements
        raise ValueError("the workspace must be contiguous")
    return workspace.numel() * workspace.element_size()


def _same_device(dev, holder):
    if holder.device is not None and holder.device != dev:
        raise ValueError(f"{type(holder).__name__}: its tensors are not on the current device cuda:{dev}")


def _dense(t, dtype, n, name):
    """Pointer of a contiguous tensor of n elements (n None: any number)."""
    if t.dtype is not dtype or (n is not None and t.numel() != n) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor" + ("" if n is None else f" of {n} elements"))
    return t.data_ptr()


def _chunks(ts, tp, n, dtype, name, dev):
    """Host array of the pointers of tp contiguous chunks of n elements (or one tensor with tp = 1)."""
    if not isinstance(ts, (list, tuple)):
        ts = (ts,)
    if len(ts) != tp:
        raise ValueError(f"{name} has {len(ts)} chunks, not tp = {tp}")
    for t in ts:
        if t.get_device() != dev:
            raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{dev}")
    return (ctypes.c_void_p * tp)(*[_dense(t, dtype, n, name) for t in ts])


def _tokens(tokens, s, b):
    """(pointer, index type, strides) of a [s, b] int32 or int64 tensor, a transposed [b, s] batch among them."""
    code = INDEX.get(tokens.dtype)
    if code is None or tokens.dim() != 2:
        raise TypeError("tokens must be a two-dimensional [s, b] int32 or int64 tensor (a [b, s] batch: tokens.t())")
    if tokens.shape != (s, b):
        raise ValueError(f"tokens are {tuple(tokens.shape)}, not [s, b] = {(s, b)}")
    return (tokens.data_ptr(), code, *tokens.stride())


def embed_forward(tokens, table, out, *, s, b, h, vocab, tp, scale=1.0, stream=None) -> None:
    """tpmlp_embed_forward.  tokens: [s, b] (any strides); out: a list of tp chunks [s/tp, b, h], or one tensor."""
    tok = _tokens(tokens, s, b)
    dt = table.dtype
    table_ptr = _dense(table, dt, vocab * h, "table")
    dev = _on_device(tokens, table)
    _check(load().tpmlp_embed_forward(*tok, table_ptr, scale, _chunks(out, tp, s // max(tp, 1) * b * h, dt, "out", dev), s,
                                      b, h, vocab, tp, DTYPE[dt], _stream(stream, dev)))


def embed_backward_workspace(s, b, h, vocab) -> int:
    return int(load().tpmlp_embed_backward_workspace(s, b, h, vocab))


def _embed_backward(fn, tokens, dx, grad, grad_dtype, s, b, h, vocab, tp, scale, workspace, stream):
    tok = _tokens(tokens, s, b)
    dt = (dx[0] if isinstance(dx, (list, tuple)) else dx).dtype
    grad_ptr = _dense(grad, grad_dtype or dt, vocab * h, "the gradient")
    dev = _on_device(tokens, grad, workspace)
    if workspace is None:
        workspace = _temporary(embed_backward_workspace(s, b, h, vocab), grad.device, stream)
    _check(fn(*tok, _chunks(dx, tp, s // max(tp, 1) * b * h, dt, "dx", dev), grad_ptr, scale, workspace.data_ptr(),
              _size(workspace), s, b, h, vocab, tp, DTYPE[dt], _stream(stream, dev)))


def embed_backward(tokens, dx, dtable, *, s, b, h, vocab, tp, scale=1.0, workspace=None, stream=None) -> None:
    """tpmlp_embed_backward: the whole gradient of the table, in dx's type."""
    _embed_backward(load().tpmlp_embed_backward, tokens, dx, dtable, None, s, b, h, vocab, tp, scale, workspace, stream)


def embed_backward_main_grad(tokens, dx, main_grad, *, s, b, h, vocab, tp, scale=1.0, workspace=None,
                             stream=None) -> None:
    """tpmlp_embed_backward_main_grad: the gradient added to a float32 main_grad [vocab, h]."""
    _embed_backward(load().tpmlp_embed_backward_main_grad, tokens, dx, main_grad, torch.float32, s, b, h, vocab, tp, scale,
                    workspace, stream)


# ---------------------------------------------------------------- QK norm and rotation, paged cache


class QKRope:
    """The norm weights [d] and the rotation tables cos, sin [max_pos, rot/2] (float32) of an attention
    layer.  Without gammas there is no norm, without tables no rotation.  Keeps the memory that the tensors have
    now (values written to it in place are seen); a tensor that is given other memory needs a new QKRope."""

    def __init__(self, *, q_gamma=None, k_gamma=None, eps=1e-6, cos=None, sin=None, interleaved=False):
        if (cos is None) != (sin is None):
            raise ValueError("cos and sin must both be given or both be None")
        for t in (cos, sin):
            if t is not None and (t.dtype != torch.float32 or t.dim() != 2 or not t.is_contiguous()):
                raise TypeError("cos and sin must be contiguous [max_pos, rot/2] float32 tensors")
        if cos is not None and cos.shape != sin.shape:
            raise ValueError("cos and sin must have the same shape")
        for t in (q_gamma, k_gamma):
            if t is not None and (t.dim() != 1 or not t.is_contiguous()):
                raise TypeError("q_gamma and k_gamma must be contiguous [d] tensors")
        if (q_gamma is None) != (k_gamma is None):
            raise ValueError("q_gamma and k_gamma must both be given or both be None")
        if q_gamma is not None and (q_gamma.shape != k_gamma.shape or q_gamma.dtype != k_gamma.dtype):
            raise ValueError("q_gamma and k_gamma must have the same shape and type")
        # aliases: `parameter.data = …` would free the memory whose address is passed on
        q_gamma, k_gamma, cos, sin = (None if t is None else t.detach() for t in (q_gamma, k_gamma, cos, sin))
        self.q_gamma, self.k_gamma, self.cos, self.sin = q_gamma, k_gamma, cos, sin
        given = [t.get_device() for t in (q_gamma, k_gamma, cos, sin) if t is not None]
        if len(set(given)) > 1:
            raise ValueError("the tensors of a QKRope must be on one device")
        self.device = given[0] if given else None
        self.kind = None if q_gamma is None else (q_gamma.numel(), DTYPE[q_gamma.dtype])
        self.c = _QKRope(_ptr(q_gamma), _ptr(k_gamma), _ptr(cos), _ptr(sin), 0 if cos is None else cos.shape[0],
                         float(eps), 0 if cos is None else 2 * cos.shape[1], int(bool(interleaved)))
        self.ref = ctypes.byref(self.c)

    def _check(self, d, dt, dev):
        _same_device(dev, self)
        if self.kind is not None and self.kind != (d, dt):
            raise ValueError("q_gamma and k_gamma must have d elements of the activations' type")


class PagedKVCache:
    """Keys and values [pages, page_size, kv_heads, d], views of any stride order whose last dimension is
    contiguous (e.g. a [pages, kv_heads, page_size, d] buffer with its middle dimensions transposed).  Keeps the
    memory that they have now."""

    def __init__(self, k, v):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError("k and v must be [pages, page_size, kv_heads, d] of one type and stride, the last contiguous")
        k, v = k.detach(), v.detach()
        self.k, self.v = k, v
        self.pages, self.page_size, self.kv_heads, self.d = k.shape
        if k.get_device() != v.get_device():
            raise ValueError("k and v must be on one device")
        self.device = k.get_device()
        self.kind = (self.kv_heads, self.d, DTYPE[k.dtype])
        self.c = _KVCache(k.data_ptr(), v.data_ptr(), self.pages, self.page_size, *k.stride()[:3])
        self.ref = ctypes.byref(self.c)

    def _check(self, kv_heads, d, dt, dev):
        _same_device(dev, self)
        if self.kind != (kv_heads, d, dt):
            raise ValueError(f"the cache holds {self.kv_heads} heads of {self.d} {self.k.dtype}")


def _rows(t, rows, width, dtype, name):
    """(pointer, row stride) of a [rows, width] tensor, or one whose further dimensions are contiguous in a row."""
    if t.dtype is not dtype or t.numel() != rows * width or t.shape[0] != rows:
        raise ValueError(f"{name} is {tuple(t.shape)} of {t.dtype}, not [{rows}, {width}] of {dtype}")
    if t.is_contiguous():
        return t.data_ptr(), width
    if not t[0].is_contiguous():
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.data_ptr(), t.stride(0) if rows > 1 else width


def _positions(positions, rows):
    if positions is None:
        return None, 0
    code = INDEX.get(positions.dtype)
    if code is None or positions.numel() != rows or not positions.is_contiguous():
        raise TypeError("positions must be a contiguous int32 or int64 tensor of one position a row")
    return positions.data_ptr(), code


def _vector(t, dtype, n, name):
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} tensor of {n} elements")
    return t.data_ptr()


def _table(t, n):
    if t.dtype is not torch.int32 or t.dim() != 2 or t.shape[0] != n:
        raise TypeError(f"block_table must be a [{n}, width] int32 tensor with contiguous rows")
    width = t.shape[1]
    if t.is_contiguous():
        return t.data_ptr(), width, width
    if width > 1 and t.stride(1) != 1:
        raise TypeError(f"block_table must be a [{n}, width] int32 tensor with contiguous rows")
    return t.data_ptr(), t.stride(0) if n > 1 else width, width


def qk_norm_rope_forward(qkv, out, rope, *, rows, b, heads, kv_heads, d, positions=None, stream=None) -> None:
    """tpmlp_qk_norm_rope_forward: qkv, out [rows, (heads + 2·kv_heads)·d] in the group layout (out may be qkv);
    positions None: row m is at position m // b."""
    t = qkv.dtype
    W = (heads + 2 * kv_heads) * d
    args = (*_rows(qkv, rows, W, t, "qkv"), *_rows(out, rows, W, t, "out"), rope.ref, *_positions(positions, rows))
    dt = DTYPE[t]
    dev = _on_device(qkv, out, positions)
    rope._check(d, dt, dev)
    _check(load().tpmlp_qk_norm_rope_forward(*args, rows, b, heads, kv_heads, d, dt, _stream(stream, dev)))


def qk_norm_rope_backward_workspace(rows, heads, kv_heads, d) -> int:
    return int(load().tpmlp_qk_norm_rope_backward_workspace(rows, heads, kv_heads, d))


def qk_norm_rope_backward(qkv, dout, dqkv, dq_gamma, dk_gamma, rope, *, rows, b, heads, kv_heads, d, positions=None,
                          workspace=None, stream=None) -> None:
    """tpmlp_qk_norm_rope_backward: qkv the forward's input (None without norms); dqkv may be dout; dq_gamma and
    dk_gamma [d] float32 (None without norms)."""
    t = dout.dtype
    W = (heads + 2 * kv_heads) * d
    norm = rope.q_gamma is not None
    args = (*(_rows(qkv, rows, W, t, "qkv") if norm else (None, 0)), *_rows(dout, rows, W, t, "dout"),
            *_rows(dqkv, rows, W, t, "dqkv"), _dense(dq_gamma, torch.float32, d, "dq_gamma") if norm else None,
            _dense(dk_gamma, torch.float32, d, "dk_gamma") if norm else None, rope.ref, *_positions(positions, rows))
    dt = DTYPE[t]
    dev = _on_device(qkv if norm else None, dout, dqkv, dq_gamma, dk_gamma, positions, workspace)
    rope._check(d, dt, dev)
    if norm and workspace is None:
        workspace = _temporary(qk_norm_rope_backward_workspace(rows, heads, kv_heads, d), dout.device, stream)
    _check(load().tpmlp_qk_norm_rope_backward(*args, rows, b, heads, kv_heads, d, dt, _ptr(workspace),
                                              _size(workspace),
                                              _stream(stream, dev)))


def qk_norm_rope_append(qkv, q, cache, slots, rope, *, rows, heads, kv_heads, d, positions, stream=None) -> None:
    """tpmlp_qk_norm_rope_append: q [rows, heads, d] out, keys and values to `slots` of the PagedKVCache."""
    t = qkv.dtype
    args = (*_rows(qkv, rows, (heads + 2 * kv_heads) * d, t, "qkv"), *_rows(q, rows, heads * d, t, "q"), cache.ref,
            _vector(slots, torch.int64, rows, "slots"), rope.ref, *_positions(positions, rows))
    dt = DTYPE[t]
    dev = _on_device(qkv, q, slots, positions)
    rope._check(d, dt, dev)
    cache._check(kv_heads, d, dt, dev)
    _check(load().tpmlp_qk_norm_rope_append(*args, rows, heads, kv_heads, d, dt, _stream(stream, dev)))


def paged_attn_workspace_size(n, heads, kv_heads, d) -> int:
    return int(load().tpmlp_paged_attn_workspace_size(n, heads, kv_heads, d))


def paged_attn_decode(q, cache, block_table, lengths, o, lse=None, *, n, heads, kv_heads, d, scale=None,
                      workspace=None, stream=None) -> None:
    """tpmlp_paged_attn_decode: q, o [n, heads, d]; block_table [n, width] and lengths [n] int32; lse [n, heads]
    float32 (base 2) or None; scale None: 1/√d."""
    t = q.dtype
    args = (*_rows(q, n, heads * d, t, "q"), cache.ref, *_table(block_table, n),
            _vector(lengths, torch.int32, n, "lengths"), d ** -0.5 if scale is None else scale,
            *_rows(o, n, heads * d, t, "o"), None if lse is None else _dense(lse, torch.float32, n * heads, "lse"))
    dt = DTYPE[t]
    dev = _on_device(q, block_table, lengths, o, lse, workspace)
    cache._check(kv_heads, d, dt, dev)
    if workspace is None:
        workspace = _temporary(paged_attn_workspace_size(n, heads, kv_heads, d), q.device, stream)
    _check(load().tpmlp_paged_attn_decode(*args, n, heads, kv_heads, d, dt, workspace.data_ptr(),
                                          _size(workspace), _stream(stream, dev)))


def attn_decode(x, wqkv, wo, rope, cache, positions, slots, block_table, lengths, qkv, q, o, z, *, n, h, heads,
                kv_heads=None, workspace=None, stream=None) -> None:
    """tpmlp_attn_decode: the attention block for one new token of each of n sequences; lengths count that token."""
    kv = heads if kv_heads is None else kv_heads
    t, d = wqkv.dtype, h // heads
    W = h + 2 * kv * d
    x_, wqkv_, wo_, qkv_, q_, o_, z_ = (
        _dense(v, t, size, name) for v, size, name in
        ((x, n * h, "x"), (wqkv, W * h, "wqkv"), (wo, h * h, "wo"), (qkv, n * W, "qkv"), (q, n * h, "q"), (o, n * h, "o"),
         (z, n * h, "z")))
    pos, slots_, table, lens = (_positions(positions, n), _vector(slots, torch.int64, n, "slots"), _table(block_table, n),
                                _vector(lengths, torch.int32, n, "lengths"))
    dt = DTYPE[t]
    dev = _on_device(x, wqkv, wo, positions, slots, block_table, lengths, qkv, q, o, z, workspace)
    rope._check(d, dt, dev)
    cache._check(kv, d, dt, dev)
    if workspace is None:
        workspace = _temporary(paged_attn_workspace_size(n, heads, kv, d), x.device, stream)
    _check(load().tpmlp_attn_decode(n, h, heads, kv, dt, x_, wqkv_, wo_, rope.ref, *pos, cache.ref, slots_, *table, lens,
                                    qkv_, q_, o_, z_, workspace.data_ptr(), _size(workspace),
                                    _stream(stream, dev)))


def attn_rope_workspace_size(s, b, h, heads, tp, sp, dtype, causal, kv_heads=None) -> int:
    kv = heads if kv_heads is None else kv_heads
    return int(load().tpmlp_attn_rope_workspace_size(s, b, h, heads, kv, tp, int(bool(sp)), _dtype_code(dtype),
                                                      int(bool(causal))))


def _rope_block(x, wqkv, wo, rope, qkv, o, lse, workspace, s, b, h, heads, kv, tp, sp, dtype, more):
    """What both directions of the block take, checked: (type code, device, chunks and their elements), the pointers
    of wqkv, wo, qkv, o and lse, and those of x's chunks.  `more`: further tensors that must be on the device."""
    t, d, n = wqkv.dtype, h // heads, tp if sp else 1
    dt, W = DTYPE[t], h + 2 * kv * d
    if dtype is not None and _dtype_code(dtype) != dt:
        raise ValueError(f"wqkv is {t}, not {dtype}")
    ptrs = [_dense(v, e, size, name) for v, e, size, name in
            ((wqkv, t, W * h, "wqkv"), (wo, t, h * h, "wo"), (qkv, t, s * b * W, "qkv"), (o, t, s * b * h, "o"),
             (lse, torch.float32, b * heads * ((s + 127) // 128 * 128), "lse"))]
    dev = _on_device(wqkv, wo, qkv, o, lse, workspace, *more)
    rope._check(d, dt, dev)
    chunk = s // max(n, 1) * b * h
    return (dt, dev, n, chunk), ptrs, _chunks(x, n, chunk, t, "x", dev)


def attn_rope_forward(x, wqkv, wo, rope, qkv_raw, qkv, o, lse, z, *, s, b, h, heads, tp, sp, causal, kv_heads=None,
                      workspace=None, dtype=None, stream=None) -> None:
    """tpmlp_attn_rope_forward: attn_forward with the QK norms and the rotation of `rope`."""
    kv = heads if kv_heads is None else kv_heads
    raw_ = _dense(qkv_raw, wqkv.dtype, s * b * (h + 2 * kv * (h // heads)), "qkv_raw")
    (dt, dev, n, chunk), (wqkv_, wo_, qkv_, o_, lse_), x_ = _rope_block(x, wqkv, wo, rope, qkv, o, lse, workspace, s, b, h,
                                                                        heads, kv, tp, sp, dtype, (qkv_raw,))
    z_ = _chunks(z, n, chunk, wqkv.dtype, "z", dev)
    _check(load().tpmlp_attn_rope_forward(s, b, h, heads, kv, tp, int(bool(sp)), dt, int(bool(causal)), x_, wqkv_, wo_,
                                          rope.ref, raw_, qkv_, o_, lse_, z_, _ptr(workspace), _size(workspace),
                                          _stream(stream, dev)))


def attn_rope_backward(x, wqkv, wo, rope, qkv_raw, qkv, o, lse, dz, dx, dwqkv, dwo, dq_gamma, dk_gamma, dqkv, dout, *,
                       s, b, h, heads, tp, sp, causal, workspace, kv_heads=None, dtype=None, stream=None) -> None:
    """tpmlp_attn_rope_backward (workspace: attn_rope_workspace_size bytes).  dq_gamma, dk_gamma: [d] float32, used
    with norms only, as is qkv_raw."""
    kv = heads if kv_heads is None else kv_heads
    t, d, norm = wqkv.dtype, h // heads, rope.q_gamma is not None
    W = h + 2 * kv * d
    raw_, dgq_, dgk_ = ((_dense(qkv_raw, t, s * b * W, "qkv_raw"), _dense(dq_gamma, torch.float32, d, "dq_gamma"),
                         _dense(dk_gamma, torch.float32, d, "dk_gamma")) if norm else (None, None, None))
    grads = ((dwqkv, W * h, "dwqkv"), (dwo, h * h, "dwo"), (dqkv, s * b * W, "dqkv"), (dout, s * b * h, "dout"))
    dwqkv_, dwo_, dqkv_, dout_ = (_dense(v, t, size, name) for v, size, name in grads)
    more = (dwqkv, dwo, dqkv, dout, *((qkv_raw, dq_gamma, dk_gamma) if norm else ()))
    (dt, dev, n, chunk), (wqkv_, wo_, qkv_, o_, lse_), x_ = _rope_block(x, wqkv, wo, rope, qkv, o, lse, workspace, s, b, h,
                                                                        heads, kv, tp, sp, dtype, more)
    dz_, dx_ = (_chunks(v, n, chunk, t, name, dev) for v, name in ((dz, "dz"), (dx, "dx")))
    _check(load().tpmlp_attn_rope_backward(s, b, h, heads, kv, tp, int(bool(sp)), dt, int(bool(causal)), x_, wqkv_, wo_,
                                           rope.ref, raw_, qkv_, o_, lse_, dz_, dx_, dwqkv_, dwo_, dgq_, dgk_, dqkv_, dout_,
                                           workspace.data_ptr(), _size(workspace), _stream(stream, dev)))


# ---------------------------------------------------------------- checkpoints in 8 bits


class Checkpoint8:
    """An activation [rows, cols] held in 8 bits: codes [rows, cols] (e4m3) and scales [rows, ceil(cols/32)], the value
    being code·2^(byte − 127), both contiguous uint8 tensors.  Keeps the memory that they have now."""

    def __init__(self, codes, scales):
        if codes.dim() != 2 or scales.dim() != 2 or scales.shape != (codes.shape[0], -(-codes.shape[1] // 32)):
            raise ValueError("codes must be [rows, cols] and scales [rows, ceil(cols/32)]")
        codes, scales = codes.detach(), scales.detach()
        self.codes, self.scales = codes, scales
        self.ptrs = (_dense(codes, torch.uint8, None, "codes"), _dense(scales, torch.uint8, None, "scales"))
        self.rows, self.cols = codes.shape
        if codes.get_device() != scales.get_device():
            raise ValueError("codes and scales must be on one device")
        self.device = codes.get_device()

    @classmethod
    def empty(cls, rows, cols, device="cuda"):
        return cls(*(torch.empty(rows, n, dtype=torch.uint8, device=device) for n in (cols, -(-cols // 32))))

    def _check(self, rows, cols, dev):
        _same_device(dev, self)
        if (self.rows, self.cols) != (rows, cols):
            raise ValueError(f"the checkpoint is of [{self.rows}, {self.cols}], not [{rows}, {cols}]")
        return self.ptrs


def checkpoint_pack(x, checkpoint, *, rows, cols, stream=None) -> None:
    """tpmlp_checkpoint_pack: x [rows, cols] (contiguous rows) into the Checkpoint8."""
    t = x.dtype
    args = _rows(x, rows, cols, t, "x")
    dt = DTYPE[t]
    dev = _on_device(x)
    _check(load().tpmlp_checkpoint_pack(*args, *checkpoint._check(rows, cols, dev), rows, cols, dt, _stream(stream, dev)))


def checkpoint_unpack(checkpoint, x, *, rows, cols, stream=None) -> None:
    """tpmlp_checkpoint_unpack: the Checkpoint8's values into x [rows, cols] (contiguous rows)."""
    t = x.dtype
    args = _rows(x, rows, cols, t, "x")
    dt = DTYPE[t]
    dev = _on_device(x)
    _check(load().tpmlp_checkpoint_unpack(*checkpoint._check(rows, cols, dev), *args, rows, cols, dt, _stream(stream, dev)))


def checkpoint_workspace_size(s, b, h, f, tp, sp, dtype, act="gelu", mode="fused") -> int:
    return int(load().tpmlp_checkpoint_workspace_size(s, b, h, f, tp, int(sp), _dtype_code(dtype), ACT[act], MODE[mode]))


def _checkpoint_block(x, w1, w2, u, workspace, s, b, h, f, tp, sp, act, more):
    """What both directions take, checked: (type, device, chunks and their elements), and the pointers of x's chunks,
    w1, w2 and the checkpoint."""
    t, n, halves = w1.dtype, tp if sp else 1, 2 if act == "swiglu" else 1
    dev = _on_device(w1, w2, workspace, *more)
    chunk = s // max(n, 1) * b * h
    return (t, dev, n, chunk), (_chunks(x, n, chunk, t, "x", dev), _dense(w1, t, halves * f * h, "w1"),
                                _dense(w2, t, h * f, "w2"), *u._check(s * b * halves, f, dev))


def forward_checkpoint(x, w1, w2, u, z, *, s, b, h, f, tp, sp, act="gelu", mode="fused", workspace=None,
                       stream=None) -> None:
    """tpmlp_forward_checkpoint: the forward that keeps U as the Checkpoint8 `u` of [s·b, f] (SwiGLU: [2·s·b, f], row 2m
    the gate and row 2m + 1 the up half of token m).  workspace: checkpoint_workspace_size bytes."""
    (t, dev, n, chunk), args = _checkpoint_block(x, w1, w2, u, workspace, s, b, h, f, tp, sp, act, ())
    z_ = _chunks(z, n, chunk, t, "z", dev)
    if workspace is None:
        workspace = _temporary(checkpoint_workspace_size(s, b, h, f, tp, sp, t, act, mode), w1.device, stream)
    _check(load().tpmlp_forward_checkpoint(s, b, h, f, tp, int(bool(sp)), DTYPE[t], ACT[act], MODE[mode], *args, z_,
                                           workspace.data_ptr(), _size(workspace), _stream(stream, dev)))


def backward_checkpoint(x, w1, w2, u, dz, dx, dw1, dw2, *, s, b, h, f, tp, sp, act="gelu", mode="fused", main_grad=False,
                        workspace=None, stream=None) -> None:
    """tpmlp_backward_checkpoint.  main_grad: dw1 and dw2 are float32 and added to."""
    (t, dev, n, chunk), args = _checkpoint_block(x, w1, w2, u, workspace, s, b, h, f, tp, sp, act, (dw1, dw2))
    gt = torch.float32 if main_grad else t
    dw1_, dw2_ = _dense(dw1, gt, w1.numel(), "dw1"), _dense(dw2, gt, h * f, "dw2")
    dz_, dx_ = _chunks(dz, n, chunk, t, "dz", dev), _chunks(dx, n, chunk, t, "dx", dev)
    if workspace is None:
        workspace = _temporary(checkpoint_workspace_size(s, b, h, f, tp, sp, t, act, mode), w1.device, stream)
    _check(load().tpmlp_backward_checkpoint(s, b, h, f, tp, int(bool(sp)), DTYPE[t], ACT[act], MODE[mode], *args, dz_, dx_,
                                            dw1_, dw2_, int(bool(main_grad)), workspace.data_ptr(), _size(workspace),
                                            _stream(stream, dev)))


# ---------------------------------------------------------------- RMS norms around a block


class RMSResidual:
    """What a layer has between two blocks: the norm weights behind the first (post_gamma) and in front of the second
    (pre_gamma), each [h] or None; the gate of the first block's branch, [h] or [b, h] or None; the branch's scale.
    Keeps the memory that the tensors have now (values written to it in place are seen); a tensor that is given other
    memory needs a new RMSResidual."""

    def __init__(self, *, post_gamma=None, pre_gamma=None, gate=None, scale=1.0, eps=1e-6):
        post_gamma, pre_gamma, gate = (None if t is None else t.detach() for t in (post_gamma, pre_gamma, gate))
        self.post_gamma, self.pre_gamma, self.gate = post_gamma, pre_gamma, gate
        given = [t for t in (post_gamma, pre_gamma, gate) if t is not None]
        for t in given:
            if t.dim() != 1 and not (t is gate and t.dim() == 2) or not t.is_contiguous():
                raise TypeError("post_gamma and pre_gamma must be contiguous [h], the gate a contiguous [h] or [b, h] tensor")
        if len({(t.shape[-1], t.dtype) for t in given}) > 1:
            raise ValueError("the tensors of an RMSResidual must have one width h and one type")
        if len({t.get_device() for t in given}) > 1:
            raise ValueError("the tensors of an RMSResidual must be on one device")
        self.device = given[0].get_device() if given else None
        self.kind = (given[0].shape[-1], given[0].dtype) if given else None
        self.per_batch = gate is not None and gate.dim() == 2
        self.gate_rows = gate.shape[0] if self.per_batch else 1
        self.scale, self.eps = float(scale), float(eps)
        self.c = _RMSResidual(_ptr(post_gamma), _ptr(pre_gamma), _ptr(gate), self.gate_rows, self.scale, self.eps)
        self.ref = ctypes.byref(self.c)

    def _check(self, b, h, t, dev):
        _same_device(dev, self)
        if self.kind is not None and self.kind != (h, t):
            raise ValueError(f"the norms are of {self.kind[0]} columns of {self.kind[1]}")
        if self.per_batch and self.gate_rows != b:
            raise ValueError(f"the gate has {self.gate_rows} rows, not b = {b}")


def _add_chunks(ptrs, ts, name, tp, n, dtype, dev):
    """Appends the pointers of tp contiguous chunks of n elements (or one tensor with tp = 1): at tp = 8 most of a
    small call's time goes into looking its chunks over, so each is asked for no more than it has to be."""
    if type(ts) is not list and not isinstance(ts, (list, tuple)):
        ts = (ts,)
    if len(ts) != tp:
        raise ValueError(f"{name} has {len(ts)} chunks, not tp = {tp}")
    for t in ts:
        if t.dtype is not dtype or t.numel() != n or t.get_device() != dev or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous {dtype} tensors of {n} elements on the current device cuda:{dev}")
        ptrs.append(t.data_ptr())


def sp_rms_residual_forward(r, z, norms, x, y, rstd_z, rstd_x, *, s, b, h, tp, checkpoint=None, stream=None) -> None:
    """tpmlp_sp_rms_residual_forward with the layer's RMSResidual.  r, z, x, y: lists of tp chunks [s/tp, b, h], or one
    tensor each with tp = 1; z None: y of r alone.  y and rstd_x are used with pre_gamma, rstd_z with post_gamma
    ([s·b] float32).  checkpoint: a Checkpoint8 of [s·b, h] that takes z."""
    t = (r[0] if isinstance(r, (list, tuple)) else r).dtype
    post, pre, block = norms.post_gamma is not None, norms.pre_gamma is not None, z is not None
    dev = torch.cuda.current_device()
    norms._check(b, h, t, dev)
    n, ptrs = s // max(tp, 1) * b * h, []
    _add_chunks(ptrs, r, "r", tp, n, t, dev)
    if block:
        _add_chunks(ptrs, z, "z", tp, n, t, dev)
        _add_chunks(ptrs, x, "x", tp, n, t, dev)
    if pre:
        _add_chunks(ptrs, y, "y", tp, n, t, dev)
    host = array("Q", ptrs)  # kept until the call has copied it
    r_, one = host.buffer_info()[0], 8 * tp
    z_, x_ = (r_ + one, r_ + 2 * one) if block else (None, None)
    y_ = (r_ + 3 * one if block else r_ + one) if pre else None
    codes, scales = (None, None) if checkpoint is None else checkpoint._check(s * b, h, dev)
    rz = _float_vector(rstd_z, s * b, "rstd_z", dev) if post else None
    rx = _float_vector(rstd_x, s * b, "rstd_x", dev) if pre else None
    _check(load().tpmlp_sp_rms_residual_forward(r_, z_, norms.ref, x_, y_, codes, scales, rz, rx, s, b, h, tp, DTYPE[t],
                                                _stream(stream, dev)))


def _float_vector(t, n, name, dev):
    """Pointer of a contiguous float32 tensor of n elements on the current device."""
    if t.dtype is not torch.float32 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of {n} elements")
    if t.get_device() != dev:
        raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{dev}")
    return t.data_ptr()


def sp_rms_residual_backward_workspace(s, b, h, gate_rows=1) -> int:
    return int(load().tpmlp_sp_rms_residual_backward_workspace(s, b, h, gate_rows))


def sp_rms_residual_backward(dx, dy, x, z, norms, rstd_z, rstd_x, dr, dz, dpost_gamma, dpre_gamma, dgate, *, s, b, h, tp,
                             workspace=None, stream=None) -> None:
    """tpmlp_sp_rms_residual_backward.  dx (None: no gradient from past the next block), dy and x (used with pre_gamma),
    dr (may be dx) and dz (None where the forward had no z): chunks as in the forward; z: chunks, or the forward's
    Checkpoint8 (used with post_gamma or a gate).  dpost_gamma, dpre_gamma [h] and dgate (the gate's shape): float32,
    None where the parameter is."""
    first = dr[0] if isinstance(dr, (list, tuple)) else dr
    t = first.dtype
    post, pre, gate = norms.post_gamma is not None, norms.pre_gamma is not None, norms.gate is not None
    past, block = dx is not None, dz is not None
    dev = torch.cuda.current_device()
    norms._check(b, h, t, dev)
    codes = scales = None
    reads_z = post or gate
    if reads_z and isinstance(z, Checkpoint8):
        codes, scales = z._check(s * b, h, dev)
        reads_z = False
    n, ptrs = s // max(tp, 1) * b * h, []
    _add_chunks(ptrs, dr, "dr", tp, n, t, dev)
    if block:
        _add_chunks(ptrs, dz, "dz", tp, n, t, dev)
    if past:
        _add_chunks(ptrs, dx, "dx", tp, n, t, dev)
    if pre:
        _add_chunks(ptrs, dy, "dy", tp, n, t, dev)
        _add_chunks(ptrs, x, "x", tp, n, t, dev)
    if reads_z:
        _add_chunks(ptrs, z, "z", tp, n, t, dev)
    host = array("Q", ptrs)  # kept until the call has copied it
    dr_, one = host.buffer_info()[0], 8 * tp
    at = dr_
    dz_ = (at := at + one) if block else None
    dx_ = (at := at + one) if past else None
    dy_ = (at := at + one) if pre else None
    x_ = (at := at + one) if pre else None
    z_ = at + one if reads_z else None
    rz = _float_vector(rstd_z, s * b, "rstd_z", dev) if post else None
    rx = _float_vector(rstd_x, s * b, "rstd_x", dev) if pre else None
    dpo = _float_vector(dpost_gamma, h, "dpost_gamma", dev) if post else None
    dpr = _float_vector(dpre_gamma, h, "dpre_gamma", dev) if pre else None
    dg = _float_vector(dgate, norms.gate_rows * h, "dgate", dev) if gate else None
    if workspace is None:
        workspace = _temporary(sp_rms_residual_backward_workspace(s, b, h, norms.gate_rows), first.device, stream)
    elif workspace.get_device() != dev:
        raise ValueError(f"a tensor is on {workspace.device}, the current device is cuda:{dev}")
    _check(load().tpmlp_sp_rms_residual_backward(dx_, dy_, x_, z_, codes, scales, norms.ref, rz, rx, dr_, dz_, dpo, dpr, dg,
                                                 workspace.data_ptr(), _size(workspace), s, b, h, tp, DTYPE[t],
                                                 _stream(stream, dev)))
