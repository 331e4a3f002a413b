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

``MLPBlock`` is a convenience holder that allocates outputs and the workspace
with ``torch.empty`` for one configuration and calls the entry points.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

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
    chunks [s/tp, b, h]; otherwise single [s, b, h] tensors.
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

    def __post_init__(self):
        self.M = self.s * self.b
        self.n1 = 2 * self.f if self.act == "swiglu" else self.f
        self.ws_bytes = workspace_size(self.s, self.b, self.h, self.f, self.tp, self.sp, self.dtype, self.act,
                                       self.mode)
        self.workspace = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=self.device)

    def act_tensor(self):
        if self.sp:
            return [torch.empty(self.s // self.tp, self.b, self.h, dtype=self.dtype, device=self.device)
                    for _ in range(self.tp)]
        return torch.empty(self.s, self.b, self.h, dtype=self.dtype, device=self.device)

    def alloc_forward(self):
        return {
            "u": torch.empty(self.M, self.n1, dtype=self.dtype, device=self.device),
            "y": torch.empty(self.M, self.f, dtype=self.dtype, device=self.device),
            "z": self.act_tensor(),
        }

    def alloc_backward(self):
        return {
            "dx": self.act_tensor(),
            "dw1": torch.empty(self.n1, self.h, dtype=self.dtype, device=self.device),
            "dw2": torch.empty(self.h, self.f, dtype=self.dtype, device=self.device),
            "du": torch.empty(self.M, self.n1, dtype=self.dtype, device=self.device),
        }

    def _kw(self):
        return dict(s=self.s, b=self.b, h=self.h, f=self.f, tp=self.tp, sp=self.sp, act=self.act, mode=self.mode,
                    workspace=self.workspace, workspace_bytes=self.workspace.numel(), dtype=self.dtype)

    def forward(self, x, w1, w2, out=None, stream=None):
        out = out or self.alloc_forward()
        forward(x, w1, w2, out["u"], out["y"], out["z"], stream=stream, **self._kw())
        return out

    def backward_main_grad(self, x, w1, w2, fwd, dz, main_grad_w1, main_grad_w2, out=None, stream=None):
        """Backward whose weight gradients are added into float32 main_grad buffers."""
        out = out or self.alloc_backward()
        backward_main_grad(x, w1, w2, fwd["u"], fwd["y"], dz, out["dx"], main_grad_w1, main_grad_w2, out["du"],
                           stream=stream, **self._kw())
        return out

    def backward(self, x, w1, w2, fwd, dz, out=None, stream=None):
        out = out or self.alloc_backward()
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
