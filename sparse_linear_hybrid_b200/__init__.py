"""Python binding of libsalad, the SALAD hybrid attention layer for B200.

Argument marshalling only: every step of the layer runs in the CUDA kernels of
``libsalad.so`` (built by ``python -m sparse_linear_hybrid_b200.build``).
PyTorch supplies device memory and streams.  There is no CPU fallback: calls
raise if the library is missing or a tensor is not on a CUDA device.

The entry points mirror ``include/salad.h``:
    mask_num_blocks, build_block_mask, validate_mask, tile_num_blocks, build_tile_mask, build_topk_mask,
    workspace_bytes, attn_forward, attn_forward_lse, attn_forward_heads, attn_forward_tiles, attn_forward_static,
    attn_backward_sparse,
    attn_backward, gate_forward, rope_inv_freq, rope_forward, rope_backward, ckpt_pack, ckpt_unpack,
    new_ckpt_backward_workspace, attn_backward_ckpt, new_diff_workspace, diff_attn_forward, diff_attn_forward_lse,
    diff_attn_backward, diff_attn_decode, linear_state, check_status, set_wait_limit_ns, set_max_ctas, set_phase_events,
    status_string
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import functools
import inspect
import math
import os
import struct

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsalad.so")
_lib = None

SALAD_OK = 0
SALAD_ERR_INVALID_ARG = -1
SALAD_ERR_UNSUPPORTED = -2
SALAD_ERR_CAPACITY = -3
SALAD_ERR_WORKSPACE = -4
SALAD_ERR_CUDA = -5
SALAD_ERR_DEVICE_TIMEOUT = -6
SALAD_ERR_OUT_OF_MEMORY = -7
SALAD_ERR_BAD_MASK = -8


# salad_type and salad_ckpt_format
_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_FORMATS = {"int8": 0, "e4m3": 1}


# salad_rope_tensor and salad_ckpt_tensor as bytes (a fraction of what filling ctypes structures costs a small call)
_ROPE_TENSOR = struct.Struct("PPi4x6q").pack
_CKPT_TENSOR = struct.Struct("PqPP").pack
_INT3 = struct.Struct("3i").pack
_NULL = contextlib.nullcontext()
_INT_MAX = 0x7FFFFFFF


class SaladError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libsalad.so (raises when it has not been built)."""
    global _lib
    if _lib is None:
        # SALAD_LIBRARY selects another build of the same library (the profiling
        # build libsalad_profile.so, the checking build libsalad_debug.so); by
        # default the in-tree libsalad.so
        path = os.environ.get("SALAD_LIBRARY") or LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -m sparse_linear_hybrid_b200.build`")
        L = ctypes.CDLL(path)
        i, p, f, sz = ctypes.c_int, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
        L.salad_mask_num_blocks.argtypes = [i, i, i, i, ctypes.POINTER(i)]
        L.salad_mask_num_blocks.restype = i
        L.salad_build_block_mask.argtypes = [i, i, i, i, i, p, p, p, ctypes.c_int64,
                                             ctypes.POINTER(ctypes.c_int64), p]
        L.salad_build_block_mask.restype = i
        L.salad_tile_num_blocks.argtypes = [i, i, i, i, i, i, ctypes.POINTER(i)]
        L.salad_tile_num_blocks.restype = i
        L.salad_build_tile_mask.argtypes = [i, i, i, i, i, i, i, p, p, p, ctypes.c_int64,
                                            ctypes.POINTER(ctypes.c_int64), p]
        L.salad_build_tile_mask.restype = i
        L.salad_transpose_block_mask.argtypes = [p, p, i, i, p, p, p]
        L.salad_transpose_block_mask.restype = i
        L.salad_validate_mask.argtypes = [p, p, ctypes.c_int64, i, ctypes.POINTER(ctypes.c_int64)]
        L.salad_validate_mask.restype = i
        L.salad_workspace_bytes.argtypes = [i, i, i, i]
        L.salad_workspace_bytes.restype = sz
        L.salad_attn_forward.argtypes = [p, p, p, i, i, i, i, i, p, p, p, p, f, f, p, p, sz, p]
        L.salad_attn_forward.restype = i
        L.salad_attn_forward_bh.argtypes = [p, p, p, i, i, i, i, i, p, p, p, p, f, f, p, p, sz, p]
        L.salad_attn_forward_bh.restype = i
        L.salad_attn_forward_lse.argtypes = [p, p, p, i, i, i, i, i, p, p, p, p, f, f, i, p, p, p, sz, p]
        L.salad_attn_forward_lse.restype = i
        L.salad_attn_forward_heads.argtypes = [p, p, p, i, i, i, i, i, i, i, p, p, p, p, f, f, p, p, sz, p]
        L.salad_attn_forward_heads.restype = i
        L.salad_attn_forward_host.argtypes = [p, p, p, p, i, i, i, i, i, p, p, p, p, f, f, i, p, p, p, p, p, sz, p, p,
                                              p]
        L.salad_attn_forward_host.restype = i
        L.salad_backward_workspace_bytes.argtypes = [i, i, i]
        L.salad_backward_workspace_bytes.restype = sz
        L.salad_attn_backward_sparse.argtypes = [p, p, p, p, p, p, i, i, i, i, i, p, p, p, p, i, f, p, p, p, p, sz,
                                                 p]
        L.salad_attn_backward_sparse.restype = i
        L.salad_layer_backward_workspace_bytes.argtypes = [i, i, i, i]
        L.salad_layer_backward_workspace_bytes.restype = sz
        L.salad_attn_backward.argtypes = [p, p, p, p, p, p, i, i, i, i, i, p, p, p, p, i, p, p, f, f, p, p, p, p, p,
                                          p, sz, p]
        L.salad_attn_backward.restype = i
        L.salad_attn_forward_tiles.argtypes = [p, p, p, i, i, i, i, i, i, i, i, i, p, p, p, p, f, f, p, p, sz,
                                               p]
        L.salad_attn_forward_tiles.restype = i
        L.salad_gate_workspace_bytes.argtypes = [i, i, i, i]
        L.salad_gate_workspace_bytes.restype = sz
        L.salad_gate_forward.argtypes = [p, i, i, i, i, p, i, p, p, p, f, p, p, p, sz, p]
        L.salad_gate_forward.restype = i
        L.salad_topk_workspace_bytes.argtypes = [i, i, i, i, i]
        L.salad_topk_workspace_bytes.restype = sz
        L.salad_build_topk_mask.argtypes = [p, p, i, i, i, i, i, i, p, p, p, sz, p]
        L.salad_build_topk_mask.restype = i
        L.salad_attn_forward_static.argtypes = [p, p, p, i, i, i, i, i, p, p, p, p, f, f, p, p]
        L.salad_attn_forward_static.restype = i
        L.salad_rope.argtypes = [p, i, i, i, i, i, i, i, i, p, p, i, p, ctypes.c_int64, i, i, p, f, i, p]
        L.salad_rope.restype = i
        for fn in (L.salad_ckpt_pack, L.salad_ckpt_unpack):
            fn.argtypes = [p, i, i, i, i, i, p]
            fn.restype = i
        L.salad_ckpt_backward_workspace_bytes.argtypes = [i, i, i, i]
        L.salad_ckpt_backward_workspace_bytes.restype = sz
        L.salad_attn_backward_ckpt.argtypes = ([p] * 6 + [i, p] + [i] * 5 + [p] * 4 + [i, p, p, f, f] + [p] * 6
                                               + [sz, p])
        L.salad_attn_backward_ckpt.restype = i
        L.salad_diff_workspace_bytes.argtypes = [i, i, i, i]
        L.salad_diff_workspace_bytes.restype = sz
        L.salad_diff_forward.argtypes = [p] * 3 + [i] * 5 + [p, p, i, p, i, f, p, p, p, p, sz, p]
        L.salad_diff_forward.restype = i
        L.salad_diff_backward.argtypes = [p] * 7 + [i] * 5 + [p] * 4 + [i, p, i, f] + [p] * 5 + [sz, p]
        L.salad_diff_backward.restype = i
        L.salad_diff_decode.argtypes = [p] * 3 + [i] * 5 + [p, p, i, f, p, p]
        L.salad_diff_decode.restype = i
        L.salad_linear_state.argtypes = [p, p, i, i, i, i, p, p, p, p, sz, p]
        L.salad_linear_state.restype = i
        L.salad_check_status.argtypes = [p, p]
        L.salad_check_status.restype = i
        L.salad_check_status_static.argtypes = [p]
        L.salad_check_status_static.restype = i
        L.salad_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
        L.salad_set_wait_limit_ns.restype = None
        L.salad_set_max_ctas.argtypes = [i]
        L.salad_set_max_ctas.restype = None
        L.salad_set_phase_events.argtypes = [p, p, p]
        L.salad_set_phase_events.restype = None
        L.salad_profile_set_buffer.argtypes = [p, sz]
        L.salad_profile_set_buffer.restype = i
        L.salad_status_string.argtypes = [i]
        L.salad_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().salad_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != SALAD_OK:
        raise SaladError(status, what)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:  # (the current stream's handle without a Stream object around it)
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()))
    return ctypes.c_void_p(stream.cuda_stream)


def _dev_ptr(t: torch.Tensor, dtype, name: str) -> ctypes.c_void_p:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor (libsalad has no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _host_ptr(t: torch.Tensor, dtype, name: str) -> ctypes.c_void_p:
    if not isinstance(t, torch.Tensor) or t.is_cuda:
        raise TypeError(f"{name} must be a host (CPU) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _of_its_stream(fn):
    """Makes a `stream` given to fn the current one: what the call allocates (outputs,
    workspace, the transposed mask) and launches beside the library's kernels is then of
    that stream, in order with them, and is not given out again while they use it."""
    at = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def call(*args, **kw):
        stream = args[at] if len(args) > at else kw.get("stream")
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


_copy_streams = {}


def mask_num_blocks(T: int, H: int, W: int, block: int) -> int:
    nb = ctypes.c_int(0)
    _check(lib().salad_mask_num_blocks(T, H, W, block, ctypes.byref(nb)), "salad_mask_num_blocks")
    return nb.value


def _build_csr(name, nb, heads, call, device):
    """Size-then-fill of a window mask CSR through `call(row_ptr, col_idx, cap, nnz)`."""
    device = torch.device("cuda") if device is None else torch.device(device)
    row_ptr = torch.empty(heads * nb + 1, dtype=torch.int32, device=device)
    nnz = ctypes.c_int64(0)
    st = call(_dev_ptr(row_ptr, torch.int32, "row_ptr"), None, 0, nnz)
    if st not in (SALAD_OK, SALAD_ERR_CAPACITY):
        _check(st, name)
    col_idx = torch.empty(max(int(nnz.value), 1), dtype=torch.int32, device=device)
    _check(call(_dev_ptr(row_ptr, torch.int32, "row_ptr"), _dev_ptr(col_idx, torch.int32, "col_idx"),
                col_idx.numel(), nnz), name)
    return row_ptr, col_idx[:int(nnz.value)]


@_of_its_stream
def build_block_mask(T: int, H: int, W: int, block: int, windows, device=None, stream=None):
    """ST-SWA block mask as a per-head CSR: (row_ptr, col_idx) int32 CUDA tensors."""
    win = np.ascontiguousarray(windows, dtype=np.int32).reshape(-1, 3)
    s = _stream(stream)

    def call(rp, ci, cap, nnz):
        return lib().salad_build_block_mask(T, H, W, block, win.shape[0], win.ctypes.data_as(ctypes.c_void_p),
                                            rp, ci, cap, ctypes.byref(nnz), s)
    return _build_csr("salad_build_block_mask", mask_num_blocks(T, H, W, block), win.shape[0], call, device)


def validate_mask(row_ptr, col_idx, nb: int) -> int:
    """Host check of a CSR mask (see salad.h): returns -1 when valid, else the
    first offending row.  Accepts numpy arrays or tensors (copied to the host)."""
    rp = np.ascontiguousarray(row_ptr.cpu().numpy() if hasattr(row_ptr, "cpu") else row_ptr, dtype=np.int32)
    ci = np.ascontiguousarray(col_idx.cpu().numpy() if hasattr(col_idx, "cpu") else col_idx, dtype=np.int32)
    bad = ctypes.c_int64(-1)
    cols = ci.ctypes.data_as(ctypes.c_void_p) if ci.size else None
    lib().salad_validate_mask(rp.ctypes.data_as(ctypes.c_void_p), cols, len(rp) - 1, int(nb), ctypes.byref(bad))
    return int(bad.value)


def tile_num_blocks(T: int, H: int, W: int, tile) -> int:
    bt, bh, bw = tile
    nb = ctypes.c_int(0)
    _check(lib().salad_tile_num_blocks(T, H, W, bt, bh, bw, ctypes.byref(nb)), "salad_tile_num_blocks")
    return nb.value


@_of_its_stream
def build_tile_mask(T: int, H: int, W: int, tile, windows, device=None, stream=None):
    """ST-SWA mask over bt x bh x bw boxes of the grid: per-head CSR (row_ptr, col_idx)."""
    bt, bh, bw = tile
    win = np.ascontiguousarray(windows, dtype=np.int32).reshape(-1, 3)
    s = _stream(stream)

    def call(rp, ci, cap, nnz):
        return lib().salad_build_tile_mask(T, H, W, bt, bh, bw, win.shape[0],
                                           win.ctypes.data_as(ctypes.c_void_p), rp, ci, cap,
                                           ctypes.byref(nnz), s)
    return _build_csr("salad_build_tile_mask", tile_num_blocks(T, H, W, tile), win.shape[0], call, device)


def workspace_bytes(B: int, N: int, heads: int, d: int) -> int:
    n = lib().salad_workspace_bytes(B, N, heads, d)
    if n == 0:
        raise SaladError(SALAD_ERR_INVALID_ARG, "salad_workspace_bytes")
    return int(n)


def new_workspace(B: int, N: int, heads: int, d: int, device=None) -> torch.Tensor:
    """A zero-filled workspace of the size salad_attn_forward needs."""
    device = torch.device("cuda") if device is None else torch.device(device)
    return torch.zeros(workspace_bytes(B, N, heads, d), dtype=torch.uint8, device=device)


@_of_its_stream
def attn_forward(q, k, v, row_ptr, col_idx, w_proj, gate, block: int, softmax_scale: float = 0.0,
                 eps: float = 1e-6, out=None, workspace=None, stream=None, mask_per_bh: bool = False) -> torch.Tensor:
    """out = block-sparse attention + gate * (ReLU linear attention @ w_proj).

    q, k, v: bf16 CUDA [B, N, Hh, d]; w_proj bf16 [d, d]; gate fp32 [B, Hh].
    The mask's rows are per head (build_block_mask), or per (b, h) with
    mask_per_bh (build_topk_mask).
    """
    B, N, Hh, d = q.shape
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = new_workspace(B, N, Hh, d, q.device)
    fn = lib().salad_attn_forward_bh if mask_per_bh else lib().salad_attn_forward
    _check(fn(
        _dev_ptr(q, torch.bfloat16, "q"), _dev_ptr(k, torch.bfloat16, "k"), _dev_ptr(v, torch.bfloat16, "v"),
        B, N, Hh, d, block, _dev_ptr(row_ptr, torch.int32, "row_ptr"),
        _dev_ptr(col_idx, torch.int32, "col_idx"), _dev_ptr(w_proj, torch.bfloat16, "w_proj"),
        _dev_ptr(gate, torch.float32, "gate"), float(softmax_scale), float(eps),
        _dev_ptr(out, torch.bfloat16, "out"), _dev_ptr(workspace, torch.uint8, "workspace"),
        workspace.numel(), _stream(stream)), "salad_attn_forward")
    return out


@_of_its_stream
def attn_forward_lse(q, k, v, row_ptr, col_idx, w_proj, gate, block: int, softmax_scale: float = 0.0,
                     eps: float = 1e-6, out=None, lse=None, workspace=None, stream=None, mask_per_bh: bool = False):
    """attn_forward that also returns each row's log-sum-exp of the sparse softmax
    (natural log, fp32 [B, Hh, N]): (out, lse)."""
    B, N, Hh, d = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, Hh, N, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = new_workspace(B, N, Hh, d, q.device)
    _check(lib().salad_attn_forward_lse(
        _dev_ptr(q, torch.bfloat16, "q"), _dev_ptr(k, torch.bfloat16, "k"), _dev_ptr(v, torch.bfloat16, "v"),
        B, N, Hh, d, block, _dev_ptr(row_ptr, torch.int32, "row_ptr"),
        _dev_ptr(col_idx, torch.int32, "col_idx"), _dev_ptr(w_proj, torch.bfloat16, "w_proj"),
        _dev_ptr(gate, torch.float32, "gate"), float(softmax_scale), float(eps), int(bool(mask_per_bh)),
        _dev_ptr(out, torch.bfloat16, "out"), _dev_ptr(lse, torch.float32, "lse"),
        _dev_ptr(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)), "salad_attn_forward_lse")
    return out, lse


@_of_its_stream
def attn_forward_heads(q, k, v, head_begin: int, head_count: int, row_ptr, col_idx, w_proj, gate, block: int,
                       softmax_scale: float = 0.0, eps: float = 1e-6, out=None, workspace=None,
                       stream=None) -> torch.Tensor:
    """attn_forward on heads [head_begin, head_begin + head_count) of full
    [B, N, Hh, d] tensors (one rank's share of a head-parallel layer): the mask
    holds the range's heads, gate is fp32 [B, head_count]; out (full shape) is
    written on those heads only."""
    B, N, Hh, d = q.shape
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = new_workspace(B, N, head_count, d, q.device)
    _check(lib().salad_attn_forward_heads(
        _dev_ptr(q, torch.bfloat16, "q"), _dev_ptr(k, torch.bfloat16, "k"), _dev_ptr(v, torch.bfloat16, "v"),
        B, N, Hh, int(head_begin), int(head_count), d, block, _dev_ptr(row_ptr, torch.int32, "row_ptr"),
        _dev_ptr(col_idx, torch.int32, "col_idx"), _dev_ptr(w_proj, torch.bfloat16, "w_proj"),
        _dev_ptr(gate, torch.float32, "gate"), float(softmax_scale), float(eps),
        _dev_ptr(out, torch.bfloat16, "out"), _dev_ptr(workspace, torch.uint8, "workspace"),
        workspace.numel(), _stream(stream)), "salad_attn_forward_heads")
    return out


@_of_its_stream
def transpose_block_mask(row_ptr, col_idx, groups: int, nb: int, stream=None):
    """The transposed mask on the GPU (salad_transpose_block_mask): for every
    group (head, or (b, h)) and key block J, the ascending query blocks whose
    row keeps J.  Returns (t_row_ptr, t_col_idx), int32 CUDA tensors."""
    t_row_ptr = torch.empty(groups * nb + 1, dtype=torch.int32, device=row_ptr.device)
    t_col_idx = torch.empty(max(1, col_idx.numel()), dtype=torch.int32, device=row_ptr.device)
    _check(lib().salad_transpose_block_mask(
        _dev_ptr(row_ptr, torch.int32, "row_ptr"), _dev_ptr(col_idx, torch.int32, "col_idx"), int(groups), int(nb),
        _dev_ptr(t_row_ptr, torch.int32, "t_row_ptr"), _dev_ptr(t_col_idx, torch.int32, "t_col_idx"),
        _stream(stream)), "salad_transpose_block_mask")
    return t_row_ptr, t_col_idx[:col_idx.numel()]


def _transposed_mask(row_ptr, col_idx, t_row_ptr, t_col_idx, build, groups=0, nb=0):
    """The transposed mask the backward walks for dk and dv: given, or with `build`
    built on the GPU (always for a mask with rows per (b, h), such as Top-K's, which
    is not symmetric), or the mask itself, as for the symmetric window masks."""
    if (t_row_ptr is None) != (t_col_idx is None):
        raise ValueError("give both t_row_ptr and t_col_idx, or neither")
    if t_row_ptr is None:
        if build:
            return transpose_block_mask(row_ptr, col_idx, groups, nb)
        return row_ptr, col_idx
    return t_row_ptr, t_col_idx


@_of_its_stream
def attn_backward_sparse(q, k, v, o, dout, lse, row_ptr, col_idx, block: int = 128, t_row_ptr=None,
                         t_col_idx=None, softmax_scale: float = 0.0, mask_per_bh: bool = False, workspace=None,
                         stream=None):
    """Gradients of the sparse branch (see salad.h): (dq, dk, dv) fp32 [B, N, Hh, d].
    o is the branch output and lse the forward's log-sum-exp (attn_forward_lse);
    the transposed mask defaults to the mask itself, which is right for the
    symmetric window masks; a mask with rows per (b, h) needs its transpose."""
    B, N, Hh, d = q.shape
    t_row_ptr, t_col_idx = _transposed_mask(row_ptr, col_idx, t_row_ptr, t_col_idx, mask_per_bh, B * Hh,
                                            (N + block - 1) // block)
    grads = [torch.empty(B, N, Hh, d, dtype=torch.float32, device=q.device) for _ in range(3)]
    if workspace is None:
        workspace = torch.zeros(lib().salad_backward_workspace_bytes(B, N, Hh), dtype=torch.uint8, device=q.device)
    i32 = lambda t, name: _dev_ptr(t, torch.int32, name)  # noqa: E731
    _check(lib().salad_attn_backward_sparse(
        _dev_ptr(q, torch.bfloat16, "q"), _dev_ptr(k, torch.bfloat16, "k"), _dev_ptr(v, torch.bfloat16, "v"),
        _dev_ptr(o, torch.bfloat16, "o"), _dev_ptr(dout, torch.bfloat16, "dout"), _dev_ptr(lse, torch.float32, "lse"),
        B, N, Hh, d, int(block), i32(row_ptr, "row_ptr"), i32(col_idx, "col_idx"), i32(t_row_ptr, "t_row_ptr"),
        i32(t_col_idx, "t_col_idx"), int(bool(mask_per_bh)), float(softmax_scale),
        *[_dev_ptr(g, torch.float32, n) for g, n in zip(grads, ("dq", "dk", "dv"))],
        _dev_ptr(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)),
        "salad_attn_backward_sparse")
    return tuple(grads)


@_of_its_stream
def attn_backward(q, k, v, out, dout, lse, row_ptr, col_idx, w_proj, gate, block: int = 128, t_row_ptr=None,
                  t_col_idx=None, softmax_scale: float = 0.0, eps: float = 1e-6, mask_per_bh: bool = False,
                  workspace=None, stream=None):
    """Gradients of the whole layer (see salad.h): dict of fp32 CUDA tensors dq, dk,
    dv [B, N, Hh, d], dw [d, d] and dgate [B, Hh].  out and lse come from
    attn_forward_lse on the same inputs."""
    B, N, Hh, d = q.shape
    t_row_ptr, t_col_idx = _transposed_mask(row_ptr, col_idx, t_row_ptr, t_col_idx, mask_per_bh, B * Hh,
                                            (N + block - 1) // block)
    res = {n: torch.empty(B, N, Hh, d, dtype=torch.float32, device=q.device) for n in ("dq", "dk", "dv")}
    res["dw"] = torch.empty(d, d, dtype=torch.float32, device=q.device)
    res["dgate"] = torch.empty(B, Hh, dtype=torch.float32, device=q.device)
    if workspace is None:
        n = lib().salad_layer_backward_workspace_bytes(B, N, Hh, d)
        if n == 0:
            raise SaladError(SALAD_ERR_INVALID_ARG, "salad_layer_backward_workspace_bytes")
        workspace = torch.zeros(n, dtype=torch.uint8, device=q.device)
    i32 = lambda t, name: _dev_ptr(t, torch.int32, name)  # noqa: E731
    f32 = lambda name: _dev_ptr(res[name], torch.float32, name)  # noqa: E731
    _check(lib().salad_attn_backward(
        _dev_ptr(q, torch.bfloat16, "q"), _dev_ptr(k, torch.bfloat16, "k"), _dev_ptr(v, torch.bfloat16, "v"),
        _dev_ptr(out, torch.bfloat16, "out"), _dev_ptr(dout, torch.bfloat16, "dout"),
        _dev_ptr(lse, torch.float32, "lse"), B, N, Hh, d, int(block), i32(row_ptr, "row_ptr"),
        i32(col_idx, "col_idx"), i32(t_row_ptr, "t_row_ptr"), i32(t_col_idx, "t_col_idx"), int(bool(mask_per_bh)),
        _dev_ptr(w_proj, torch.bfloat16, "w_proj"), _dev_ptr(gate, torch.float32, "gate"), float(softmax_scale),
        float(eps), f32("dq"), f32("dk"), f32("dv"), f32("dw"), f32("dgate"),
        _dev_ptr(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)), "salad_attn_backward")
    return res


@_of_its_stream
def attn_forward_host(q, k, v, row_ptr, col_idx, w_proj, gate, block: int, out=None, staging=None,
                      heads_per_chunk: int = 0, softmax_scale: float = 0.0, eps: float = 1e-6, workspace=None,
                      stream=None, copy_streams=None, device=None):
    """The layer forward on host tensors (see salad_attn_forward_host): q, k, v
    bf16 CPU [B, N, Hh, d] (pinned for the copies to overlap the compute), the
    mask, w_proj and gate on the GPU.  `staging` is (q_dev, k_dev, v_dev, out_dev)
    bf16 CUDA tensors of the same shape (allocated when None); `copy_streams` two
    CUDA streams for the copies (two per device are kept for reuse when None).
    Returns the host output tensor (pinned when allocated here)."""
    B, N, Hh, d = q.shape
    dev = torch.device("cuda") if device is None else torch.device(device)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16).pin_memory()
    if staging is None:
        staging = tuple(torch.empty(q.shape, dtype=torch.bfloat16, device=dev) for _ in range(4))
    if copy_streams is None:
        key = dev.index if dev.index is not None else torch.cuda.current_device()
        if key not in _copy_streams:
            _copy_streams[key] = (torch.cuda.Stream(device=key), torch.cuda.Stream(device=key))
        copy_streams = _copy_streams[key]
    hpc = int(heads_per_chunk) if heads_per_chunk > 0 else (Hh + 5) // 6
    if workspace is None:
        workspace = new_workspace(1, N, min(hpc, Hh), d, dev)
    h = lambda t, n: _host_ptr(t, torch.bfloat16, n)  # noqa: E731
    g = lambda t, n: _dev_ptr(t, torch.bfloat16, n)  # noqa: E731
    _check(lib().salad_attn_forward_host(
        h(q, "q"), h(k, "k"), h(v, "v"), h(out, "out"), B, N, Hh, d, int(block),
        _dev_ptr(row_ptr, torch.int32, "row_ptr"), _dev_ptr(col_idx, torch.int32, "col_idx"),
        g(w_proj, "w_proj"), _dev_ptr(gate, torch.float32, "gate"), float(softmax_scale), float(eps),
        int(heads_per_chunk), g(staging[0], "q_dev"), g(staging[1], "k_dev"), g(staging[2], "v_dev"),
        g(staging[3], "out_dev"), _dev_ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
        _stream(stream), _stream(copy_streams[0]), _stream(copy_streams[1])), "salad_attn_forward_host")
    return out


@_of_its_stream
def attn_forward_tiles(q, k, v, grid, tile, row_ptr, col_idx, w_proj, gate, softmax_scale: float = 0.0,
                       eps: float = 1e-6, out=None, workspace=None, stream=None) -> torch.Tensor:
    """attn_forward with 3-D tile blocks: grid = (T, H, W), tile = (bt, bh, bw)
    with bt * bh * bw == 128; the mask from build_tile_mask."""
    B, N, Hh, d = q.shape
    T, H, W = grid
    bt, bh, bw = tile
    if N != T * H * W:
        raise ValueError(f"q has {N} tokens, the grid {T * H * W}")
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = new_workspace(B, N, Hh, d, q.device)
    _check(lib().salad_attn_forward_tiles(
        _dev_ptr(q, torch.bfloat16, "q"), _dev_ptr(k, torch.bfloat16, "k"), _dev_ptr(v, torch.bfloat16, "v"),
        B, T, H, W, bt, bh, bw, Hh, d, _dev_ptr(row_ptr, torch.int32, "row_ptr"),
        _dev_ptr(col_idx, torch.int32, "col_idx"), _dev_ptr(w_proj, torch.bfloat16, "w_proj"),
        _dev_ptr(gate, torch.float32, "gate"), float(softmax_scale), float(eps),
        _dev_ptr(out, torch.bfloat16, "out"), _dev_ptr(workspace, torch.uint8, "workspace"),
        workspace.numel(), _stream(stream)), "salad_attn_forward_tiles")
    return out


@_of_its_stream
def gate_forward(q, t_emb, w_t, w_x, beta, threshold: float, gate_out=None, s_out=None, workspace=None,
                 stream=None) -> torch.Tensor:
    """Dynamic gate with branch dropping (see salad.h): fp32 [B, Hh] CUDA tensor,
    0 where the sigmoid gate falls below `threshold`.  t_emb fp32 [B, E], w_t
    [Hh, E], w_x [Hh, d], beta [Hh]."""
    B, N, Hh, d = q.shape
    E = t_emb.shape[1] if t_emb is not None else 0
    if gate_out is None:
        gate_out = torch.empty(B, Hh, dtype=torch.float32, device=q.device)
    if workspace is None:
        n = lib().salad_gate_workspace_bytes(B, N, Hh, d)
        if n == 0:
            raise SaladError(SALAD_ERR_INVALID_ARG, "salad_gate_workspace_bytes")
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    opt = lambda t, name: None if t is None else _dev_ptr(t, torch.float32, name)  # noqa: E731
    _check(lib().salad_gate_forward(
        _dev_ptr(q, torch.bfloat16, "q"), B, N, Hh, d, opt(t_emb, "t_emb"), E, opt(w_t, "w_t"),
        _dev_ptr(w_x, torch.float32, "w_x"), _dev_ptr(beta, torch.float32, "beta"), float(threshold),
        opt(s_out, "s_out"), _dev_ptr(gate_out, torch.float32, "gate_out"),
        _dev_ptr(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)), "salad_gate_forward")
    return gate_out


@_of_its_stream
def build_topk_mask(q, k, block: int, keep: int, workspace=None, stream=None):
    """Top-K dynamic block mask (see salad.h) as a per-(b, h) CSR: (row_ptr,
    col_idx) int32 CUDA tensors, min(keep, nb) ascending key blocks per row."""
    B, N, Hh, d = q.shape
    nb = (N + block - 1) // block
    kk = min(int(keep), nb)
    row_ptr = torch.empty(B * Hh * nb + 1, dtype=torch.int32, device=q.device)
    col_idx = torch.empty(max(B * Hh * nb * kk, 1), dtype=torch.int32, device=q.device)
    if workspace is None:
        n = lib().salad_topk_workspace_bytes(B, N, Hh, d, block)
        if n == 0:
            raise SaladError(SALAD_ERR_INVALID_ARG, "salad_topk_workspace_bytes")
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    _check(lib().salad_build_topk_mask(
        _dev_ptr(q, torch.bfloat16, "q"), _dev_ptr(k, torch.bfloat16, "k"), B, N, Hh, d, int(block), int(keep),
        _dev_ptr(row_ptr, torch.int32, "row_ptr"), _dev_ptr(col_idx, torch.int32, "col_idx"),
        _dev_ptr(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)),
        "salad_build_topk_mask")
    return row_ptr, col_idx[:B * Hh * nb * kk]


@_of_its_stream
def attn_forward_static(q, k, v, row_ptr, col_idx, w_proj, gate, block: int, softmax_scale: float = 0.0,
                        eps: float = 1e-6, out=None, stream=None) -> torch.Tensor:
    """attn_forward for callers that cannot allocate device memory: the
    scratch is the library's static device array (see salad.h)."""
    B, N, Hh, d = q.shape
    if out is None:
        out = torch.empty_like(q)
    _check(lib().salad_attn_forward_static(
        _dev_ptr(q, torch.bfloat16, "q"), _dev_ptr(k, torch.bfloat16, "k"), _dev_ptr(v, torch.bfloat16, "v"),
        B, N, Hh, d, block, _dev_ptr(row_ptr, torch.int32, "row_ptr"),
        _dev_ptr(col_idx, torch.int32, "col_idx"), _dev_ptr(w_proj, torch.bfloat16, "w_proj"),
        _dev_ptr(gate, torch.float32, "gate"), float(softmax_scale), float(eps),
        _dev_ptr(out, torch.bfloat16, "out"), _stream(stream)), "salad_attn_forward_static")
    return out


def _on(*tensors):
    """(context that makes the tensors' device current, that device); all have to be on one CUDA device."""
    dev = None
    for t in tensors:
        try:
            d = t.get_device()  # (-1: not a CUDA tensor)
        except AttributeError:
            d = -1
        if d != dev:
            if d < 0:
                raise TypeError("the tensors must be CUDA tensors (libsalad has no CPU path)")
            if dev is not None:
                raise ValueError(f"the tensors lie on several devices: cuda:{dev} and cuda:{d}")
            dev = d
    return (_NULL if dev == torch._C._cuda_getDevice() else torch.cuda.device(dev)), tensors[0].device


def _at(ctx, dev, stream):
    """_on's context, or with a stream of the caller's the one that makes it
    current: outputs and workspaces that the call allocates are then of that
    stream, and are not given out again while its kernels use them."""
    if stream is None:
        return ctx
    if stream.device != dev:
        raise ValueError(f"the stream is of {stream.device}, the tensors of {dev}")
    return torch.cuda.stream(stream)


def _ptr(t, dtype, name) -> int:
    """_dev_ptr's checks for a tensor that _on has seen; the bare address."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _int32(name, *sizes):
    """Refuses sizes that the C interface's int would silently cut."""
    if max(sizes) > _INT_MAX:
        raise SaladError(SALAD_ERR_UNSUPPORTED, f"{name}: sizes {sizes}")


def _new_like(x, dtype):
    """Contiguous memory of x's shape."""
    return torch.empty_like(x, dtype=dtype, memory_format=torch.contiguous_format)


def rope_inv_freq(rot: int, base: float = 10000.0, sections=None, scaling: str | None = None, factor: float = 1.0,
                  original_length: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """(frequencies fp64 CUDA [rot/2], scale) of rotary positions.

    Every axis with n = sections[a] pairs has base^(-j/n), j = 0 ... n-1 (sections
    sum to rot/2; one axis by default).  Long contexts, `factor` times the trained
    length: "linear" divides every frequency by it; "ntk" raises the base by
    factor^(n/(n-1)), so that the slowest pair is divided by it and the fastest
    kept; "yarn" keeps pairs that turn more than beta_fast times within
    original_length tokens, divides those below beta_slow turns, blends between,
    and scales the turned pairs by 0.1 ln(factor) + 1."""
    sections = [rot // 2] if sections is None else [int(n) for n in sections]
    if rot < 2 or rot % 2 or min(sections) < 0 or sum(sections) != rot // 2:
        raise ValueError(f"sections {sections} do not sum to rot / 2 = {rot / 2}")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if not (base > 0 and factor >= 1 and math.isfinite(base) and math.isfinite(factor)):
        raise ValueError("base must be positive and factor at least 1")
    if scaling == "yarn" and not (original_length > 0 and beta_fast > beta_slow > 0):
        raise ValueError("yarn needs original_length > 0 and beta_fast > beta_slow > 0")
    freq, scale = [], 1.0
    for n in sections:
        b = base * factor ** (n / (n - 1)) if scaling == "ntk" and n > 1 else base
        f = np.float64(b) ** (-np.arange(n, dtype=np.float64) / max(n, 1))
        if scaling == "linear":
            f = f / factor
        elif scaling == "yarn":
            keep = np.clip((original_length * f / (2 * math.pi) - beta_slow) / (beta_fast - beta_slow), 0, 1)
            f = f * keep + f / factor * (1 - keep)
            scale = 0.1 * math.log(factor) + 1.0
        freq.append(f)
    device = torch.device("cuda") if device is None else torch.device(device)
    return torch.from_numpy(np.concatenate(freq)).to(device), scale


def _rope(q, k, inv_freq, sections, interleaved, scale, positions, grid, origin, q_out, k_out, out_dtype, inverse,
          stream):
    xs = (q,) if k is None else (q, k)
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    ctx, dev = _on(*xs, inv_freq) if positions is None else _on(*xs, inv_freq, positions)
    if q.dim() != 4:
        raise ValueError("q and k must be [B, N, heads, d] with the same B, N and d")
    B, N, _, d = q.shape
    if q.numel() > _INT_MAX:
        _int32("salad_rope", *q.shape)
    kind = q.dtype
    if kind not in _TYPES or (out_dtype is not None and out_dtype not in _TYPES):
        raise TypeError("q, k and the outputs must be fp32, bf16 or fp16")
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise TypeError("inv_freq must be a contiguous fp64 vector")
    rot = 2 * inv_freq.numel()
    sections = [rot // 2] if sections is None else [int(n) for n in sections]
    axes = len(sections)
    if not 1 <= axes <= 3:
        raise ValueError("one to three sections")
    pos_ptr, pos_b, gh, gw = None, 0, 1, 1
    if positions is not None:
        if grid is not None:
            raise ValueError("give positions or a grid, not both")
        if positions.dtype != torch.int32:
            raise TypeError(f"positions must be int32, got {positions.dtype}")
        shape = tuple(positions.shape)
        one = (N,) if axes == 1 else (N, axes)
        if shape not in (one, (1, *one), (B, *one)) or not positions.is_contiguous():
            raise ValueError(f"positions must be contiguous [B, N{', axes' if axes > 1 else ''}] or without B")
        pos_ptr, pos_b = positions.data_ptr(), (N * axes if len(shape) > len(one) and shape[0] > 1 else 0)
    elif grid is not None:
        T, gh, gw = (int(n) for n in grid)
        if axes != 3 or T * gh * gw != N:
            raise ValueError(f"a grid needs three sections and {T} * {gh} * {gw} tokens, got {axes} and {N}")
    elif axes != 1:
        raise ValueError("several sections need positions or a grid")
    ys, packed = [], b""
    with _at(ctx, dev, stream):
        for x, y in zip(xs, (q_out, k_out)):
            if x.dim() != 4 or x.shape[0] != B or x.shape[1] != N or x.shape[3] != d:
                raise ValueError("q and k must be [B, N, heads, d] with the same B, N and d")
            if x.dtype != kind:
                raise TypeError("q and k must share one of fp32, bf16, fp16")
            if y is None:
                y = _new_like(x, out_dtype or (ys[0].dtype if ys else kind))
            else:
                _on(q, y)
                if y.shape != x.shape or y.dtype not in _TYPES or (ys and y.dtype != ys[0].dtype):
                    raise ValueError("outputs must have their input's shape, and one type")
                if out_dtype is not None and y.dtype != out_dtype:
                    raise TypeError(f"the output is {y.dtype}, not {out_dtype}")
            xb, xn, xh, xf = x.stride()
            yb, yn, yh, yf = y.stride()
            if d > 1 and (xf != 1 or yf != 1):
                raise ValueError("the features of a head must be contiguous")
            packed += _ROPE_TENSOR(x.data_ptr(), y.data_ptr(), x.shape[2], xb, xn, xh, yb, yn, yh)
            ys.append(y)
        if B and N:
            o = tuple(origin)
            _check(lib().salad_rope(packed, len(xs), _TYPES[kind], _TYPES[ys[0].dtype], B, N, d, rot, bool(interleaved),
                                    inv_freq.data_ptr(), _INT3(*sections, *(0,) * (3 - axes)), axes, pos_ptr, pos_b, gh,
                                    gw, _INT3(*o, *(0,) * (3 - len(o))), scale, inverse, _stream(stream)), "salad_rope")
    return ys


def rope_forward(q, k, inv_freq, sections=None, interleaved: bool = False, scale: float = 1.0, positions=None,
                 grid=None, origin=(0, 0, 0), q_out=None, k_out=None, out_dtype=None, stream=None):
    """q and k (k may be None) turned by their tokens' positions (see salad_rope): (q_out, k_out).

    q, k: CUDA [B, N, heads, d], fp32, bf16 or fp16, any strides with contiguous
    features (views of a fused projection); inv_freq fp64 [rot/2] and scale from
    rope_inv_freq.  Positions: int32 CUDA [B, N] or [N] (with several sections
    [.., N, axes]), or a grid (T, H, W) in raster order from `origin`, or by
    default origin[0] + n.  Outputs may be q and k themselves."""
    ys = _rope(q, k, inv_freq, sections, interleaved, scale, positions, grid, origin, q_out, k_out, out_dtype, 0, stream)
    return ys[0], (ys[1] if k is not None else None)


def rope_backward(dq, dk, inv_freq, sections=None, interleaved: bool = False, scale: float = 1.0, positions=None,
                  grid=None, origin=(0, 0, 0), dq_out=None, dk_out=None, out_dtype=None, stream=None):
    """Gradients of rope_forward's q and k from those of its outputs (the turn by
    the opposite angles); attn_backward's fp32 gradients may be stored as bf16."""
    ys = _rope(dq, dk, inv_freq, sections, interleaved, scale, positions, grid, origin, dq_out, dk_out, out_dtype, 1,
               stream)
    return ys[0], (ys[1] if dk is not None else None)


@dataclasses.dataclass
class Checkpoint:
    """8-bit codes and scale bytes of one tensor (see salad.h): codes uint8 of the
    tensor's shape, scales uint8 [..., ceil(C/32)] for its last dimension C."""
    codes: torch.Tensor
    scales: torch.Tensor
    fmt: str
    dtype: torch.dtype

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


def _rows_of(x):
    """(rows, cols, row stride) of a tensor whose groups run along its last
    dimension; trailing dimensions that lie one after another are taken as one row
    where that keeps whole groups."""
    shape, st = x.shape, x.stride()
    cols, i = shape[-1], x.dim() - 2
    if cols > 1 and st[-1] != 1:
        raise ValueError("the last dimension must be contiguous")
    while i >= 0 and cols % 32 == 0 and (st[i] == cols or shape[i] == 1) and cols * shape[i] < 1 << 30:
        cols *= shape[i]
        i -= 1
    rows, stride = 1, cols
    first = True
    while i >= 0:
        if shape[i] != 1:
            if first:
                stride, first = st[i], False
            elif st[i] != stride * rows:
                raise ValueError("the rows must lie at one distance from each other")
            rows *= shape[i]
        i -= 1
    return rows, cols, stride


def _ckpt_call(fn, name, xs, cks, fmt, stream, packed_as=None):
    """One launch for tensors of the same layout, else one each; a checkpoint is of
    the format packed_as once its launch has been taken."""
    groups, filled = {}, {}
    for x, c in zip(xs, cks):
        if x.numel():
            rows, cols, stride = _rows_of(x)
            if x.numel() > _INT_MAX:
                _int32(name, rows, cols)
            key = (rows, cols, x.dtype)
            groups.setdefault(key, []).append(_CKPT_TENSOR(x.data_ptr(), stride, c.codes.data_ptr(), c.scales.data_ptr()))
            if packed_as is not None:
                filled.setdefault(key, []).append(c)
        elif packed_as is not None:
            c.fmt, c.dtype = packed_as, x.dtype
    s = _stream(stream)
    for (rows, cols, dtype), packed in groups.items():
        for i in range(0, len(packed), 4):
            _check(fn(b"".join(packed[i:i + 4]), len(packed[i:i + 4]), rows, cols, _TYPES[dtype], _FORMATS[fmt], s), name)
            if filled:
                for c in filled[rows, cols, dtype][i:i + 4]:
                    c.fmt, c.dtype = packed_as, dtype


def _ckpt_scales_shape(shape):
    return (*shape[:-1], (shape[-1] + 31) // 32)


def _once(outs):
    given = [id(c) for c in outs if c is not None]
    if len(set(given)) < len(given):
        raise ValueError("the same output is given twice")


def ckpt_pack(x, fmt: str = "int8", out=None, stream=None):
    """8-bit checkpoint of a CUDA tensor (fp32, bf16 or fp16), or of each of a list
    of them (one launch where their layouts agree): groups of 32 along the last
    dimension share a power-of-two scale (see salad_ckpt_pack).  Rows may lie
    apart (a view of a fused projection).  fmt "int8" or "e4m3"; `out` reuses
    earlier checkpoints' memory."""
    if fmt not in _FORMATS:
        raise ValueError(f"unknown format {fmt!r}")
    many = isinstance(x, (list, tuple))
    xs = x if many else (x,)
    outs = (None,) * len(xs) if out is None else out if many else (out,)
    if not xs or len(outs) != len(xs):
        raise ValueError("one output for each tensor")
    if out is not None:
        _once(outs)
    ctx, dev = _on(*xs)
    res = []
    with _at(ctx, dev, stream):
        for t, c in zip(xs, outs):
            if t.dtype not in _TYPES or t.dim() < 1:
                raise TypeError("tensors of fp32, bf16 or fp16 with one dimension at least")
            scales = _ckpt_scales_shape(t.shape)
            if c is None:
                codes = torch.empty_like(t, dtype=torch.uint8, memory_format=torch.contiguous_format)
                c = Checkpoint(codes, codes.new_empty(scales), fmt, t.dtype)
            else:
                if c.codes.shape != t.shape or c.scales.shape != scales:
                    raise ValueError("the checkpoint's memory has another shape")
                _on(t, c.codes, c.scales)
                _ptr(c.codes, torch.uint8, "codes"), _ptr(c.scales, torch.uint8, "scales")
            res.append(c)
        _ckpt_call(lib().salad_ckpt_pack, "salad_ckpt_pack", xs, res, fmt, stream, None if out is None else fmt)
    return res if many else res[0]


def ckpt_unpack(ckpt, dtype=None, out=None, stream=None):
    """The values of a Checkpoint, or of each of a list, in `dtype` (by default the
    packed tensor's); exact for bf16 and fp32 (see salad.h for bf16's smallest)."""
    many = isinstance(ckpt, (list, tuple))
    cks = ckpt if many else (ckpt,)
    outs = (None,) * len(cks) if out is None else out if many else (out,)
    if not cks or len(outs) != len(cks):
        raise ValueError("one output for each checkpoint")
    if out is not None:
        _once(outs)
    fmt = cks[0].fmt
    if fmt not in _FORMATS or any(c.fmt != fmt for c in cks):
        raise ValueError("the checkpoints have several formats")
    ctx, dev = _on(*(t for c in cks for t in (c.codes, c.scales)))
    res = []
    with _at(ctx, dev, stream):
        for c, y in zip(cks, outs):
            _ptr(c.codes, torch.uint8, "codes"), _ptr(c.scales, torch.uint8, "scales")
            if c.scales.shape != _ckpt_scales_shape(c.codes.shape):
                raise ValueError("scales and codes have shapes that do not agree")
            if y is None:
                y = torch.empty_like(c.codes, dtype=dtype or c.dtype)
            else:
                _on(c.codes, y)
            if y.shape != c.codes.shape:
                raise ValueError("the output has another shape")
            if y.dtype not in _TYPES or (dtype is not None and y.dtype != dtype):
                raise TypeError("outputs of fp32, bf16 or fp16, as asked for")
            res.append(y)
        _ckpt_call(lib().salad_ckpt_unpack, "salad_ckpt_unpack", res, cks, fmt, stream)
    return res if many else res[0]


def new_ckpt_backward_workspace(B: int, N: int, heads: int, d: int, device=None) -> torch.Tensor:
    """A zero-filled workspace for attn_backward_ckpt."""
    n = lib().salad_ckpt_backward_workspace_bytes(B, N, heads, d)
    if n == 0:
        raise SaladError(SALAD_ERR_INVALID_ARG, "salad_ckpt_backward_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=torch.device("cuda") if device is None else torch.device(device))


def attn_backward_ckpt(q, k, v, dout, row_ptr, col_idx, w_proj, gate, block: int = 128, t_row_ptr=None,
                       t_col_idx=None, softmax_scale: float = 0.0, eps: float = 1e-6, mask_per_bh: bool = False,
                       workspace=None, stream=None):
    """The whole layer's gradients from 8-bit checkpoints of q, k and v
    (ckpt_pack of [B, N, Hh, d] tensors): out and lse are computed again from the
    decoded values.  A dict of CUDA tensors: dq, dk, dv bf16 [B, N, Hh, d], dw fp32
    [d, d], dgate fp32 [B, Hh]; the other arguments as attn_backward.  The transposed
    mask is built on the GPU when none is given (about 20 us); a symmetric mask, such
    as build_block_mask's, may be given as its own transpose."""
    if not (q.fmt == k.fmt == v.fmt) or not (q.codes.shape == k.codes.shape == v.codes.shape) or q.codes.dim() != 4:
        raise ValueError("checkpoints of q, k and v: one format, one shape [B, N, Hh, d]")
    B, N, Hh, d = q.codes.shape
    for c in (q, k, v):
        if c.scales.shape != _ckpt_scales_shape(c.codes.shape):
            raise ValueError("scales and codes have shapes that do not agree")
    if dout.shape != q.codes.shape or w_proj.shape != (d, d) or gate.shape != (B, Hh):
        raise ValueError("dout, w_proj or gate has another shape than the checkpoints ask for")
    ctx, dev = _on(q.codes, q.scales, k.codes, k.scales, v.codes, v.scales, dout, row_ptr, col_idx, w_proj, gate,
                   *(t for t in (t_row_ptr, t_col_idx, workspace) if t is not None))
    with _at(ctx, dev, stream):
        nb = (N + block - 1) // block
        if row_ptr.numel() != (B * Hh if mask_per_bh else Hh) * nb + 1:
            raise ValueError(f"row_ptr has {row_ptr.numel()} entries, not {(B * Hh if mask_per_bh else Hh) * nb + 1}")
        t_row_ptr, t_col_idx = _transposed_mask(row_ptr, col_idx, t_row_ptr, t_col_idx, col_idx.numel(),
                                                B * Hh if mask_per_bh else Hh, nb)
        if t_row_ptr.shape != row_ptr.shape:
            raise ValueError("the transposed mask has another number of rows")
        res = {n: torch.empty(B, N, Hh, d, dtype=torch.bfloat16, device=dev) for n in ("dq", "dk", "dv")}
        res["dw"] = torch.empty(d, d, dtype=torch.float32, device=dev)
        res["dgate"] = torch.empty(B, Hh, dtype=torch.float32, device=dev)
        if workspace is None:
            workspace = new_ckpt_backward_workspace(B, N, Hh, d, dev)
        u8 = lambda t, name: _dev_ptr(t, torch.uint8, name)  # noqa: E731
        i32 = lambda t, name: _dev_ptr(t, torch.int32, name)  # noqa: E731
        _check(lib().salad_attn_backward_ckpt(
            u8(q.codes, "q.codes"), u8(q.scales, "q.scales"), u8(k.codes, "k.codes"), u8(k.scales, "k.scales"),
            u8(v.codes, "v.codes"), u8(v.scales, "v.scales"), _FORMATS[q.fmt], _dev_ptr(dout, torch.bfloat16, "dout"),
            B, N, Hh, d, int(block), i32(row_ptr, "row_ptr"), _cols(col_idx, row_ptr), i32(t_row_ptr, "t_row_ptr"),
            _cols(t_col_idx, t_row_ptr), int(bool(mask_per_bh)), _dev_ptr(w_proj, torch.bfloat16, "w_proj"),
            _dev_ptr(gate, torch.float32, "gate"), float(softmax_scale), float(eps),
            *[_dev_ptr(res[n], torch.bfloat16, n) for n in ("dq", "dk", "dv")],
            *[_dev_ptr(res[n], torch.float32, n) for n in ("dw", "dgate")],
            u8(workspace, "workspace"), workspace.numel(), _stream(stream)), "salad_attn_backward_ckpt")
    return res


def new_diff_workspace(B: int, N: int, heads: int, d: int, device=None) -> torch.Tensor:
    """A zero-filled workspace for the forward and backward of differential attention."""
    n = lib().salad_diff_workspace_bytes(B, N, heads, d)
    if n == 0:
        raise SaladError(SALAD_ERR_INVALID_ARG, "salad_diff_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=torch.device("cuda") if device is None else torch.device(device))


def _bf16_like(q, *named):
    shape = q.shape
    for t, name in named:
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    return [_ptr(t, torch.bfloat16, name) for t, name in named]


def _lam(lam, heads):
    if lam.shape != (heads,):
        raise ValueError(f"lam has shape {tuple(lam.shape)}, not ({heads},)")
    if lam.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"lam must be fp32 or bf16, got {lam.dtype}")
    return _ptr(lam, lam.dtype, "lam"), _TYPES[lam.dtype]


def _cols(col_idx, row_ptr):
    """The column list's pointer; a mask that keeps nothing has none, and none is read."""
    return _ptr(col_idx, torch.int32, "col_idx") or _ptr(row_ptr, torch.int32, "row_ptr")


def _mask_rows(row_ptr, B, N, heads, mask_per_bh):
    rows = (B * heads if mask_per_bh else heads) * ((N + 127) // 128)
    if row_ptr.numel() != rows + 1:
        raise ValueError(f"row_ptr has {row_ptr.numel()} entries, not {rows + 1}")


def _diff_forward(q, k, v, row_ptr, col_idx, lam, softmax_scale, mask_per_bh, out, out2, lse, train, workspace, stream):
    ctx, dev = _on(q, k, v, row_ptr, col_idx, lam, *(t for t in (out, out2, lse, workspace) if t is not None))
    with _at(ctx, dev, stream):
        B, N, Hh, d = q.shape
        _mask_rows(row_ptr, B, N, Hh, mask_per_bh)
        if out is None:
            out = torch.empty_like(q)
        if train:
            out2 = torch.empty_like(q) if out2 is None else out2
            lse = torch.empty(2, B, Hh, N, dtype=torch.float32, device=dev) if lse is None else lse
            if lse.shape != (2, B, Hh, N):
                raise ValueError(f"lse has shape {tuple(lse.shape)}, not {(2, B, Hh, N)}")
        if workspace is None:
            workspace = new_diff_workspace(B, N, Hh, d, dev)
        ptrs = _bf16_like(q, (q, "q"), (k, "k"), (v, "v"), (out, "out"), *([(out2, "out2")] if train else []))
        _check(lib().salad_diff_forward(
            *ptrs[:3], B, N, Hh, d, 128, _ptr(row_ptr, torch.int32, "row_ptr"), _cols(col_idx, row_ptr),
            int(bool(mask_per_bh)), *_lam(lam, Hh), float(softmax_scale),
            ptrs[3], ptrs[4] if train else None, _ptr(lse, torch.float32, "lse") if train else None,
            _ptr(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)), "salad_diff_forward")
    return out, out2, lse


def diff_attn_forward(q, k, v, row_ptr, col_idx, lam, softmax_scale: float = 0.0, mask_per_bh: bool = False, out=None,
                      workspace=None, stream=None) -> torch.Tensor:
    """Differential attention over a mask of 128-token blocks (see salad_diff_forward):
    out = (softmax(q_1 k_1^T) - lam softmax(q_2 k_2^T)) v with q_1, k_1 the first and
    q_2, k_2 the second half of each head's features.

    q, k, v: bf16 CUDA [B, N, Hh, d]; lam fp32 or bf16 [Hh]; mask rows per head, or
    per (b, h) with mask_per_bh; softmax_scale 0 is 1/sqrt(d/2)."""
    return _diff_forward(q, k, v, row_ptr, col_idx, lam, softmax_scale, mask_per_bh, out, None, None, False, workspace,
                         stream)[0]


def diff_attn_forward_lse(q, k, v, row_ptr, col_idx, lam, softmax_scale: float = 0.0, mask_per_bh: bool = False,
                          out=None, out2=None, lse=None, workspace=None, stream=None):
    """diff_attn_forward that also returns what diff_attn_backward needs: (out, out2,
    lse) with out2 bf16 [B, N, Hh, d] the second map's output and lse fp32 [2, B, Hh, N]."""
    return _diff_forward(q, k, v, row_ptr, col_idx, lam, softmax_scale, mask_per_bh, out, out2, lse, True, workspace,
                         stream)


def diff_attn_backward(q, k, v, out, out2, dout, lse, row_ptr, col_idx, lam, t_row_ptr=None, t_col_idx=None,
                       softmax_scale: float = 0.0, mask_per_bh: bool = False, workspace=None, stream=None):
    """Gradients of differential attention (see salad_diff_backward): dict of dq, dk,
    dv bf16 [B, N, Hh, d] and dlam [Hh] of lam's type.  out, out2 and lse come from
    diff_attn_forward_lse on the same inputs (with q, k, v decoded from a checkpoint: of
    a forward on the decoded ones).  The transposed mask is built on the GPU when none
    is given (about 20 us); a symmetric mask, such as build_block_mask's, may be given
    as its own transpose."""
    ctx, dev = _on(q, k, v, out, out2, dout, lse, row_ptr, col_idx, lam,
                   *(t for t in (t_row_ptr, t_col_idx, workspace) if t is not None))
    with _at(ctx, dev, stream):
        B, N, Hh, d = q.shape
        _mask_rows(row_ptr, B, N, Hh, mask_per_bh)
        t_row_ptr, t_col_idx = _transposed_mask(row_ptr, col_idx, t_row_ptr, t_col_idx, col_idx.numel(),
                                                B * Hh if mask_per_bh else Hh, (N + 127) // 128)
        _mask_rows(t_row_ptr, B, N, Hh, mask_per_bh)
        if lse.shape != (2, B, Hh, N):
            raise ValueError(f"lse has shape {tuple(lse.shape)}, not {(2, B, Hh, N)}")
        res = {n: torch.empty_like(q) for n in ("dq", "dk", "dv")}
        res["dlam"] = torch.empty_like(lam)
        if workspace is None:
            workspace = new_diff_workspace(B, N, Hh, d, dev)
        ptrs = _bf16_like(q, (q, "q"), (k, "k"), (v, "v"), (out, "out"), (out2, "out2"), (dout, "dout"))
        i32 = lambda t, name: _ptr(t, torch.int32, name)  # noqa: E731
        _check(lib().salad_diff_backward(
            *ptrs, _ptr(lse, torch.float32, "lse"), B, N, Hh, d, 128, i32(row_ptr, "row_ptr"),
            _cols(col_idx, row_ptr), i32(t_row_ptr, "t_row_ptr"), _cols(t_col_idx, t_row_ptr), int(bool(mask_per_bh)),
            *_lam(lam, Hh), float(softmax_scale), *[_ptr(res[n], torch.bfloat16, n) for n in ("dq", "dk", "dv")],
            res["dlam"].data_ptr(), _ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
            _stream(stream)), "salad_diff_backward")
    return res


def diff_attn_decode(q, k_cache, v_cache, lens, lam, softmax_scale: float = 0.0, out=None, stream=None) -> torch.Tensor:
    """Differential attention of a few queries against a cache (see salad_diff_decode):
    q bf16 [B, Nq, Hh, d], k_cache and v_cache bf16 [B, capacity, Hh, d], lens int32
    CUDA [B]; every query of sequence b sees keys [0, lens[b])."""
    ctx, dev = _on(q, k_cache, v_cache, lens, lam, *(() if out is None else (out,)))
    with _at(ctx, dev, stream):
        B, Nq, Hh, d = q.shape
        cap = k_cache.shape[1]
        if k_cache.shape != (B, cap, Hh, d) or v_cache.shape != k_cache.shape or lens.shape != (B,):
            raise ValueError("k_cache, v_cache [B, capacity, Hh, d] and lens [B] must fit q")
        if out is None:
            out = torch.empty_like(q)
        ptrs = _bf16_like(q, (q, "q"), (out, "out"))
        _check(lib().salad_diff_decode(
            ptrs[0], _ptr(k_cache, torch.bfloat16, "k_cache"), _ptr(v_cache, torch.bfloat16, "v_cache"), B, Nq,
            cap, Hh, d, _ptr(lens, torch.int32, "lens"), *_lam(lam, Hh), float(softmax_scale), ptrs[1],
            _stream(stream)), "salad_diff_decode")
    return out


@_of_its_stream
def linear_state(k, v, gate=None, workspace=None, stream=None):
    """(S fp32 [B*Hh, d, d], z fp32 [B*Hh, d]) of the ReLU linear branch."""
    B, N, Hh, d = k.shape
    if workspace is None:
        workspace = new_workspace(B, N, Hh, d, k.device)
    S = torch.zeros(B * Hh, d, d, dtype=torch.float32, device=k.device)
    z = torch.zeros(B * Hh, d, dtype=torch.float32, device=k.device)
    g = None if gate is None else _dev_ptr(gate, torch.float32, "gate")
    _check(lib().salad_linear_state(
        _dev_ptr(k, torch.bfloat16, "k"), _dev_ptr(v, torch.bfloat16, "v"), B, N, Hh, d, g,
        _dev_ptr(S, torch.float32, "S"), _dev_ptr(z, torch.float32, "z"),
        _dev_ptr(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)),
        "salad_linear_state")
    return S, z


def check_status(workspace, stream=None) -> int:
    """Synchronise and return (and clear) the workspace status; see salad.h."""
    return int(lib().salad_check_status(_dev_ptr(workspace, torch.uint8, "workspace"), _stream(stream)))


def set_wait_limit_ns(limit_ns: int) -> None:
    lib().salad_set_wait_limit_ns(int(limit_ns))


def set_max_ctas(max_ctas: int) -> None:
    """Test hook: cap the persistent attention grid (0: one CTA per SM)."""
    lib().salad_set_max_ctas(int(max_ctas))


def set_phase_events(before_linear=None, before_attention=None, after_attention=None) -> None:
    """Record these CUDA events (raw cudaEvent_t handles, or objects with a
    ``cuda_event`` handle) inside later attn_forward calls: before the
    linear-branch kernels, before and after the attention kernel."""
    def handle(e):
        if e is None or isinstance(e, ctypes.c_void_p):
            return e
        return ctypes.c_void_p(e.cuda_event if hasattr(e, "cuda_event") else int(e))
    h = [handle(e) for e in (before_linear, before_attention, after_attention)]
    lib().salad_set_phase_events(*h)
