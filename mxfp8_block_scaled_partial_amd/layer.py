"""Python binding of the training-layer operators: the C ABI of include/layer/mxfp8_layer.h under the
same names, for torch tensors.

As in :mod:`.binding`, this is marshalling only: a ``make_*`` function describes a call once
(tensors become device pointers and leading dimensions; the description keeps its tensors
alive and, where the call needs one, a workspace), and the entry point of the same name runs it
on torch's current stream as often as wanted.  Calls of one description share its buffers and
workspace, so they have to be ordered like any calls that share buffers.  There is no CPU
fallback.

8-bit matrices are uint8 tensors (or ``torch.float8_e4m3fn`` / ``float8_e8m0fnu`` views) of E4M3
codes and E8M0 scale bytes; tensors of any other type are refused.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as B
from .binding import Buf, Mxfp8Error  # noqa: F401  (re-exported with the calls that raise it)

ALONG_COLS, ALONG_ROWS = 0, 1
ALONG = {"cols": ALONG_COLS, "rows": ALONG_ROWS}
ACT_NONE, ACT_GELU, ACT_SWIGLU = range(3)
ACT_FUNCS = {"none": ACT_NONE, "gelu": ACT_GELU, "swiglu": ACT_SWIGLU}
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
BLOCK = 128  # values that share a scale in the 8-bit matrices these operators write

# every entry point declared in include/layer/mxfp8_layer.h
EXPORTS = ("mxfp8_matmul", "mxfp8_matmul_workspace", "mxfp8_act_forward", "mxfp8_act_backward",
           "mxfp8_layernorm_forward", "mxfp8_layernorm_backward", "mxfp8_layernorm_workspace")


class Operand(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("scale", ctypes.c_void_p), ("scale_ld", ctypes.c_int64),
                ("along", ctypes.c_int32), ("block", ctypes.c_int32),
                ("across", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class Product(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("a", Operand), ("b", Operand), ("out", Buf), ("addend", Buf),
                ("out_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)]


class Mat8(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("scale", ctypes.c_void_p), ("scale_ld", ctypes.c_int64)]


class Act(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("func", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("input", Buf * 2), ("grad", Buf), ("saved", Mat8 * 2), ("out", Buf * 2),
                ("row", Mat8 * 2), ("col", Mat8 * 2)]


class LayerNorm(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("x", Buf), ("gamma", ctypes.c_void_p), ("beta", ctypes.c_void_p),
                ("y", Buf), ("mean", ctypes.c_void_p), ("rstd", ctypes.c_void_p),
                ("dy", Buf), ("dx", Buf), ("dgamma", ctypes.c_void_p),
                ("dbeta", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)]


_lib = None


def lib():
    """The library with the argument and result types of this header's entry points set."""
    global _lib
    if _lib is None:
        L = B.lib()
        for name, struct in (("mxfp8_matmul", Product), ("mxfp8_act_forward", Act),
                             ("mxfp8_act_backward", Act), ("mxfp8_layernorm_forward", LayerNorm),
                             ("mxfp8_layernorm_backward", LayerNorm)):
            f = getattr(L, name)
            f.argtypes = [ctypes.POINTER(struct), ctypes.c_void_p]
            f.restype = ctypes.c_int
        for name, struct in (("mxfp8_matmul_workspace", Product),
                             ("mxfp8_layernorm_workspace", LayerNorm)):
            f = getattr(L, name)
            f.argtypes = [ctypes.POINTER(struct)]
            f.restype = ctypes.c_int64
        _lib = L
    return _lib


# ------------------------------------------------------------------ tensor marshalling


def _matrix(t, rows, cols, what, dtype=None) -> Buf:
    """A row-major [rows, cols] tensor with unit column stride; an absent one (None, or without
    elements) is an empty handle."""
    if not B._present(t):
        return Buf(None, 0)
    if t.dim() != 2 or (t.shape[0], t.shape[1]) != (rows, cols):
        raise ValueError(f"{what} must be [{rows}, {cols}], got shape {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{what} must have unit stride along its last dimension")
    ld = t.stride(0) if rows > 1 else cols
    if ld < cols:
        raise ValueError(f"{what} has overlapping rows")
    return Buf(B._dev_ptr(t, what), ld)


def _vector(t, length, what):
    if t is None or (length == 0 and t.numel() == 0):
        return None
    if t.dim() != 1 or t.numel() != length or t.dtype != torch.float32 or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous float32 tensor of {length} elements")
    return B._dev_ptr(t, what)


def _blocks(n: int, block: int) -> int:
    return (n + block - 1) // block


def _bytes(t, kind, what):
    """Refuses an 8-bit tensor of another format, whose bytes would be read as this one's."""
    if t is not None and t.dtype not in (torch.uint8, kind):
        raise ValueError(f"{what} must be uint8 or {kind}, got {t.dtype}")


def _mat8(pair, rows, cols, by_cols, what) -> Mat8:
    """A (data, scale) pair in row-wise or column-wise blocks of 128; None is absent."""
    if pair is None:
        return Mat8(None, 0, None, 0)
    data, scale = pair
    _bytes(data, E4M3, f"{what} data")
    _bytes(scale, E8M0, f"{what} scale")
    d = _matrix(data, rows, cols, f"{what} data")
    s = _matrix(scale, _blocks(rows, BLOCK) if by_cols else rows,
                cols if by_cols else _blocks(cols, BLOCK), f"{what} scale")
    return Mat8(d.ptr, d.ld, s.ptr, s.ld)


def _workspace(need: int, workspace, device, struct):
    """Checks the caller's workspace or makes one, and puts it into the description."""
    if need < 0:
        raise Mxfp8Error(-need, B.mxfp8_last_error())
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        struct.own = workspace, {B._stream(None)}
    if workspace is not None:
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        struct.workspace = B._dev_ptr(workspace, "workspace")
        struct.workspace_bytes = workspace.numel() * workspace.element_size()
    return workspace


def _stream_of(struct, stream) -> int:
    """The call's stream.  A workspace that the description made belongs to the stream that was
    current then; the allocator learns of every other one that uses it, so that the memory is not
    given away while such a call still runs after the description is gone."""
    handle = B._stream(stream)
    workspace, known = getattr(struct, "own", (None, ()))
    if workspace is not None and handle not in known:
        workspace.record_stream(torch.cuda.ExternalStream(handle, device=workspace.device))
        known.add(handle)
    return handle


# ------------------------------------------------------------------ matrix product


def make_operand(data, scale, *, along: str = "cols", block: int = BLOCK,
                 across: int = 1) -> Operand:
    """An 8-bit operand of a product.

    ``data`` is [outer, k] with ``along="cols"`` and [k, outer] with ``along="rows"``; one scale
    byte covers ``block`` (32 or 128) values along the sum and ``across`` (1 or 128) outer
    values.  A weight of the writeback is ``make_operand(st.data_row, st.scale_row, block=32)``
    or ``make_operand(st.data_col, st.scale_col, along="rows", block=32)`` with its data viewed
    as [rows, cols]."""
    if along not in ALONG:
        raise ValueError(f"along must be 'cols' or 'rows', got {along!r}")
    if block not in (32, 128) or across not in (1, 128):
        raise ValueError(f"block must be 32 or 128 and across 1 or 128, got {block}, {across}")
    _bytes(data, E4M3, "data")
    _bytes(scale, E8M0, "scale")
    if data.dim() != 2:
        raise ValueError(f"data must be 2-D, got shape {tuple(data.shape)}")
    d = _matrix(data, data.shape[0], data.shape[1], "data")
    sr, sc = (across, block) if along == "cols" else (block, across)
    rows, cols = _blocks(data.shape[0], sr), _blocks(data.shape[1], sc)
    if scale.dim() != 2 or scale.shape[0] < rows or scale.shape[1] < cols:
        raise ValueError(f"scale shape {tuple(scale.shape)} is smaller than [{rows}, {cols}]")
    s = _matrix(scale[:rows, :cols], rows, cols, "scale")
    o = Operand(d.ptr, d.ld, s.ptr, s.ld, ALONG[along], block, across, 0)
    o.outer, o.k = (data.shape if along == "cols" else data.shape[::-1])
    o.tensors = (data, scale)
    return o


def make_product(a: Operand, b: Operand, out, *, addend=None, workspace=None) -> Product:
    """out = a b^T (+ addend): ``out`` [m, n] float32 or bfloat16, ``addend`` [m, n] float32
    (``out`` itself adds in place).  ``workspace`` defaults to one that the description owns."""
    if a.k != b.k:
        raise ValueError(f"the operands' sums have {a.k} and {b.k} values")
    if out.dim() != 2 or out.shape[0] != a.outer or out.shape[1] != b.outer:
        raise ValueError(f"out must be [{a.outer}, {b.outer}], got shape {tuple(out.shape)}")
    p = Product(a.outer, b.outer, a.k, a, b, _matrix(out, a.outer, b.outer, "out"),
                _matrix(addend, a.outer, b.outer, "addend", torch.float32),
                B.dtype_code(out.dtype), 0, None, 0)
    workspace = _workspace(lib().mxfp8_matmul_workspace(ctypes.byref(p)), workspace, out.device, p)
    p.tensors = (a.tensors, b.tensors, out, addend, workspace)
    return p


def mxfp8_matmul_workspace(product: Product) -> int:
    """Bytes of workspace the product needs; negative: the status code, negated."""
    return lib().mxfp8_matmul_workspace(ctypes.byref(product))


def mxfp8_matmul(product: Product, stream=None) -> None:
    B._check(lib().mxfp8_matmul(ctypes.byref(product), _stream_of(product, stream)))


# ------------------------------------------------------- activation with 8-bit checkpoint


def make_act(func: str, *, inputs=(), grad=None, saved=(), out=(), row=(), col=()) -> Act:
    """An activation: ``func`` is "none", "gelu" or "swiglu" (inputs gate, up).

    Forward: ``inputs`` are the [rows, cols] tensors; backward: ``grad`` is the gradient of the
    result.  ``saved`` are (data, scale) pairs of the inputs in 8 bits, row-wise blocks of 128.
    ``out`` (tensors of the inputs' dtype), ``row`` and ``col`` ((data, scale) pairs in row-wise
    and column-wise blocks of 128) receive the result, or in a backward call the gradient of
    each input; None, or a shorter list, leaves one out."""
    if func not in ACT_FUNCS:
        raise ValueError(f"func must be one of {', '.join(ACT_FUNCS)}, got {func!r}")
    inputs, saved, out, row, col = (list(x) for x in (inputs, saved, out, row, col))
    if any(len(x) > 2 for x in (inputs, saved, out, row, col)):
        raise ValueError("at most two inputs, saved, out, row and col each")
    like = grad if grad is not None else inputs[0] if inputs else None
    if like is None:
        raise ValueError("an activation needs its inputs (forward) or grad (backward)")
    if like.dim() != 2:
        raise ValueError(f"values must be 2-D, got shape {tuple(like.shape)}")
    rows, cols, dtype = like.shape[0], like.shape[1], like.dtype
    a = Act(rows, cols, ACT_FUNCS[func], B.dtype_code(dtype))
    a.grad = _matrix(grad, rows, cols, "grad", dtype)
    for i, t in enumerate(inputs):
        a.input[i] = _matrix(t, rows, cols, f"inputs[{i}]", dtype)
    for i, t in enumerate(out):
        a.out[i] = _matrix(t, rows, cols, f"out[{i}]", dtype)
    for i, t in enumerate(saved):
        a.saved[i] = _mat8(t, rows, cols, False, f"saved[{i}]")
    for i, t in enumerate(row):
        a.row[i] = _mat8(t, rows, cols, False, f"row[{i}]")
    for i, t in enumerate(col):
        a.col[i] = _mat8(t, rows, cols, True, f"col[{i}]")
    a.tensors = (inputs, grad, saved, out, row, col)
    return a


def mxfp8_act_forward(act: Act, stream=None) -> None:
    B._check(lib().mxfp8_act_forward(ctypes.byref(act), B._stream(stream)))


def mxfp8_act_backward(act: Act, stream=None) -> None:
    B._check(lib().mxfp8_act_backward(ctypes.byref(act), B._stream(stream)))


# ------------------------------------------------------------------ layer norm


def make_layernorm(x, gamma=None, beta=None, *, mean=None, rstd=None, y=None, dy=None, dx=None,
                   dgamma=None, dbeta=None, eps: float = 1e-5, workspace=None) -> LayerNorm:
    """A layer norm over the last dimension of x [rows, cols]; forward fills y, mean and rstd,
    backward reads mean, rstd and dy and fills dx, dgamma and dbeta (each may be left out).
    Parameters and statistics are float32 vectors."""
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D, got shape {tuple(x.shape)}")
    rows, cols, dtype = x.shape[0], x.shape[1], x.dtype
    p = LayerNorm(rows, cols, B.dtype_code(dtype), eps, _matrix(x, rows, cols, "x"),
                  _vector(gamma, cols, "gamma"), _vector(beta, cols, "beta"),
                  _matrix(y, rows, cols, "y", dtype), _vector(mean, rows, "mean"),
                  _vector(rstd, rows, "rstd"), _matrix(dy, rows, cols, "dy", dtype),
                  _matrix(dx, rows, cols, "dx", dtype), _vector(dgamma, cols, "dgamma"),
                  _vector(dbeta, cols, "dbeta"), None, 0)
    if dgamma is not None or dbeta is not None:
        workspace = _workspace(lib().mxfp8_layernorm_workspace(ctypes.byref(p)), workspace,
                               x.device, p)
    p.tensors = (x, gamma, beta, mean, rstd, y, dy, dx, dgamma, dbeta, workspace)
    return p


def mxfp8_layernorm_workspace(norm: LayerNorm) -> int:
    """Bytes of workspace the backward pass needs; negative: the status code, negated."""
    return lib().mxfp8_layernorm_workspace(ctypes.byref(norm))


def mxfp8_layernorm_forward(norm: LayerNorm, stream=None) -> None:
    B._check(lib().mxfp8_layernorm_forward(ctypes.byref(norm), B._stream(stream)))


def mxfp8_layernorm_backward(norm: LayerNorm, stream=None) -> None:
    B._check(lib().mxfp8_layernorm_backward(ctypes.byref(norm), _stream_of(norm, stream)))
