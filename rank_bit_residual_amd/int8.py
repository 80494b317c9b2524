"""8-bit tensors with a scale for each row, and the operators on them.

An Int8Tensor holds Q(x) of a matrix x [rows, K]: for each row a float32 scale, max|x| / 127, and the nearest integers to
x / scale. Its products sum over K, so a row is a token of activations or an output channel of a weight, each with a scale
of its own; a matrix that enters products along both axes is quantised along both.

A linear layer with x [M, K] and weight w [K, N], in training (the quantisers pass gradients straight through):

    x_rows, x_cols = int8_quantize(x, axis=None)
    w_rows, w_cols = int8_quantize(w, axis=None)
    y = int8_matmul(x_rows, w_cols, bias=b)
    dx, dw, db = int8_backward(dy, w_rows, x_cols, bias=True)

and in serving `y = int8_matmul(x, w_cols, bias=b)`, with w_cols kept, or behind a norm
`y = int8_matmul(layer_norm(x, weight, bias, quantize="int8"), w_cols)`. Every arithmetic step runs in libsvdq; tensors are
float32, bfloat16 or float16 on a GPU. The calls record no autograd graph, like those of mx.py.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib as L
from .api import _check_int
from .mx import _call, _check_axis, _dtype_code, _matrix, _no_graph, _output, _parts, _rows, _same_device, _workspace_bytes


@functools.lru_cache(maxsize=4096)
def _bytes(rows: int, cols: int) -> tuple:
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    L.check(L.load().svdq_i8_layout(rows, cols, ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


class Int8Tensor:
    """An 8-bit tensor on the device: the values Q(x) of a [rows, cols] matrix, a scale for each row.

    data: one uint8 array, the codes and behind them the scales, in the layout of svdq_i8_layout. It may be saved and
    restored with torch; the padding rows of its last tiles hold nothing.
    """

    __slots__ = ("data", "rows", "cols", "_at")

    def __init__(self, data: torch.Tensor, rows: int, cols: int):
        _check_int("rows", rows)
        _check_int("cols", cols)
        code_bytes, scale_bytes = _bytes(rows, cols)
        if not isinstance(data, torch.Tensor) or data.dtype != torch.uint8 or data.dim() != 1 or not data.is_contiguous():
            raise TypeError("data must be a contiguous uint8 vector")
        if data.numel() < code_bytes + scale_bytes:
            raise ValueError(f"data holds {data.numel()} bytes, a [{rows}, {cols}] tensor needs {code_bytes + scale_bytes}")
        self.data, self.rows, self.cols, self._at = data, rows, cols, code_bytes

    @classmethod
    def _empty(cls, rows: int, cols: int, device) -> "Int8Tensor":
        code_bytes, scale_bytes = _bytes(rows, cols)
        t = cls.__new__(cls)
        t.data = torch.empty(code_bytes + scale_bytes, dtype=torch.uint8, device=device)
        t.rows, t.cols, t._at = rows, cols, code_bytes
        return t

    @property
    def shape(self) -> tuple:
        return (self.rows, self.cols)

    @property
    def device(self) -> torch.device:
        return self.data.device

    @property
    def codes(self) -> torch.Tensor:
        """The tiled codes, as bytes."""
        return self.data[: self._at]

    @property
    def scales(self) -> torch.Tensor:
        """The rows' scales, float32 [rows]."""
        return self.data[self._at: self._at + 4 * self.rows].view(torch.float32)

    def __repr__(self) -> str:
        return f"Int8Tensor([{self.rows}, {self.cols}], device={self.data.device})"


def _i8(t, name: str) -> None:
    if not isinstance(t, Int8Tensor):
        raise TypeError(f"{name}: expected an Int8Tensor")
    if not t.data.is_cuda:
        raise RuntimeError("libsvdq device calls need tensors on an AMD GPU (HIP device)")


def _scratch(need: int, device) -> tuple:
    """(the workspace, which has to live until the call, its address, its size)."""
    if not need:
        return None, None, 0
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    return ws, ws.data_ptr(), need


def int8_quantize(x: torch.Tensor, axis: int | None = 1):
    """Q(x) of x [R, C] (any strides): with axis=1 the [R, C] Int8Tensor with a scale for each row of x, with axis=0 the
    [C, R] Int8Tensor of its transpose, with a scale for each column; with axis=None both. A row (column) with an infinity or a
    NaN reads as NaN."""
    dt = _matrix(x, "x")
    _check_axis(axis)
    (R, C), (sr, sc), device = x.shape, x.stride(), x.device
    rows = Int8Tensor._empty(R, C, device) if axis != 0 else None
    cols = Int8Tensor._empty(C, R, device) if axis != 1 else None
    ws, at, need = _scratch(_workspace_bytes("svdq_i8_quantize_workspace_bytes", R, C, sr, sc, axis != 0, axis != 1), device)
    _call(L.load().svdq_i8_quantize, device.index, x.data_ptr(), R, C, sr, sc, dt, *_parts(rows), *_parts(cols), at, need)
    return (rows, cols) if axis is None else (rows if axis == 1 else cols)


def int8_dequantize(t: Int8Tensor, dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values of an Int8Tensor as a [rows, cols] tensor: code times scale in float32, rounded to dtype."""
    _i8(t, "t")
    code = _dtype_code(dtype)
    device = t.data.device
    out = _output(out, t.rows, t.cols, dtype, device, t.data)
    _call(L.load().svdq_i8_dequantize, device.index, *_parts(t), t.rows, t.cols, code, out.data_ptr(), _rows(out)[1])
    return out


def int8_matmul(a, b: Int8Tensor, bias: torch.Tensor | None = None, dtype: torch.dtype | None = None,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """Y = A B^T (+ bias) [M, N] of a [M, K] and b [N, K]: exact integer sums, times the scales of their row and column plus the bias in
    float32 (float64 where a scale is far from 1), rounded once to dtype; an output depends on its row of a and of b and its bias
    alone, bit for bit, whatever M and N. a: an Int8Tensor, or a matrix, which is quantised along
    its rows. dtype: a matrix's own, else bfloat16. bias: [N] of that dtype. For a layer with weight [K, N],
    b = int8_quantize(weight, axis=0)."""
    _i8(b, "b")
    raw = isinstance(a, torch.Tensor)
    if raw:
        _matrix(a, "a")
        if dtype is None:
            dtype = a.dtype
        elif dtype != a.dtype:
            a, raw = int8_quantize(a), False
    else:
        _i8(a, "a")
        dtype = dtype or torch.bfloat16
    code = _dtype_code(dtype)
    (M, K), device, N = a.shape, a.device, b.rows
    if K != b.cols:
        raise ValueError(f"a [{M}, {K}] and b [{N}, {b.cols}] must share their second dimension")
    at_bias = None
    if bias is not None:
        if not isinstance(bias, torch.Tensor):
            raise TypeError("bias: expected a torch.Tensor")
        if bias.dim() != 1 or bias.shape[0] != N or bias.dtype != dtype:
            raise ValueError(f"bias must be a [{N}] tensor of the output's dtype")
        _no_graph(bias, "bias")
        bias = bias.contiguous()
        at_bias = bias.data_ptr()
    _same_device(device, b, bias)
    y = _output(out, M, N, dtype, device, a if raw else a.data, b.data, bias)
    lib = L.load()
    if raw:
        sr, sc = a.stride()
        sc = 1 if K == 1 else sc
        ws, at, need = _scratch(_workspace_bytes("svdq_i8_linear_workspace_bytes", M, N, K, sr, sc, code), device)
        _call(lib.svdq_i8_linear, device.index, a.data_ptr(), M, K, sr, sc, *_parts(b), N, at_bias, code, y.data_ptr(), _rows(y)[1],
              at, need)
    else:
        ws, at, need = _scratch(_workspace_bytes("svdq_i8_workspace_bytes", M, N, K), device)
        _call(lib.svdq_i8_matmul, device.index, *_parts(a), M, *_parts(b), N, K, at_bias, code, y.data_ptr(), _rows(y)[1], at, need)
    return y


def int8_backward(dy: torch.Tensor, w_rows: Int8Tensor, x_cols: Int8Tensor, bias: bool = False, dtype: torch.dtype | None = None):
    """(dx [M, K], dw [K, N]) of y = int8_matmul(x, w) from dy [M, N]: dx = Q(dy) Q(w)^T and dw = Q(x^T) Q(dy^T)^T; with bias=True
    also db [N], the sums of dy's columns. w_rows: the weight [K, N] quantised along its rows (axis=1); x_cols: the input quantised
    along its columns (axis=0), [K, M]. dtype: of the gradients, dy's by default."""
    dt = _matrix(dy, "dy")
    _i8(w_rows, "w_rows")
    _i8(x_cols, "x_cols")
    (M, N), K, device = dy.shape, w_rows.rows, dy.device
    if w_rows.cols != N or x_cols.cols != M or x_cols.rows != K:
        raise ValueError(f"w_rows must be [K, {N}] and x_cols [K, {M}]")
    _same_device(device, w_rows, x_cols)
    dtype = dtype or dy.dtype
    out = _dtype_code(dtype)
    dy, ldy = _rows(dy)
    dx = torch.empty(M, K, dtype=dtype, device=device)
    dw = torch.empty(K, N, dtype=dtype, device=device)
    db = torch.empty(N, dtype=dtype, device=device) if bias else None
    ws, at, need = _scratch(_workspace_bytes("svdq_i8_backward_workspace_bytes", M, N, K), device)
    _call(L.load().svdq_i8_backward, device.index, dy.data_ptr(), ldy, M, N, dt, *_parts(w_rows), *_parts(x_cols), K, out,
          dx.data_ptr(), K, dw.data_ptr(), N, db.data_ptr() if bias else None, at, need)
    return (dx, dw, db) if bias else (dx, dw)
