"""MXFP4 tensors made on the device, and the operators on them.

An MxTensor holds Q(x) of a matrix x [rows, K]: for each run of 32 elements along K a power of two
and 4-bit E2M1 codes, the format of `linear`'s residual weights (without a smoothing scale or
low-rank factors). Its products sum over K, so a matrix that enters products along both axes (a
weight in a forward and a backward pass) is quantised along both, in one pass over it.

A gated feed-forward block with x [B, K] and the merged weight w = [gate | up] of [K, 2F], in
training (the quantisers pass gradients straight through):

    x_rows, x_cols = mx_quantize(x, axis=None)
    w_rows, w_cols = mx_quantize(w, axis=None)
    h, gu = mx_gated(x_rows, w_cols, act="silu", save=True)       # h [B, F]
    dx, dw = mx_gated_backward(dh, gu, w_rows, x_cols, act="silu")

and in serving `h = mx_gated(x, w_cols)`, with w_cols kept. Every arithmetic step runs in libsvdq;
tensors are float32, bfloat16 or float16 on a GPU. The calls record no autograd graph: a training step runs them
under torch.no_grad() or inside a torch.autograd.Function, and an input that requires grad is refused elsewhere.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib as L
from .api import _check_int

_DT = {torch.float32: L.SVDQ_F32, torch.bfloat16: L.SVDQ_BF16, torch.float16: L.SVDQ_F16}
_ACT = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}


@functools.lru_cache(maxsize=4096)
def _bytes(rows: int, cols: int) -> tuple:
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    L.check(L.load().svdq_mx_layout(rows, cols, ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


class MxTensor:
    """An MXFP4 tensor on the device: the values Q(x) of a [rows, cols] matrix, blocks along cols.

    data: one uint8 array, the codes and behind them the scale bytes, in the layout of svdq_mx_layout. It
    may be saved and restored with torch; the padding rows of its last tiles hold nothing.
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
    def _empty(cls, rows: int, cols: int, device) -> "MxTensor":
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
        return self.data[: self._at]

    @property
    def scales(self) -> torch.Tensor:
        return self.data[self._at: sum(_bytes(self.rows, self.cols))]

    def __repr__(self) -> str:
        return f"MxTensor([{self.rows}, {self.cols}], device={self.data.device})"


def _dtype_code(dtype) -> int:
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}: float32, bfloat16 or float16")
    return _DT[dtype]


def _act_code(act: str) -> int:
    if act not in _ACT:
        raise ValueError(f"act must be one of {sorted(_ACT)}, got {act!r}")
    return _ACT[act]


def _matrix(t, name: str) -> int:
    """The dtype code of a nonempty matrix on a GPU."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise RuntimeError("libsvdq device calls need tensors on an AMD GPU (HIP device)")
    if t.dim() != 2 or t.numel() == 0:
        raise ValueError(f"{name} must be a nonempty matrix")
    _no_graph(t, name)
    return _dtype_code(t.dtype)


def _no_graph(t: torch.Tensor, name: str) -> None:
    """Refuses an input whose gradient would be lost in silence."""
    if t.requires_grad and torch.is_grad_enabled():
        raise RuntimeError(f"{name} requires grad, and this call records no graph: detach it, or call under torch.no_grad() or in a "
                           "torch.autograd.Function, whose backward calls mx_gated_backward, int8_backward or layer_norm_backward")


def _mx(t, name: str) -> None:
    if not isinstance(t, MxTensor):
        raise TypeError(f"{name}: expected an MxTensor")
    if not t.data.is_cuda:
        raise RuntimeError("libsvdq device calls need tensors on an AMD GPU (HIP device)")


def _same_device(device, *ts) -> None:
    for t in ts:
        if t is not None and t.device != device:
            raise ValueError("all tensors of a call must be on one device")


def _call(fn, index: int, *args) -> None:
    """A libsvdq call on the current stream of device `index`, which is the current device meanwhile."""
    # the stream's handle and the device's index as torch's own wrappers read them, without their objects
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status:
        L.check(status)


def _parts(t) -> tuple:
    if t is None:
        return None, None
    at = t.data.data_ptr()
    return at, at + t._at


def _overlap(out: torch.Tensor, t: torch.Tensor) -> bool:
    """Whether an element of t may lie in out (a checked output)."""
    size, other = out.element_size(), t.element_size()
    a, b = out.data_ptr(), t.data_ptr()
    ld, cols = out.stride(0) * size, out.shape[1] * size
    if a + (out.shape[0] - 1) * ld + cols <= b or b + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * other <= a:
        return False
    # columns beside the output's in the rows of one buffer (whose rows do not overlap: a single row's stride may be anything)
    beside = t.dim() == 2 and t.stride(1) == 1 and t.stride(0) * other == ld >= cols
    return not (beside and cols <= (b - a) % ld and (b - a) % ld + t.shape[1] * other <= ld)


def _output(out, rows: int, cols: int, dtype, device, *inputs) -> torch.Tensor:
    if out is None:
        return torch.empty(rows, cols, dtype=dtype, device=device)
    if not isinstance(out, torch.Tensor) or out.shape != (rows, cols) or out.dtype != dtype or out.device != device:
        raise ValueError(f"out must be a [{rows}, {cols}] {dtype} tensor on {device}")
    if (cols > 1 and out.stride(1) != 1) or (rows > 1 and out.stride(0) < cols):
        raise ValueError("out must have unit column stride and rows that do not overlap")
    _no_graph(out, "out")
    if any(t is not None and _overlap(out, t) for t in inputs):
        raise ValueError("out must not overlap an input")
    return out


def _rows(t: torch.Tensor) -> tuple:
    """(t or a copy of it with unit column stride and rows that do not overlap, its row stride)."""
    (rows, cols), (ld, step) = t.shape, t.stride()
    if step == 1 or cols == 1:
        if ld >= cols:
            return t, ld
        if rows == 1:
            return t, cols  # a single row may have any stride
    return t.contiguous(), cols


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(name: str, *sizes) -> int:
    need = ctypes.c_size_t()
    L.check(getattr(L.load(), name)(*sizes, ctypes.byref(need)))
    return need.value


def _check_axis(axis) -> None:
    if axis is not None and (isinstance(axis, bool) or axis not in (0, 1)):
        raise ValueError("axis must be 0, 1 or None")


def mx_quantize(x: torch.Tensor, axis: int | None = 1):
    """Q(x) of x [R, C] (any strides): with axis=1 the [R, C] MxTensor whose blocks run along the rows of
    x, with axis=0 the [C, R] MxTensor of its transpose, whose blocks run along its columns; with
    axis=None both, from one pass over x. A block with an infinity or a NaN reads as NaN."""
    dt = _matrix(x, "x")
    _check_axis(axis)
    (R, C), (sr, sc), device = x.shape, x.stride(), x.device
    rows = MxTensor._empty(R, C, device) if axis != 0 else None
    cols = MxTensor._empty(C, R, device) if axis != 1 else None
    _call(L.load().svdq_mx_quantize, device.index, x.data_ptr(), R, C, sr, sc, dt, *_parts(rows), *_parts(cols))
    return (rows, cols) if axis is None else (rows if axis == 1 else cols)


def mx_dequantize(t: MxTensor, dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values of an MxTensor as a [rows, cols] tensor (exact in float32 and bfloat16)."""
    _mx(t, "t")
    code = _dtype_code(dtype)
    device = t.data.device
    out = _output(out, t.rows, t.cols, dtype, device, t.data)
    _call(L.load().svdq_mx_dequantize, device.index, *_parts(t), t.rows, t.cols, code, out.data_ptr(), _rows(out)[1])
    return out


def _product(a, b, names, dtype, out, bias=None, act=None, save=False) -> tuple:
    """(y or h, gu or None) of the four product calls: gated with an activation's code in `act`."""
    _mx(b, names[1])
    raw = isinstance(a, torch.Tensor)
    if raw:
        _matrix(a, names[0])
        if dtype is None:
            dtype = a.dtype
        elif dtype != a.dtype:
            a, raw = mx_quantize(a), False
    else:
        _mx(a, names[0])
        dtype = dtype or torch.bfloat16
    code = _dtype_code(dtype)
    (M, K), device, gated = a.shape, a.device, act is not None
    if K != b.cols:
        raise ValueError(f"{names[0]} [{M}, {K}] and {names[1]} [{b.rows}, {b.cols}] must share their second dimension")
    _same_device(device, b, bias)
    N, extra, gu, at_gu = b.rows, act, None, None
    if gated:
        if N % 2:
            raise ValueError(f"{names[1]} must hold as many up rows as gate rows")
        N //= 2
        if save:
            gu = torch.empty(M, 2 * N, dtype=dtype, device=device)
            at_gu = gu.data_ptr()
    elif bias is not None:
        if bias.dim() != 1 or bias.shape[0] != N or bias.dtype != dtype:
            raise ValueError(f"bias must be a [{N}] tensor of the output's dtype")
        _no_graph(bias, "bias")
        bias = bias.contiguous()
        extra = bias.data_ptr()
    y = _output(out, M, N, dtype, device, a if raw else a.data, b.data, bias)
    if raw:
        sr, sc = a.stride()
        need = _workspace_bytes("svdq_mx_linear_workspace_bytes_of", M, N, K, 1 if K == 1 else sc, gated, code)
    else:
        need = _workspace_bytes("svdq_mx_workspace_bytes", M, N, K, gated)
    ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    tail = (y.data_ptr(), _rows(y)[1]) + ((at_gu, 2 * N) if gated else ()) + (ws.data_ptr() if need else None, need)
    lib = L.load()
    if raw:
        _call(lib.svdq_mx_gated_linear if gated else lib.svdq_mx_linear, device.index, a.data_ptr(), M, K, sr,
              1 if K == 1 else sc, *_parts(b), N, extra, code, *tail)
    else:
        _call(lib.svdq_mx_gated if gated else lib.svdq_mx_matmul, device.index, *_parts(a), M, *_parts(b), N, K, extra, code,
              *tail)
    return y, gu


def mx_matmul(a, b: MxTensor, bias: torch.Tensor | None = None, dtype: torch.dtype | None = None,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """Y = A B^T (+ bias) [M, N] of a [M, K] and b [N, K]: MXFP4 products summed in float32, rounded once.
    a: an MxTensor, or a matrix, which is quantised along its rows. dtype: a matrix's own, else
    bfloat16. bias: [N] of that dtype. For a layer with weight [K, N], b = mx_quantize(weight, axis=0)."""
    if bias is not None and not isinstance(bias, torch.Tensor):
        raise TypeError("bias: expected a torch.Tensor")
    return _product(a, b, ("a", "b"), dtype, out, bias=bias)[0]


def mx_gated(x, w: MxTensor, act: str = "silu", dtype: torch.dtype | None = None, save: bool = False,
             out: torch.Tensor | None = None):
    """h = act(x Wg^T) * (x Wu^T) [M, F], both projections in one kernel. x: an MxTensor or a matrix
    [M, K], as in mx_matmul. w: [2F, K], the F gate rows, then the F up rows: mx_quantize(weight, axis=0) of
    the merged weight [K, 2F]. act: "silu", "gelu", "gelu_tanh" or "relu". With save=True also returns the
    pre-activations [M, 2F] (gate, then up), rounded to the dtype, for mx_gated_backward."""
    h, gu = _product(x, w, ("x", "w"), dtype, out, act=_act_code(act), save=save)
    return (h, gu) if save else h


def _pre_activations(dh, gu) -> tuple:
    """(dtype code, M, F, device, dh, its row stride, gu, its row stride) of a backward call's gradient and saved
    pre-activations."""
    dt = _matrix(dh, "dh")
    _matrix(gu, "gu")
    M, F = dh.shape
    if gu.shape != (M, 2 * F) or gu.dtype != dh.dtype:
        raise ValueError(f"gu must be a [{M}, {2 * F}] tensor of dh's dtype")
    device = dh.device
    _same_device(device, gu)
    return dt, M, F, device, *_rows(dh), *_rows(gu)


def mx_gated_grad(dh: torch.Tensor, gu: torch.Tensor, act: str = "silu", axis: int | None = None):
    """The gradients d = [dg | du] of a gated block's pre-activations, dg = dh * u * act'(g) and
    du = dh * act(g), from dh [M, F] and gu [M, 2F]: Q(d) [M, 2F] and Q(d^T) [2F, M], from one pass; with axis=1
    Q(d) alone (all that dx needs), with axis=0 Q(d^T) alone (all that dw needs)."""
    code = _act_code(act)
    _check_axis(axis)
    dt, M, F, device, dh, ldh, gu, ldgu = _pre_activations(dh, gu)
    rows = MxTensor._empty(M, 2 * F, device) if axis != 0 else None
    cols = MxTensor._empty(2 * F, M, device) if axis != 1 else None
    _call(L.load().svdq_mx_gated_grad, device.index, dh.data_ptr(), ldh, gu.data_ptr(), ldgu, M, F, code, dt, *_parts(rows),
          *_parts(cols))
    return (rows, cols) if axis is None else (rows if axis == 1 else cols)


def mx_gated_backward(dh: torch.Tensor, gu: torch.Tensor, w_rows: MxTensor, x_cols: MxTensor, act: str = "silu",
                      dtype: torch.dtype | None = None):
    """(dx [M, K], dw [K, 2F]) of h = mx_gated(x, w): dx = Q(d) Q(w)^T and dw = Q(x^T) Q(d^T)^T with the d of
    mx_gated_grad. w_rows: the merged weight [K, 2F] quantised along its rows (axis=1); x_cols: the input
    quantised along its columns (axis=0), [K, M]. dtype: of the gradients, dh's by default."""
    code = _act_code(act)
    _mx(w_rows, "w_rows")
    _mx(x_cols, "x_cols")
    dt, M, F, device, dh, ldh, gu, ldgu = _pre_activations(dh, gu)
    K = w_rows.rows
    if w_rows.cols != 2 * F or x_cols.cols != M or x_cols.rows != K:
        raise ValueError(f"w_rows must be [K, {2 * F}] and x_cols [K, {M}]")
    _same_device(device, w_rows, x_cols)
    dtype = dtype or dh.dtype
    out = _dtype_code(dtype)
    dx = torch.empty(M, K, dtype=dtype, device=device)
    dw = torch.empty(K, 2 * F, dtype=dtype, device=device)
    need = _workspace_bytes("svdq_mx_gated_backward_workspace_bytes", M, F, K)
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    _call(L.load().svdq_mx_gated_backward, device.index, dh.data_ptr(), ldh, gu.data_ptr(), ldgu, M, F, code, dt,
          *_parts(w_rows), *_parts(x_cols), K, out, dx.data_ptr(), K, dw.data_ptr(), 2 * F, ws.data_ptr(), need)
    return dx, dw
