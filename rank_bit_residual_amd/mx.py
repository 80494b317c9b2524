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
tensors are float32, bfloat16 or float16 on a GPU.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib as L

_DT = {torch.float32: L.SVDQ_F32, torch.bfloat16: L.SVDQ_BF16, torch.float16: L.SVDQ_F16}
_ACT = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}


@dataclass(frozen=True, eq=False)
class MxTensor:
    """An MXFP4 tensor on the device: the values Q(x) of a [rows, cols] matrix, blocks along cols.

    codes, scales: uint8 arrays in the layout of svdq_mx_layout (they may be saved and restored
    with torch; rows past `rows` of the last tiles hold nothing).
    """

    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int

    @property
    def shape(self) -> tuple:
        return (self.rows, self.cols)

    @property
    def device(self) -> torch.device:
        return self.codes.device


def _dtype_code(dtype) -> int:
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}: float32, bfloat16 or float16")
    return _DT[dtype]


def _act_code(act: str) -> int:
    if act not in _ACT:
        raise ValueError(f"act must be one of {sorted(_ACT)}, got {act!r}")
    return _ACT[act]


def _matrix(t, name: str) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise RuntimeError("libsvdq device calls need tensors on an AMD GPU (HIP device)")
    if t.dim() != 2 or t.shape[0] < 1 or t.shape[1] < 1:
        raise ValueError(f"{name} must be a nonempty matrix")
    _dtype_code(t.dtype)


def _mx(t, name: str) -> None:
    if not isinstance(t, MxTensor):
        raise TypeError(f"{name}: expected an MxTensor")
    code_bytes, scale_bytes = _bytes(t.rows, t.cols)
    for part, need in ((t.codes, code_bytes), (t.scales, scale_bytes)):
        if not isinstance(part, torch.Tensor) or part.dtype != torch.uint8 or not part.is_contiguous():
            raise TypeError(f"{name}: codes and scales must be contiguous uint8 tensors")
        if part.numel() < need:
            raise ValueError(f"{name}: codes or scales shorter than its shape needs")
    if not t.codes.is_cuda:
        raise RuntimeError("libsvdq device calls need tensors on an AMD GPU (HIP device)")
    if t.scales.device != t.codes.device:
        raise ValueError(f"{name}: codes and scales must be on one device")


def _same_device(*ts) -> torch.device:
    dev = ts[0].device
    for t in ts[1:]:
        if t is not None and t.device != dev:
            raise ValueError("all tensors of a call must be on one device")
    return dev


def _bytes(rows: int, cols: int) -> tuple:
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    L.check(L.load().svdq_mx_layout(rows, cols, ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def _empty(rows: int, cols: int, device) -> MxTensor:
    code_bytes, scale_bytes = _bytes(rows, cols)
    return MxTensor(torch.empty(code_bytes, dtype=torch.uint8, device=device),
                    torch.empty(scale_bytes, dtype=torch.uint8, device=device), rows, cols)


def _call(name: str, device, *args) -> None:
    """libsvdq's `name` on the current stream of `device`, which is the current device meanwhile."""
    fn = getattr(L.load(), name)
    if torch.cuda.current_device() == device.index:
        L.check(fn(*args, torch.cuda.current_stream(device).cuda_stream))
    else:
        with torch.cuda.device(device):
            L.check(fn(*args, torch.cuda.current_stream(device).cuda_stream))


def _parts(t) -> tuple:
    return (None, None) if t is None else (t.codes.data_ptr(), t.scales.data_ptr())


def _output(out, rows: int, cols: int, dtype, device, name: str = "out") -> torch.Tensor:
    if out is None:
        return torch.empty((rows, cols), dtype=dtype, device=device)
    if not isinstance(out, torch.Tensor) or out.shape != (rows, cols) or out.dtype != dtype or out.device != device:
        raise ValueError(f"{name} must be a [{rows}, {cols}] {dtype} tensor on {device}")
    if (cols > 1 and out.stride(1) != 1) or (rows > 1 and out.stride(0) < cols):
        raise ValueError(f"{name} must have unit column stride and rows that do not overlap")
    return out


def _row_stride(t: torch.Tensor) -> int:
    return max(t.stride(0), t.shape[1])  # a single row may have any stride


def _unit_columns(t: torch.Tensor) -> torch.Tensor:
    if (t.shape[1] == 1 or t.stride(1) == 1) and (t.shape[0] == 1 or t.stride(0) >= t.shape[1]):
        return t
    return t.contiguous()


def mx_quantize(x: torch.Tensor, axis: int | None = 1):
    """Q(x) of x [R, C] (any strides): with axis=1 the [R, C] MxTensor whose blocks run along the rows of
    x, with axis=0 the [C, R] MxTensor of its transpose, whose blocks run along its columns; with
    axis=None both, from one pass over x. A block with an infinity or a NaN reads as NaN."""
    _matrix(x, "x")
    if axis is not None and (isinstance(axis, bool) or axis not in (0, 1)):
        raise ValueError("axis must be 0, 1 or None")
    R, C = x.shape
    rows = _empty(R, C, x.device) if axis != 0 else None
    cols = _empty(C, R, x.device) if axis != 1 else None
    _call("svdq_mx_quantize", x.device, x.data_ptr(), R, C, x.stride(0), x.stride(1), _DT[x.dtype], *_parts(rows),
          *_parts(cols))
    return (rows, cols) if axis is None else (rows if axis == 1 else cols)


def mx_dequantize(t: MxTensor, dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values of an MxTensor as a [rows, cols] tensor (exact in float32 and bfloat16)."""
    _mx(t, "t")
    code = _dtype_code(dtype)
    out = _output(out, t.rows, t.cols, dtype, t.device)
    _call("svdq_mx_dequantize", t.device, *_parts(t), t.rows, t.cols, code, out.data_ptr(), _row_stride(out))
    return out


def _workspace(M: int, N: int, K: int, gated: bool, device) -> tuple:
    """(tensor, address, bytes) of a product's scratch, from the current stream's memory."""
    need = ctypes.c_size_t()
    L.check(L.load().svdq_mx_workspace_bytes(M, N, K, gated, ctypes.byref(need)))
    if not need.value:
        return None, None, 0
    ws = torch.empty(need.value, dtype=torch.uint8, device=device)
    return ws, ws.data_ptr(), need.value


def _operand(a, name: str, dtype):
    """An MxTensor and the output dtype: a matrix is quantised along its rows, its dtype the default."""
    if isinstance(a, torch.Tensor):
        return mx_quantize(a), dtype or a.dtype
    _mx(a, name)
    return a, dtype or torch.bfloat16


def mx_matmul(a, b: MxTensor, bias: torch.Tensor | None = None, dtype: torch.dtype | None = None,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """Y = A B^T (+ bias) [M, N] of a [M, K] and b [N, K]: MXFP4 products summed in float32, rounded once.
    a: an MxTensor, or a matrix, which is quantised along its rows first. dtype: a matrix's own, else
    bfloat16. bias: [N] of that dtype. For a layer with weight [K, N], b = mx_quantize(weight, axis=0)."""
    _mx(b, "b")
    a, dtype = _operand(a, "a", dtype)
    code = _dtype_code(dtype)
    if a.cols != b.cols:
        raise ValueError(f"a [{a.rows}, {a.cols}] and b [{b.rows}, {b.cols}] must share their second dimension")
    device = _same_device(a, b, bias)
    if bias is not None:
        if bias.dim() != 1 or bias.shape[0] != b.rows or bias.dtype != dtype:
            raise ValueError(f"bias must be a [{b.rows}] tensor of the output's dtype")
        bias = bias.contiguous()
    y = _output(out, a.rows, b.rows, dtype, device)
    _keep, *ws = _workspace(a.rows, b.rows, a.cols, False, device)
    _call("svdq_mx_matmul", device, *_parts(a), a.rows, *_parts(b), b.rows, a.cols,
          None if bias is None else bias.data_ptr(), code, y.data_ptr(), _row_stride(y), *ws)
    return y


def mx_gated(x, w: MxTensor, act: str = "silu", dtype: torch.dtype | None = None, save: bool = False,
             out: torch.Tensor | None = None):
    """h = act(x Wg^T) * (x Wu^T) [M, F], both projections in one kernel. x: an MxTensor or a matrix
    [M, K], as in mx_matmul. w: [2F, K], the F gate rows, then the F up rows: mx_quantize(weight, axis=0) of
    the merged weight [K, 2F]. act: "silu", "gelu", "gelu_tanh" or "relu". With save=True also returns the
    pre-activations [M, 2F] (gate, then up), rounded to the dtype, for mx_gated_backward."""
    code = _act_code(act)
    _mx(w, "w")
    x, dtype = _operand(x, "x", dtype)
    dt = _dtype_code(dtype)
    if w.rows % 2:
        raise ValueError("w must hold as many up rows as gate rows")
    if x.cols != w.cols:
        raise ValueError(f"x [{x.rows}, {x.cols}] and w [{w.rows}, {w.cols}] must share their second dimension")
    device = _same_device(x, w)
    M, F = x.rows, w.rows // 2
    h = _output(out, M, F, dtype, device)
    gu = torch.empty((M, 2 * F), dtype=dtype, device=device) if save else None
    _keep, *ws = _workspace(M, F, x.cols, True, device)
    _call("svdq_mx_gated", device, *_parts(x), M, *_parts(w), F, x.cols, code, dt, h.data_ptr(), _row_stride(h),
          None if gu is None else gu.data_ptr(), 2 * F, *ws)
    return (h, gu) if save else h


def mx_gated_grad(dh: torch.Tensor, gu: torch.Tensor, act: str = "silu"):
    """The gradients d = [dg | du] of a gated block's pre-activations, dg = dh * u * act'(g) and
    du = dh * act(g), from dh [M, F] and gu [M, 2F]: Q(d) [M, 2F] and Q(d^T) [2F, M], from one pass."""
    code = _act_code(act)
    _matrix(dh, "dh")
    _matrix(gu, "gu")
    M, F = dh.shape
    if gu.shape != (M, 2 * F) or gu.dtype != dh.dtype:
        raise ValueError(f"gu must be a [{M}, {2 * F}] tensor of dh's dtype")
    device = _same_device(dh, gu)
    dh, gu = _unit_columns(dh), _unit_columns(gu)
    rows, cols = _empty(M, 2 * F, device), _empty(2 * F, M, device)
    _call("svdq_mx_gated_grad", device, dh.data_ptr(), _row_stride(dh), gu.data_ptr(), _row_stride(gu), M, F, code,
          _DT[dh.dtype], *_parts(rows), *_parts(cols))
    return rows, cols


def mx_gated_backward(dh: torch.Tensor, gu: torch.Tensor, w_rows: MxTensor, x_cols: MxTensor, act: str = "silu",
                      dtype: torch.dtype | None = None):
    """(dx [M, K], dw [K, 2F]) of h = mx_gated(x, w): dx = Q(d) Q(w)^T and dw = Q(x^T) Q(d^T)^T with the d of
    mx_gated_grad. w_rows: the merged weight [K, 2F] quantised along its rows (axis=1); x_cols: the input
    quantised along its columns (axis=0), [K, M]. dtype: of the gradients, dh's by default."""
    _mx(w_rows, "w_rows")
    _mx(x_cols, "x_cols")
    _matrix(dh, "dh")
    M, F = dh.shape
    if w_rows.cols != 2 * F or x_cols.cols != M or w_rows.rows != x_cols.rows:
        raise ValueError(f"w_rows must be [K, {2 * F}] and x_cols [K, {M}]")
    _same_device(dh, w_rows, x_cols)
    dtype = dtype or dh.dtype
    _dtype_code(dtype)
    rows, cols = mx_gated_grad(dh, gu, act)
    return mx_matmul(rows, w_rows, dtype=dtype), mx_matmul(x_cols, cols, dtype=dtype)
