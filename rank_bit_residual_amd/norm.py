"""Layer norm, with an 8-bit or MXFP4 tensor as its output where a product follows, and its backward pass.

A pre-norm block's first layer, in serving (w_cols = int8_quantize(w, axis=0), or mx_quantize(w, axis=0)):

    y = int8_matmul(layer_norm(x, weight, bias, quantize="int8"), w_cols)
    h = mx_gated(layer_norm(x, weight, bias, quantize="mx"), w_cols)

and in training

    y, mean, rstd = layer_norm(x, weight, bias, save=True)
    dx, dweight, dbias = layer_norm_backward(dy, x, mean, rstd, weight)

Every arithmetic step runs in libsvdq; x is float32, bfloat16 or float16 on a GPU, weight and bias are of its type or float32.
The calls record no autograd graph, like those of mx.py.
"""
from __future__ import annotations

import torch

from . import _lib as L
from .int8 import Int8Tensor, _scratch
from .mx import _DT, MxTensor, _call, _matrix, _no_graph, _output, _parts, _rows, _same_device, _workspace_bytes


def _param(t, name: str, K: int, dtype, device) -> torch.Tensor:
    """A [K] vector of x's dtype or float32, with unit stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dim() != 1 or t.shape[0] != K or (t.dtype != dtype and t.dtype != torch.float32):
        raise ValueError(f"{name} must be a [{K}] tensor of x's dtype or float32")
    if t.device != device:
        raise ValueError("all tensors of a call must be on one device")
    _no_graph(t, name)
    return t if t.is_contiguous() else t.contiguous()


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, eps: float = 1e-5,
               quantize: str | None = None, save: bool = False, out: torch.Tensor | None = None):
    """y = (x - mean) / sqrt(var + eps) * weight + bias of each row of x [M, K] (var: the mean square of x - mean), computed in
    float64, rounded to float32 and then to x's dtype; with quantize="int8" or "mx" the Int8Tensor or MxTensor of the float32
    values instead. weight, bias: [K], both of x's dtype or both float32; a bias needs a weight. With save=True also returns
    mean and rstd = 1 / sqrt(var + eps), float32 [M], for layer_norm_backward."""
    dt = _matrix(x, "x")
    if quantize not in (None, "int8", "mx"):
        raise ValueError(f"quantize must be None, 'int8' or 'mx', got {quantize!r}")
    if quantize is not None and out is not None:
        raise ValueError("a quantised norm takes no out")
    if isinstance(eps, bool) or not isinstance(eps, (int, float)):
        raise TypeError("eps must be a number")
    if bias is not None and weight is None:
        raise ValueError("a bias needs a weight")
    (M, K), device = x.shape, x.device
    pt = dt
    if weight is not None:
        weight = _param(weight, "weight", K, x.dtype, device)
        pt = _DT[weight.dtype]
        if bias is not None:
            bias = _param(bias, "bias", K, x.dtype, device)
            if bias.dtype != weight.dtype:
                raise ValueError("weight and bias must share one dtype")
    x, ldx = _rows(x)
    if quantize is None:
        y = _output(out, M, K, x.dtype, device, x, weight, bias)
        fn, result, tail = L.load().svdq_layer_norm, y, (y.data_ptr(), _rows(y)[1])
    elif quantize == "int8":
        result = Int8Tensor._empty(M, K, device)
        fn, tail = L.load().svdq_layer_norm_i8, _parts(result)
    else:
        result = MxTensor._empty(M, K, device)
        fn, tail = L.load().svdq_layer_norm_mx, _parts(result)
    mean = rstd = None
    if save:
        mean = torch.empty(M, dtype=torch.float32, device=device)
        rstd = torch.empty(M, dtype=torch.float32, device=device)
    _call(fn, device.index, x.data_ptr(), ldx, M, K, weight.data_ptr() if weight is not None else None,
          bias.data_ptr() if bias is not None else None, pt, float(eps), dt, *tail, mean.data_ptr() if save else None,
          rstd.data_ptr() if save else None)
    return (result, mean, rstd) if save else result


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor | None = None):
    """(dx [M, K], dweight [K], dbias [K]) of y = layer_norm(x, weight, bias) from dy [M, K], with the mean and rstd that it saved:
    with xh = (x - mean) rstd and g = dy weight, dx = rstd (g - mean of g - xh times the mean of g xh) over each row, dweight the
    sum of dy xh and dbias the sum of dy over the rows, in weight's dtype (None without a weight). A row's sums are float32, those over
    the rows float32 in groups, through 1030 additions at most, and float64 from there."""
    dt = _matrix(dy, "dy")
    _matrix(x, "x")
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("dy and x must share one shape and dtype")
    (M, K), device = x.shape, x.device
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor")
        if t.shape != (M,) or t.dtype != torch.float32:
            raise ValueError(f"{name} must be a [{M}] float32 tensor")
        _no_graph(t, name)
    _same_device(device, dy, mean, rstd)
    mean = mean if mean.is_contiguous() else mean.contiguous()
    rstd = rstd if rstd.is_contiguous() else rstd.contiguous()
    pt, dweight, dbias = dt, None, None
    if weight is not None:
        weight = _param(weight, "weight", K, x.dtype, device)
        pt = _DT[weight.dtype]
        dweight, dbias = torch.empty_like(weight), torch.empty_like(weight)
    dy, lddy = _rows(dy)
    x, ldx = _rows(x)
    dx = torch.empty(M, K, dtype=x.dtype, device=device)
    ws, at, need = _scratch(_workspace_bytes("svdq_layer_norm_backward_workspace_bytes", M, K, weight is not None), device)
    given = weight is not None
    _call(L.load().svdq_layer_norm_backward, device.index, dy.data_ptr(), lddy, x.data_ptr(), ldx, mean.data_ptr(), rstd.data_ptr(), M,
          K, weight.data_ptr() if given else None, pt, dt, dx.data_ptr(), K, dweight.data_ptr() if given else None,
          dbias.data_ptr() if given else None, at, need)
    return dx, dweight, dbias
