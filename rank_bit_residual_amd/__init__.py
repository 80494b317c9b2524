"""SVDQuant linear operator for AMD Instinct MI355X (gfx950).

Y = (X^ L1) L2 + Q(X^) Q(R): smoothed activations X^ = x / scale, a rank-r truncated
SVD L1 L2 of the smoothed weight, and the 4-bit (per-tensor INT or MXFP4) residual R.
The per-call path is hand-written HIP in libsvdq.so; this package is its ctypes binding.
MXFP4 tensors made on the device, their products and a gated feed-forward block's projections
with their backward pass are the mx_* functions (mx.py); 8-bit tensors with a scale for each row,
their products and a linear layer's backward pass the int8_* functions (int8.py); layer norm, which
makes either kind of tensor, and its backward pass are in norm.py.
"""
from .api import (Prepared, calibrate_scale, fake_quantize, linear, prepare, prepared_layout, quantize_activations,
                  smooth_inputs, split_weight, svdquant_linear, workspace_bytes)
from .int8 import Int8Tensor, int8_backward, int8_dequantize, int8_matmul, int8_quantize
from .mx import MxTensor, mx_dequantize, mx_gated, mx_gated_backward, mx_gated_grad, mx_matmul, mx_quantize
from .norm import layer_norm, layer_norm_backward

__all__ = ["Int8Tensor", "MxTensor", "Prepared", "calibrate_scale", "fake_quantize", "int8_backward", "int8_dequantize",
           "int8_matmul", "int8_quantize", "layer_norm", "layer_norm_backward", "linear", "mx_dequantize", "mx_gated",
           "mx_gated_backward", "mx_gated_grad", "mx_matmul", "mx_quantize", "prepare", "prepared_layout",
           "quantize_activations", "smooth_inputs", "split_weight", "svdquant_linear", "workspace_bytes"]
