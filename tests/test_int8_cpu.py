"""8-bit tensor and layer norm operators without a GPU: the oracle's own checks, the queries and every refusal."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import rank_bit_residual_amd as R
from oracle import int8 as X
from rank_bit_residual_amd import _lib

A = 1 << 20  # a 256-byte aligned address that no refused call reads
F32, BF16, F64, F16 = _lib.SVDQ_F32, _lib.SVDQ_BF16, _lib.SVDQ_F64, _lib.SVDQ_F16
EINVAL, EDTYPE = _lib.SVDQ_EINVAL, _lib.SVDQ_EDTYPE


# ----------------------------------------------------------------------------- oracle
def test_oracle_codes_are_the_nearest_to_the_real_quotient():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((4, 50)).astype(np.float32)
    x[1] = (np.arange(50) - 25 + 0.5) * np.float32(2.0**-3)
    x[1, 0] = np.float32(127 * 2.0**-3)
    x[2] = 0
    x[3, 7] = np.inf
    codes, s = X.quantize(x.astype(np.float64))
    assert s[2] == 0 and np.isnan(s[3]) and not codes[2:].any()
    for r in (0, 1):
        assert s[r] == np.float32(np.float64(np.abs(x[r]).max()) / 127)
        for v, c in zip(x[r], codes[r]):
            q = Fraction(float(v)) / Fraction(float(s[r]))
            assert abs(q - int(c)) <= Fraction(1, 2) and (abs(q - int(c)) < Fraction(1, 2) or c % 2 == 0)
    v = X.values(x.astype(np.float64))
    assert np.isnan(v[3]).all() and (np.abs(v[:2] - x[:2]) <= s[:2, None] / 2 * 1.0001).all()


def test_oracle_unpack():
    rows, K = 18, 130
    kq = 4
    codes = np.zeros((2, kq, 16, 64), np.int8)
    for r in range(rows):
        for k in range(K):
            codes[r // 16, k // 64, r % 16, k % 64] = (7 * r + 3 * k) % 251 - 125
    got, past = X.unpack(codes.view(np.uint8), rows, K)
    assert np.array_equal(got, (7 * np.arange(rows)[:, None] + 3 * np.arange(K)) % 251 - 125) and not past.any()


def test_oracle_norm_gradient_against_differences():
    rng = np.random.default_rng(3)
    x, dy, w = rng.standard_normal((3, 9)), rng.standard_normal((3, 9)), rng.standard_normal(9)
    _, mean, rstd = X.layer_norm(x)
    dx, dw, db = X.layer_norm_grad(dy, x, mean, rstd, w)
    h = 1e-5
    loss = lambda x, w, b: (dy * X.layer_norm(x, w, b)[0]).sum()  # noqa: E731
    for k in range(9):
        e = np.zeros(9)
        e[k] = h
        assert abs((loss(x, w + e, e * 0) - loss(x, w - e, e * 0)) / (2 * h) - dw[k]) < 1e-8
        assert abs((loss(x, w, e) - loss(x, w, -e)) / (2 * h) - db[k]) < 1e-8
        for m in range(3):
            d = np.zeros_like(x)
            d[m, k] = h
            assert abs((loss(x + d, w, None) - loss(x - d, w, None)) / (2 * h) - dx[m, k]) < 1e-8


# ----------------------------------------------------------------------------- C ABI
def _layout(rows, K):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    st = _lib.load().svdq_i8_layout(rows, K, ctypes.byref(a), ctypes.byref(b))
    return st, a.value, b.value


def test_layout():
    assert _layout(1, 1) == (0, 2 * 1024, 256)
    assert _layout(17, 128) == (0, 2 * 2 * 1024, 256)
    assert _layout(65, 129) == (0, 5 * 4 * 1024, 512)
    assert _layout(1 << 20, 1 << 16) == (0, 1 << 36, 1 << 22)  # past 32 bits
    for rows, K in ((0, 4), (4, 0), (-1, 4), ((1 << 30) + 1, 4), (4, (1 << 30) + 1)):
        assert _layout(rows, K)[0] == EINVAL
    assert _lib.load().svdq_i8_layout(4, 4, None, None) == EINVAL


def _refused(status, st):
    assert st == status, (st, _lib.load().svdq_last_error())
    assert _lib.load().svdq_last_error()


@pytest.mark.parametrize("change,status", [
    (dict(dtype=F64), EDTYPE), (dict(dtype=7), EDTYPE), (dict(R=0), EINVAL), (dict(C=0), EINVAL), (dict(C=(1 << 30) + 1), EINVAL),
    (dict(x=None), EINVAL), (dict(x=A + 1), EINVAL), (dict(sr=-1), EINVAL), (dict(sc=-4), EINVAL), (dict(codes=None), EINVAL),
    (dict(scales=None), EINVAL), (dict(codes=A + 16), EINVAL), (dict(scales_t=None), EINVAL), (dict(codes_t=A + 128), EINVAL),
    (dict(codes=None, scales=None, codes_t=None, scales_t=None), EINVAL), (dict(work=None), EINVAL), (dict(work=A + 64), EINVAL),
    (dict(bytes=256), EINVAL), (dict(C=1 << 29, sr=1 << 29), EINVAL),
])
def test_quantize_refusals(change, status):
    a = dict(x=A, R=4, C=40, sr=40, sc=1, dtype=BF16, codes=A, scales=A, codes_t=A, scales_t=A, work=A, bytes=1 << 50)
    a.update(change)
    _refused(status, _lib.load().svdq_i8_quantize(*a.values(), None))


def _quantize_bytes(R, C, sr, sc, rows, cols):
    n = ctypes.c_size_t()
    assert _lib.load().svdq_i8_quantize_workspace_bytes(R, C, sr, sc, rows, cols, ctypes.byref(n)) == 0
    return n.value


def test_quantize_workspace_query():
    assert _quantize_bytes(100, 300, 300, 1, 1, 0) == 0 and _quantize_bytes(100, 300, 300, 1, 1, 1) >= 300 * 4
    # contiguous columns: the other direction reads the matrix once
    assert _quantize_bytes(100, 300, 1, 100, 0, 1) == 0 and _quantize_bytes(100, 300, 1, 100, 1, 0) >= 100 * 4
    n = ctypes.c_size_t()
    for bad in ((0, 4, 4, 1), (4, 0, 4, 1), (4, 4, -1, 1), (4, 4, 1, -1)):
        _refused(EINVAL, _lib.load().svdq_i8_quantize_workspace_bytes(*bad, 1, 1, ctypes.byref(n)))
    _refused(EINVAL, _lib.load().svdq_i8_quantize_workspace_bytes(4, 4, 4, 1, 1, 1, None))


@pytest.mark.parametrize("change,status", [
    (dict(dtype=F64), EDTYPE), (dict(rows=0), EINVAL), (dict(K=-3), EINVAL), (dict(codes=None), EINVAL), (dict(scales=A + 4), EINVAL),
    (dict(out=None), EINVAL), (dict(out=A + 1), EINVAL), (dict(ldo=39), EINVAL),
])
def test_dequantize_refusals(change, status):
    a = dict(codes=A, scales=A, rows=4, K=40, dtype=F16, out=A, ldo=40)
    a.update(change)
    _refused(status, _lib.load().svdq_i8_dequantize(*a.values(), None))


@pytest.mark.parametrize("change,status", [
    (dict(dtype=F64), EDTYPE), (dict(M=0), EINVAL), (dict(N=0), EINVAL), (dict(K=0), EINVAL), (dict(ac=None), EINVAL),
    (dict(asc=None), EINVAL), (dict(bc=A + 8), EINVAL), (dict(bs=None), EINVAL), (dict(bias=A + 2), EINVAL), (dict(y=None), EINVAL),
    (dict(y=A + 2), EINVAL), (dict(ldy=7), EINVAL), (dict(K=(1 << 26) + 1), EINVAL), (dict(K=1 << 18), EINVAL),
    (dict(K=1 << 18, work=A, bytes=16), EINVAL), (dict(K=1 << 18, work=A + 8, bytes=1 << 40), EINVAL),
    (dict(M=1 << 30, N=1 << 30, ldy=1 << 30), EINVAL),
])
def test_matmul_refusals(change, status):
    a = dict(ac=A, asc=A, M=4, bc=A, bs=A, N=8, K=40, bias=None, dtype=F32, y=A, ldy=8, work=None, bytes=0)
    a.update(change)
    _refused(status, _lib.load().svdq_i8_matmul(*a.values(), None))


@pytest.mark.parametrize("change,status", [
    (dict(dtype=F64), EDTYPE), (dict(M=0), EINVAL), (dict(N=0), EINVAL), (dict(K=0), EINVAL), (dict(x=None), EINVAL),
    (dict(x=A + 2), EINVAL), (dict(sr=-1), EINVAL), (dict(sc=-1), EINVAL), (dict(bc=None), EINVAL), (dict(bs=A + 4), EINVAL),
    (dict(bias=A + 2), EINVAL), (dict(y=None), EINVAL), (dict(ldy=7), EINVAL), (dict(K=(1 << 26) + 1), EINVAL), (dict(M=100), EINVAL),
    (dict(sc=2), EINVAL), (dict(M=100, work=A, bytes=64), EINVAL), (dict(M=100, work=A + 1, bytes=1 << 40), EINVAL),
    (dict(M=1 << 24, N=1 << 17, ldy=1 << 17, work=A, bytes=1 << 60), EINVAL),
])
def test_linear_refusals(change, status):
    a = dict(x=A, M=4, K=40, sr=40, sc=1, bc=A, bs=A, N=8, bias=None, dtype=F32, y=A, ldy=8, work=None, bytes=0)
    a.update(change)
    _refused(status, _lib.load().svdq_i8_linear(*a.values(), None))


@pytest.mark.parametrize("change,status", [
    (dict(dtype=F64), EDTYPE), (dict(out=F64), EDTYPE), (dict(M=0), EINVAL), (dict(N=0), EINVAL), (dict(K=0), EINVAL), (dict(dy=None), EINVAL),
    (dict(lddy=7), EINVAL), (dict(dy=A + 1), EINVAL), (dict(wc=None), EINVAL), (dict(ws=A + 4), EINVAL), (dict(xc=A + 16), EINVAL),
    (dict(xs=None), EINVAL), (dict(dx=None), EINVAL), (dict(lddx=39), EINVAL), (dict(dw=A + 1), EINVAL), (dict(lddw=7), EINVAL),
    (dict(db=A + 2), EINVAL), (dict(work=None), EINVAL), (dict(work=A + 8), EINVAL), (dict(bytes=4096), EINVAL),
    (dict(M=(1 << 26) + 1), EINVAL), (dict(N=(1 << 26) + 1, lddy=1 << 27, lddw=1 << 27), EINVAL),
    (dict(M=1 << 24, K=1 << 17, lddx=1 << 17), EINVAL), (dict(N=1 << 20, K=1 << 24, lddy=1 << 20, lddw=1 << 20, lddx=1 << 24), EINVAL),
])
def test_backward_refusals(change, status):
    """Among them calls of which only one product does not fit a launch: nothing runs (without a GPU a launch that was tried would give
    EHIP)."""
    a = dict(dy=A, lddy=8, M=4, N=8, dtype=BF16, wc=A, ws=A, xc=A, xs=A, K=40, out=F32, dx=A, lddx=40, dw=A, lddw=8, db=A, work=A,
             bytes=1 << 60)
    a.update(change)
    _refused(status, _lib.load().svdq_i8_backward(*a.values(), None))


def _form(M, N, K):
    got = (ctypes.c_int * 4)()
    assert _lib.load().svdq_i8_product_form(M, N, K, got) == 0
    return tuple(got)


def test_product_queries():
    lib, got, n = _lib.load(), (ctypes.c_int * 4)(), ctypes.c_size_t()
    for bad in ((0, 4, 4), (4, 0, 4), (4, 4, 0), (4, 4, (1 << 26) + 1)):
        _refused(EINVAL, lib.svdq_i8_product_form(*bad, got))
        _refused(EINVAL, lib.svdq_i8_workspace_bytes(*bad, ctypes.byref(n)))
    _refused(EINVAL, lib.svdq_i8_product_form(4, 4, 4, None))
    _refused(EINVAL, lib.svdq_i8_workspace_bytes(4, 4, 4, None))
    for M, N, K in ((1, 100, 512), (300, 5000, 4096), (1024, 1024, 65536), (130, 151, 33000), (1, 64, 1 << 20), (500, 500, 1 << 26)):
        bm, bn, splits, waves = _form(M, N, K)
        assert lib.svdq_i8_workspace_bytes(M, N, K, ctypes.byref(n)) == 0
        assert n.value == (splits * M * N * 4 if splits > 1 else 0)
        # int32 holds 2^17 products of 127^2: no block sums more
        pairs = -(-K // 128)
        assert -(-pairs // splits) * 128 <= 1 << 17 and splits <= pairs
        assert waves == 1 or splits == 1


def test_linear_workspace_query():
    lib, n = _lib.load(), ctypes.c_size_t()
    codes, scales = _layout(100, 512)[1:]
    assert lib.svdq_i8_linear_workspace_bytes(100, 256, 512, 512, 1, BF16, ctypes.byref(n)) == 0 and n.value >= codes + scales
    assert lib.svdq_i8_linear_workspace_bytes(1, 256, 512, 512, 1, BF16, ctypes.byref(n)) == 0 and n.value == 0  # one launch
    # contiguous columns: the rows' maxima come first
    assert lib.svdq_i8_linear_workspace_bytes(100, 256, 512, 1, 100, BF16, ctypes.byref(n)) == 0
    assert n.value >= codes + scales + _quantize_bytes(100, 512, 1, 100, 1, 0)
    _refused(EDTYPE, lib.svdq_i8_linear_workspace_bytes(4, 4, 4, 4, 1, F64, ctypes.byref(n)))
    for bad in ((0, 4, 4, 4, 1), (4, 4, 4, -4, 1), (4, 4, 4, 4, -1), (4, 4, (1 << 26) + 1, 4, 1)):
        _refused(EINVAL, lib.svdq_i8_linear_workspace_bytes(*bad, BF16, ctypes.byref(n)))


def test_backward_form_query():
    lib, form = _lib.load(), (ctypes.c_int * 2)()
    for sizes, want in (((4096, 12288, 4096), (256, 256)), ((1, 1, 1), (64, 64)), ((16, 12288, 4096), (0, 0)), ((1 << 26, 64, 64), (0, 0))):
        assert lib.svdq_i8_backward_form(*sizes, form) == 0
        assert tuple(form) == want
    for bad in ((0, 4, 4), (4, 0, 4), (4, 4, 0), ((1 << 26) + 1, 4, 4), (4, (1 << 26) + 1, 4)):
        _refused(EINVAL, lib.svdq_i8_backward_form(*bad, form))
    _refused(EINVAL, lib.svdq_i8_backward_form(4, 4, 4, None))


def test_backward_workspace_query():
    lib, n = _lib.load(), ctypes.c_size_t()
    d = sum(_layout(100, 96)[1:]) + sum(_layout(96, 100)[1:])
    assert lib.svdq_i8_backward_workspace_bytes(100, 96, 512, ctypes.byref(n)) == 0 and n.value >= d and n.value % 256 == 0
    for bad in ((0, 4, 4), (4, 0, 4), (4, 4, 0), ((1 << 26) + 1, 4, 4), (4, (1 << 26) + 1, 4)):
        _refused(EINVAL, lib.svdq_i8_backward_workspace_bytes(*bad, ctypes.byref(n)))
    _refused(EINVAL, lib.svdq_i8_backward_workspace_bytes(4, 4, 4, None))


@pytest.mark.parametrize("change,status", [
    (dict(dtype=F64), EDTYPE), (dict(M=0), EINVAL), (dict(K=0), EINVAL), (dict(x=None), EINVAL), (dict(ldx=39), EINVAL), (dict(x=A + 1), EINVAL),
    (dict(weight=None), EINVAL), (dict(pt=F64), EDTYPE), (dict(pt=F16), EDTYPE), (dict(weight=A + 1), EINVAL), (dict(bias=A + 1), EINVAL),
    (dict(eps=-1e-9), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(eps=float("inf")), EINVAL), (dict(mean=None), EINVAL),
    (dict(rstd=None), EINVAL), (dict(mean=A + 2), EINVAL),
])
@pytest.mark.parametrize("name,out", [("svdq_layer_norm", (A, 40)), ("svdq_layer_norm_i8", (A, A)), ("svdq_layer_norm_mx", (A, A))])
def test_norm_refusals(name, out, change, status):
    a = dict(x=A, ldx=40, M=4, K=40, weight=A, bias=A, pt=BF16, eps=1e-5, dtype=BF16)
    b = dict(mean=A, rstd=A)
    for k, v in change.items():
        (b if k in b else a)[k] = v
    _refused(status, getattr(_lib.load(), name)(*a.values(), *out, *b.values(), None))


@pytest.mark.parametrize("name,out", [("svdq_layer_norm", (None, 40)), ("svdq_layer_norm", (A, 39)), ("svdq_layer_norm", (A + 1, 40)),
                                      ("svdq_layer_norm_i8", (None, A)), ("svdq_layer_norm_i8", (A, A + 4)),
                                      ("svdq_layer_norm_mx", (A, None)), ("svdq_layer_norm_mx", (A + 16, A))])
def test_norm_refuses_outputs(name, out):
    _refused(EINVAL, getattr(_lib.load(), name)(A, 40, 4, 40, A, A, BF16, 1e-5, BF16, *out, None, None, None))


@pytest.mark.parametrize("change,status", [
    (dict(dtype=F64), EDTYPE), (dict(M=0), EINVAL), (dict(K=0), EINVAL), (dict(dy=None), EINVAL), (dict(lddy=39), EINVAL), (dict(x=None), EINVAL),
    (dict(ldx=39), EINVAL), (dict(mean=None), EINVAL), (dict(rstd=A + 1), EINVAL), (dict(pt=F16), EDTYPE), (dict(weight=A + 1), EINVAL),
    (dict(weight=None), EINVAL), (dict(dx=None), EINVAL), (dict(lddx=39), EINVAL), (dict(dweight=None), EINVAL), (dict(dbias=None), EINVAL),
    (dict(dbias=A + 1), EINVAL), (dict(work=None), EINVAL), (dict(work=A + 8), EINVAL), (dict(bytes=64), EINVAL),
])
def test_norm_backward_refusals(change, status):
    a = dict(dy=A, lddy=40, x=A, ldx=40, mean=A, rstd=A, M=4, K=40, weight=A, pt=F32, dtype=BF16, dx=A, lddx=40, dweight=A, dbias=A, work=A,
             bytes=1 << 50)
    a.update(change)
    _refused(status, _lib.load().svdq_layer_norm_backward(*a.values(), None))


def test_norm_backward_workspace_query():
    lib, n = _lib.load(), ctypes.c_size_t()
    assert lib.svdq_layer_norm_backward_workspace_bytes(100, 512, 0, ctypes.byref(n)) == 0 and n.value == 0
    for M, K in ((1, 1), (100, 512), (8192, 8192), (100000, 64), (10, 100000)):
        assert lib.svdq_layer_norm_backward_workspace_bytes(M, K, 1, ctypes.byref(n)) == 0
        assert n.value >= 8 * K and n.value % 256 == 0
    for bad in ((0, 4), (4, 0), (4, (1 << 30) + 1)):
        _refused(EINVAL, lib.svdq_layer_norm_backward_workspace_bytes(*bad, 1, ctypes.byref(n)))
    _refused(EINVAL, lib.svdq_layer_norm_backward_workspace_bytes(4, 4, 1, None))


# ----------------------------------------------------------------------------- binding
def _fake(rows, cols, short=0):
    _, a, b = _layout(rows, cols)
    return R.Int8Tensor(torch.zeros(a + b - short, dtype=torch.uint8), rows, cols)


def test_binding_refuses_cpu_tensors_and_wrong_types():
    x, m = torch.zeros(4, 64), torch.zeros(4)
    for call in (lambda: R.int8_quantize(x), lambda: R.int8_dequantize(_fake(4, 64)), lambda: R.int8_matmul(x, _fake(4, 64)),
                 lambda: R.int8_backward(x, _fake(4, 64), _fake(4, 4)), lambda: R.layer_norm(x), lambda: R.layer_norm_backward(x, x, m, m)):
        with pytest.raises(RuntimeError):
            call()
    for call in (lambda: R.int8_quantize(x.numpy()), lambda: R.int8_dequantize(x), lambda: R.int8_matmul(x, x),
                 lambda: R.layer_norm(x.numpy()), lambda: R.layer_norm_backward(x.numpy(), x, m, m)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        _fake(20, 64, short=1)
    with pytest.raises(ValueError):
        R.Int8Tensor(torch.zeros(1 << 20, dtype=torch.uint8), 0, 4)
    for data in (torch.zeros(1 << 20), torch.zeros(4, 1 << 20, dtype=torch.uint8), torch.zeros(1 << 21, dtype=torch.uint8)[::2]):
        with pytest.raises(TypeError):
            R.Int8Tensor(data, 4, 4)
    t = _fake(20, 64)
    assert t.shape == (20, 64) and t.scales.shape == (20,) and t.scales.dtype == torch.float32 and "20, 64" in repr(t)


@pytest.mark.parametrize("rows,cols", [(4.0, 64), (4, 64.0), (True, 64), ("4", 64), (None, 4)])
def test_tensor_sizes_are_whole_numbers(rows, cols):
    data = torch.zeros(1 << 16, dtype=torch.uint8)
    assert R.Int8Tensor(data, 4, 64).shape == (4, 64) and R.Int8Tensor(data, 1, 64).shape == (1, 64)
    with pytest.raises(ValueError, match="int"):
        R.Int8Tensor(data, rows, cols)
