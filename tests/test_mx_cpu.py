"""MXFP4 tensor operators without a GPU: the oracle's own checks, the layout query and every refusal."""
import ctypes
import math

import numpy as np
import pytest
import torch

import rank_bit_residual_amd as R
from oracle import mx as X
from rank_bit_residual_amd import _lib

A = 1 << 20  # a 256-byte aligned address that no refused call reads


# ----------------------------------------------------------------------------- oracle
def test_oracle_blocks():
    x = np.zeros((3, 70))
    x[0, 3] = 6.0
    x[1, 40] = 6.0000001
    x[2, 69] = np.inf
    codes, s = X.quantize(x)
    assert s.tolist() == [[127, 0, 0], [0, 128, 0], [0, 0, 255]]
    assert codes[0, 3] == 7 and codes[1, 40] == 5 and not codes[2].any()
    v = X.values(x)
    assert np.isnan(v[2, 64:]).all() and not np.isnan(v[:2]).any() and v[0, 3] == 6


@pytest.mark.parametrize("name", X.ACTS)
def test_oracle_gradient_against_differences(name):
    """act' against a central difference: its error is h^2 / 6 |act'''| (below 1 here) plus the rounding
    2^-52 |act| / h."""
    g = np.linspace(-6, 6, 193) + 1e-3
    h = 1e-4
    diff = (X.act(name, g + h) - X.act(name, g - h)) / (2 * h)
    assert np.abs(diff - X.act_grad(name, g)).max() < h * h / 2 + 2.0**-52 * 6 / h


def test_oracle_gated_gradient_against_differences():
    rng = np.random.default_rng(3)
    gu, dh = rng.standard_normal((4, 10)), rng.standard_normal((4, 5))
    h = 1e-5
    for name in X.ACTS:
        d = X.gated_grad(dh, gu, name)
        for j in range(10):
            step = np.zeros_like(gu)
            step[:, j] = h
            f = lambda z: (dh * X.act(name, z[:, :5]) * z[:, 5:]).sum(1)  # noqa: E731
            assert np.allclose((f(gu + step) - f(gu - step)) / (2 * h), d[:, j], atol=1e-8)


# ----------------------------------------------------------------------------- C ABI
def _layout(rows, K):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    st = _lib.load().svdq_mx_layout(rows, K, ctypes.byref(a), ctypes.byref(b))
    return st, a.value, b.value


def test_layout():
    assert _layout(1, 1) == (0, 2 * 1024, 2 * 256)
    assert _layout(17, 256) == (0, 2 * 2 * 1024, 2 * 256)
    assert _layout(65, 257) == (0, 5 * 4 * 1024, 2 * 4 * 256)
    assert _layout(1 << 20, 1 << 16) == (0, 1 << 35, 1 << 31)  # past 32 bits
    for rows, K in ((0, 4), (4, 0), (-1, 4), ((1 << 30) + 1, 4), (4, (1 << 30) + 1)):
        assert _layout(rows, K)[0] == _lib.SVDQ_EINVAL
    assert _lib.load().svdq_mx_layout(4, 4, None, None) == _lib.SVDQ_EINVAL


def _refused(status, st):
    assert st == status, (st, _lib.load().svdq_last_error())
    assert _lib.load().svdq_last_error()


F32, BF16, F64, F16 = _lib.SVDQ_F32, _lib.SVDQ_BF16, _lib.SVDQ_F64, _lib.SVDQ_F16
EINVAL, EDTYPE = _lib.SVDQ_EINVAL, _lib.SVDQ_EDTYPE


@pytest.mark.parametrize("change,status", [
    (dict(dtype=F64), EDTYPE), (dict(dtype=7), EDTYPE), (dict(R=0), EINVAL), (dict(C=0), EINVAL),
    (dict(C=(1 << 30) + 1), EINVAL), (dict(x=None), EINVAL), (dict(x=A + 1), EINVAL), (dict(sr=-1), EINVAL),
    (dict(sc=-4), EINVAL), (dict(codes=None), EINVAL), (dict(scales=None), EINVAL), (dict(codes=A + 16), EINVAL),
    (dict(scales_t=None), EINVAL), (dict(codes_t=A + 128), EINVAL),
    (dict(codes=None, scales=None, codes_t=None, scales_t=None), EINVAL),
])
def test_quantize_refusals(change, status):
    a = dict(x=A, R=4, C=40, sr=40, sc=1, dtype=BF16, codes=A, scales=A, codes_t=A, scales_t=A)
    a.update(change)
    _refused(status, _lib.load().svdq_mx_quantize(*a.values(), None))


@pytest.mark.parametrize("change,status", [
    (dict(dtype=F64), EDTYPE), (dict(rows=0), EINVAL), (dict(K=-3), EINVAL), (dict(codes=None), EINVAL),
    (dict(scales=A + 4), EINVAL), (dict(out=None), EINVAL), (dict(out=A + 1), EINVAL), (dict(ldo=39), EINVAL),
])
def test_dequantize_refusals(change, status):
    a = dict(codes=A, scales=A, rows=4, K=40, dtype=F16, out=A, ldo=40)
    a.update(change)
    _refused(status, _lib.load().svdq_mx_dequantize(*a.values(), None))


@pytest.mark.parametrize("change,status", [
    (dict(dtype=F64), EDTYPE), (dict(M=0), EINVAL), (dict(N=0), EINVAL), (dict(K=0), EINVAL), (dict(ac=None), EINVAL),
    (dict(asc=None), EINVAL), (dict(bc=A + 8), EINVAL), (dict(bs=None), EINVAL), (dict(bias=A + 2), EINVAL),
    (dict(y=None), EINVAL), (dict(y=A + 2), EINVAL), (dict(ldy=7), EINVAL), (dict(K=(1 << 27) + 1), EINVAL),
    (dict(M=256, N=256, K=1 << 16, ldy=256), EINVAL), (dict(M=256, N=256, K=1 << 16, ldy=256, work=A, bytes=1024), EINVAL),
    (dict(M=256, N=256, K=1 << 16, ldy=256, work=A + 8, bytes=1 << 40), EINVAL),
])
def test_matmul_refusals(change, status):
    a = dict(ac=A, asc=A, M=4, bc=A, bs=A, N=8, K=40, bias=None, dtype=F32, y=A, ldy=8, work=None, bytes=0)
    a.update(change)
    _refused(status, _lib.load().svdq_mx_matmul(*a.values(), None))


@pytest.mark.parametrize("change,status", [
    (dict(dtype=F64), EDTYPE), (dict(M=0), EINVAL), (dict(F=0), EINVAL), (dict(F=1 << 30), EINVAL), (dict(K=0), EINVAL),
    (dict(act=4), EINVAL), (dict(act=-1), EINVAL), (dict(ac=None), EINVAL), (dict(ws=None), EINVAL), (dict(h=None), EINVAL),
    (dict(ldh=7), EINVAL), (dict(gu=A, ldgu=15), EINVAL), (dict(gu=A + 1, ldgu=16), EINVAL),
])
def test_gated_refusals(change, status):
    a = dict(ac=A, asc=A, M=4, wc=A, ws=A, F=8, K=40, act=0, dtype=BF16, h=A, ldh=8, gu=None, ldgu=0, work=None, bytes=0)
    a.update(change)
    _refused(status, _lib.load().svdq_mx_gated(*a.values(), None))


@pytest.mark.parametrize("change,status", [
    (dict(dtype=F64), EDTYPE), (dict(M=0), EINVAL), (dict(N=0), EINVAL), (dict(K=0), EINVAL), (dict(x=None), EINVAL),
    (dict(x=A + 2), EINVAL), (dict(sr=-1), EINVAL), (dict(sc=-1), EINVAL), (dict(bc=None), EINVAL), (dict(bs=A + 4), EINVAL),
    (dict(bias=A + 2), EINVAL), (dict(y=None), EINVAL), (dict(ldy=7), EINVAL), (dict(K=(1 << 27) + 1), EINVAL),
    (dict(M=100), EINVAL), (dict(sc=2), EINVAL), (dict(M=100, work=A, bytes=64), EINVAL),
    (dict(M=100, work=A + 1, bytes=1 << 40), EINVAL),
])
def test_linear_refusals(change, status):
    a = dict(x=A, M=4, K=40, sr=40, sc=1, bc=A, bs=A, N=8, bias=None, dtype=F32, y=A, ldy=8, work=None, bytes=0)
    a.update(change)
    _refused(status, _lib.load().svdq_mx_linear(*a.values(), None))


@pytest.mark.parametrize("change,status", [
    (dict(dtype=F64), EDTYPE), (dict(M=0), EINVAL), (dict(F=0), EINVAL), (dict(F=1 << 30), EINVAL), (dict(act=4), EINVAL),
    (dict(x=None), EINVAL), (dict(wc=None), EINVAL), (dict(h=None), EINVAL), (dict(ldh=7), EINVAL),
    (dict(gu=A, ldgu=15), EINVAL), (dict(M=100), EINVAL), (dict(sc=0), EINVAL),
])
def test_gated_linear_refusals(change, status):
    a = dict(x=A, M=4, K=40, sr=40, sc=1, wc=A, ws=A, F=8, act=0, dtype=BF16, h=A, ldh=8, gu=None, ldgu=0, work=None, bytes=0)
    a.update(change)
    _refused(status, _lib.load().svdq_mx_gated_linear(*a.values(), None))


@pytest.mark.parametrize("change,status", [
    (dict(dtype=F64), EDTYPE), (dict(M=0), EINVAL), (dict(F=0), EINVAL), (dict(F=1 << 30), EINVAL), (dict(act=9), EINVAL),
    (dict(dh=None), EINVAL), (dict(ldh=7), EINVAL), (dict(gu=None), EINVAL), (dict(ldgu=15), EINVAL), (dict(gu=A + 1), EINVAL),
    (dict(codes=None), EINVAL), (dict(scales_t=A + 1), EINVAL),
    (dict(codes=None, scales=None, codes_t=None, scales_t=None), EINVAL),
])
def test_gated_grad_refusals(change, status):
    a = dict(dh=A, ldh=8, gu=A, ldgu=16, M=4, F=8, act=0, dtype=BF16, codes=A, scales=A, codes_t=A, scales_t=A)
    a.update(change)
    _refused(status, _lib.load().svdq_mx_gated_grad(*a.values(), None))


@pytest.mark.parametrize("change,status", [
    (dict(dtype=F64), EDTYPE), (dict(out=F64), EDTYPE), (dict(M=0), EINVAL), (dict(F=0), EINVAL), (dict(F=1 << 30), EINVAL),
    (dict(F=1 << 62), EINVAL), (dict(K=0), EINVAL), (dict(act=7), EINVAL), (dict(dh=None), EINVAL), (dict(ldh=7), EINVAL),
    (dict(gu=None), EINVAL), (dict(ldgu=15), EINVAL), (dict(wc=None), EINVAL), (dict(ws=A + 4), EINVAL), (dict(xc=A + 16), EINVAL),
    (dict(xs=None), EINVAL), (dict(dx=None), EINVAL), (dict(lddx=39), EINVAL), (dict(dw=A + 1), EINVAL), (dict(lddw=15), EINVAL),
    (dict(work=None), EINVAL), (dict(work=A + 8), EINVAL), (dict(bytes=4096), EINVAL), (dict(M=(1 << 27) + 1), EINVAL),
    (dict(F=1 << 27, ldh=1 << 27, ldgu=1 << 28, lddw=1 << 28), EINVAL),
])
def test_gated_backward_refusals(change, status):
    a = dict(dh=A, ldh=8, gu=A, ldgu=16, M=4, F=8, act=0, dtype=BF16, wc=A, ws=A, xc=A, xs=A, K=40, out=F32, dx=A, lddx=40, dw=A,
             lddw=16, work=A, bytes=1 << 50)
    a.update(change)
    _refused(status, _lib.load().svdq_mx_gated_backward(*a.values(), None))


def test_backward_workspace_query():
    lib, n = _lib.load(), ctypes.c_size_t()
    d = sum(_layout(100, 2 * 96)[1:]) + sum(_layout(2 * 96, 100)[1:])
    assert lib.svdq_mx_gated_backward_workspace_bytes(100, 96, 512, ctypes.byref(n)) == 0 and n.value == d
    assert lib.svdq_mx_gated_backward_workspace_bytes(1 << 16, 64, 128, ctypes.byref(n)) == 0
    assert n.value > sum(_layout(1 << 16, 128)[1:]) + sum(_layout(128, 1 << 16)[1:])  # dw's sum over many rows is shared out
    for bad in ((0, 4, 4), (4, 0, 4), (4, 4, 0), (4, 1 << 29, 4), ((1 << 27) + 1, 4, 4), (4, 1 << 27, 4), (4, 1 << 62, 4)):
        _refused(EINVAL, lib.svdq_mx_gated_backward_workspace_bytes(*bad, ctypes.byref(n)))
    _refused(EINVAL, lib.svdq_mx_gated_backward_workspace_bytes(4, 4, 4, None))


def test_workspace_query():
    lib, n = _lib.load(), ctypes.c_size_t(7)
    assert lib.svdq_mx_workspace_bytes(256, 256, 512, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.svdq_mx_workspace_bytes(256, 256, 1 << 16, 0, ctypes.byref(n)) == 0
    assert n.value >= 2 * 256 * 256 * 4
    for bad in ((0, 4, 4, 0), (4, 0, 4, 0), (4, 4, 0, 0), (4, 1 << 30, 4, 1), (4, 4, (1 << 27) + 1, 0)):
        _refused(EINVAL, lib.svdq_mx_workspace_bytes(*bad, ctypes.byref(n)))
    _refused(EINVAL, lib.svdq_mx_workspace_bytes(4, 4, 4, 0, None))
    codes, scales = _layout(100, 512)[1:]
    assert lib.svdq_mx_linear_workspace_bytes(100, 256, 512, 1, 0, ctypes.byref(n)) == 0 and n.value == codes + scales
    assert lib.svdq_mx_linear_workspace_bytes(1, 256, 512, 1, 1, ctypes.byref(n)) == 0 and n.value == 0
    _refused(EINVAL, lib.svdq_mx_linear_workspace_bytes(4, 4, 4, -1, 0, ctypes.byref(n)))
    _refused(EINVAL, lib.svdq_mx_linear_workspace_bytes(4, 0, 4, 1, 0, ctypes.byref(n)))


def test_launches_past_the_grid_are_refused():
    """2^32 threads along a dimension of a grid: refused before anything is launched."""
    lib, big = _lib.load(), 1 << 30
    _refused(EINVAL, lib.svdq_mx_quantize(A, big, 4, 4, 1, BF16, A, A, None, None, None))
    _refused(EINVAL, lib.svdq_mx_quantize(A, 4, big, 1, 4, BF16, None, None, A, A, None))
    _refused(EINVAL, lib.svdq_mx_dequantize(A, A, big, 4, BF16, A, 4, None))
    _refused(EINVAL, lib.svdq_mx_gated_grad(A, 1, A, 2, big, 1, 0, BF16, A, A, A, A, None))
    _refused(EINVAL, lib.svdq_mx_gated_grad(A, 32, A, 64, big, 32, 0, BF16, A, A, A, A, None))
    _refused(EINVAL, lib.svdq_mx_matmul(A, A, big, A, A, 4, 64, None, BF16, A, 4, None, 0, None))
    _refused(EINVAL, lib.svdq_mx_matmul(A, A, 1, A, A, big, 64, None, BF16, A, big, None, 0, None))


def test_calls_of_several_launches_are_refused_whole():
    """Every launch's grid is checked before the first one: where only the last does not fit, nothing runs. (Without a GPU a
    launch that was tried would give EHIP.)"""
    lib, room = _lib.load(), 1 << 60
    M, N = 1 << 24, 1 << 17  # 2^24 tiles of 256 x 256
    _refused(EINVAL, lib.svdq_mx_linear(A, M, 64, 64, 1, A, A, N, None, BF16, A, N, A, room, None))
    _refused(EINVAL, lib.svdq_mx_gated_linear(A, M, 64, 64, 1, A, A, N // 2, 0, BF16, A, N // 2, None, 0, A, room, None))
    # dx [M, K] does not fit, then dw [K, 2F] does not
    F, K = 64, 1 << 17
    _refused(EINVAL, lib.svdq_mx_gated_backward(A, F, A, 2 * F, M, F, 0, BF16, A, A, A, A, K, BF16, A, K, A, 2 * F, A, room, None))
    F, K, M = 1 << 20, 1 << 24, 32
    _refused(EINVAL, lib.svdq_mx_gated_backward(A, F, A, 2 * F, M, F, 0, BF16, A, A, A, A, K, BF16, A, K, A, 2 * F, A, room, None))


def _linear_workspace(M, N, K, gated=0, dtype=None, sc=1):
    n, lib = ctypes.c_size_t(), _lib.load()
    if dtype is None:
        assert lib.svdq_mx_linear_workspace_bytes(M, N, K, sc, gated, ctypes.byref(n)) == 0
    else:
        assert lib.svdq_mx_linear_workspace_bytes_of(M, N, K, sc, gated, dtype, ctypes.byref(n)) == 0
    return n.value


def test_long_rows_are_quantised_before_the_product():
    """A few rows are quantised inside the product (no workspace) while K is short, one row always, many never."""
    for gated in (0, 1):
        for M in (2, 4, 8, 16):
            for dtype in (BF16, F16, F32):
                fused = [_linear_workspace(M, 64, K, gated, dtype) == 0 for K in (64, 512, 1024, 16384, 28672, 1 << 17)]
                assert fused == [True, True, True, False, False, False]
            assert _linear_workspace(M, 64, 4096, gated, F32) >= _linear_workspace(M, 64, 4096, gated, BF16)
            for K in (64, 2048, 4096, 16384):
                widest = max(_linear_workspace(M, 64, K, gated, d) for d in (F32, BF16, F16))
                assert _linear_workspace(M, 64, K, gated) == widest
        for K in (64, 4096):
            assert _linear_workspace(1, 8192, K, gated, F32) == _linear_workspace(1, 8192, K, gated, BF16) == 0
            assert _linear_workspace(1, 64, K, gated, F32, sc=2) > 0 and _linear_workspace(17, 64, K, gated, BF16) > 0
    n = ctypes.c_size_t()
    _refused(EDTYPE, _lib.load().svdq_mx_linear_workspace_bytes_of(4, 4, 4, 1, 0, F64, ctypes.byref(n)))
    _refused(EINVAL, _lib.load().svdq_mx_linear_workspace_bytes_of(4, 4, 4, -1, 0, F32, ctypes.byref(n)))


def _form(M, N, K, gated=0):
    got = (ctypes.c_int * 4)()
    assert _lib.load().svdq_mx_product_form(M, N, K, gated, got) == 0
    return tuple(got)


def test_product_form_query():
    lib, got = _lib.load(), (ctypes.c_int * 4)()
    for bad in ((0, 4, 4, 0), (4, 0, 4, 0), (4, 4, 0, 0), (4, 1 << 30, 4, 1), (4, 4, (1 << 27) + 1, 0)):
        _refused(EINVAL, lib.svdq_mx_product_form(*bad, got))
    _refused(EINVAL, lib.svdq_mx_product_form(4, 4, 4, 0, None))
    n = ctypes.c_size_t()
    for M, N, K, gated in ((1, 100, 512, 0), (300, 5000, 4096, 1), (1024, 1024, 65536, 0), (130, 151, 33000, 1)):
        bm, bn, splits, waves = _form(M, N, K, gated)
        assert lib.svdq_mx_workspace_bytes(M, N, K, gated, ctypes.byref(n)) == 0
        assert n.value == (splits * M * N * (2 if gated else 1) * 4 if splits > 1 else 0)
        assert (waves == 1) == (bm >= 128) and bn % 16 == 0


@pytest.mark.parametrize("M", [1, 16, 32, 64])
@pytest.mark.parametrize("K", [512, 8192])
def test_few_row_blocks_change_with_the_tiles_a_compute_unit_gets(M, K):
    """The block shape is one over each range of column tiles: up to 256, to 512, and more; no width has its own."""
    for widths in ((16, 1000, 4080, 4096), (4097, 5000, 8000, 8176, 8177, 8192), (8193, 8208, 9000, 16384, 16400)):
        forms = {f for f in (_form(M, n, K) for n in widths) if f[3] > 1}
        assert len(forms) <= 1, forms



@pytest.mark.parametrize("N,K,gated", [(12288, 4096, 1), (28672, 8192, 1), (8192, 28672, 0), (1024, 28672, 0), (128256, 4096, 0),
                                       (16384, 16384, 0), (4096, 65536, 0), (140000, 65536, 0), (72000, 65536, 1)])
def test_one_row_is_one_launch(N, K, gated):
    """However large the weight: its bytes take as long in any form, and tiles would need two or three launches."""
    bm, _, splits, waves = _form(1, N, K, gated)
    assert bm == 16 and splits == 1 and waves > 1
    for dtype in (F32, BF16, F16):
        assert _linear_workspace(1, N, K, gated, dtype) == 0


# ----------------------------------------------------------------------------- binding
@pytest.mark.parametrize("out,x,want", [
    ((0, 4, 8, 8), (32, 4, 8, 8), False),  # (offset, rows, columns, row stride)
    ((0, 4, 8, 8), (31, 4, 8, 8), True),
    ((40, 4, 8, 8), (8, 4, 8, 8), False),
    ((40, 4, 8, 8), (9, 4, 8, 8), True),
    ((0, 4, 8, 8), (0, 4, 8, 8), True),
    ((0, 4, 8, 16), (8, 4, 8, 16), False),  # beside it in one buffer
    ((8, 4, 8, 16), (0, 4, 8, 16), False),
    ((0, 4, 8, 16), (7, 4, 8, 16), True),
    ((0, 4, 8, 16), (8, 4, 9, 16), True),
    ((8, 4, 8, 16), (24, 2, 8, 16), True),
    ((0, 4, 8, 16), (10, 4, 4, 12), True),  # other strides: taken to overlap
    ((5, 1, 8, 8), (12, 1, 1, 1), True),
    ((5, 1, 8, 8), (13, 1, 1, 1), False),
])
def test_overlap(out, x, want):
    from rank_bit_residual_amd import mx

    buf = torch.zeros(200)
    out, x = (torch.as_strided(buf, (r, c), (ld, 1), at) for at, r, c, ld in (out, x))
    assert mx._overlap(out, x) is want
    assert not mx._overlap(out, torch.zeros(4, 8)) and not mx._overlap(out, torch.zeros(8))


def test_overlap_of_an_output_row_without_a_stride():
    """A row may have any row stride, 0 too (a view made by expand)."""
    from rank_bit_residual_amd import mx

    buf = torch.zeros(200)
    out = torch.as_strided(buf, (1, 8), (0, 1), 5)
    for at, want in ((0, True), (12, True), (13, False)):
        assert mx._overlap(out, torch.as_strided(buf, (1, 8), (0, 1), at)) is want
        assert mx._overlap(out, torch.as_strided(buf, (3, 8), (0, 1), at)) is want
        assert mx._overlap(out, torch.as_strided(buf, (2, 8), (8, 1), at)) is want


def _fake(rows, cols, short=0):
    _, a, b = _layout(rows, cols)
    return R.MxTensor(torch.zeros(a + b - short, dtype=torch.uint8), rows, cols)


def test_binding_refuses_cpu_tensors_and_wrong_types():
    x = torch.zeros(4, 64)
    for call in (lambda: R.mx_quantize(x), lambda: R.mx_dequantize(_fake(4, 64)), lambda: R.mx_matmul(x, _fake(4, 64)),
                 lambda: R.mx_gated(x, _fake(8, 64)), lambda: R.mx_gated_grad(x, torch.zeros(4, 128))):
        with pytest.raises(RuntimeError):
            call()
    for call in (lambda: R.mx_quantize(x.numpy()), lambda: R.mx_dequantize(x), lambda: R.mx_matmul(x, x),
                 lambda: R.mx_gated(x, x), lambda: R.mx_gated_backward(x, x, x, x)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        _fake(20, 64, short=1)
    with pytest.raises(ValueError):
        R.MxTensor(torch.zeros(1 << 20, dtype=torch.uint8), 0, 4)
    for data in (torch.zeros(1 << 20), torch.zeros(4, 1 << 20, dtype=torch.uint8), torch.zeros(1 << 21, dtype=torch.uint8)[::2]):
        with pytest.raises(TypeError):
            R.MxTensor(data, 4, 4)
    t = _fake(20, 64)
    assert t.shape == (20, 64) and t.codes.numel() + t.scales.numel() == t.data.numel() and "20, 64" in repr(t)
    with pytest.raises(ValueError):
        R.mx_gated(x, _fake(8, 64), act="swish")
    with pytest.raises(ValueError):
        R.mx_gated_grad(x, x, act="tanh")


@pytest.mark.parametrize("axis", [2, -1, True, "rows"])
def test_axes_are_refused(axis):
    x = torch.zeros(4, 64)
    with pytest.raises((ValueError, RuntimeError)):
        R.mx_quantize(x, axis=axis)
    with pytest.raises(ValueError):
        R.mx_gated_grad(x, torch.zeros(4, 128), axis=axis)


@pytest.mark.parametrize("rows,cols", [(4.0, 64), (4, 64.0), (True, 64), ("4", 64), (None, 4)])
def test_tensor_sizes_are_whole_numbers(rows, cols):
    data = torch.zeros(1 << 16, dtype=torch.uint8)
    assert R.MxTensor(data, 4, 64).shape == (4, 64) and R.MxTensor(data, 1, 64).shape == (1, 64)
    with pytest.raises(ValueError, match="int"):
        R.MxTensor(data, rows, cols)
