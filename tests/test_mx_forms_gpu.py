"""Every kernel form of the MXFP4 products on an MI355X, with the form asserted before it is run.

Operands are codes of blocks whose largest is 6, so they are their own Q, and every partial sum is a multiple of 1/4 below
2^22 (36 K <= 2^22): one value in float32, whatever the order of the sum and the form of the product.
"""
import ctypes

import pytest
import torch

import rank_bit_residual_amd as R
from rank_bit_residual_amd import _lib

pytestmark = pytest.mark.gpu

TD = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
GRID = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def _form(M, N, K, gated=False):
    got = (ctypes.c_int * 4)()
    _lib.check(_lib.load().svdq_mx_product_form(M, N, K, gated, got))
    return tuple(got)


def _gen(seed):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.Generator(device="cuda").manual_seed(seed)


def _on_grid(gen, rows, cols):
    x = torch.tensor(GRID, device="cuda")[torch.randint(0, 8, (rows, cols), generator=gen, device="cuda")]
    x[:, ::32] = 6.0
    return x * (1 - 2 * torch.randint(0, 2, (rows, cols), generator=gen, device="cuda"))


def _product(a, b):
    return a.double() @ b.double().t().contiguous()


# ----------------------------------------------------------------------------- few rows
# one-tile blocks of eight waves, two-tile blocks, and past 512 column tiles four waves or eight
@pytest.mark.parametrize("M,N,K,form", [
    (1, 4096, 1000, (16, 16, 1, 8)), (16, 4097, 1000, (16, 32, 1, 8)), (1, 8176, 1000, (16, 32, 1, 8)),
    (4, 8177, 1000, (16, 32, 1, 8)), (16, 8192, 1000, (16, 32, 1, 8)), (1, 8192, 8000, (16, 32, 1, 8)),
    (1, 8193, 1000, (16, 16, 1, 4)), (16, 16400, 1000, (16, 16, 1, 4)), (4, 8193, 1000, (16, 16, 1, 4)),
    (1, 8193, 8000, (16, 16, 1, 8)), (16, 8208, 8000, (16, 16, 1, 8)),
    (17, 300, 1000, (32, 16, 1, 8)), (32, 4112, 1000, (32, 32, 1, 8)), (32, 8193, 1100, (32, 32, 1, 8)), (20, 8193, 1000, (32, 16, 1, 4)),
    (33, 300, 1000, (64, 16, 1, 8)), (64, 4112, 512, (64, 32, 1, 8)), (70, 300, 1000, (64, 16, 1, 8)),
])
def test_few_row_forms(M, N, K, form):
    assert _form(M, N, K) == form
    gen = _gen(M + N + K)
    a, b = _on_grid(gen, M, K), _on_grid(gen, N, K)
    ref = _product(a, b)
    bq, aq = R.mx_quantize(b), R.mx_quantize(a)
    bias = torch.randint(-8, 8, (N,), generator=gen, device="cuda").float()
    for dtype in TD.values():
        want = ref.float().to(dtype)
        assert torch.equal(R.mx_matmul(aq, bq, dtype=dtype), want)
        assert torch.equal(R.mx_matmul(a.to(dtype), bq), want)
        assert torch.equal(R.mx_matmul(a.to(dtype), bq, bias=bias.to(dtype)), (ref + bias.double()).float().to(dtype))


def _fused(M, N, K, dtype, gated=False):
    n = ctypes.c_size_t()
    code = {torch.float32: _lib.SVDQ_F32, torch.bfloat16: _lib.SVDQ_BF16, torch.float16: _lib.SVDQ_F16}[dtype]
    _lib.check(_lib.load().svdq_mx_linear_workspace_bytes_of(M, N, K, 1, gated, code, ctypes.byref(n)))
    return n.value == 0


# rows quantised inside the product and before it, on either side of each type's border
@pytest.mark.parametrize("M,N,K,fused", [(2, 64, 1000, "f32 bf16 f16"), (16, 200, 2048, "bf16 f16"), (8, 40, 4096, "bf16 f16"),
                                         (16, 40, 4096, ""), (2, 33, 28672, ""), (4, 8000, 8192, "bf16 f16"), (1, 33, 8192, "f32 bf16 f16"),
                                         (1, 33, 28672, "f32 bf16 f16")])
def test_quantised_inside_the_product_or_before(M, N, K, fused):
    gen = _gen(M + N + K)
    a, b = _on_grid(gen, M, K), _on_grid(gen, N, K)
    ref = _product(a, b)
    bq = R.mx_quantize(b)
    for name, dtype in TD.items():
        assert _fused(M, N, K, dtype) == (name in fused.split())
        assert torch.equal(R.mx_matmul(a.to(dtype), bq), ref.float().to(dtype))


def test_few_rows_of_a_tensor_past_32_bits():
    """Few rows against 4.6 GB of codes, in the few-row kernel's own addressing: the first and the last columns."""
    rows, cols = 140_000, 65_536
    assert all(_form(M, rows, cols)[3] > 1 and _form(M, rows // 2, cols, True)[3] > 1 for M in (1, 4))
    gen = _gen(79)
    x = torch.randint(-3, 4, (rows, cols), generator=gen, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    x[:, ::32] = 3
    r = R.mx_quantize(x)
    assert r.data.numel() > 2**32
    for M in (1, 4):
        a = torch.randint(-3, 4, (M, cols), generator=gen, device="cuda", dtype=torch.int8).to(torch.bfloat16)
        a[:, ::32] = 3
        y = R.mx_matmul(a.float(), r)
        for part in (slice(0, 300), slice(rows - 300, rows)):
            assert torch.equal(y[:, part], a.float() @ x[part].float().t().contiguous())
        g = R.mx_gated(a.float(), r, act="relu")
        gate, up = slice(rows // 2 - 300, rows // 2), slice(rows - 300, rows)
        ref = (a.float() @ x[gate].float().t().contiguous()).relu() * (a.float() @ x[up].float().t().contiguous())
        assert torch.equal(g[:, -300:], ref)
