"""Every kernel form of the MXFP4 products on an MI355X, with the form asserted before it is run.

Operands are codes of blocks whose largest is 6, so they are their own Q, and every partial sum is a multiple of 1/4 below
2^22 (36 K <= 2^22): one value in float32, whatever the order of the sum and the form of the product.
"""
import ctypes
import math

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


# ----------------------------------------------------------------------------- tiles
TILES = [(333, 2501, 1000, (128, 128, False)), (515, 12290, 100, (128, 256, False)), (1030, 12290, 1030, (256, 256, False)),
         (129, 2501, 9000, (128, 128, True)), (65, 8200, 9000, (128, 256, True)), (129, 8200, 33000, (256, 256, True))]


def _tile_form(*sizes):
    bm, bn, splits, waves = _form(*sizes)
    assert waves == 1
    return bm, bn, splits > 1


def _view(rows, cols, dtype):
    """A matrix inside a larger one, off its alignment, and a check that the rest of that stays."""
    big = torch.full((rows + 3, cols + 5), 7.0, dtype=dtype, device="cuda")

    def rest_stays():
        big[1:-2, 3:-2] = 7.0
        return bool((big == 7.0).all())

    return big[1:-2, 3:-2], rest_stays


@pytest.mark.parametrize("M,N,K,form", TILES)
def test_tile_forms(M, N, K, form):
    """Every tile, whole and with K shared out, in every type: a bias, a strided output, quantised and unquantised rows."""
    assert _tile_form(M, N, K) == form
    gen = _gen(M + N + K)
    a, b = _on_grid(gen, M, K), _on_grid(gen, N, K)
    ref = _product(a, b)
    bq, aq = R.mx_quantize(b), R.mx_quantize(a)
    bias = torch.randint(-8, 8, (N,), generator=gen, device="cuda").float()
    for dtype in TD.values():
        want = ref.float().to(dtype)
        assert torch.equal(R.mx_matmul(a.to(dtype), bq), want)
        got = R.mx_matmul(aq, bq, bias=bias.to(dtype), dtype=dtype)
        assert torch.equal(got, (ref + bias.double()).float().to(dtype))
        out, rest_stays = _view(M, N, dtype)
        assert R.mx_matmul(aq, bq, dtype=dtype, out=out) is out and torch.equal(out, want)
        assert rest_stays()


GATED = [(33, 300, 512, (64, 32, None)), (300, 2001, 1000, (128, 128, False)), (1000, 4090, 1000, (128, 256, False)),
         (1500, 5000, 1000, (256, 256, False)), (257, 1000, 4096, (128, 128, True)), (130, 2050, 9000, (128, 256, True)),
         (129, 5000, 33000, (256, 256, True))]
HALF = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}  # half a step, relative
TINY = {torch.float32: 1e-37, torch.bfloat16: 1e-37, torch.float16: 2.0**-24}


def _act(name, g):
    """act(g) in float64, and the bound on the float32 activation's relative error."""
    if name == "relu":
        return g.clamp_min(0), torch.zeros_like(g)
    if name == "gelu":
        return 0.5 * g * torch.special.erfc(-g / 2**0.5), (3 + g * g) * 2.0**-20
    w = g if name == "silu" else 2 * (2 / torch.pi) ** 0.5 * (g + 0.044715 * g**3)
    return g / (1 + torch.exp(-w)), (3 + w.abs()) * 2.0**-21


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("M,F,K,form", GATED)
def test_gated_forms(M, F, K, form, act):
    """Every form in every type and activation, with and without the pre-activations, into a strided output: exact sums,
    so g and u come rounded once, and h is off by the activation's error, the product's 2^-24 and the store's half step."""
    bm, bn, splits, waves = _form(M, F, K, True)
    assert (bm, bn, splits > 1 if waves == 1 else None) == form
    gen = _gen(M + F + K)
    scale = 2.0**-round(math.log2(7 * K**0.5) / 2)  # pre-activations of about unit scale
    x, w = _on_grid(gen, M, K) * scale, _on_grid(gen, 2 * F, K) * scale
    gu = _product(x, w)
    a, ew = _act(act, gu[:, :F])
    ref = a * gu[:, F:]
    wq, xq = R.mx_quantize(w), R.mx_quantize(x)
    for dtype in TD.values():
        h, saved = R.mx_gated(x.to(dtype), wq, act=act, save=True)
        assert torch.equal(saved, gu.float().to(dtype))
        bound = (ew + 2.0**-23 + 1.01 * HALF[dtype]) * ref.abs() + TINY[dtype]
        assert ((h.double() - ref).abs() <= bound).all()
        out, rest_stays = _view(M, F, dtype)
        assert R.mx_gated(xq, wq, act=act, dtype=dtype, out=out) is out and torch.equal(out, h)
        assert rest_stays()


# ----------------------------------------------------------------------------- streams and graphs, with workspaces
SPLIT = dict(M=257, K=16384, F=1000)  # K is shared out in the projections
LONG = dict(M=20000, K=260, F=64)  # in the weights' gradient
WIDE = dict(M=1100, K=512, F=2600)  # in the input's gradient


def _inputs(seed, M, K, F):
    gen = _gen(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    return randn(M, K), randn(K, 2 * F), randn(M, F)


def _step(x, w, dh):
    xr, xc = R.mx_quantize(x, axis=None)
    wr, wc = R.mx_quantize(w, axis=None)
    h, gu = R.mx_gated(xr, wc, save=True)
    return (h, gu, *R.mx_gated_backward(dh, gu, wr, xc), R.mx_matmul(x, wc, dtype=torch.float32), R.mx_gated(x, wc, act="gelu"))


def _assert_shares(size):
    M, K, F = size["M"], size["K"], size["F"]
    shared = [_tile_form(*p)[2] for p in ((M, F, K, True), (M, 2 * F, K), (M, K, 2 * F), (K, 2 * F, M))]
    assert shared == [size is SPLIT, size is SPLIT, size is WIDE, size is LONG]


@pytest.mark.parametrize("size", [SPLIT, LONG, WIDE])
def test_two_streams_at_once(size):
    """Products with workspaces on two streams, each on its own inputs, without a wait between them."""
    _assert_shares(size)
    sets = [_inputs(31, **size), _inputs(32, **size)]
    want = [_step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(4):
        for s, ins in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(_step(*ins))
    torch.cuda.synchronize()
    for k, g in enumerate(got):
        assert all(torch.equal(p, q) for p, q in zip(want[k % 2], g)), k


@pytest.mark.parametrize("size", [SPLIT, LONG, WIDE])
def test_captured_and_replayed(size):
    """Two graphs that live at the same time, replayed in turn with other inputs, eager calls between them."""
    _assert_shares(size)
    sets = [_inputs(41, **size), _inputs(42, **size)]
    for ins in sets:
        _step(*ins)
    torch.cuda.synchronize()
    graphs = []
    for ins in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _step(*ins)
        graphs.append((g, out))
    for k in range(4):
        for i, ((g, out), ins) in enumerate(zip(graphs, sets)):
            for dst, src in zip(ins, _inputs(60 + 2 * k + i, **size)):
                dst.copy_(src)
            g.replay()
        want = [_step(*ins) for ins in sets]
        torch.cuda.synchronize()
        for (_, out), w in zip(graphs, want):
            assert all(torch.equal(p, q) for p, q in zip(out, w)), k


FIRST_TILES = """
import ctypes, torch, rank_bit_residual_amd as R
from rank_bit_residual_amd import _lib
sizes = [(333, 2501, 1000), (515, 12290, 100), (1030, 12290, 1030), (129, 2501, 9000), (65, 8200, 9000)]
form, seen = (ctypes.c_int * 4)(), set()
for s in sizes:
    _lib.check(_lib.load().svdq_mx_product_form(*s, 0, form))
    seen.add((form[0], form[1], form[2] > 1))
    assert form[3] == 1
assert len(seen) == 5
g = torch.Generator(device="cuda").manual_seed(3)
ops = [(torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16),
        torch.randn(N, K, generator=g, device="cuda", dtype=torch.bfloat16)) for M, N, K in sizes]
step = lambda: [f(a, R.mx_quantize(b)) for a, b in ops for f in (R.mx_matmul, R.mx_gated) if f is R.mx_matmul or len(b) % 2 == 0]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = step()
for k in range(3):
    for a, _ in ops:
        a.mul_(-0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, step())), k
print("same")
"""


def test_first_call_of_a_process_captured():
    """Each tile kernel's one-time set-up happens inside the capture."""
    import os
    import subprocess
    import sys

    _gen(0)
    r = subprocess.run([sys.executable, "-c", FIRST_TILES], capture_output=True, text=True, timeout=100,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


# ----------------------------------------------------------------------------- ends of the range
@pytest.mark.parametrize("e", [-127, -126, -125, -124, -60, 100, 124])
def test_values_at_the_ends_of_the_range(e):
    """Blocks of the lowest scale bytes (0 stands for 2^-127, a float32 subnormal) and of high ones, read back along both axes."""
    gen = _gen(e + 200)
    x = _on_grid(gen, 70, 96)
    x[::32] = 6.0
    want = x.double() * 2.0**e
    assert torch.equal(want.float().double(), want)
    rows, cols = R.mx_quantize(want.float(), axis=None)
    bytes_of = lambda t: t.scales.view(-1, 64, 4)[0, :32, :3]  # noqa: E731
    assert (bytes_of(rows) == e + 127).all()
    for dtype in TD.values():
        assert torch.equal(R.mx_dequantize(rows, dtype), want.to(dtype))
        back = R.mx_dequantize(cols, dtype)
        assert torch.equal(back[:, :64], want.t()[:, :64].to(dtype))


@pytest.mark.parametrize("e,f", [(-127, 100), (-127, 0), (-127, -8), (-126, 2), (-125, -1), (-120, -10), (100, 10), (-60, -60)])
@pytest.mark.parametrize("M,N,K", [(3, 64, 160), (300, 2500, 160), (129, 300, 9000)])
def test_products_at_the_ends_of_the_range(M, N, K, e, f):
    """Terms down to 2^-140 and their sums, subnormal float32 numbers among them, are exact in every kernel."""
    gen = _gen(M + K)
    a, b = _on_grid(gen, M, K).double(), _on_grid(gen, N, K).double()
    ref = a @ b.t().contiguous() * 2.0 ** (e + f)
    y = R.mx_matmul((a * 2.0**e).float(), R.mx_quantize((b * 2.0**f).float()))
    assert torch.equal(y.double(), ref)
    assert torch.equal(R.mx_matmul(R.mx_quantize((a * 2.0**e).float()), R.mx_quantize((b * 2.0**f).float()), dtype=torch.bfloat16),
                       ref.float().to(torch.bfloat16))
