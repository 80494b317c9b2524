"""MXFP4 tensor operators on an MI355X against plain float64 implementations (oracle/mx.py).

Codes, scale bytes and dequantised values must be equal. Products: every term is exact, and a float32
sum of K terms in any order is off by at most K steps of 2^-23 of the sum of the terms' sizes (a matrix
core may cut off instead of rounding); the output adds half a step of its type.
"""
import os

import numpy as np
import pytest
import torch

import rank_bit_residual_amd as R
from oracle import mx as X
from oracle import svdquant as O

pytestmark = pytest.mark.gpu

TD = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
STEP = {"f32": 2.0**-24, "bf16": 2.0**-8, "f16": 2.0**-11}  # half a step, relative
TINY = {"f32": 2.0**-149, "bf16": 2.0**-133, "f16": 2.0**-24}  # the smallest magnitude of the type


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _round(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, np.float64)).to(TD[dtype])


def _gpu(a, dtype):
    return _round(a, dtype).to(dev())


def _np(t):
    return t.detach().cpu().double().numpy()


def _parts(t):
    return X.unpack(t.codes.cpu().numpy(), t.scales.cpu().numpy(), t.rows, t.cols)


def _check_tensor(t, want):
    """t holds Q(want): equal codes and bytes, zeros past the last element."""
    assert t.shape == want.shape
    codes, s, past, spast = _parts(t)
    wc, ws = X.quantize(want)
    assert np.array_equal(s, ws), np.argwhere(s != ws)[:4]
    assert np.array_equal(codes, wc), (np.argwhere(codes != wc)[:4], want[tuple(np.argwhere(codes != wc)[0])])
    assert not past.any() and not spast.any()


def _wide(rng, rows, cols):
    """Values whose rows and columns differ by many powers of two, with ties, zeros and a zero block."""
    x = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-6, 7, (rows, 1)) * 2.0 ** rng.integers(-3, 4, (1, cols))
    x[rng.random((rows, cols)) < 0.05] = 0
    x[rng.random((rows, cols)) < 0.05] = 2.5
    x[0, : min(cols, 32)] = 0
    return x


# ----------------------------------------------------------------------------- quantise
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (1, 4096), (3, 31), (33, 33), (128, 128), (130, 255), (65, 257),
                                       (300, 70), (257, 1000)])
def test_quantize(dtype, rows, cols):
    x = _gpu(_wide(np.random.default_rng(rows * 1009 + cols), rows, cols), dtype)
    both = R.mx_quantize(x, axis=None)
    want = _np(x)
    for t, w in ((R.mx_quantize(x), want), (R.mx_quantize(x, axis=0), want.T), (both[0], want), (both[1], want.T)):
        _check_tensor(t, w)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_quantize_strides(dtype):
    rng = np.random.default_rng(5)
    big = _gpu(_wide(rng, 200, 301), dtype)
    odd = _gpu(_wide(rng, 1, 200 * 301 + 1), dtype).reshape(-1)[1:].reshape(200, 301)  # not 4-byte aligned in 16 bits
    for x in (big.t(), big[3:150, 5:222], big[::2, ::3], big[7:8].expand(40, 301), big[:, 9:10].expand(200, 50),
              odd, odd.t(), big[:, :96].t()):
        rows, cols = R.mx_quantize(x, axis=None)
        _check_tensor(rows, _np(x))
        _check_tensor(cols, _np(x).T)
        _check_tensor(R.mx_quantize(x, axis=0), _np(x).T)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_quantize_ends_of_the_range(dtype):
    """Subnormals, the largest values, negative zeros, and every border between two codes at many scales."""
    info = torch.finfo(TD[dtype])
    rng = np.random.default_rng(6)
    x = np.zeros((8, 96))
    x[0, :32] = rng.integers(-7, 8, 32) * TINY[dtype]
    x[0, 32:64] = rng.integers(-700, 700, 32) * TINY[dtype]
    x[0, 64:] = -0.0
    x[1] = rng.choice([-1.0, 1.0], 96) * info.max
    x[2] = info.max * rng.random(96)
    x[3] = info.tiny * (1 + rng.random(96))
    x[4] = info.tiny / 2 * rng.random(96)
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    for r in range(5, 8):
        x[r] = np.tile(borders, 12) * 2.0 ** np.repeat(rng.integers(-10, 8, 3), 32) * rng.choice([-1.0, 1.0], 96)
    x = _gpu(x, dtype)
    rows, cols = R.mx_quantize(x, axis=None)
    _check_tensor(rows, _np(x))
    _check_tensor(cols, _np(x).T)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_infinities_and_nan_poison_their_block_alone(dtype):
    x = np.random.default_rng(8).standard_normal((70, 100))
    x[1, 40], x[2, 99], x[50, 0], x[51, 64] = np.inf, np.nan, -np.inf, np.nan
    x = _gpu(x, dtype)
    rows, cols = R.mx_quantize(x, axis=None)
    _check_tensor(rows, _np(x))
    _check_tensor(cols, _np(x).T)
    got = _np(R.mx_dequantize(rows, torch.float32))
    assert np.array_equal(got, X.values(_np(x)), equal_nan=True)
    w = R.mx_quantize(_gpu(np.random.default_rng(9).standard_normal((40, 100)), dtype))
    for y in (R.mx_matmul(rows, w), R.mx_matmul(w, rows).t(), R.mx_gated(rows, w)):
        bad = np.isnan(_np(y)).all(1)
        assert np.array_equal(np.isnan(_np(y)).any(1), bad)
        assert np.flatnonzero(bad).tolist() == [1, 2, 50, 51]


def test_nan_blocks_in_tiles():
    """The tiled product: rows of A and of b with a NaN block give NaN rows and columns, nothing else."""
    gen = _gen(4)
    a, b = _on_grid(gen, 2000, 512), _on_grid(gen, 4096, 512)
    ref = a @ b.t().contiguous()
    a[7, 100], a[1999, 511], b[3, 0], b[4095, 300] = float("nan"), float("inf"), float("-inf"), float("nan")
    y = R.mx_matmul(a, R.mx_quantize(b))
    bad = torch.zeros(2000, 4096, dtype=torch.bool, device=a.device)
    bad[[7, 1999]] = True
    bad[:, [3, 4095]] = True
    assert torch.equal(y.isnan(), bad) and torch.equal(y[~bad], ref[~bad])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 33), (64, 128), (70, 300)])
def test_dequantize(dtype, rows, cols):
    x = _gpu(_wide(np.random.default_rng(rows + cols), rows, cols), "f32")
    t = R.mx_quantize(x)
    want = _np(_round(X.values(_np(x)), dtype))
    assert np.array_equal(_np(R.mx_dequantize(t, TD[dtype])), want)
    # into a view: unit columns, rows apart; what lies between stays
    big = torch.full((rows + 2, cols + 3), 7.0, dtype=TD[dtype], device=x.device)
    view = big[1:-1, 2:-1]
    assert R.mx_dequantize(t, TD[dtype], out=view) is view
    assert np.array_equal(_np(view), want)
    big[1:-1, 2:-1] = 7.0
    assert (big == 7.0).all()


# ----------------------------------------------------------------------------- products
SIZES = [(1, 1, 1), (1, 64, 33), (2, 300, 17), (16, 1024, 64), (17, 257, 100), (33, 96, 250), (64, 512, 256), (65, 512, 256),
         (130, 1000, 301), (256, 256, 512), (300, 2048, 130), (512, 768, 640)]


def _matmul_bound(a, b, ref, dtype):
    return STEP[dtype] * np.abs(ref) * 1.001 + a.shape[1] * 2.0**-23 * (np.abs(a) @ np.abs(b).T) + TINY[dtype]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_matmul(dtype, M, K, N):
    rng = np.random.default_rng(M + K + N)
    a, b = _gpu(rng.standard_normal((M, K)), dtype), _gpu(rng.standard_normal((N, K)) / 8, dtype)
    bias = _gpu(rng.standard_normal(N), dtype)
    va, vb = X.values(_np(a)), X.values(_np(b))
    ref = va @ vb.T
    bq = R.mx_quantize(b)
    y = R.mx_matmul(a, bq)
    assert y.dtype == TD[dtype] and y.shape == (M, N)
    assert (np.abs(_np(y) - ref) <= _matmul_bound(va, vb, ref, dtype)).all()
    yb = R.mx_matmul(R.mx_quantize(a), bq, bias=bias, dtype=TD[dtype])
    refb = ref + _np(bias)
    assert (np.abs(_np(yb) - refb) <= _matmul_bound(va, vb, refb, dtype) + 2.0**-23 * np.abs(refb)).all()
    assert torch.equal(R.mx_matmul(R.mx_quantize(a), bq, dtype=TD[dtype]), y)


@pytest.mark.parametrize("M,K,N", SIZES)
def test_matmul_exact(M, K, N):
    """Codes times common powers of two: every partial sum is a multiple of 1/4 below 2^22, so the float32
    result has one value, whatever the order."""
    rng = np.random.default_rng(M * 3 + K + N)
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    pick = lambda n: rng.choice(grid, (n, K)) * rng.choice([-1.0, 1.0], (n, K))  # noqa: E731
    a, b = pick(M), pick(N)
    assert K * 36 < 2**20
    y = R.mx_matmul(_gpu(a, "f32"), R.mx_quantize(_gpu(b, "f32")))
    assert np.array_equal(_np(y), X.values(a) @ X.values(b).T)


def test_matmul_far_scales():
    """Blocks whose powers of two lie far apart: each output is one block's product."""
    a, b = np.zeros((40, 128)), np.zeros((50, 128))
    for j in range(4):
        a[j::4, 32 * j:32 * j + 32] = 2.0 ** (30 * j - 60)
        b[:, 32 * j:32 * j + 32] = 2.0 ** (20 - 25 * j)
    y = R.mx_matmul(_gpu(a, "f32"), R.mx_quantize(_gpu(b, "f32")))
    assert np.array_equal(_np(y), a @ b.T)


@pytest.mark.parametrize("M,K,N", [(3, 256, 40), (100, 300, 301), (300, 512, 520)])
def test_matmul_into_a_view(M, K, N):
    rng = np.random.default_rng(1)
    a, b = _gpu(rng.standard_normal((M, K)), "bf16"), R.mx_quantize(_gpu(rng.standard_normal((N, K)), "bf16"))
    big = torch.full((M + 5, N + 7), 3.0, dtype=torch.bfloat16, device=a.device)
    view = big[2:M + 2, 3:N + 3]
    assert R.mx_matmul(a, b, out=view) is view
    assert torch.equal(view, R.mx_matmul(a, b))
    view.fill_(3.0)
    assert (big == 3.0).all()


# ----------------------------------------------------------------------------- every form of the product
GRID = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def _on_grid(gen, rows, cols):
    """Values that are their own Q: codes of a block whose largest is 6, signs included."""
    x = torch.tensor(GRID, device=dev())[torch.randint(0, 8, (rows, cols), generator=gen, device=dev())]
    x[:, ::32] = 6.0
    return x * (1 - 2 * torch.randint(0, 2, (rows, cols), generator=gen, device=dev()))


def _gen(seed):
    g = torch.Generator(device=dev())
    g.manual_seed(seed)
    return g


# rows of A from one to many, K long enough to be shared out, tiles of each shape, last tiles of a row or a column
@pytest.mark.parametrize("M,K,N", [(1, 1024, 8200), (1, 4097, 100), (3, 4097, 100), (16, 65536, 20), (17, 520, 9000),
                                   (40, 512, 9001), (64, 65536, 64), (70, 8192, 8192), (97, 40000, 300), (130, 40000, 301),
                                   (200, 1030, 3000), (300, 4096, 5000), (513, 4096, 12290), (2000, 1030, 4090),
                                   (1030, 4096, 12300), (1, 32768, 1300), (33, 128, 8192), (300, 128, 20000), (700, 65536, 1300)])
def test_every_form_of_the_product(M, K, N):
    """Sums of multiples of 1/4 below 2^22 (65536 * 36): one value in float32 whatever the order."""
    gen = _gen(M + K + N)
    a, b = _on_grid(gen, M, K), _on_grid(gen, N, K)
    ref = a.double() @ b.double().t().contiguous()
    bq = R.mx_quantize(b)
    for x in (a, R.mx_quantize(a)):
        y = R.mx_matmul(x, bq, dtype=torch.float32)
        assert torch.equal(y.double(), ref)
    bias = torch.randint(-8, 8, (N,), generator=gen, device=dev()).to(torch.bfloat16)
    y = R.mx_matmul(a.to(torch.bfloat16), bq, bias=bias)
    assert torch.equal(y, (ref + bias.double()).float().to(torch.bfloat16))


@pytest.mark.parametrize("save", [False, True])
@pytest.mark.parametrize("M,K,F", [(1, 4096, 600), (1, 1023, 9000), (5, 520, 333), (33, 33000, 40), (130, 33000, 151), (200, 1030, 3001),
                                   (300, 4096, 6000), (500, 2048, 12290), (1500, 512, 2050), (1, 65536, 300), (100, 128, 4096),
                                   (400, 1024, 8192), (700, 65536, 700), (3000, 1024, 2500)])
def test_every_form_of_the_gated_product(M, K, F, save):
    gen = _gen(M + K + F)
    x, w = _on_grid(gen, M, K) / 64, _on_grid(gen, 2 * F, K) / 64
    gu = x.double() @ w.double().t().contiguous()
    wq = R.mx_quantize(w)
    for a in (x, R.mx_quantize(x)):
        got = R.mx_gated(a, wq, act="silu", dtype=torch.float32, save=save)
        h = got[0] if save else got
        if save:
            assert torch.equal(got[1].double(), gu)  # exact sums, as above
        g, u = gu[:, :F], gu[:, F:]
        ref = g / (1 + torch.exp(-g)) * u
        # the float32 activation's relative error (3 + |g|) 2^-21, the product's and the store's 2^-24 each
        bound = ((3 + g.abs()) * 2.0**-21 + 2.0**-23) * ref.abs() + 1e-37
        assert ((h.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M", [1, 3, 20, 200])
def test_unquantised_rows_at_any_place(dtype, M):
    """Rows that start off every vector's alignment, with any row stride and with strided columns."""
    gen = _gen(M)
    big = _on_grid(gen, 2 * M + 1, 700).to(TD[dtype])
    b = R.mx_quantize(_on_grid(gen, 50, 333))
    w = R.mx_quantize(_on_grid(gen, 24, 333))
    for x in (big[1:M + 1, 1:334], big[::2, 3:336][:M], big[:M, :666:2], big[:1, 5:338].expand(M, 333)):
        c = x.contiguous().clone()
        assert torch.equal(R.mx_matmul(x, b), R.mx_matmul(c, b))
        assert torch.equal(R.mx_gated(x, w), R.mx_gated(c, w))


# ----------------------------------------------------------------------------- far offsets
def test_offsets_past_32_bits():
    """A tensor of 4.6 GB of codes from 18 GB of values in {-3 .. 3}, which are their own Q along either axis (a block's
    largest of 3 is 6 halves): values back, and products with its last rows."""
    rows, cols = 140_000, 65_536
    gen = _gen(77)
    x = torch.randint(-3, 4, (rows, cols), generator=gen, device=dev(), dtype=torch.int8).to(torch.bfloat16)
    x[:, ::32] = 3
    x[::32] = 3
    r, c = R.mx_quantize(x, axis=None)
    assert r.data.numel() > 2**32
    assert torch.equal(R.mx_dequantize(r), x)
    back = R.mx_dequantize(c)
    assert all(torch.equal(back[k:k + 8192], x[:, k:k + 8192].t()) for k in range(0, cols, 8192))
    del back
    for M in (1, 40, 200):
        a = torch.randint(-3, 4, (M, cols), generator=gen, device=dev(), dtype=torch.int8).to(torch.bfloat16)
        a[:, ::32] = 3
        y = R.mx_matmul(R.mx_quantize(a), r, dtype=torch.float32)
        for part in (slice(0, 300), slice(rows - 300, rows)):
            assert torch.equal(y[:, part], a.float() @ x[part].float().t().contiguous())
        g = R.mx_gated(R.mx_quantize(a), r, act="relu", dtype=torch.float32)
        up = slice(rows - 300, rows)
        gate = slice(rows // 2 - 300, rows // 2)
        ref = (a.float() @ x[gate].float().t().contiguous()).relu() * (a.float() @ x[up].float().t().contiguous())
        assert torch.equal(g[:, -300:], ref)  # two exact factors, one rounding


def test_gated_grad_offsets_past_32_bits():
    M, F = 70_016, 32_768
    gen = _gen(78)
    dh = torch.randn(M, F, generator=gen, device=dev(), dtype=torch.bfloat16)
    gu = torch.randn(M, 2 * F, generator=gen, device=dev(), dtype=torch.bfloat16)
    rows, cols = R.mx_gated_grad(dh, gu)
    want_r, want_c = R.mx_gated_grad(dh[-128:].clone(), gu[-128:].clone())
    assert torch.equal(R.mx_dequantize(rows)[-128:], R.mx_dequantize(want_r))
    assert torch.equal(R.mx_dequantize(cols)[:, -128:], R.mx_dequantize(want_c))


# ----------------------------------------------------------------------------- gated block
REL_ACT = 2.0**-18  # the float32 activation: (3 + |w|) 2^-21 with |w| below 5 where it counts


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("act", X.ACTS)
@pytest.mark.parametrize("M,K,F", [(1, 64, 1), (1, 512, 100), (7, 300, 33), (40, 256, 65), (70, 100, 130), (129, 512, 128),
                                   (300, 768, 257)])
def test_gated(dtype, act, M, K, F):
    rng = np.random.default_rng(M + K + F)
    x, w = _gpu(rng.standard_normal((M, K)), dtype), _gpu(rng.standard_normal((K, 2 * F)) / np.sqrt(K), dtype)
    wq = R.mx_quantize(w, axis=0)
    vx, vw = X.values(_np(x)), X.values(_np(w).T)
    g, u = vx @ vw[:F].T, vx @ vw[F:].T
    h, gu = R.mx_gated(x, wq, act=act, save=True)
    assert h.shape == (M, F) and gu.shape == (M, 2 * F) and h.dtype == gu.dtype == TD[dtype]
    # the sums' errors without the output's half step
    sums = K * 2.0**-23
    eg, eu = sums * (np.abs(vx) @ np.abs(vw[:F]).T), sums * (np.abs(vx) @ np.abs(vw[F:]).T)
    for got, ref, e in ((_np(gu)[:, :F], g, eg), (_np(gu)[:, F:], u, eu)):
        assert (np.abs(got - ref) <= STEP[dtype] * np.abs(ref) * 1.001 + e + TINY[dtype]).all()
    a = X.act(act, g)
    ref = a * u
    # |act'| is below 1.2 everywhere; gelu's bound has twice the constant
    ea = 1.2 * eg + 2 * REL_ACT * np.abs(a)
    bound = STEP[dtype] * np.abs(ref) * 1.01 + ea * (np.abs(u) + eu) + np.abs(a) * eu + TINY[dtype] + 2.0**-23 * np.abs(ref)
    assert (np.abs(_np(h) - ref) <= bound).all()
    assert torch.equal(R.mx_gated(R.mx_quantize(x), wq, act=act, dtype=TD[dtype]), h)


@pytest.mark.parametrize("act", X.ACTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,F", [(1, 1), (1, 96), (33, 31), (130, 64), (70, 129), (129, 260)])
def test_gated_grad(dtype, act, M, F):
    rng = np.random.default_rng(M + F)
    dh, gu = _gpu(rng.standard_normal((M, F)), dtype), _gpu(2 * rng.standard_normal((M, 2 * F)), dtype)
    want = X.gated_grad(_np(dh), _np(gu), act)
    rows, cols = R.mx_gated_grad(dh, gu, act=act)
    _check_tensor(rows, want)
    _check_tensor(cols, want.T)


@pytest.mark.parametrize("act", X.ACTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,F", [(1, 1), (1, 96), (33, 31), (130, 64), (70, 129), (129, 260), (40, 32), (300, 416)])
def test_gated_grad_in_one_direction(dtype, act, M, F):
    """Each direction alone: the same codes and scale bytes as both from one pass, padding and all."""
    rng = np.random.default_rng(M + F)
    dh, gu = _gpu(rng.standard_normal((M, F)), dtype), _gpu(2 * rng.standard_normal((M, 2 * F)), dtype)
    want = X.gated_grad(_np(dh), _np(gu), act)
    _check_tensor(R.mx_gated_grad(dh, gu, act=act, axis=1), want)
    _check_tensor(R.mx_gated_grad(dh, gu, act=act, axis=0), want.T)


@pytest.mark.parametrize("act", X.ACTS)
def test_gated_grad_far_pre_activations(act):
    """Pre-activations at both ends, where a sigmoid or its complement has few digits in float32, and around
    the zero of act', in blocks of their own so that each decides its block's scale."""
    rng = np.random.default_rng(12)
    dh = rng.standard_normal((64, 320))
    gu = rng.standard_normal((64, 640))
    for k, at in enumerate([-100.0, -70.0, -30.0, -12.0, -9.0, -5.0, 5.0, 9.0, 30.0, 100.0]):
        gu[:, 32 * k:32 * k + 32] = at + rng.random((64, 32))
    gu[32:, :320] = -1.2784645427610738 + 1e-3 * rng.standard_normal((32, 320))
    gu[48:, :320] = -0.7517916243494656 + 1e-3 * rng.standard_normal((16, 320))
    for dtype in ("f32", "bf16", "f16"):
        d, z = _gpu(dh, dtype), _gpu(gu, dtype)
        want = X.gated_grad(_np(d), _np(z), act)
        # below 2^-100 of float32 a gradient's own value is not kept to the last digit; f32 keeps these
        rows, cols = R.mx_gated_grad(d, z, act=act)
        _check_tensor(rows, want)
        _check_tensor(cols, want.T)


def test_gated_grad_on_borders():
    """relu makes the gradients exact products: gradients on a border between two codes take the even one,
    and gradients a float32 step beside one do not."""
    F = 128
    dh = np.ones((32, F))
    gu = np.ones((32, 2 * F))
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    at = np.tile(borders, F // 8)
    near = np.stack([at, np.nextafter(at.astype(np.float32), np.float32(9)), np.nextafter(at.astype(np.float32), np.float32(0)), -at])
    gu[:, F:] = near[np.arange(32) % 4]
    gu[1::4, F + 7::8] = 6.0
    d, z = _gpu(dh, "f32"), _gpu(gu, "f32")
    rows, cols = R.mx_gated_grad(d, z, act="relu")
    want = X.gated_grad(_np(d), _np(z), "relu")
    _check_tensor(rows, want)
    _check_tensor(cols, want.T)


def test_gated_grad_not_finite():
    rng = np.random.default_rng(2)
    dh, gu = rng.standard_normal((70, 100)), rng.standard_normal((70, 200))
    dh[3, 5], gu[20, 40], gu[40, 150], gu[60, 99] = np.nan, np.nan, np.inf, -np.inf
    d, z = _gpu(dh, "bf16"), _gpu(gu, "bf16")
    with np.errstate(invalid="ignore"):
        want = X.gated_grad(_np(d), _np(z), "silu")
    assert (~np.isfinite(want)).sum() >= 6
    rows, cols = R.mx_gated_grad(d, z)
    _check_tensor(rows, want)
    _check_tensor(cols, want.T)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_relu_of_a_negative_zero(dtype):
    """max(-0, 0) is +0: the gradients are zeros with dh's sign, codes and all."""
    dh = np.where(np.arange(96 * 40).reshape(40, 96) % 3 == 0, -1.5, 1.5)
    gu = np.full((40, 192), -0.0)
    gu[:, 96:] = 2.0
    d, z = _gpu(dh, dtype), _gpu(gu, dtype)
    want = np.concatenate([dh * 2.0 * 0.0, dh * 0.0], axis=1)
    rows, cols = R.mx_gated_grad(d, z, act="relu")
    _check_tensor(rows, want)
    _check_tensor(cols, want.T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", X.ACTS)
@pytest.mark.parametrize("F", [64, 70])
def test_gated_grad_of_an_overflowing_product(dtype, act, F):
    """dh * u past the float32 range where act' brings the gradient back: below relu's zero, beside the zeros of the
    other derivatives, and far out on their tails. The formula's gradient is finite there, and small or zero."""
    rng = np.random.default_rng(F)
    dh = rng.standard_normal((40, F))
    gu = rng.standard_normal((40, 2 * F))
    big = np.zeros((40, F), bool)
    big[2, 7] = big[9, 33:40] = big[33, F - 1] = big[39, 0] = True
    big[:, 50] = True
    dh[big] = 1.5e30 * rng.choice([-1, 1], big.sum())
    gu[:, F:][big] = 1e10
    root = {"silu": -1.2784645427610738, "gelu": -0.7517915246935645, "gelu_tanh": -0.7524614220710163, "relu": -0.0}[act]
    gu[:, :F][big] = root - rng.integers(0, 5, big.sum()) * 2.0**-23
    far = {"silu": -55.0, "gelu": -9.0, "gelu_tanh": -8.0, "relu": -1.0}[act]
    gu[:, 5], dh[:, 5], gu[:, F + 5] = far, 1.5e30, 1e10
    d, z = _gpu(dh, dtype), _gpu(gu, dtype)
    want = X.gated_grad(_np(d), _np(z), act)
    assert np.abs(want).max() < 2.0**127
    rows, cols = R.mx_gated_grad(d, z, act=act)
    _check_tensor(rows, want)
    _check_tensor(cols, want.T)


@pytest.mark.parametrize("F", [64, 70])
def test_gated_grad_just_below_infinity(F):
    """Gradients between the largest float32 and 2^128, which float32 would round up to infinity, are finite; from 2^128
    on a block is NaN."""
    dh, gu = np.ones((33, F)), np.ones((33, 2 * F))
    dh[3, 5], gu[3, F + 5] = (2 - 2.0**-22) * 2.0**64, (1 + 2.0**-23) * 2.0**63  # (2 - 2^-44 (1 + ..)) 2^127
    dh[7, 9], gu[7, F + 9] = -(2 - 2.0**-22) * 2.0**63, (1 + 2.0**-23) * 2.0**64
    dh[20, 40], gu[20, F + 40] = 2.0**64, 2.0**64
    d, z = _gpu(dh, "f32"), _gpu(gu, "f32")
    want = X.gated_grad(_np(d), _np(z), "relu")
    high = np.abs(want[[3, 7], [5, 9]])
    with np.errstate(over="ignore"):
        assert (high < 2.0**128).all() and np.isinf(high.astype(np.float32)).all() and want[20, 40] == 2.0**128
    want[20, 40] = np.inf
    rows, cols = R.mx_gated_grad(d, z, act="relu")
    _check_tensor(rows, want)
    _check_tensor(cols, want.T)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K,F", [(5, 40, 33), (70, 256, 64), (130, 300, 100)])
def test_training_step_together(dtype, M, K, F):
    """The operators as a training step uses them, against the formulas on the same inputs."""
    rng = np.random.default_rng(M)
    x, w = _gpu(rng.standard_normal((M, K)), dtype), _gpu(rng.standard_normal((K, 2 * F)) / np.sqrt(K), dtype)
    dh = _gpu(rng.standard_normal((M, F)), dtype)
    xr, xc = R.mx_quantize(x, axis=None)
    wr, wc = R.mx_quantize(w, axis=None)
    h, gu = R.mx_gated(xr, wc, act="gelu_tanh", dtype=TD[dtype], save=True)
    dx, dw = R.mx_gated_backward(dh, gu, wr, xc, act="gelu_tanh")
    assert dx.shape == (M, K) and dw.shape == (K, 2 * F) and dx.dtype == dw.dtype == TD[dtype]
    d = X.gated_grad(_np(dh), _np(gu), "gelu_tanh")
    for got, a, b in ((dx, X.values(d), X.values(_np(w))), (dw, X.values(_np(x).T), X.values(d.T))):
        ref = a @ b.T
        assert (np.abs(_np(got) - ref) <= _matmul_bound(a, b, ref, dtype)).all()


@pytest.mark.parametrize("M,K,F", [(1, 64, 17), (40, 300, 96), (2000, 520, 700), (40_000, 128, 48)])
def test_backward_is_its_parts(M, K, F):
    """The one call against the gradients and the two products one by one, in both output types."""
    gen = _gen(M)
    dh = torch.randn(M, F, generator=gen, device=dev()).to(torch.bfloat16)
    gu = torch.randn(M, 2 * F, generator=gen, device=dev()).to(torch.bfloat16)
    w = R.mx_quantize(torch.randn(K, 2 * F, generator=gen, device=dev()))
    x = R.mx_quantize(torch.randn(M, K, generator=gen, device=dev()), axis=0)
    rows, cols = R.mx_gated_grad(dh, gu, act="gelu")
    for dtype in (torch.bfloat16, torch.float32):
        dx, dw = R.mx_gated_backward(dh, gu, w, x, act="gelu", dtype=dtype)
        assert torch.equal(dx, R.mx_matmul(rows, w, dtype=dtype))
        assert torch.equal(dw, R.mx_matmul(x, cols, dtype=dtype))


def test_gradients_against_differences():
    """With x, w and the gradients on exact grids the quantisers change nothing they are differentiated
    through: dx and dw of sum(dh * h) against central differences of the float64 block, to the rounding of
    d to four bits: each element of d is off by at most half a step, a sixth of its block's maximum."""
    rng = np.random.default_rng(21)
    M, K, F = 32, 32, 16
    x = rng.choice([-1.0, -0.5, 0.5, 1.0], (M, K))
    w = rng.choice([-1.0, -0.5, 0.5, 1.0], (K, 2 * F)) / 8
    x[:, 0] = 6.0
    x[0] = 6.0
    w[:, 0] = w[0] = 6.0 / 8
    assert np.array_equal(X.values(x), x) and np.array_equal(X.values(x.T).T, x)
    assert np.array_equal(X.values(w), w) and np.array_equal(X.values(w.T).T, w)
    dh = rng.standard_normal((M, F))
    dhq = _np(_round(dh, "f32"))
    xr, xc = R.mx_quantize(_gpu(x, "f32"), axis=None)
    wr, wc = R.mx_quantize(_gpu(w, "f32"), axis=None)
    _, gu = R.mx_gated(xr, wc, dtype=torch.float32, save=True)
    dx, dw = (_np(t) for t in R.mx_gated_backward(_gpu(dh, "f32"), gu, wr, xc))

    def loss(x_, w_):
        gu_ = x_ @ w_
        return (dhq * X.act("silu", gu_[:, :F]) * gu_[:, F:]).sum()

    d = X.gated_grad(dhq, x @ w, "silu")
    off_rows = np.abs(X.values(d) - d) @ np.abs(w).T
    off_cols = np.abs(x).T @ np.abs(X.values(d.T).T - d)
    step = 1e-4
    for i, j in ((0, 0), (3, 7), (31, 31), (12, 20)):
        for arr, got, off, first in ((x, dx, off_rows, True), (w, dw, off_cols, False)):
            e = np.zeros_like(arr)
            e[i, j] = step
            diff = (loss(x + e, w) - loss(x - e, w) if first else loss(x, w + e) - loss(x, w - e)) / (2 * step)
            assert abs(got[i, j] - diff) <= off[i, j] * 1.01 + 1e-4 * (1 + abs(diff)), (i, j, first)


# ----------------------------------------------------------------------------- streams, graphs, repeats
def _step(x, w, dh):
    xr, xc = R.mx_quantize(x, axis=None)
    wr, wc = R.mx_quantize(w, axis=None)
    h, gu = R.mx_gated(xr, wc, dtype=x.dtype, save=True)
    return (h, *R.mx_gated_backward(dh, gu, wr, xc), R.mx_matmul(x, wc), R.mx_dequantize(xr))


def _step_inputs(seed, M=100, K=512, F=96):
    rng = np.random.default_rng(seed)
    return (_gpu(rng.standard_normal((M, K)), "bf16"), _gpu(rng.standard_normal((K, 2 * F)), "bf16"),
            _gpu(rng.standard_normal((M, F)), "bf16"))


def test_repeats_are_equal():
    ins = _step_inputs(1)
    first = _step(*ins)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, _step(*ins)))


def test_another_stream():
    ins = _step_inputs(2)
    want = _step(*ins)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = _step(*ins)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_two_streams_at_once():
    a, b = _step_inputs(3), _step_inputs(4, M=3)
    want = _step(*a), _step(*b)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(3):
        with torch.cuda.stream(s):
            x = _step(*a)
        with torch.cuda.stream(t):
            y = _step(*b)
        got.append((x, y))
    torch.cuda.synchronize()
    for x, y in got:
        assert all(torch.equal(p, q) for p, q in zip(want[0] + want[1], x + y))


@pytest.mark.parametrize("M", [1, 100, 300])
def test_captured_and_replayed(M):
    """Two graphs that live at the same time, replayed in turn with other inputs, against eager calls."""
    sets = [_step_inputs(5, M=M), _step_inputs(6, M=M)]
    graphs = []
    for ins in sets:
        _step(*ins)
    torch.cuda.synchronize()
    for ins in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _step(*ins)
        graphs.append((g, out))
    for k in range(4):
        for (g, out), ins in zip(graphs, sets):
            for dst, src in zip(ins, _step_inputs(50 + k, M=M)):
                dst.copy_(src)
            g.replay()
        torch.cuda.synchronize()
        want = _step(*sets[0])
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(want, out)), k


FIRST_CALL = """
import torch, rank_bit_residual_amd as R
g = torch.Generator(device="cuda").manual_seed(3)
x, w = (torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16) for s in ((100, 512), (512, 192)))
dh = torch.randn(100, 96, generator=g, device="cuda", dtype=torch.bfloat16)
def step():
    xr, xc = R.mx_quantize(x, axis=None)
    wr, wc = R.mx_quantize(w, axis=None)
    h, gu = R.mx_gated(xr, wc, save=True)
    return h, *R.mx_gated_backward(dh, gu, wr, xc), R.mx_matmul(x[:1], wc)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = step()
for k in range(3):
    x.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, step())), k
print("same")
"""


def test_first_call_of_a_process_captured():
    import subprocess
    import sys

    r = subprocess.run([sys.executable, "-c", FIRST_CALL], capture_output=True, text=True, timeout=100,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


def test_output_beside_the_input():
    """Input and output as columns of one buffer."""
    buf = torch.randn(100, 64 + 40, device=dev(), dtype=torch.bfloat16)
    b = R.mx_quantize(torch.randn(40, 64, device=dev()))
    want = R.mx_matmul(buf[:, :64], b)
    assert torch.equal(R.mx_matmul(buf[:, :64], b, out=buf[:, 64:]), want) and torch.equal(buf[:, 64:], want)


# ----------------------------------------------------------------------------- refusals that need device tensors
def test_binding_refusals():
    d = dev()
    x = torch.randn(4, 64, device=d)
    t = R.mx_quantize(x)
    with pytest.raises(TypeError):
        R.mx_quantize(x.double())
    with pytest.raises(TypeError):
        R.mx_dequantize(t, torch.float64)
    with pytest.raises(TypeError):
        R.mx_matmul(x, t, dtype=torch.int32)
    for call in (lambda: R.mx_quantize(x[0]), lambda: R.mx_quantize(x[:0]), lambda: R.mx_quantize(x, axis=2),
                 lambda: R.mx_quantize(x, axis=True), lambda: R.mx_matmul(x[:, :32], t),
                 lambda: R.mx_matmul(x, t, bias=torch.zeros(5, device=d)),
                 lambda: R.mx_matmul(x, t, bias=torch.zeros(4, device=d, dtype=torch.bfloat16)),
                 lambda: R.mx_matmul(x, t, bias=torch.zeros(4)),
                 lambda: R.mx_matmul(x, t, out=torch.zeros(4, 5, device=d)),
                 lambda: R.mx_matmul(x, t, out=torch.zeros(4, 4, device=d).t()),
                 lambda: R.mx_matmul(x, t, out=torch.zeros(1, 4, device=d).expand(4, 4)),
                 lambda: R.mx_matmul(x, t, out=torch.zeros(4, 4, device=d, dtype=torch.bfloat16)),
                 lambda: R.mx_matmul(x, R.mx_quantize(torch.randn(64, 64, device=d)), out=x),
                 lambda: R.mx_dequantize(t, torch.bfloat16, out=t.data[:512].view(torch.bfloat16).view(4, 64)),
                 lambda: R.mx_matmul(x, R.MxTensor(torch.zeros(1 << 14, dtype=torch.uint8, device=d)[16:], 4, 64)),
                 lambda: R.mx_gated(x, R.mx_quantize(x[:3])), lambda: R.mx_gated(x[:, :60], t),
                 lambda: R.mx_gated(x, t, act="tanh"), lambda: R.mx_gated_grad(x, x),
                 lambda: R.mx_gated_grad(x, torch.zeros(4, 128, device=d, dtype=torch.float16)),
                 lambda: R.mx_gated_backward(x, torch.zeros(4, 128, device=d), t, t)):
        with pytest.raises(ValueError):
            call()


def test_inputs_that_require_grad():
    """Refused where autograd would lose their gradient; taken under no_grad, in inference mode and in a Function."""
    d = dev()
    x, w = torch.randn(40, 64, device=d, requires_grad=True), torch.randn(64, 96, device=d, requires_grad=True)
    bias, out = torch.zeros(96, device=d, requires_grad=True), torch.zeros(40, 96, device=d)
    with torch.no_grad():
        xr, xc = R.mx_quantize(x, axis=None)
        wr, wc = R.mx_quantize(w, axis=None)
        h, gu = R.mx_gated(x, wc, save=True)
        dh = torch.randn_like(h)
        want = R.mx_gated_backward(dh, gu, wr, xc)
        y = R.mx_matmul(x, wc, bias=bias, out=out)
    assert not h.requires_grad and not y.requires_grad
    with torch.inference_mode():
        assert torch.equal(R.mx_gated(x, wc), h)
    assert torch.equal(R.mx_gated(x.detach(), wc), h)
    leaf = dh.clone().requires_grad_()
    for call in (lambda: R.mx_quantize(w), lambda: R.mx_matmul(x, wc), lambda: R.mx_matmul(x, wc, dtype=torch.bfloat16),
                 lambda: R.mx_matmul(xr, wc, bias=bias, dtype=torch.float32), lambda: R.mx_gated(x, wc),
                 lambda: R.mx_gated_grad(leaf, gu), lambda: R.mx_gated_backward(leaf, gu, wr, xc),
                 lambda: R.mx_dequantize(xr, torch.float32, out=x)):
        with pytest.raises(RuntimeError, match="requires grad"):
            call()

    class Gated(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            xr, ctx.x = R.mx_quantize(x, axis=None)
            ctx.w, wc = R.mx_quantize(w, axis=None)
            h, gu = R.mx_gated(xr, wc, dtype=x.dtype, save=True)
            ctx.save_for_backward(gu)
            return h

        @staticmethod
        def backward(ctx, dh):
            return R.mx_gated_backward(dh, ctx.saved_tensors[0], ctx.w, ctx.x)

    Gated.apply(x, w).backward(dh)
    assert torch.equal(x.grad, want[0]) and torch.equal(w.grad, want[1])


def test_float64_oracle_matches_the_library_rule():
    """The operators' codes are those of quantize_activations with a unit scale."""
    x = _gpu(_wide(np.random.default_rng(4), 20, 300), "bf16")
    codes, scales, _ = R.quantize_activations(x, torch.ones(300, device=x.device), "mx")
    got, s, _, _ = _parts(R.mx_quantize(x))
    assert np.array_equal(codes.cpu().numpy()[:, :150], O.pack_nibbles(got))
    assert np.array_equal(scales.cpu().numpy()[:, :s.shape[1]], s)
