"""8-bit tensor operators on an MI355X against plain float64 implementations (oracle/int8.py).

Codes, scales and dequantised values must be equal. Products: the integer sum S is exact; y is float32(S) times
float32(sa sb), each off by half a step, plus the bias with one rounding, then the output's own: together
2^-23 |S sa sb| + (2^-24 + STEP) |y|, and a small multiple of the smallest magnitude below the normal range.
"""
import ctypes
import threading

import numpy as np
import pytest
import torch

import rank_bit_residual_amd as R
from oracle import int8 as X
from rank_bit_residual_amd import _lib

pytestmark = pytest.mark.gpu

TD = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
STEP = {"f32": 2.0**-24, "bf16": 2.0**-8, "f16": 2.0**-11}  # half a step, relative
TINY = {"f32": 2.0**-149, "bf16": 2.0**-133, "f16": 2.0**-24}  # the smallest magnitude of the type


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _gpu(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, np.float64)).to(TD[dtype]).to(dev())


def _np(t):
    return t.detach().cpu().double().numpy()


def _form(M, N, K):
    got = (ctypes.c_int * 4)()
    assert _lib.load().svdq_i8_product_form(M, N, K, got) == 0
    return tuple(got)


def _check_tensor(t, want):
    """t holds Q(want): equal codes and scales, zeros past the last element."""
    assert t.shape == want.shape
    codes, past = X.unpack(t.codes.cpu().numpy(), t.rows, t.cols)
    wc, ws = X.quantize(want)
    s = t.scales.cpu().numpy()
    assert np.array_equal(s, ws, equal_nan=True), np.argwhere(s != ws)[:4]
    assert np.array_equal(codes, wc), (np.argwhere(codes != wc)[:4], want[tuple(np.argwhere(codes != wc)[0])])
    assert not past.any()


def _wide(rng, rows, cols):
    """Values whose rows and columns differ by many powers of two, with zeros, ties, a zero row and a zero column."""
    x = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-6, 7, (rows, 1)) * 2.0 ** rng.integers(-3, 4, (1, cols))
    x[rng.random((rows, cols)) < 0.05] = 0
    if rows > 4:
        x[1] = 0
        x[2] = np.where(np.arange(cols) % 7 == 0, 127.0, (rng.integers(-127, 127, cols) + 0.5))  # ties of a scale of 1
    if cols > 4:
        x[:, 3] = 0
    return x


# ----------------------------------------------------------------------------- quantise
QUANT_SIZES = [(1, 1), (1, 64), (1, 4096), (3, 31), (33, 33), (128, 128), (130, 255), (65, 257), (300, 70), (257, 1000), (20, 1030),
               (17, 2500), (9, 5003), (5, 9001), (3, 20000), (2, 40000), (1100, 40)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", QUANT_SIZES)
def test_quantize(dtype, rows, cols):
    x = _gpu(_wide(np.random.default_rng(rows * 1009 + cols), rows, cols), dtype)
    both = R.int8_quantize(x, axis=None)
    want = _np(x)
    for t, w in ((R.int8_quantize(x), want), (R.int8_quantize(x, axis=0), want.T), (both[0], want), (both[1], want.T)):
        _check_tensor(t, w)


@pytest.mark.parametrize("rows,cols,dtype", [(9001, 64, "bf16"), (9001, 300, "f16"), (4500, 1000, "f32"), (4999, 1500, "bf16"), (2100, 4000, "f16"),
                                             (1100, 5003, "f32"), (1100, 8195, "bf16"), (5001, 4200, "bf16"), (4500, 8190, "f16"), (1030, 12300, "bf16"), (600, 16500, "f16"),
                                             (9, 5, "f32"), (700, 7, "bf16"), (5, 8, "f16"), (2000, 9, "bf16")])
def test_quantize_many_rows(rows, cols, dtype):
    """More rows than the blocks of a launch, so that each takes several, and a last one that is not full."""
    x = _gpu(_wide(np.random.default_rng(rows + cols), rows, cols), dtype)
    want = _np(x)
    _check_tensor(R.int8_quantize(x), want)
    r, c = R.int8_quantize(x, axis=None)
    _check_tensor(r, want)
    _check_tensor(c, want.T)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_quantize_strides(dtype):
    rng = np.random.default_rng(5)
    big = _gpu(_wide(rng, 200, 301), dtype)
    odd = _gpu(_wide(rng, 1, 200 * 301 + 1), dtype).reshape(-1)[1:].reshape(200, 301)  # not 4-byte aligned in 16 bits
    for x in (big.t(), big[3:150, 5:222], big[::2, ::3], big[7:8].expand(40, 301), big[:, 9:10].expand(200, 50), odd, odd.t(),
              big[:, :96].t(), big[:, 4:5], big[4:5].t(), big[::3, ::2].t()):
        rows, cols = R.int8_quantize(x, axis=None)
        _check_tensor(rows, _np(x))
        _check_tensor(cols, _np(x).T)
        _check_tensor(R.int8_quantize(x), _np(x))
        _check_tensor(R.int8_quantize(x, axis=0), _np(x).T)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_quantize_ends_of_the_range(dtype):
    """Subnormals, the largest values, negative zeros, and values around every border between two codes."""
    info = torch.finfo(TD[dtype])
    rng = np.random.default_rng(6)
    x = np.zeros((9, 256))
    x[0] = rng.integers(-7, 8, 256) * TINY[dtype]
    x[1] = rng.integers(-700, 700, 256) * TINY[dtype]
    x[2] = -0.0
    x[3] = rng.choice([-1.0, 1.0], 256) * info.max
    x[4] = info.max * rng.random(256)
    x[5] = info.tiny * (1 + rng.random(256))
    x[6] = info.tiny / 2 * rng.random(256)
    for r, s in ((7, 2.0**-9), (8, 3.0)):
        x[r] = (np.arange(256) - 127.5).clip(-127, 127) * s  # every tie
    x = _gpu(x, dtype)
    rows, cols = R.int8_quantize(x, axis=None)
    _check_tensor(rows, _np(x))
    _check_tensor(cols, _np(x).T)


def test_codes_next_to_a_border():
    """float32 values a step from (k + 1/2) s for every k, with scales of every mantissa: what x times 1 / s cannot tell apart."""
    rng = np.random.default_rng(11)
    most = (1 + rng.random(400)).astype(np.float32) * np.float32(127) * 2.0 ** rng.integers(-40, 40, 400).astype(np.float32)
    s = (most.astype(np.float64) / 127).astype(np.float32)
    x = ((np.arange(127) + 0.5) * s[:, None].astype(np.float64)).astype(np.float32)
    x = np.concatenate([x, np.nextafter(x, np.float32(np.inf)), np.nextafter(x, np.float32(0)), most[:, None]], 1)
    x = np.where(np.abs(x) > most[:, None], most[:, None], x)
    _check_tensor(R.int8_quantize(torch.from_numpy(x).to(dev())), x.astype(np.float64))
    _check_tensor(R.int8_quantize(torch.from_numpy(x).to(dev()), axis=None)[1], x.T.astype(np.float64))
    _check_tensor(R.int8_quantize(torch.from_numpy(np.ascontiguousarray(x.T)).to(dev()), axis=0), x.astype(np.float64))


def _smallest_scales(dtype):
    """[90, 382] values whose rows' scales fill [2^-126, 2^-124): those next to every border between two codes, and the row's largest. (Half
    of such a scale may be no float32.)"""
    rng = np.random.default_rng(31)
    step = {"f32": 2.0**-23, "bf16": 2.0**-7}[dtype]
    most = np.concatenate([127 * (1 + rng.random(60)) * 2.0**-126, 127 * (1 + rng.random(20)) * 2.0**-125,
                           127 * 2.0**-126 * (1 + step * np.arange(9)), [2.0**-119]])
    most = _gpu(most, dtype)
    s = (_np(most) / 127).astype(np.float32)
    t = _gpu((np.arange(127) + 0.5) * s[:, None].astype(np.float64), dtype)
    x = torch.cat([t, torch.nextafter(t, t * 0), -torch.nextafter(t, t + 1), most[:, None]], 1)
    x = torch.minimum(x.abs(), x[:, -1:]) * torch.where(x < 0, -1, 1)
    x[0, :-1:2] = x[0, -1:] / 2
    return x.to(TD[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_codes_next_to_a_border_of_the_smallest_scales(dtype):
    x = _smallest_scales(dtype)
    want = _np(x)
    s = X.quantize(want)[1]
    assert (s >= 2.0**-126).all() and (s < 2.0**-124).all() and ((s > 2.0**-126) & (s < 2.0**-125)).sum() >= 60
    both = R.int8_quantize(x, axis=None)
    _check_tensor(both[0], want)
    _check_tensor(both[1], want.T)
    _check_tensor(R.int8_quantize(x), want)
    _check_tensor(R.int8_quantize(x.t().contiguous(), axis=0), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_codes_of_the_smallest_scales_in_a_norm_and_a_product(dtype):
    x = _smallest_scales(dtype)
    want = _np(x)
    # a norm's output is its bias where the weight is zero
    z = torch.randn(3, x.shape[1], device=x.device, dtype=x.dtype)
    for r in range(0, x.shape[0], 7):
        _check_tensor(R.layer_norm(z, torch.zeros_like(x[r]), x[r], quantize="int8"), np.tile(want[r], (3, 1)))
    # times 127 I the codes come back, rounded once
    eye = R.int8_quantize(127 * torch.eye(x.shape[1], device=x.device))
    codes, s = X.quantize(want)
    y = (127.0 * codes * s[:, None].astype(np.float64)).astype(np.float32)
    for M in (1, 2, 40, 90):
        assert np.array_equal(R.int8_matmul(x[:M].float(), eye).cpu().numpy(), y[:M])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_infinities_and_nan_poison_their_row_alone(dtype):
    x = np.random.default_rng(8).standard_normal((70, 300))
    x[1, 40], x[2, 299], x[50, 0], x[51, 64] = np.inf, np.nan, -np.inf, np.nan
    x = _gpu(x, dtype)
    rows, cols = R.int8_quantize(x, axis=None)
    _check_tensor(rows, _np(x))
    _check_tensor(cols, _np(x).T)
    got = _np(R.int8_dequantize(rows, torch.float32))
    assert np.array_equal(np.isnan(got), np.isnan(X.values(_np(x))))
    w = R.int8_quantize(_gpu(np.random.default_rng(9).standard_normal((40, 300)), dtype))
    for y in (R.int8_matmul(rows, w), R.int8_matmul(w, rows).t(), R.int8_matmul(x, w), R.int8_matmul(x[:3], w)):
        bad = np.isnan(_np(y)).all(1)
        assert np.array_equal(np.isnan(_np(y)).any(1), bad)
        assert np.flatnonzero(bad).tolist() == [r for r in (1, 2, 50, 51) if r < y.shape[0]]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 33), (64, 128), (70, 300)])
def test_dequantize(dtype, rows, cols):
    x = _gpu(_wide(np.random.default_rng(rows + cols), rows, cols), "f32")
    t = R.int8_quantize(x)
    codes, s = X.quantize(_np(x))
    want = _np(torch.from_numpy(codes.astype(np.float32) * s[:, None]).to(TD[dtype]))
    assert np.array_equal(_np(R.int8_dequantize(t, TD[dtype])), want)
    # into a view: unit columns, rows apart; what lies between stays
    big = torch.full((rows + 2, cols + 3), 7.0, dtype=TD[dtype], device=x.device)
    view = big[1:-1, 2:-1]
    assert R.int8_dequantize(t, TD[dtype], out=view) is view
    assert np.array_equal(_np(view), want)
    big[1:-1, 2:-1] = 7.0
    assert (big == 7.0).all()


# ----------------------------------------------------------------------------- products
SIZES = [(1, 1, 1), (1, 64, 33), (2, 300, 17), (4, 4096, 100), (16, 1024, 64), (17, 257, 100), (33, 96, 250), (64, 512, 256),
         (65, 512, 256), (130, 1000, 301), (256, 256, 512), (300, 2048, 130), (512, 768, 640), (70, 33000, 90), (1, 33000, 130),
         (3, 12288, 40), (1000, 130, 1500), (260, 8192, 260)]


def _product(a, b):
    """(float64 product of the 8-bit values, the size that rounding errors are relative to)."""
    (ca, sa), (cb, sb) = X.quantize(a), X.quantize(b)
    y = (ca.astype(np.float64) @ cb.astype(np.float64).T) * (sa.astype(np.float64)[:, None] * sb.astype(np.float64))
    return y


def _bound(y, plain, dtype):
    return 2.0**-23 * 1.001 * np.abs(plain) + (2.0**-24 + STEP[dtype]) * 1.001 * np.abs(y) + 2 * TINY[dtype]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_matmul(dtype, M, K, N):
    rng = np.random.default_rng(M + K + N)
    a, b = _gpu(rng.standard_normal((M, K)), dtype), _gpu(rng.standard_normal((N, K)) / 8, dtype)
    bias = _gpu(rng.standard_normal(N), dtype)
    ref = _product(_np(a), _np(b))
    aq, bq = R.int8_quantize(a), R.int8_quantize(b)
    y = R.int8_matmul(a, bq)
    assert y.dtype == TD[dtype] and y.shape == (M, N)
    assert (np.abs(_np(y) - ref) <= _bound(ref, ref, dtype)).all()
    yb = R.int8_matmul(aq, bq, bias=bias, dtype=TD[dtype])
    refb = ref + _np(bias)
    assert (np.abs(_np(yb) - refb) <= _bound(refb, ref, dtype)).all()
    # quantised inside the product or before it: the same
    assert torch.equal(R.int8_matmul(aq, bq, dtype=TD[dtype]), y)
    assert torch.equal(R.int8_matmul(a, bq, bias=bias), yb)
    # another output type than the matrix's
    other = "f32" if dtype != "f32" else "bf16"
    assert (np.abs(_np(R.int8_matmul(a, bq, dtype=TD[other])) - ref) <= _bound(ref, ref, other)).all()


def _near(got, ref, bound, dtype):
    """got is ref within bound, or the infinity that ref rounds to past the type's range (from half a step above its largest)."""
    most = torch.finfo(TD[dtype]).max
    over = np.isinf(got) & (np.sign(got) == np.sign(ref)) & (np.abs(ref) + bound >= most * (1 + STEP[dtype] / 2))
    return (over | (np.abs(np.where(np.isinf(got), 0, got) - ref) <= bound)).all()


def _exact_sums(M, K, N, seed):
    """Whole numbers as they are (a 127 in every row makes the scale 1): float32 results with one value while the sums stay below
    2^24."""
    gen = torch.Generator().manual_seed(seed)
    a, b = (torch.randint(-3, 4, (n, K), generator=gen).float() for n in (M, N))
    a[:, 0] = 127
    b[:, -1] = -127
    return a.to(dev()), b.to(dev())


FORMS = [(1000, 130, 1500), (65, 128, 64), (129, 4096, 100), (2048, 256, 2048), (4096, 128, 4096), (4096, 1024, 2100), (1024, 16384, 1024),
         (300, 65536, 300), (3000, 640, 5000), (513, 8192, 700), (4000, 2048, 4090), (100, 2368, 3500),
         (128, 4465, 1205), (3, 12000, 5690), (355, 123, 3788), (600, 45000, 78), (1467, 3134, 583)]


@pytest.mark.parametrize("M,K,N", FORMS)
def test_matmul_exact(M, K, N):
    """Equal bits in every form: tiles of each shape, whole and shared out, ragged edges in both directions."""
    a, b = _exact_sums(M, K, N, M + K + N)
    ref = (a.double() @ b.double().t().contiguous()).float()
    assert ref.abs().max() < 2**24
    y = R.int8_matmul(R.int8_quantize(a), R.int8_quantize(b), dtype=torch.float32)
    assert torch.equal(y, ref)
    assert torch.equal(R.int8_matmul(a, R.int8_quantize(b)), ref)


def test_every_form_is_met():
    forms = {_form(M, N, K) for M, K, N in FORMS + SIZES}
    want = {(16, 16), (16, 32), (32, 32), (64, 32), (64, 64), (64, 128), (128, 128), (256, 256)}
    assert want == {f[:2] for f in forms}
    for shared in (False, True):
        assert {(64, 64), (64, 128), (128, 128)} <= {f[:2] for f in forms if (f[2] > 1) == shared}


@pytest.mark.parametrize("M,K,N", [(1024, 65536, 1024), (199, 53501, 4423), (700, 90001, 900)])
def test_matmul_exact_in_shares_of_the_largest_tiles(M, K, N):
    assert _form(M, N, K)[:2] == (256, 256) and _form(M, N, K)[2] > 1
    a, b = _exact_sums(M, K, N, M + K + N)
    ref = (a.double() @ b.double().t().contiguous()).float()
    assert ref.abs().max() < 2**24
    y = R.int8_matmul(R.int8_quantize(a), R.int8_quantize(b), dtype=torch.float32)
    assert torch.equal(y, ref)
    assert torch.equal(R.int8_matmul(a, R.int8_quantize(b)), ref)
    half = R.int8_matmul(R.int8_quantize(a), R.int8_quantize(b), bias=torch.ones(N, device=a.device, dtype=torch.bfloat16))
    assert torch.equal(half, (ref + 1).to(torch.bfloat16))


def test_sums_past_32_bits():
    """K past 2^17 with every product at 127^2: the sums leave int32, and are exact all the same."""
    K = 140001
    for M, N in ((2, 5), (70, 130)):
        a = torch.full((M, K), 127.0, device=dev())
        b = torch.full((N, K), -127.0, device=dev())
        b[:, 1::2] = 127.0
        b[1, :] = 127.0
        y = R.int8_matmul(R.int8_quantize(a), R.int8_quantize(b), dtype=torch.float32)
        want = torch.full((M, N), -127.0 * 127.0, device=dev())
        want[:, 1] = float(np.float32(127 * 127 * K))
        assert torch.equal(y, want)


def test_largest_sums_in_one_share():
    """2^17 products of 127^2 fill int32 to 1.5 %."""
    K = 1 << 17
    for M in (1, 64, 65, 300):
        a = torch.full((M, K), -127.0, device=dev())
        b = torch.full((80, K), 127.0, device=dev())
        y = R.int8_matmul(R.int8_quantize(a), R.int8_quantize(b), dtype=torch.float32)
        assert (y == float(np.float32(-127 * 127 * K))).all()


@pytest.mark.parametrize("M", [1, 3, 40, 200])
def test_far_scales(M):
    """Rows whose scales lie at the ends of the range: an infinite product of scales makes no NaN of a zero sum, a vanished one no
    zero of a value that the type holds, and rows of zeros stay zeros."""
    K, N = 256, 70
    a, b = np.zeros((M, K)), np.zeros((N, K))
    a[:, :128] = np.random.default_rng(M).integers(-127, 128, (M, 128))
    a[:, 0] = 127
    a *= 2.0 ** np.linspace(-130, 120, M)[:, None] if M > 1 else 2.0**100
    b[:, 64:] = np.random.default_rng(M + 1).integers(-127, 128, (N, 192))
    b[::2, :128] = 0  # these meet a in zeros only
    b[:, 200] = 127
    b *= 2.0 ** np.linspace(-120, 120, N)[:, None]
    b[5] = 0
    a, b = _gpu(a, "f32"), _gpu(b, "f32")
    ref = _product(_np(a), _np(b))
    y = _np(R.int8_matmul(a, R.int8_quantize(b)))
    big = np.abs(ref) >= 2.0**128
    assert (ref[:, ::2] == 0).all() and (y[:, ::2] == 0).all() and big.any()
    assert np.isinf(y[np.abs(ref) > 2.0**128 * 1.001]).all()
    ok = np.abs(ref) < 2.0**127
    assert (np.abs(y - ref)[ok] <= _bound(ref, ref, "f32")[ok]).all()


def test_out_and_strides():
    rng = np.random.default_rng(3)
    big = _gpu(rng.standard_normal((150, 400)), "bf16")
    w = R.int8_quantize(_gpu(rng.standard_normal((90, 130)), "bf16"))
    for x in (big[3:100, 5:135], big[:130, :77].t(), big[::3, 1::3][:, :130], big[4:5, :130].expand(33, 130), big[9:10, 7:137]):
        want = R.int8_matmul(x.contiguous(), w)
        assert torch.equal(R.int8_matmul(x, w), want)
        room = torch.full((x.shape[0] + 2, 100), 7.0, dtype=torch.bfloat16, device=x.device)
        view = room[1:-1, 4:94]
        assert R.int8_matmul(x, w, out=view) is view and torch.equal(view, want)
        view.fill_(7.0)
        assert (room == 7.0).all()
    with pytest.raises(ValueError, match="overlap"):
        R.int8_matmul(big[:90, :130], w, out=big[:90, :90])


@pytest.mark.parametrize("K,N", [(40, 300), (1500, 2000), (12000, 130), (140_000, 65)])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_an_output_depends_on_its_own_rows_alone(dtype, K, N):
    """The same bits from whatever form the numbers of rows and columns lead to."""
    rng = np.random.default_rng(K)
    a, w, bias = _gpu(rng.standard_normal((1500, K)), dtype), _gpu(rng.standard_normal((K, N)), dtype), _gpu(rng.standard_normal(N), dtype)
    a[3] *= 2.0**-24  # f32: a scale far below the others
    b = R.int8_quantize(w, axis=0)
    y = R.int8_matmul(a, b, bias=bias)
    forms = {_form(1500, N, K)}
    for M in (1, 3, 17, 64, 200, 700):
        forms.add(_form(M, N, K))
        assert torch.equal(R.int8_matmul(a[:M], b, bias=bias), y[:M])
        assert torch.equal(R.int8_matmul(R.int8_quantize(a[:M]), b, bias=bias, dtype=a.dtype), y[:M])
    c = R.int8_quantize(w[:, :33], axis=0)
    assert torch.equal(R.int8_matmul(a, c, bias=bias[:33]), y[:, :33])
    assert len(forms) > 2


# ----------------------------------------------------------------------------- backward
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (3, 70, 33), (100, 96, 130), (515, 333, 144), (64, 2731, 100), (2000, 65, 70), (300, 512, 4000), (300, 5000, 64), (4200, 4100, 20),
                                   (100, 9000, 30)])
def test_backward(dtype, M, N, K):
    rng = np.random.default_rng(M + N + K)
    dy, x, w = (_gpu(_wide(rng, *shape), dtype) for shape in ((M, N), (M, K), (K, N)))
    wr, xc = R.int8_quantize(w, axis=1), R.int8_quantize(x, axis=0)
    dx, dw, db = R.int8_backward(dy, wr, xc, bias=True)
    ndy, nx, nw = _np(dy), _np(x), _np(w)
    for got, ref in ((dx, _product(ndy, nw)), (dw, _product(nx.T, ndy.T))):
        assert got.dtype == TD[dtype] and _near(_np(got), ref, _bound(ref, ref, dtype), dtype)
    ref = ndy.sum(0)
    # at most M - 1 float32 additions, each off by half a step of a partial sum
    bound = M * 2.0**-24 * np.abs(ndy).sum(0) + STEP[dtype] * 1.01 * np.abs(ref) + TINY[dtype]
    assert _near(_np(db), ref, bound, dtype)
    # the same as the calls that it stands for
    r, c = R.int8_quantize(dy, axis=None)
    assert torch.equal(dx, R.int8_matmul(r, wr, dtype=TD[dtype])) and torch.equal(dw, R.int8_matmul(xc, c, dtype=TD[dtype]))
    two = R.int8_backward(dy, wr, xc)
    assert len(two) == 2 and torch.equal(two[0], dx) and torch.equal(two[1], dw)
    f = R.int8_backward(dy, wr, xc, bias=True, dtype=torch.float32)
    assert all(t.dtype == torch.float32 for t in f)
    # rows apart
    room = torch.zeros(M, N + 5, dtype=TD[dtype], device=dy.device)
    room[:, 2: N + 2] = dy
    assert all(torch.equal(p, q) for p, q in zip(R.int8_backward(room[:, 2: N + 2], wr, xc, bias=True), (dx, dw, db)))


@pytest.mark.parametrize("M,N,c", [(1 << 25, 8, 1 + 2.0**-10 - 2.0**-23), (1 << 25, 4, 1 + 2.0**-10 - 2.0**-23), (1 << 23, 600, 1 + 2.0**-12 - 2.0**-23),
                                   (1 << 22, 2, 1 + 2.0**-14 - 2.0**-23)])
def test_sums_over_many_rows(M, N, c):
    """dy = c: a running sum of some thousand c rounds every addition to the same side. No sum goes through more than 1030 float32
    additions, and the result is rounded once."""
    dy = torch.full((M, N), c, device=dev())
    w, xc = R.int8_quantize(torch.ones(1, N, device=dev())), R.int8_quantize(torch.ones(1, M, device=dev()))
    want = M * float(dy[0, 0])
    db = R.int8_backward(dy, w, xc, bias=True)[2]
    assert bool(((db.double() - want).abs() <= 1031 * 2.0**-24 * want).all())


def test_backward_of_more_rows_than_a_launch_sums():
    """270000 rows of 8200 are read in two launches, whose codes, scales and maxima make one tensor of each direction."""
    M, N, K = 270_000, 8200, 3
    gen = torch.Generator(device=dev())
    gen.manual_seed(80)
    dy = torch.randn(M, N, generator=gen, device=dev(), dtype=torch.bfloat16)
    wr, xc = (R.int8_quantize(torch.randn(K, n, generator=gen, device=dev())) for n in (N, M))
    dx, dw, db = R.int8_backward(dy, wr, xc, bias=True)
    assert torch.equal(dx, R.int8_matmul(R.int8_quantize(dy), wr)) and torch.equal(dw, R.int8_matmul(xc, R.int8_quantize(dy, axis=0)))
    want, size = (sum(f(dy[k: k + 30_000].double()).sum(0) for k in range(0, M, 30_000)) for f in (lambda t: t, torch.abs))
    assert bool(((db.double() - want).abs() <= 1031 * 2.0**-24 * size + STEP["bf16"] * 1.01 * want.abs()).all())


BACKWARD_SIZES = {(512, 512, 2048): (64, 64), (700, 700, 1100): (64, 64), (10, 300, 500): (64, 64), (2000, 500, 4000): (64, 128),
                  (515, 1440, 2731): (64, 128), (800, 800, 8000): (64, 128), (3000, 1000, 5000): (128, 128), (1024, 4096, 1024): (128, 128),
                  (2048, 4096, 4096): (256, 256), (4096, 2000, 8190): (256, 256), (16, 4096, 12288): (0, 0), (1000, 100, 12000): (0, 0)}  # M, K, N: the tiles that both products share


@pytest.mark.parametrize("M,K,N", list(BACKWARD_SIZES))
def test_both_products_in_one_launch(M, K, N):
    """Bit for bit those of two calls, in every form; values beside a float64 product of the same codes."""
    got = (ctypes.c_int * 2)()
    assert _lib.load().svdq_i8_backward_form(M, N, K, got) == 0
    assert tuple(got) == BACKWARD_SIZES[(M, K, N)]
    rng = np.random.default_rng(M + K)
    dy, x, w = (_gpu(rng.standard_normal(shape), "bf16") for shape in ((M, N), (M, K), (K, N)))
    dy[:, 7] *= 2.0**-100  # a column of dw whose scales are far from 1
    wr, xc = R.int8_quantize(w, axis=1), R.int8_quantize(x, axis=0)
    r, c = R.int8_quantize(dy, axis=None)
    for dtype in (torch.bfloat16, torch.float32, torch.float16):
        dx, dw = R.int8_backward(dy, wr, xc, dtype=dtype)
        assert torch.equal(dx, R.int8_matmul(r, wr, dtype=dtype)) and torch.equal(dw, R.int8_matmul(xc, c, dtype=dtype))
        if dtype == torch.float32:
            for y, a, b in ((dx, r, wr), (dw, xc, c)):
                rows, cols = slice(y.shape[0] - 70, None), slice(y.shape[1] - 70, None)
                ref = _np(R.int8_dequantize(a, torch.float32)[rows]) @ _np(R.int8_dequantize(b, torch.float32)[cols]).T
                mass = np.abs(_np(R.int8_dequantize(a, torch.float32)[rows])) @ np.abs(_np(R.int8_dequantize(b, torch.float32)[cols])).T
                assert (np.abs(_np(y[rows, cols]) - ref) <= 5.1 * 2.0**-24 * mass).all()  # three roundings, and two of the values'


# ----------------------------------------------------------------------------- far offsets
def test_offsets_past_32_bits():
    """A tensor of 4.6 GB of codes from whole numbers that are their own codes along either axis (a largest of 127 in every row and column):
    values back, products with its first and last rows on either side, and an output past 2^31 elements. The sums stay below 2^24, so that
    float32 holds them all and a product in any order."""
    rows, cols = 140_000, 32_768
    gen = torch.Generator(device=dev())
    gen.manual_seed(78)
    small = lambda *size: torch.randint(-3, 4, size, generator=gen, device=dev(), dtype=torch.int8).to(torch.bfloat16)  # noqa: E731
    x = small(rows, cols)
    x[:, ::1024] = 127
    x[::1024] = 127
    r, c = R.int8_quantize(x, axis=None)
    assert r.data.numel() > 2**32 and bool((r.scales == 1).all()) and bool((c.scales == 1).all())
    assert torch.equal(R.int8_dequantize(r), x)
    back = R.int8_dequantize(c)
    assert all(torch.equal(back[k:k + 4096], x[:, k:k + 4096].t()) for k in range(0, cols, 4096))
    del back, c
    ends = (slice(1, 300), slice(rows - 300, rows))
    for M in (1, 40, 200):
        a = small(M, cols)
        a[:, 5] = 127
        want = [a.float() @ x[part].float().t().contiguous() for part in ends]
        for left in (R.int8_quantize(a), a):
            y = R.int8_matmul(left, r, dtype=torch.bfloat16)
            assert all(torch.equal(y[:, part], w.to(torch.bfloat16)) for part, w in zip(ends, want))
        y = R.int8_matmul(r, R.int8_quantize(a), dtype=torch.float32)
        assert all(torch.equal(y[part], w.t()) for part, w in zip(ends, want))
    del y, r
    a, b = x[:, :128], small(16_384, 128)
    b[:, 7] = 127
    y = R.int8_matmul(a, R.int8_quantize(b))
    assert y.numel() > 2**31
    assert all(torch.equal(y[part], (a[part].float() @ b.float().t().contiguous()).to(torch.bfloat16)) for part in ends)


# ----------------------------------------------------------------------------- streams and graphs
def _calls():
    rng = np.random.default_rng(21)
    x = _gpu(rng.standard_normal((300, 500)), "bf16")
    w = _gpu(rng.standard_normal((500, 700)), "bf16")
    dy = _gpu(rng.standard_normal((300, 700)), "bf16")
    weight, bias = _gpu(1 + 0.1 * rng.standard_normal(500), "bf16"), _gpu(rng.standard_normal(500), "bf16")
    w_rows, w_cols = R.int8_quantize(w, axis=None)
    m_cols = R.mx_quantize(w, axis=0)

    def step():
        y, mean, rstd = R.layer_norm(x, weight, bias, save=True)
        y_rows, y_cols = R.int8_quantize(y, axis=None)
        z = R.int8_matmul(y_rows, w_cols)
        dh, dw, db = R.int8_backward(dy, w_rows, y_cols, bias=True)
        grads = R.layer_norm_backward(dh, x, mean, rstd, weight)
        served = R.int8_matmul(R.layer_norm(x[:2], weight, bias, quantize="int8"), w_cols)
        gated = R.mx_gated(R.layer_norm(x, weight, bias, quantize="mx"), m_cols)
        long = R.int8_matmul(dy.t()[:1], R.int8_quantize(x, axis=0))
        return [y, mean, rstd, R.int8_dequantize(y_cols), z, dh, dw, db, *grads, served, gated, long]

    return step


def test_training_step_and_serving_together_on_a_stream_and_in_a_graph():
    """A pre-norm layer's calls as a program makes them, with the same results alone, on another stream, and captured and replayed
    several times with eager work between."""
    step = _calls()
    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(4):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(step(), want))


def test_two_streams_and_two_graphs_at_once():
    """Calls that overlap in time share nothing: two streams without a wait between them, then two graphs replayed in turn."""
    steps = [_calls(), _calls()]
    want = [s() for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                got[k].append(steps[k]())
    torch.cuda.synchronize()
    for k in (0, 1):
        for out in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[k]))
    graphs, outs = [], []
    for k in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(steps[k]())
        graphs.append(g)
    for _ in range(3):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                graphs[k].replay()
        torch.cuda.synchronize()
        for k in (0, 1):
            assert all(torch.equal(a, b) for a, b in zip(outs[k], want[k]))


def test_calls_from_several_threads_at_once():
    """Host threads, each on a stream of its own, with sizes of their own, so that nothing that one thread's call planned serves another's."""
    def step(k):
        rng = np.random.default_rng(90 + k)
        x, w, dy = (_gpu(rng.standard_normal(s), "bf16") for s in ((200 + 61 * k, 700), (700, 500 + 40 * k), (200 + 61 * k, 500 + 40 * k)))
        g = _gpu(1 + 0.1 * rng.standard_normal(700), "f32")
        torch.cuda.synchronize()  # the inputs are made on the default stream

        def call():
            wr, wc = R.int8_quantize(w, axis=None)
            y, mean, rstd = R.layer_norm(x, g, save=True)
            xr, xc = R.int8_quantize(y, axis=None)
            z = R.int8_matmul(xr, wc)
            dh, dw, db = R.int8_backward(dy, wr, xc, bias=True)
            one = R.int8_matmul(R.layer_norm(x[:1 + k], g, quantize="int8"), wc)
            return [y, z, dh, dw, db, one, R.int8_matmul(x[:1 + k], wc), *R.layer_norm_backward(dh, x, mean, rstd, g)]

        return call

    steps = [step(k) for k in range(4)]
    want = [s() for s in steps]
    torch.cuda.synchronize()
    got, errors = [[] for _ in steps], []

    def go(k):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(10):
                    got[k].append(steps[k]())
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=go, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for k in range(4):
        assert len(got[k]) == 10 and all(torch.equal(a, b) for out in got[k] for a, b in zip(out, want[k]))


def test_calls_refuse_what_they_cannot_record():
    x = _gpu(np.ones((4, 64)), "f32").requires_grad_()
    w = R.int8_quantize(torch.ones(8, 64, device=x.device))
    for call in (lambda: R.int8_quantize(x), lambda: R.int8_matmul(x, w), lambda: R.int8_matmul(w, w, bias=x[0, :8], dtype=torch.float32)):
        with pytest.raises(RuntimeError, match="grad"):
            call()
    with torch.no_grad():
        assert (R.int8_matmul(x, w) == 64).all()


def test_refusals_of_the_binding():
    d = dev()
    x, w = torch.ones(4, 64, device=d), R.int8_quantize(torch.ones(8, 64, device=d))
    for bad in (torch.ones(4, 63, device=d), torch.ones(64, device=d), torch.ones(0, 64, device=d), torch.ones(4, 0, device=d)):
        with pytest.raises(ValueError):
            R.int8_matmul(bad, w)
    with pytest.raises(TypeError):
        R.int8_matmul(x.double(), w)
    with pytest.raises(TypeError):
        R.int8_matmul(x, R.mx_quantize(torch.ones(8, 64, device=d)))
    with pytest.raises(ValueError):
        R.int8_matmul(x, w, bias=torch.ones(7, device=d))
    with pytest.raises(ValueError):
        R.int8_matmul(x, w, bias=torch.ones(8, device=d, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        R.int8_matmul(x, w, out=torch.ones(4, 9, device=d))
    with pytest.raises(ValueError):
        R.int8_backward(torch.ones(4, 8, device=d), w, w)
    with pytest.raises(ValueError):
        R.int8_quantize(torch.ones(0, 4, device=d))
