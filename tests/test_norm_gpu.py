"""Layer norm and its backward pass on an MI355X against plain float64 implementations (oracle/int8.py).

Forward: y is float64's, rounded to float32 and then to its type. Float64 sums of K terms and one subtraction of squares leave an
error far below 2^-30 of (|xh| + 1) |weight| + |bias| at these sizes (K 2^-52 of the spread, times sqrt(K) where x[0] is the row's
far outlier); the two roundings are 2^-24 and half a step.

Backward: with the saved mean and rstd taken as they are, xh carries 2^-23, g 2^-24, a product of the two 2^-22; a mean of K terms adds
one half step of its partial sums for each addition in its longest chain (at most D below).
"""
import numpy as np
import pytest
import torch

import rank_bit_residual_amd as R
from oracle import int8 as X

pytestmark = pytest.mark.gpu

TD = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
STEP = {"f32": 2.0**-24, "bf16": 2.0**-8, "f16": 2.0**-11}  # half a step, relative
TINY = {"f32": 2.0**-149, "bf16": 2.0**-133, "f16": 2.0**-24}  # the smallest magnitude of the type
SIZES = [(1, 1), (1, 8), (3, 31), (5, 64), (200, 33), (7, 512), (6, 513), (1, 4096), (9, 2048), (6, 2500), (17, 4099), (33, 5003), (4, 8192),
         (5, 8200), (3, 16384), (3, 16390), (2, 40001)]


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _gpu(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, np.float64)).to(TD[dtype]).to(dev())


def _np(t):
    return t.detach().cpu().double().numpy()


def _inputs(rng, M, K, dtype, params):
    x = rng.standard_normal((M, K)) * 2.0 ** rng.integers(-4, 5, (M, 1)) + 3 * rng.standard_normal((M, 1))
    x[:, K // 2] *= 30
    w, b = 1 + 0.5 * rng.standard_normal(K), rng.standard_normal(K)
    pt = "f32" if params == "f32" else dtype
    return _gpu(x, dtype), _gpu(w, pt), _gpu(b, pt)


def _forward_bound(x, w, b, y, dtype):
    xh, _, _ = X.layer_norm(x)
    w = 1.0 if w is None else np.abs(w)
    b = 0.0 if b is None else np.abs(b)
    return 2.0**-30 * ((np.abs(xh) + 1) * w + b) + (2.0**-24 + STEP[dtype]) * 1.001 * np.abs(y) + 2 * TINY[dtype]


@pytest.mark.parametrize("params", ["same", "f32"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K", SIZES)
def test_layer_norm(M, K, dtype, params):
    x, w, b = _inputs(np.random.default_rng(M * 7 + K), M, K, dtype, params)
    for weight, bias in ((w, b), (w, None), (None, None)):
        nw, nb = (None if t is None else _np(t) for t in (weight, bias))
        ref, mean, rstd = X.layer_norm(_np(x), nw, nb)
        y, mu, rs = R.layer_norm(x, weight, bias, save=True)
        assert y.dtype == TD[dtype]
        assert (np.abs(_np(y) - ref) <= _forward_bound(_np(x), nw, nb, ref, dtype)).all()
        spread = np.sqrt(_np(x).var(1)) + 1e-30
        assert (np.abs(_np(mu) - mean) <= 2.0**-24 * 1.001 * np.abs(mean) + 2.0**-30 * spread).all()
        assert (np.abs(_np(rs) - rstd) <= (2.0**-24 + 2.0**-30) * rstd).all()
        assert torch.equal(R.layer_norm(x, weight, bias), y)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K", SIZES)
def test_quantised_norm_is_the_quantised_float32_norm(M, K, dtype):
    """The 8-bit and MXFP4 outputs are the tensors of the float32 result, bit for bit, in every path (a float32 copy of x and its
    parameters holds the same values)."""
    x, w, b = _inputs(np.random.default_rng(M * 5 + K), M, K, dtype, "same")
    y = R.layer_norm(x.float(), w.float(), b.float())
    for how, make, back in (("int8", R.int8_quantize, R.int8_dequantize), ("mx", R.mx_quantize, R.mx_dequantize)):
        t, mean, rstd = R.layer_norm(x, w, b, quantize=how, save=True)
        want = make(y)
        assert t.shape == (M, K)
        assert torch.equal(back(t, torch.float32), back(want, torch.float32))
        ones = R.int8_quantize(torch.ones(3, K, device=x.device)) if how == "int8" else R.mx_quantize(torch.ones(3, K, device=x.device))
        product = R.int8_matmul if how == "int8" else R.mx_matmul
        assert torch.equal(product(t, ones), product(want, ones))  # the padding along K is in place
        _, mu, rs = R.layer_norm(x, w, b, save=True)
        assert torch.equal(mean, mu) and torch.equal(rstd, rs)
    codes, past = X.unpack(R.layer_norm(x, w, b, quantize="int8").codes.cpu().numpy(), M, K)
    assert not past.any() and (np.abs(codes).max(1) == 127).sum() == (np.abs(_np(y)).max(1) > 0).sum()


@pytest.mark.parametrize("M,K,dtype", [(5001, 300, "bf16"), (4999, 1000, "f16"), (2501, 1500, "f32"), (1100, 4000, "bf16"), (2100, 5003, "f32"),
                                       (2100, 8190, "bf16"), (600, 8000, "f16"), (600, 9001, "bf16"), (700, 12288, "f32"), (300, 16384, "bf16"), (300, 16390, "f32"), (1100, 5, "bf16"),
                                       (2000, 8, "f32"), (40, 7, "f16")])
def test_many_rows(M, K, dtype):
    """More rows than the blocks of a launch, so that each takes several, and a last one that is not full; forward, quantised and backward."""
    rng = np.random.default_rng(M + K)
    x, w, b = _inputs(rng, M, K, dtype, "f32")
    nx, nw, nb = _np(x), _np(w), _np(b)
    ref, mean, rstd = X.layer_norm(nx, nw, nb)
    y, mu, rs = R.layer_norm(x, w, b, save=True)
    assert (np.abs(_np(y) - ref) <= _forward_bound(nx, nw, nb, ref, dtype)).all()
    assert (np.abs(_np(rs) - rstd) <= (2.0**-24 + 2.0**-30) * rstd).all()
    full = R.layer_norm(x.float(), w, b)
    for how, make, back in (("int8", R.int8_quantize, R.int8_dequantize), ("mx", R.mx_quantize, R.mx_dequantize)):
        assert torch.equal(back(R.layer_norm(x, w, b, quantize=how), torch.float32), back(make(full), torch.float32))
    dy = _gpu(rng.standard_normal((M, K)), dtype)
    got = R.layer_norm_backward(dy, x, mu, rs, w)
    refs = X.layer_norm_grad(_np(dy), nx, _np(mu), _np(rs), nw)
    for g, r, bound in zip(got, refs, _grad_bounds(_np(dy), nx, _np(mu), _np(rs), nw, refs, dtype, "f32")):
        assert (np.abs(_np(g) - r) <= bound).all()


@pytest.mark.parametrize("M,K,dtype", [(5200, 4500, "bf16"), (6100, 8190, "f16"), (3100, 5003, "bf16"), (8300, 4200, "f32")])
def test_many_rows_of_four_vectors_a_thread(M, K, dtype):
    """The form of many rows of 4096 to 8192 columns, of 16-bit values and of MXFP4 tensors."""
    test_many_rows(M, K, dtype)


def test_far_means_and_outliers():
    """Means 10^4 standard deviations off, a first element that is the row's outlier, constant rows, and the ends of the range."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((8, 3000))
    x[0] += 1e4
    x[1] = 1e4 + x[1] * 1e-2
    x[2, 0] = 1e6
    x[3] = 5.0
    x[4] = 0.0
    x[5] *= 1e-30
    x[6] *= 1e30
    x[7] = -3e38
    x = _gpu(x, "f32")
    ref, mean, rstd = X.layer_norm(_np(x))
    y, mu, rs = R.layer_norm(x, save=True)
    assert (np.abs(_np(y) - ref) <= 2.0**-30 * (np.abs(ref) + 1) + 2.0**-23 * np.abs(ref)).all()
    assert (np.abs(_np(mu) - mean) <= 2.0**-24 * 1.001 * np.abs(mean)+ 2.0**-30 * np.sqrt(_np(x).var(1))).all()
    assert (_np(y)[[3, 4, 7]] == 0).all()
    assert (R.int8_dequantize(R.layer_norm(x, quantize="int8"))[3] == 0).all()


@pytest.mark.parametrize("eps", [0.0, 1e-12, 1e-3, 1, 2.5])
def test_eps(eps):
    x = _gpu(np.random.default_rng(4).standard_normal((5, 300)) * 1e-2, "f32")
    ref = X.layer_norm(_np(x), eps=eps)[0]
    assert (np.abs(_np(R.layer_norm(x, eps=eps)) - ref) <= _forward_bound(_np(x), None, None, ref, "f32") + 2.0**-24 * np.abs(ref)).all()


@pytest.mark.parametrize("K", [40, 3000, 9000, 20000])
def test_infinities_and_nan_stay_in_their_rows(K):
    x = torch.randn(12, K, device=dev(), generator=torch.Generator(device="cuda").manual_seed(K))
    clean = R.layer_norm(x)
    x[2, K - 1], x[5, 0], x[7, K // 2] = float("inf"), float("nan"), float("-inf")
    good = [r for r in range(12) if r not in (2, 5, 7)]
    for y in (R.layer_norm(x), R.int8_dequantize(R.layer_norm(x, quantize="int8"), torch.float32),
              R.mx_dequantize(R.layer_norm(x, quantize="mx"), torch.float32)):
        assert y[[2, 5, 7]].isnan().all() and y[good].isfinite().all()
    assert torch.equal(R.layer_norm(x)[good], clean[good])
    y, mean, rstd = R.layer_norm(x, save=True)
    dy = torch.ones_like(x)
    dx, _, _ = R.layer_norm_backward(dy, x, mean, rstd)
    assert dx[[2, 5, 7]].isnan().all() and dx[good].isfinite().all()


def test_views_of_inputs_and_outputs():
    rng = np.random.default_rng(6)
    big = _gpu(rng.standard_normal((60, 700)), "bf16")
    w, b = _gpu(rng.standard_normal(2 * 300), "bf16")[::2], _gpu(rng.standard_normal(300), "bf16")
    dy = _gpu(rng.standard_normal((700, 60)), "bf16")
    for x, g in ((big[3:50, 7:307], dy[:300, 5:52].t()), (big[::2, ::2][:, :300], dy[50:350, ::2].t()),
                 (big[5:6, :300].expand(40, 300), dy[:300, 3:4].t().expand(40, 300)), (big[4:5, 11:311], dy[:300, :1].t())):
        plain = x.contiguous()
        want = R.layer_norm(plain, w.contiguous(), b, save=True)
        assert all(torch.equal(p, q) for p, q in zip(R.layer_norm(x, w, b, save=True), want))
        room = torch.full((x.shape[0] + 2, 310), 7.0, dtype=torch.bfloat16, device=x.device)
        view = room[1:-1, 3:303]
        assert R.layer_norm(x, w, b, out=view) is view and torch.equal(view, want[0])
        view.fill_(7.0)
        assert (room == 7.0).all()
        back = R.layer_norm_backward(g.contiguous(), plain, want[1], want[2], w.contiguous())
        assert all(torch.equal(p, q) for p, q in zip(R.layer_norm_backward(g, x, want[1], want[2], w), back))
    with pytest.raises(ValueError, match="overlap"):
        R.layer_norm(big, out=big)


# ----------------------------------------------------------------------------- backward
def _grad_bounds(dy, x, mean, rstd, w, refs, dtype, ptype):
    M, K = x.shape
    D = 64 + 8 * (K // 8192)  # additions in a row sum's longest chain
    u = 2.0**-24
    r = rstd[:, None]
    xh = np.abs((x - mean[:, None]) * r)
    g = np.abs(dy) * (1.0 if w is None else np.abs(w))
    gm, gx = g.mean(1, keepdims=True), (g * xh).mean(1, keepdims=True)
    dx = r * u * (8 * (g + gm + xh * gx) + D * (gm + xh * gx)) + STEP[dtype] * 1.01 * np.abs(refs[0]) + 2 * TINY[dtype]
    # M - 1 additions at most, and a product with two roundings in it
    dw = (M + 4) * u * (np.abs(dy) * xh).sum(0) + STEP[ptype] * 1.01 * np.abs(refs[1]) + 2 * TINY[ptype]
    db = M * u * np.abs(dy).sum(0) + STEP[ptype] * 1.01 * np.abs(refs[2]) + 2 * TINY[ptype]
    return dx, dw, db


@pytest.mark.parametrize("params", ["same", "f32"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K", SIZES + [(600, 100), (70, 600), (2100, 65), (130, 3000), (1500, 513), (40, 12000), (300, 9001), (300, 13001), (70, 17000)])
def test_layer_norm_backward(M, K, dtype, params):
    rng = np.random.default_rng(M * 3 + K)
    x, w, _ = _inputs(rng, M, K, dtype, params)
    dy = _gpu(rng.standard_normal((M, K)), dtype)
    _, mean, rstd = R.layer_norm(x, save=True)
    ptype = "f32" if params == "f32" else dtype
    for weight in (w, None):
        got = R.layer_norm_backward(dy, x, mean, rstd, weight)
        nw = None if weight is None else _np(weight)
        refs = X.layer_norm_grad(_np(dy), _np(x), _np(mean), _np(rstd), nw)
        bounds = _grad_bounds(_np(dy), _np(x), _np(mean), _np(rstd), nw, refs, dtype, ptype)
        assert got[0].dtype == TD[dtype] and (got[1] is None) == (got[2] is None) == (weight is None)
        for g, ref, bound in zip(got, refs, bounds):
            if g is not None:
                assert (np.abs(_np(g) - ref) <= bound).all()
        assert all(a is b or torch.equal(a, b) for a, b in zip(R.layer_norm_backward(dy, x, mean, rstd, weight), got))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [3, 40, 512, 1001, 2731, 5003, 9001, 13001, 17003])
def test_backward_of_rows_whose_mean_times_rstd_is_infinite(K, dtype):
    """Constant rows far from zero: x - mean is 0 in them, and what lies past a row's end must not count as if it were x = 0."""
    rng = np.random.default_rng(K)
    x, w, _ = _inputs(rng, 9, K, dtype, "f32")
    x[2], x[7] = 2e36, -2e36
    dy = _gpu(rng.standard_normal((9, K)), dtype)
    _, mean, rstd = R.layer_norm(x, save=True)
    assert (mean.abs() * rstd)[[2, 7]].isinf().all()
    for weight in (w, None):
        got = R.layer_norm_backward(dy, x, mean, rstd, weight)
        nw = None if weight is None else _np(weight)
        refs = X.layer_norm_grad(_np(dy), _np(x), _np(mean), _np(rstd), nw)
        for g, ref, bound in zip(got, refs, _grad_bounds(_np(dy), _np(x), _np(mean), _np(rstd), nw, refs, dtype, "f32")):
            if g is not None:
                assert (np.abs(_np(g) - ref) <= bound).all()


@pytest.mark.parametrize("M,K,c", [(1 << 25, 8, 1 + 2.0**-11 - 2.0**-23), (7_000_000, 520, 1 + 2.0**-11 - 2.0**-23), (1 << 25, 4, 1 + 2.0**-9 - 2.0**-23),
                                   (1 << 20, 4100, 1 + 2.0**-12 - 2.0**-23), (3_000_001, 2, 1 + 2.0**-11 - 2.0**-23)])
def test_sums_over_many_rows(M, K, c):
    """dy = c and xh = 1: a running sum of some thousand c rounds every addition to the same side. No sum goes through more than 1030
    float32 additions, and the result is rounded once."""
    dy, x = torch.full((M, K), c, device=dev()), torch.ones(M, K, device=dev())
    rstd, w = torch.ones(M, device=dev()), torch.ones(K, device=dev())
    _, dw, db = R.layer_norm_backward(dy, x, torch.zeros_like(rstd), rstd, w)
    want = M * float(dy[0, 0])
    for g in (dw, db):
        assert bool(((g.double() - want).abs() <= 1032 * 2.0**-24 * want).all())


def test_backward_against_differences():
    """The loss sum(dy y) moves as the gradients say: central differences of the float64 oracle at the inputs of the call. Their error is
    h^2 / 6 of the third derivative (a few units here) plus 2^-52 / h of the loss's terms; the call adds float32 roundings."""
    rng = np.random.default_rng(9)
    M, K, h = 3, 40, 1e-4
    x, w, b, dy = (rng.standard_normal(s).astype(np.float32).astype(np.float64) for s in ((M, K), K, K, (M, K)))
    xt, wt, dyt = (_gpu(t, "f32") for t in (x, w, dy))
    _, mean, rstd = R.layer_norm(xt, wt, _gpu(b, "f32"), save=True)
    dx, dw, db = (_np(t) for t in R.layer_norm_backward(dyt, xt, mean, rstd, wt))
    loss = lambda x, w, b: (dy * X.layer_norm(x, w, b)[0]).sum()  # noqa: E731
    for k in range(0, K, 3):
        for m in range(M):
            step = np.zeros_like(x)
            step[m, k] = h
            assert abs((loss(x + step, w, b) - loss(x - step, w, b)) / (2 * h) - dx[m, k]) < 1e-5
        step = np.zeros(K)
        step[k] = h
        assert abs((loss(x, w + step, b) - loss(x, w - step, b)) / (2 * h) - dw[k]) < 1e-5
        assert abs((loss(x, w, b + step) - loss(x, w, b - step)) / (2 * h) - db[k]) < 1e-5


@pytest.mark.parametrize("M,K", [(280_000, 16_384), (140_000, 32_768), (5_000_000, 900)])
def test_offsets_past_32_bits(M, K):
    """More than 2^32 elements: every row's results are those of the row alone, to the last."""
    gen = torch.Generator(device=dev())
    gen.manual_seed(79)
    x = torch.randn(M, K, generator=gen, device=dev(), dtype=torch.bfloat16)
    w, b = (torch.randn(K, generator=gen, device=dev()) for _ in range(2))
    assert x.numel() > 2**32
    ends = (slice(0, 99), slice(M - 99, M))
    y, mean, rstd = R.layer_norm(x, w, b, save=True)
    for part in ends:
        assert all(torch.equal(p[part], q) for p, q in zip((y, mean, rstd), R.layer_norm(x[part], w, b, save=True)))
    del y
    for how, back in (("int8", R.int8_dequantize), ("mx", R.mx_dequantize)):
        t = back(R.layer_norm(x, w, b, quantize=how))
        assert all(torch.equal(t[part], back(R.layer_norm(x[part], w, b, quantize=how))) for part in ends)
        del t
    dx, dw, db = R.layer_norm_backward(x, x, mean, rstd, w)
    for part in ends:
        assert torch.equal(dx[part], R.layer_norm_backward(x[part], x[part], mean[part], rstd[part], w)[0])
    # sums over M rows: each row's part of dbias is of spread 1, float32 sums in parts of M / 256 rows or fewer
    want = sum(x[k:k + 20_000].double().sum(0) for k in range(0, M, 20_000))
    size = sum(x[k:k + 20_000].double().abs().sum(0) for k in range(0, M, 20_000))
    assert bool(((db.double() - want).abs() <= (M / 64 + 300) * 2.0**-24 * size).all())


@pytest.mark.parametrize("M,K", [(280_000, 16_384), (140_000, 32_768), (5_000_000, 900)])
def test_weight_gradients_past_32_bits(M, K):
    """More than 2^32 elements of dy and of another x: both sums over all rows, in float64 chunk by chunk beside them. No sum goes through more
    than 1030 float32 additions; a term of dweight has three roundings, the result one."""
    gen = torch.Generator(device=dev())
    gen.manual_seed(81)
    x, dy = (torch.randn(M, K, generator=gen, device=dev(), dtype=torch.bfloat16) for _ in range(2))
    mean, rstd = torch.randn(M, generator=gen, device=dev()), 1 + torch.rand(M, generator=gen, device=dev())
    dx, dw, db = R.layer_norm_backward(dy, x, mean, rstd, torch.ones(K, device=dev()))
    del dx
    assert x.numel() > 2**32
    want, size = torch.zeros(2, K, dtype=torch.float64, device=dev()), torch.zeros(2, K, dtype=torch.float64, device=dev())
    step = 2**28 // K
    for k in range(0, M, step):
        d = dy[k: k + step].double()
        for i, t in enumerate(((x[k: k + step].double() - mean[k: k + step, None]).mul_(rstd[k: k + step, None]).mul_(d), d)):
            want[i] += t.sum(0)
            size[i] += t.abs_().sum(0)
    for i, g in enumerate((dw, db)):
        assert bool(((g.double() - want[i]).abs() <= 1034 * 2.0**-24 * size[i]).all())


def test_refusals_of_the_binding():
    d = dev()
    x, w = torch.ones(4, 64, device=d), torch.ones(64, device=d)
    for bad in (dict(weight=w[:63]), dict(weight=w.half()), dict(bias=w), dict(weight=w, bias=w[1:]), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(quantize="fp8"), dict(quantize="int8", out=x), dict(out=torch.ones(4, 63, device=d))):
        with pytest.raises(ValueError):
            R.layer_norm(x, **bad)
    with pytest.raises(ValueError):
        R.layer_norm(x.bfloat16(), w, w.bfloat16())
    for bad in (dict(weight=3.0), dict(eps="a"), dict(eps=True)):
        with pytest.raises(TypeError):
            R.layer_norm(x, **bad)
    with pytest.raises(TypeError):
        R.layer_norm(x.double())
    m = torch.ones(4, device=d)
    for args in ((x[:3], x, m, m), (x, x, m[:3], m), (x, x, m, m.half()), (x.half(), x, m, m), (x, x, m, m, w[:3])):
        with pytest.raises(ValueError):
            R.layer_norm_backward(*args)
    with pytest.raises(TypeError):
        R.layer_norm_backward(x, x, None, m)
    g = torch.ones(4, 64, device=d, requires_grad=True)
    for call in (lambda: R.layer_norm(g), lambda: R.layer_norm_backward(g, x, m, m), lambda: R.layer_norm(x, g[0])):
        with pytest.raises(RuntimeError, match="grad"):
            call()
