"""Operators on 8-bit tensors with a scale for each row, and layer norm: their measured cases and their plain forms.

An 8-bit tensor holds, for each row of a matrix whose products sum along its rows, one float32 scale s, the
row's largest magnitude / 127, and whole numbers, the quotients x / s rounded to nearest, ties to even (s is
2^-126 at least; a row of zeros has only zeros). Write Q(x) for the values that stand for x. A token's row of
activations has a scale of its own, and so has a channel's row of a weight's transpose.

  quantize     Q(x), Q(x^T), or both
  linear       y = Q(x) Q(w^T)^T (+ b), w [k, n], quantised once and kept; with a norm, x is the layer norm of x
  linear_grad  dx = Q(dy) Q(w)^T, dw = Q(x^T) Q(dy^T)^T and db = the sum of dy's rows
  norm         y = (x - mean) / sqrt(variance + eps) * weight + bias of each row, as it is, as an 8-bit tensor or as
               an MXFP4 tensor (of y as float32); for training with the mean and 1 / sqrt(variance + eps)
  norm_grad    the gradients of x, weight and bias
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
_EPS = 1e-5


def listed():
    return [
        # a weight (or a batch of activations) of odd size, in float32, for both products of a training step
        {"name": "quantize_ragged", "op": "quantize", "rows": 777, "cols": 5003, "dtype": "f32", "axis": "both"},
        # a feed-forward weight (or a batch of its activations) before a training step
        {"name": "quantize_train", "op": "quantize", "rows": 8192, "cols": 12288, "dtype": "bf16", "axis": "both"},
        # one token through a square 8-bit layer: a decode step
        {"name": "linear_token", "op": "linear", "m": 1, "k": 8192, "n": 8192, "dtype": "bf16", "bias": False, "norm": False},
        # a short prompt through a small layer of odd sizes, with a bias
        {"name": "linear_ragged", "op": "linear", "m": 333, "k": 1000, "n": 2501, "dtype": "f16", "bias": True, "norm": False},
        # a batch of 4096 tokens through a pre-norm block's up-projection: the norm writes the product's operand
        {"name": "linear_prefill", "op": "linear", "m": 4096, "k": 4096, "n": 12288, "dtype": "bf16", "bias": True, "norm": True},
        # the backward pass of a small layer of odd sizes
        {"name": "linear_grad_ragged", "op": "linear_grad", "m": 515, "k": 1440, "n": 2731, "dtype": "f16", "bias": True},
        # the backward pass of a training step's up-projection
        {"name": "linear_grad_train", "op": "linear_grad", "m": 4096, "k": 4096, "n": 12288, "dtype": "bf16", "bias": True},
        # one token's activations before an 8-bit layer: nothing but latency
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "params": "same", "to": "int8", "save": False},
        # a prompt of odd sizes, in float32, before an MXFP4 layer
        {"name": "norm_ragged", "op": "norm", "rows": 777, "cols": 5003, "dtype": "f32", "params": "same", "to": "mx", "save": False},
        # the forward pass of a training step, with float32 parameters, statistics kept for the backward pass
        {"name": "norm_train", "op": "norm", "rows": 8192, "cols": 8192, "dtype": "bf16", "params": "f32", "to": "same", "save": True},
        # the backward pass of a small batch of odd sizes
        {"name": "norm_grad_ragged", "op": "norm_grad", "rows": 515, "cols": 2731, "dtype": "f16", "params": "same"},
        # the backward pass of a training step, with float32 parameters
        {"name": "norm_grad_train", "op": "norm_grad", "rows": 8192, "cols": 8192, "dtype": "bf16", "params": "f32"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear_grad", "norm", "norm_grad"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": _log(rng, 32, 12288), "dtype": dtype, "axis": rng.choice(["rows", "cols", "both"])}
    if op == "linear":
        return {"op": op, "m": _log(rng, 1, 4096), "k": _log(rng, 64, 8192), "n": _log(rng, 16, 12288), "dtype": dtype,
                "bias": rng.random() < 0.5, "norm": rng.random() < 0.5}
    if op == "linear_grad":
        return {"op": op, "m": _log(rng, 16, 4096), "k": _log(rng, 64, 4096), "n": _log(rng, 16, 12288), "dtype": dtype, "bias": rng.random() < 0.5}
    params = rng.choice(["same", "f32"])
    size = {"rows": _log(rng, 1, 8192), "cols": _log(rng, 32, 8192)}
    if op == "norm":
        return {"op": op, **size, "dtype": dtype, "params": params, "to": rng.choice(["same", "int8", "mx"]), "save": rng.random() < 0.5}
    return {"op": op, **size, "dtype": dtype, "params": params}


# ------------------------------------------------------------------------------------------------ inputs
def _activations(gen, rows, cols, dtype):
    """Rows of unit scale with a few channels far above the others and a shift of their own, as activations have them."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    loud = 1 + 15 * (torch.rand(cols, generator=gen, device="cuda") < 0.01).float()
    return (x * loud + 0.5 * torch.randn(rows, 1, generator=gen, device="cuda")).to(_DT[dtype])


def _weight(gen, k, n, dtype):
    return (torch.randn(k, n, generator=gen, device="cuda") / math.sqrt(k)).to(_DT[dtype])


def _vector(gen, n, middle, spread, dtype):
    return (middle + spread * torch.randn(n, generator=gen, device="cuda")).to(dtype)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt = case["op"], case["dtype"]
    if op == "quantize":
        return {"x": _activations(gen, case["rows"], case["cols"], dt)}
    if op in ("linear", "linear_grad"):
        got = {"x": _activations(gen, case["m"], case["k"], dt), "w": _weight(gen, case["k"], case["n"], dt), "b": None}
        if op == "linear_grad":
            got["dy"] = torch.randn(case["m"], case["n"], generator=gen, device="cuda").to(_DT[dt])
            return got
        if case["bias"]:
            got["b"] = _vector(gen, case["n"], 0.0, 1.0, _DT[dt])
        if case["norm"]:
            got["weight"] = _vector(gen, case["k"], 1.0, 0.1, _DT[dt])
            got["bias"] = _vector(gen, case["k"], 0.0, 0.1, _DT[dt])
        return got
    pt = torch.float32 if case["params"] == "f32" else _DT[dt]
    got = {"x": _activations(gen, case["rows"], case["cols"], dt), "weight": _vector(gen, case["cols"], 1.0, 0.1, pt)}
    if op == "norm":
        got["bias"] = _vector(gen, case["cols"], 0.0, 0.1, pt)
    else:
        got["dy"] = torch.randn(case["rows"], case["cols"], generator=gen, device="cuda").to(_DT[dt])
    return got


def prepare(case, seed):
    """The inputs, and what a program has made before the call: the weights' 8-bit tensors and what a forward pass left.
    The plain forms keep the values of those tensors in float32, the framework's calls keep its tensors."""
    state = dict(_inputs(case, seed), case=case)
    op = case["op"]
    if own:
        import rank_bit_residual_amd as R

        rows = lambda t: R.int8_quantize(t, axis=1)  # noqa: E731
        cols = lambda t: R.int8_quantize(t, axis=0)  # noqa: E731
    else:
        rows = _values
        cols = lambda t: _values(t.t())  # noqa: E731
    if op == "linear":
        state["w"] = cols(state["w"])
    elif op == "linear_grad":
        state["w"], state["x"] = rows(state["w"]), cols(state["x"])
    elif op == "norm_grad":
        x = state["x"].double()
        mean = x.mean(1)
        state["mean"], state["rstd"] = mean.float(), (1 / torch.sqrt((x - mean[:, None]).square().mean(1) + _EPS)).float()
    return state


# ------------------------------------------------------------------------------------------------ plain forms
def _values(x):
    """Q(x) in float32. A code is decided by comparing with a border, so the quotients are taken in float64."""
    x = x.double()
    s = (x.abs().amax(1, keepdim=True) / 127).float().clamp_min(2.0**-126)
    return torch.round(x / s.double()).float() * s


def _mx_values(y):
    """The MXFP4 values of y (float32): blocks of 32 along the rows, a power of two and the sizes 0 .. 6 for each."""
    n, k = y.shape
    y = torch.nn.functional.pad(y, (0, -k % 32)).reshape(n, -1, 32)
    part, e = torch.frexp(y.abs().amax(-1, keepdim=True))
    e = (e - 3 + (part > 0.75)).clamp(-126, 127)
    up, down = (((v.to(torch.int32) + 127) << 23).view(torch.float32) for v in (e, -e))
    z = y * down
    size = z.abs()
    step = torch.where(size < 2, 0.5, torch.where(size < 4, 1.0, 2.0))
    return (torch.round(z / step) * step * up).reshape(n, -1)[:, :k]


def _norm(x, weight, bias, dtype):
    """(y, mean, 1 / sqrt(variance + eps)) in `dtype`."""
    x = x.to(dtype)
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + _EPS)
    return d * rstd * weight.to(dtype) + bias.to(dtype), mean[:, 0], rstd[:, 0]


def _plain(state):
    case = state["case"]
    op, dt = case["op"], _DT[case["dtype"]]
    if op == "quantize":
        x, axis = state["x"], case["axis"]
        return [_values(x).bfloat16() if axis != "cols" else None, _values(x.t()).bfloat16() if axis != "rows" else None]
    if op == "linear":
        x = state["x"]
        if case["norm"]:
            x = _norm(x, state["weight"], state["bias"], torch.float64)[0].float()
        y = torch.matmul(_values(x), state["w"].t())
        return (y if state["b"] is None else y + state["b"].float()).to(dt)
    if op == "linear_grad":
        dy = state["dy"]
        dx = torch.matmul(_values(dy), state["w"].t()).to(dt)
        dw = torch.matmul(state["x"], _values(dy.t()).t()).to(dt)
        return [dx, dw, dy.float().sum(0).to(dt)] if case["bias"] else [dx, dw]
    if op == "norm":
        to = case["to"]
        # a code is decided by comparing with a border, so the values come from float64
        y, mean, rstd = _norm(state["x"], state["weight"], state["bias"], torch.float32 if to == "same" else torch.float64)
        y = y.float()
        got = [y.to(dt) if to == "same" else (_values(y) if to == "int8" else _mx_values(y)).bfloat16()]
        return got + [mean.float(), rstd.float()] if case["save"] else got
    x, dy, w = state["x"].float(), state["dy"].float(), state["weight"].float()
    rstd = state["rstd"][:, None]
    xh = (x - state["mean"][:, None]) * rstd
    g = dy * w
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    pt = state["weight"].dtype
    return [dx.to(dt), (dy * xh).sum(0).to(pt), dy.sum(0).to(pt)]


# ------------------------------------------------------------------------------------------------ the framework's calls
def _own(state):
    import rank_bit_residual_amd as R

    case = state["case"]
    op = case["op"]
    if op == "quantize":
        if case["axis"] == "both":
            rows, cols = R.int8_quantize(state["x"], axis=None)
            return [R.int8_dequantize(rows), R.int8_dequantize(cols)]
        if case["axis"] == "rows":
            return [R.int8_dequantize(R.int8_quantize(state["x"], axis=1)), None]
        return [None, R.int8_dequantize(R.int8_quantize(state["x"], axis=0))]
    if op == "linear":
        x = state["x"]
        if case["norm"]:
            x = R.layer_norm(x, state["weight"], state["bias"], eps=_EPS, quantize="int8")
        return R.int8_matmul(x, state["w"], bias=state["b"], dtype=_DT[case["dtype"]])
    if op == "linear_grad":
        return list(R.int8_backward(state["dy"], state["w"], state["x"], bias=case["bias"]))
    if op == "norm":
        to = None if case["to"] == "same" else case["to"]
        got = R.layer_norm(state["x"], state["weight"], state["bias"], eps=_EPS, quantize=to, save=case["save"])
        got = list(got) if case["save"] else [got]
        if to is not None:
            got[0] = (R.int8_dequantize if to == "int8" else R.mx_dequantize)(got[0])
        return got
    return list(R.layer_norm_backward(state["dy"], state["x"], state["mean"], state["rstd"], state["weight"]))


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------------ work
def work(case):
    op, s = case["op"], _SIZE[case["dtype"]]
    if op == "quantize":
        # x in, and bfloat16 values out for each direction
        n = case["rows"] * case["cols"]
        return {"bytes": n * (s + (4 if case["axis"] == "both" else 2)), "flops": 0}
    if op in ("linear", "linear_grad"):
        m, k, n = case["m"], case["k"], case["n"]
        if op == "linear":
            more = (n * s if case["bias"] else 0) + (2 * k * s if case["norm"] else 0)
            return {"bytes": m * k * s + k * n + 4 * n + m * n * s + more, "flops": 2 * m * k * n}
        return {"bytes": m * n * s + (m + n) * k + 8 * k + m * k * s + k * n * s + (n * s if case["bias"] else 0), "flops": 4 * m * k * n}
    m, k = case["rows"], case["cols"]
    p = 4 if case["params"] == "f32" else s
    if op == "norm":
        out = s if case["to"] == "same" else 2
        return {"bytes": m * k * (s + out) + 2 * k * p + (8 * m if case["save"] else 0), "flops": 8 * m * k}
    return {"bytes": 3 * m * k * s + 3 * k * p + 8 * m, "flops": 14 * m * k}


# ------------------------------------------------------------------------------------------------ the definition, in 64 bits
def _exact_q8(x):
    most = x.abs().max(-1, keepdim=True).values
    s = torch.maximum((most / 127).float(), torch.tensor(2.0**-126, device=x.device)).double()
    size = x.abs() / s
    low = torch.floor(size)
    rest = size - low
    up = (rest > 0.5) | ((rest == 0.5) & (low % 2 == 1))  # a tie goes to the even number
    return (low + up) * torch.sign(x) * s


_BORDERS = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]  # between the sizes 0, 0.5, 1, 1.5, 2, 3, 4, 6
_STEPS = [0.5, 0.5, 0.5, 0.5, 1.0, 1.0, 2.0]


def _exact_q4(x):
    n, k = x.shape
    full = torch.zeros(n, -(-k // 32) * 32, dtype=torch.float64, device=x.device)
    full[:, :k] = x
    full = full.view(n, -1, 32)
    most = full.abs().max(-1, keepdim=True).values
    scale = torch.exp2(torch.ceil(torch.log2(most.clamp_min(2.0**-120) / 6)))
    scale = torch.where(most > 6 * scale, 2 * scale, scale)
    scale = torch.where(most <= 3 * scale, scale / 2, scale)
    size, got = full.abs() / scale, torch.zeros_like(full)
    for i, (border, step) in enumerate(zip(_BORDERS, _STEPS)):
        got += step * (size > border if i % 2 == 0 else size >= border)  # a tie goes to the even code
    return (got * torch.sign(full) * scale).reshape(n, -1)[:, :k]


def _exact_norm(x, weight, bias):
    k = x.shape[1]
    mean = x.sum(1) / k
    rstd = torch.rsqrt((x - mean[:, None]).pow(2).sum(1) / k + _EPS)
    return (x - mean[:, None]) * rstd[:, None] * weight + bias, mean, rstd


def exact(case, seed):
    v = {n: t.double() if isinstance(t, torch.Tensor) else t for n, t in _inputs(case, seed).items()}
    op = case["op"]
    if op == "quantize":
        return [_exact_q8(v["x"]) if case["axis"] != "cols" else None, _exact_q8(v["x"].t()) if case["axis"] != "rows" else None]
    if op == "linear":
        # what a norm leaves is quantised from float32
        x = _exact_norm(v["x"], v["weight"], v["bias"])[0].float().double() if case["norm"] else v["x"]
        y = _exact_q8(x) @ _exact_q8(v["w"].t()).t().contiguous()
        return y if v["b"] is None else y + v["b"]
    if op == "linear_grad":
        dx = _exact_q8(v["dy"]) @ _exact_q8(v["w"]).t().contiguous()
        dw = _exact_q8(v["x"].t()) @ _exact_q8(v["dy"].t()).t().contiguous()
        return [dx, dw, v["dy"].sum(0)] if case["bias"] else [dx, dw]
    if op == "norm":
        y, mean, rstd = _exact_norm(v["x"], v["weight"], v["bias"])
        if case["to"] != "same":
            y = (_exact_q8 if case["to"] == "int8" else _exact_q4)(y.float().double())
        return [y, mean, rstd] if case["save"] else [y]
    x, dy, w = v["x"], v["dy"], v["weight"]
    k = x.shape[1]
    xh, _, rstd = _exact_norm(x, torch.ones_like(w), torch.zeros_like(w))
    g = dy * w
    dx = g * rstd[:, None] - (g.sum(1) * rstd / k)[:, None] - xh * ((g * xh).sum(1) * rstd / k)[:, None]
    return [dx, (dy * xh).sum(0), dy.sum(0)]
