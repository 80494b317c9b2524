"""Operators on MXFP4 tensors made on the device: their measured cases and their plain forms.

An MXFP4 tensor holds, for each run of 32 elements along the axis that a product sums over, one power of two
2^e (the smallest with max|x| <= 6 * 2^e) and 32 values of {0, 0.5, 1, 1.5, 2, 3, 4, 6} with a sign, rounded to
nearest, ties to the even code. Write Q(x) for the values that stand for x, quantised along its last axis.

  quantize   Q(x) and Q(x^T), from one pass over x
  linear     y = Q(x) Q(w^T)^T (+ b), w [k, n], quantised once and kept
  product    y = A B^T of two MXFP4 tensors
  gated      g = Q(x) Q(wg^T)^T, u = Q(x) Q(wu^T)^T, h = act(g) * u, with w = [wg | wu] of [k, 2 f]
  grad       [dg | du] = [dh * u * act'(g) | dh * act(g)], as Q of it and of its transpose
  backward   the same, then dx = Q([dg | du]) Q(w)^T and dw = Q(x^T) Q([dg | du]^T)^T
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
_MX = 17 / 32  # bytes for each element of an MXFP4 tensor: half a byte and a 32nd of its scale byte
_TANH = 2 * math.sqrt(2 / math.pi)


def listed():
    return [
        # one token's activations, on their way into a 4-bit layer: nothing but latency
        {"name": "quantize_token", "op": "quantize", "rows": 1, "cols": 4096, "dtype": "bf16", "axis": "rows"},
        # a float32 tensor of odd size, for both products of a training step
        {"name": "quantize_ragged", "op": "quantize", "rows": 777, "cols": 5003, "dtype": "f32", "axis": "both"},
        # a feed-forward weight (or a batch of its activations) before a training step
        {"name": "quantize_train", "op": "quantize", "rows": 8192, "cols": 12288, "dtype": "bf16", "axis": "both"},
        # a decode step of 16 sequences through a square 4-bit layer
        {"name": "linear_decode", "op": "linear", "m": 16, "k": 8192, "n": 8192, "dtype": "bf16", "bias": False},
        # a short prompt through a small layer of odd sizes, with a bias
        {"name": "linear_ragged", "op": "linear", "m": 333, "k": 1000, "n": 2501, "dtype": "f16", "bias": True},
        # a batch of 4096 tokens through an up-projection
        {"name": "linear_prefill", "op": "linear", "m": 4096, "k": 4096, "n": 12288, "dtype": "bf16", "bias": False},
        # a weight's gradient over many tokens: a long sum, few outputs, kept in float32
        {"name": "weight_grad", "op": "product", "m": 1024, "k": 65536, "n": 1024, "dtype": "f32"},
        # one token through the gated projections of a feed-forward block
        {"name": "gated_token", "op": "gated", "m": 1, "k": 4096, "f": 12288, "dtype": "bf16", "act": "silu", "save": False},
        # a training batch of odd sizes through a small gated block, pre-activations kept
        {"name": "gated_ragged", "op": "gated", "m": 515, "k": 1440, "f": 2731, "dtype": "f16", "act": "gelu_tanh", "save": True},
        # the forward pass of a training step, pre-activations kept for the backward pass
        {"name": "gated_train", "op": "gated", "m": 4096, "k": 4096, "f": 12288, "dtype": "bf16", "act": "silu", "save": True},
        # the gradients of a small block's pre-activations, ready for the products behind them
        {"name": "grad_ragged", "op": "grad", "m": 515, "f": 2731, "dtype": "f16", "act": "gelu_tanh"},
        # the backward pass of a training step
        {"name": "backward_train", "op": "backward", "m": 4096, "k": 4096, "f": 12288, "dtype": "bf16", "act": "silu"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "product", "gated", "grad", "backward"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": _log(rng, 32, 12288), "dtype": dtype, "axis": rng.choice(["rows", "cols", "both"])}
    if op == "linear":
        return {"op": op, "m": _log(rng, 1, 4096), "k": _log(rng, 64, 8192), "n": _log(rng, 16, 12288), "dtype": dtype, "bias": rng.random() < 0.5}
    if op == "product":
        return {"op": op, "m": _log(rng, 16, 4096), "k": _log(rng, 64, 65536), "n": _log(rng, 16, 4096), "dtype": dtype}
    act = rng.choice(["silu", "gelu_tanh"])
    if op == "gated":
        return {"op": op, "m": _log(rng, 1, 4096), "k": _log(rng, 64, 4096), "f": _log(rng, 16, 12288), "dtype": dtype, "act": act, "save": rng.random() < 0.5}
    if op == "grad":
        return {"op": op, "m": _log(rng, 1, 4096), "f": _log(rng, 16, 12288), "dtype": dtype, "act": act}
    return {"op": op, "m": _log(rng, 16, 4096), "k": _log(rng, 64, 4096), "f": _log(rng, 16, 12288), "dtype": dtype, "act": act}


# ------------------------------------------------------------------------------------------------ inputs
def _activations(gen, rows, cols, dtype):
    """Rows of unit scale with a few channels far above the others, as activations have them."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    loud = 1 + 15 * (torch.rand(cols, generator=gen, device="cuda") < 0.01).float()
    return (x * loud).to(_DT[dtype])


def _weight(gen, k, n, dtype):
    return (torch.randn(k, n, generator=gen, device="cuda") / math.sqrt(k)).to(_DT[dtype])


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt = case["op"], case["dtype"]
    if op == "quantize":
        return {"x": _activations(gen, case["rows"], case["cols"], dt)}
    if op == "linear":
        b = torch.randn(case["n"], generator=gen, device="cuda").to(_DT[dt]) if case["bias"] else None
        return {"x": _activations(gen, case["m"], case["k"], dt), "w": _weight(gen, case["k"], case["n"], dt), "b": b}
    if op == "product":
        return {"a": _activations(gen, case["m"], case["k"], "bf16"), "b": _activations(gen, case["n"], case["k"], "bf16")}
    if op == "gated":
        return {"x": _activations(gen, case["m"], case["k"], dt), "w": _weight(gen, case["k"], 2 * case["f"], dt)}
    got = {"dh": torch.randn(case["m"], case["f"], generator=gen, device="cuda").to(_DT[dt]),
           "gu": (1.5 * torch.randn(case["m"], 2 * case["f"], generator=gen, device="cuda")).to(_DT[dt])}
    if op == "backward":
        got["x"] = _activations(gen, case["m"], case["k"], dt)
        got["w"] = _weight(gen, case["k"], 2 * case["f"], dt)
    return got


def prepare(case, seed):
    """The inputs, and what a program has quantised before the call: the weights, and what an earlier step left.
    The plain forms keep the values of those in float32, the framework's calls keep its tensors."""
    state = dict(_inputs(case, seed), case=case)
    if own:
        import rank_bit_residual_amd as R

        rows = lambda t: R.mx_quantize(t, axis=1)  # noqa: E731
        cols = lambda t: R.mx_quantize(t, axis=0)  # noqa: E731
    else:
        rows = _values
        cols = lambda t: _values(t.t())  # noqa: E731
    op = case["op"]
    if op in ("linear", "gated"):
        state["w"] = cols(state["w"])
    elif op == "product":
        state["a"], state["b"] = rows(state["a"]), rows(state["b"])
    elif op == "backward":
        state["w"], state["x"] = rows(state["w"]), cols(state["x"])
    return state


# ------------------------------------------------------------------------------------------------ plain forms
def _pow2(e, dtype):
    """2^e of whole numbers e, from the bits of a float."""
    if dtype == torch.float64:
        return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)
    return ((e.to(torch.int32).clamp(-126, 127) + 127) << 23).view(torch.float32)


def _values(x):
    """Q(x) in float32 (computed in float64 where x is)."""
    n, k = x.shape
    x = x if x.dtype == torch.float64 else x.float()
    x = torch.nn.functional.pad(x, (0, -k % 32)).reshape(n, -1, 32)
    part, e = torch.frexp(x.abs().amax(-1, keepdim=True))
    e = e - 3 + (part > 0.75)
    z = x * _pow2(-e, x.dtype)
    size = z.abs()
    step = torch.where(size < 2, 0.5, torch.where(size < 4, 1.0, 2.0))
    z = torch.round(z / step) * step * _pow2(e, x.dtype)
    return z.reshape(n, -1)[:, :k].float()


def _act(name, g):
    """act(g) and act'(g); both activations are g times a sigmoid of some z(g)."""
    z = g if name == "silu" else _TANH * (g + 0.044715 * g * g * g)
    dz = 1.0 if name == "silu" else _TANH * (1 + 0.134145 * g * g)
    s = 1 / (1 + torch.exp(-z))
    return g * s, s * (1 + g * (1 - s) * dz)


def _plain(state):
    case = state["case"]
    op, dt = case["op"], _DT[case["dtype"]]
    if op == "quantize":
        x, axis = state["x"], case["axis"]
        return [_values(x).bfloat16() if axis != "cols" else None, _values(x.t()).bfloat16() if axis != "rows" else None]
    if op == "linear":
        y = torch.matmul(_values(state["x"]), state["w"].t())
        return (y if state["b"] is None else y + state["b"].float()).to(dt)
    if op == "product":
        return torch.matmul(state["a"], state["b"].t()).to(dt)
    f = case["f"]
    if op == "gated":
        gu = torch.matmul(_values(state["x"]), state["w"].t())
        h = (_act(case["act"], gu[:, :f])[0] * gu[:, f:]).to(dt)
        return [h, gu.to(dt)] if case["save"] else [h]
    # a code is decided by comparing with a border, so the values come in float64
    dh, g, u = state["dh"].double(), state["gu"][:, :f].double(), state["gu"][:, f:].double()
    a, da = _act(case["act"], g)
    d = torch.cat([dh * u * da, dh * a], 1)
    if op == "grad":
        return [_values(d).bfloat16(), _values(d.t()).bfloat16()]
    return [torch.matmul(_values(d), state["w"].t()).to(dt), torch.matmul(state["x"], _values(d.t()).t()).to(dt)]


# ------------------------------------------------------------------------------------------------ the framework's calls
def _own(state):
    import rank_bit_residual_amd as R

    case = state["case"]
    op, dt = case["op"], _DT[case["dtype"]]
    if op == "quantize":
        if case["axis"] == "both":
            rows, cols = R.mx_quantize(state["x"], axis=None)
            return [R.mx_dequantize(rows), R.mx_dequantize(cols)]
        if case["axis"] == "rows":
            return [R.mx_dequantize(R.mx_quantize(state["x"], axis=1)), None]
        return [None, R.mx_dequantize(R.mx_quantize(state["x"], axis=0))]
    if op == "linear":
        return R.mx_matmul(state["x"], state["w"], bias=state["b"])
    if op == "product":
        return R.mx_matmul(state["a"], state["b"], dtype=dt)
    if op == "gated":
        if case["save"]:
            return list(R.mx_gated(state["x"], state["w"], act=case["act"], save=True))
        return [R.mx_gated(state["x"], state["w"], act=case["act"])]
    if op == "grad":
        rows, cols = R.mx_gated_grad(state["dh"], state["gu"], act=case["act"])
        return [R.mx_dequantize(rows), R.mx_dequantize(cols)]
    return list(R.mx_gated_backward(state["dh"], state["gu"], state["w"], state["x"], act=case["act"]))


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------------ work
def work(case):
    op, s = case["op"], _SIZE[case["dtype"]]
    if op == "quantize":
        # x in, and bfloat16 values out for each direction
        n = case["rows"] * case["cols"]
        return {"bytes": n * (s + (4 if case["axis"] == "both" else 2)), "flops": 0}
    if op == "grad":
        n = case["m"] * case["f"]
        return {"bytes": n * (3 * s + 8), "flops": 0}
    m, k = case["m"], case["k"]
    if op == "linear":
        n = case["n"]
        return {"bytes": m * k * s + _MX * k * n + m * n * s + (n * s if case["bias"] else 0), "flops": 2 * m * k * n}
    if op == "product":
        n = case["n"]
        return {"bytes": _MX * k * (m + n) + m * n * s, "flops": 2 * m * k * n}
    f = case["f"]
    if op == "gated":
        return {"bytes": m * k * s + _MX * k * 2 * f + m * f * s * (3 if case["save"] else 1), "flops": 4 * m * k * f}
    return {"bytes": 3 * m * f * s + _MX * k * (2 * f + m) + m * k * s + 2 * k * f * s, "flops": 8 * m * k * f}


# ------------------------------------------------------------------------------------------------ the definition, in 64 bits
_BORDERS = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]  # between the sizes 0, 0.5, 1, 1.5, 2, 3, 4, 6
_STEPS = [0.5, 0.5, 0.5, 0.5, 1.0, 1.0, 2.0]


def _exact_q(x):
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


def _exact_act(name, g):
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    # (1 + tanh z) / 2 loses its digits where tanh nears -1; it is the sigmoid of 2 z
    c = math.sqrt(2 / math.pi)
    s = torch.sigmoid(2 * c * (g + 0.044715 * g**3))
    return g * s, s + 2 * g * s * (1 - s) * c * (1 + 3 * 0.044715 * g**2)


def exact(case, seed):
    v = {n: t.double() if isinstance(t, torch.Tensor) else t for n, t in _inputs(case, seed).items()}
    op = case["op"]
    if op == "quantize":
        return [_exact_q(v["x"]) if case["axis"] != "cols" else None, _exact_q(v["x"].t()) if case["axis"] != "rows" else None]
    if op == "linear":
        y = _exact_q(v["x"]) @ _exact_q(v["w"].t()).t().contiguous()
        return y if v["b"] is None else y + v["b"]
    if op == "product":
        return _exact_q(v["a"]) @ _exact_q(v["b"]).t().contiguous()
    f = case["f"]
    if op == "gated":
        x = _exact_q(v["x"])
        g, u = (x @ _exact_q(w.t()).t().contiguous() for w in (v["w"][:, :f], v["w"][:, f:]))
        h = _exact_act(case["act"], g)[0] * u
        return [h, torch.cat([g, u], 1)] if case["save"] else [h]
    g, u = v["gu"][:, :f], v["gu"][:, f:]
    a, da = _exact_act(case["act"], g)
    d = torch.cat([v["dh"] * u * da, v["dh"] * a], 1)
    rows, cols = _exact_q(d), _exact_q(d.t())
    if op == "grad":
        return [rows, cols]
    return [rows @ _exact_q(v["w"]).t().contiguous(), _exact_q(v["x"].t()) @ cols.t().contiguous()]
