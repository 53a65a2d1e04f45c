"""Performance cases of the 8-bit integer operators: tokens quantised to int8 with one scale each,
the root-mean-square norm that adds the residual and quantises its output the same way, and the
product of such tokens with a layer held in int8 with one scale per output channel.

`run` computes a case in its plain form (elementary torch operations) or, where `own` is true, with
the calls of `post_weight_quantization_27_b200.gq`.  Shapes are those of the framework's layer sets
(GPT-2-small, a 2048-wide stack, 4096- and 8192-wide stacks) with token counts from one to a long
prompt.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}

# The most elements (quantisers), multiply-adds and output bytes (product) that a drawn case may
# have: those of the largest listed ones.
_MOST_QUANT = 16384 * 28672
_MOST_NORM = 32768 * 8192
_MOST_MM = 8192 * 8192 * 28672
_MOST_OUT = 8192 * 28672 * 2 * 2


def listed():
    return [
        # one token of a decode step, the input of an attention output projection
        dict(name="quant 1x4096 bf16", op="quant", n=1, d=4096, dt="bf16", col=False, sums=True),
        # a small calibration set of fp32 activations
        dict(name="quant 2560x768 f32", op="quant", n=2560, d=768, dt="f32", col=False, sums=True),
        # a long prompt at the input of a wide down projection, with per-channel smoothing factors
        dict(name="quant 16384x28672 bf16 col", op="quant", n=16384, d=28672, dt="bf16", col=True,
             sums=False),
        # one token of a decode step: norm before the attention of a 4096-wide block
        dict(name="norm 1x4096 bf16", op="norm", n=1, d=4096, dt="bf16", wdt="bf16", res=True,
             sums=False),
        # an odd number of fp16 tokens without a residual (a first block), fp32 norm weights
        dict(name="norm 2047x2048 f16", op="norm", n=2047, d=2048, dt="f16", wdt="f32", res=False,
             sums=True),
        # a long batch through an 8192-wide block
        dict(name="norm 32768x8192 bf16", op="norm", n=32768, d=8192, dt="bf16", wdt="bf16",
             res=True, sums=False),
        # one decode token through a small attention input projection with bias
        dict(name="mm 1x768x2304 bf16", op="mm", n=1, k=768, m=2304, dt="bf16", affine=False,
             bias=True, act="none", mul=False, res=False),
        # one decode token through a gate projection: the weights' bytes are all the time
        dict(name="mm 1x4096x11008 bf16", op="mm", n=1, k=4096, m=11008, dt="bf16", affine=False,
             bias=False, act="silu", mul=False, res=False),
        # a decode batch through an affine layer, added to the residual
        dict(name="mm 33x8192x8192 f16 affine", op="mm", n=33, k=8192, m=8192, dt="f16",
             affine=True, bias=False, act="none", mul=False, res=True),
        # logits of a ragged batch: an odd number of output channels, fp32 out
        dict(name="mm 251x768x50257 f32", op="mm", n=251, k=768, m=50257, dt="f32", affine=False,
             bias=False, act="none", mul=False, res=False),
        # a calibration-sized batch through the first half of a GELU MLP
        dict(name="mm 2560x2048x8192 bf16 gelu", op="mm", n=2560, k=2048, m=8192, dt="bf16",
             affine=False, bias=True, act="gelu", mul=False, res=False),
        # a long prompt through the gate projection of a wide gated MLP, times the up projection
        dict(name="mm 8192x8192x28672 bf16 gated", op="mm", n=8192, k=8192, m=28672, dt="bf16",
             affine=False, bias=False, act="silu", mul=True, res=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "norm", "mm", "mm"])
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "mm":
        while True:
            n, k, m = _log(rng, 1, 16384), 16 * _log(rng, 4, 1792), _log(rng, 1, 50257)
            mul, res = rng.random() < 0.25, rng.random() < 0.35
            if n * k * m <= _MOST_MM and n * m * _SIZE[dt] * (1 + mul + res) <= _MOST_OUT:
                break
        return dict(op=op, n=n, k=k, m=m, dt=dt, affine=rng.random() < 0.4,
                    bias=rng.random() < 0.4, act=rng.choice(["none", "none", "relu", "gelu", "silu"]),
                    mul=mul, res=res)
    most = _MOST_QUANT if op == "quant" else _MOST_NORM
    while True:
        n, d = _log(rng, 1, 65536), 16 * _log(rng, 2, 1792)
        if n * d * _SIZE[dt] <= most * 2:
            break
    if op == "quant":
        return dict(op=op, n=n, d=d, dt=dt, col=rng.random() < 0.5, sums=rng.random() < 0.5)
    return dict(op=op, n=n, d=d, dt=dt, wdt=rng.choice([dt, "f32"]), res=rng.random() < 0.6,
                sums=rng.random() < 0.5)


def _tokens(n, d, dt, g):
    """Activations: N(0,1) times a log-normal factor per channel, a few channels 20 times larger."""
    sigma = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
    sigma[torch.randint(d, (4,), generator=g, device="cuda")] *= 20.0
    return torch.randn(n, d, generator=g, device="cuda").mul_(sigma).to(dt)


def _codes(n, d, g):
    """Tokens already quantised: (int8 codes, fp32 scales, int32 sums)."""
    x = _tokens(n, d, torch.float32, g)
    s = x.abs().amax(1).div_(127.0)
    c = x.div_(s[:, None]).round_().clamp_(-127, 127).to(torch.int8)
    return c, s, c.sum(1, dtype=torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _DT[case["dt"]]
    if case["op"] == "mm":
        n, k, m = case["n"], case["k"], case["m"]
        w = torch.randn(m, k, generator=g, device="cuda").mul_(0.02)
        if case["affine"]:   # 8-bit codes 0 .. 255 held less 128, the zero-point likewise
            lo, hi = w.amin(1).clamp_(max=0.0), w.amax(1).clamp_(min=0.0)
            s = ((hi - lo) / 255.0).to(torch.float16)
            z = (-lo / s.float()).round().clamp_(0, 255)
            w = w.div_(s.float()[:, None]).round_().add_(z[:, None]).clamp_(0, 255).sub_(128.0)
            z = (z - 128.0).to(torch.int32)
        else:
            s, z = (w.abs().amax(1) / 127.0).to(torch.float16), None
            w = w.div_(s.float()[:, None]).round_().clamp_(-127, 127)
        layer = dict(codes=w.to(torch.int8), scales=s.view(m, 1), zpoint=z)
        c, xs, sums = _codes(n, k, g)
        bias = torch.randn(m, generator=g, device="cuda") if case["bias"] else None
        mul = torch.randn(n, m, generator=g, device="cuda").to(dt) if case["mul"] else None
        res = torch.randn(n, m, generator=g, device="cuda").to(dt) if case["res"] else None
        return dict(case=case, layer=layer, x=dict(codes=c, scales=xs, sums=sums), bias=bias,
                    mul=mul, res=res, y=torch.empty(n, m, dtype=dt, device="cuda"),
                    ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    n, d = case["n"], case["d"]
    out = dict(codes=torch.empty(n, d, dtype=torch.int8, device="cuda"),
               scales=torch.empty(n, device="cuda"),
               sums=torch.empty(n, dtype=torch.int32, device="cuda") if case["sums"] else None)
    st = dict(case=case, x=_tokens(n, d, dt, g), out=out)
    if case["op"] == "quant":
        st["col"] = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda")) if case["col"] else None
    else:
        st["w"] = (1.0 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(_DT[case["wdt"]])
        st["r"] = _tokens(n, d, dt, g) if case["res"] else None
        st["h"] = torch.empty(n, d, dtype=dt, device="cuda") if case["res"] else None
    return st


_EPS = 1e-5


def _quantise(v):
    """Codes of the rows of v (fp32) on a grid of 255 levels, and the grid's step.  The divisor is a
    tensor: a division by a Python number is done as a product with its reciprocal."""
    amax = v.abs().amax(1)
    s = amax / amax.new_full((1,), 127.0)
    s = torch.where(s == 0, torch.ones_like(s), s)
    return (v / s[:, None]).round_().clamp_(-127, 127).to(torch.int8), s


def _act(v, act):
    if act == "relu":
        return v.clamp_(min=0.0)
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        u = math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)
        return v / (1.0 + torch.exp(-2.0 * u))
    return v


def run(state):
    case = state["case"]
    if own:
        from post_weight_quantization_27_b200 import gq
        if case["op"] == "mm":
            return gq.w8a8_matmul(state["layer"], state["x"], bias=state["bias"], act=case["act"],
                                  mul=state["mul"], R=state["res"], Y=state["y"], ws=state["ws"])
        if case["op"] == "quant":
            return gq.quantize_tokens_int8(state["x"], col_mul=state["col"], out=state["out"])
        q = gq.rmsnorm_quantize_int8(state["x"], state["w"], eps=_EPS, R=state["r"], H=state["h"],
                                     out=state["out"])
        return dict(q, h=state["h"])
    if case["op"] == "mm":
        w, x = state["layer"], state["x"]
        c = w["codes"].float()
        if w["zpoint"] is not None:
            c = c.sub_(w["zpoint"].float()[:, None])
        y = (x["codes"].float() @ c.t()).mul_(w["scales"].float().view(1, -1)).mul_(x["scales"][:, None])
        if state["bias"] is not None:
            y = y.add_(state["bias"])
        y = _act(y, case["act"])
        if state["mul"] is not None:
            y = y.mul_(state["mul"].float())
        if state["res"] is not None:
            y = y.add_(state["res"].float())
        return y.to(state["y"].dtype)
    v, scale, h = state["x"].float(), 1.0, None
    if case["op"] == "quant":
        if state["col"] is not None:
            v = v.mul_(state["col"]) if case["dt"] != "f32" else v * state["col"]
    else:
        if state["r"] is not None:
            h = (v + state["r"].float()).to(state["x"].dtype)
            v = h.float()
        scale = torch.rsqrt(v.double().square().mean(1) + _EPS).float()
        v = v * state["w"].float()
    codes, s = _quantise(v)
    out = dict(codes=codes, scales=s * scale,
               sums=codes.sum(1, dtype=torch.int32) if case["sums"] else None)
    return out if case["op"] == "quant" else dict(out, h=h)


def work(case):
    if case["op"] == "mm":
        n, k, m, e = case["n"], case["k"], case["m"], _SIZE[case["dt"]]
        b = n * k + m * k + 4 * n + 2 * m + (4 * m + 4 * n if case["affine"] else 0)
        b += 4 * m if case["bias"] else 0
        b += n * m * e * (1 + case["mul"] + case["res"])
        return {"bytes": b, "flops": 2 * n * k * m}
    n, d, e = case["n"], case["d"], _SIZE[case["dt"]]
    b = n * d * (e + 1) + 4 * n + (4 * n if case["sums"] else 0)
    if case["op"] == "quant":
        return {"bytes": b + (4 * d if case["col"] else 0), "flops": 0}
    return {"bytes": b + (2 * n * d * e if case["res"] else 0) + d * _SIZE[case["wdt"]], "flops": 0}


def exact(case, seed):
    """The definitions in 64 bits, a block of rows at a time.  Codes and their sums have no such
    value: which code a value takes is decided in 32 bits."""
    st = prepare(case, seed)
    if case["op"] == "mm":
        w, x = st["layer"], st["x"]
        wd = (w["codes"].double() - (0 if w["zpoint"] is None else w["zpoint"].double()[:, None]))
        wd = wd * w["scales"].double().view(-1, 1)
        rows = []
        step = max(1, 2 ** 28 // case["m"])
        for i in range(0, case["n"], step):
            sl = slice(i, i + step)
            y = torch.einsum("nk,mk->nm", x["codes"][sl].double() * x["scales"][sl].double()[:, None], wd)
            if st["bias"] is not None:
                y += st["bias"].double()
            if case["act"] == "relu":
                y = torch.where(y > 0, y, torch.zeros_like(y))
            elif case["act"] == "silu":
                y = y * torch.sigmoid(y)
            elif case["act"] == "gelu":
                y = 0.5 * y * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (y + 0.044715 * y ** 3)))
            if st["mul"] is not None:
                y *= st["mul"][sl].double()
            if st["res"] is not None:
                y += st["res"][sl].double()
            rows.append(y)
        return torch.cat(rows)
    scales, hs = [], []
    step = max(1, 2 ** 27 // case["d"])
    for i in range(0, case["n"], step):
        v = st["x"][i:i + step].double()
        f = torch.ones(v.shape[0], dtype=torch.float64, device="cuda")
        if case["op"] == "quant":
            if st["col"] is not None:
                v = v * st["col"].double()
        else:
            if st["r"] is not None:
                v = v + st["r"][i:i + step].double()
                hs.append(v)
                v = v.to(_DT[case["dt"]]).double()   # the norm is that of the rounded sum
            f = 1.0 / torch.sqrt((v * v).sum(1) / case["d"] + _EPS)
            v = v * st["w"].double()
        top = v.abs().max(1).values
        scales.append(torch.where(top > 0, top / 127.0, torch.ones_like(top)) * f)
    out = dict(codes=None, scales=torch.cat(scales), sums=None)
    return out if case["op"] == "quant" else dict(out, h=torch.cat(hs) if hs else None)
