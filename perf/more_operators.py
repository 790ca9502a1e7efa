"""What a decoder layer does in 8 bits around its attention, as cases for measurement.

Four operators: ``norm`` adds the residual, normalises by the root mean square
and gives fp16 values or 8-bit codes with scales; ``linear`` is the layer in
8-bit floats (e4m3 codes, one power-of-two scale for every 128 elements of a
row); ``gated`` is both projections of a feed-forward block with the activation
and the product, from codes; ``ffn`` is the whole block.  With ``own`` true the
framework's entry points run, otherwise a plain form in elementary torch
operations.

e4m3 format of a row: group g holds elements 128 g .. 128 g + 127 (the last may
be shorter); its scale is the smallest power of two s with max|x| / s <= 448 (1
for a group of zeros, never below 2^-126), a code is x / s rounded to e4m3; scales are e8m0 bytes.
"""
import math

import torch

own = False


# ---------------------------------------------------------------- cases ----

def listed():
    return [
        # one new token, the values go on to a layer that quantizes its own row
        dict(name="norm 1x4096 fp16", op="norm", rows=1, dim=4096, out="fp16", group=0, residual=True),
        # a small batch without a residual (the first layer), INT8 codes in groups
        dict(name="norm 129x2560 int8 g128", op="norm", rows=129, dim=2560, out="int8", group=128, residual=False),
        # a prompt of 4516 tokens, per-token codes in the form that the INT8 product reads
        dict(name="norm 4516x4096 half", op="norm", rows=4516, dim=4096, out="half", group=0, residual=True),
        # a long batch in front of 8-bit float layers, an odd token count
        dict(name="norm 16383x2560 fp8", op="norm", rows=16383, dim=2560, out="fp8", group=128, residual=True),
        # one token through a projection
        dict(name="linear 1x10240x2560", op="linear", rows=1, n=10240, k=2560),
        # a step of a small serving batch, the contraction long
        dict(name="linear 13x4096x14336", op="linear", rows=13, n=4096, k=14336),
        # a larger batch, odd count
        dict(name="linear 131x10240x2560", op="linear", rows=131, n=10240, k=2560),
        # a long batch
        dict(name="linear 8192x10240x2560", op="linear", rows=8192, n=10240, k=2560),
        # gate and up of a batch, fp16 values out
        dict(name="gated 100x10240x2560 fp16", op="gated", rows=100, f=10240, k=2560, out="fp16"),
        # gate and up of a ragged prompt, codes for the next product out
        dict(name="gated 2049x14336x4096 fp8", op="gated", rows=2049, f=14336, k=4096, out="fp8"),
        # one token through the whole block
        dict(name="ffn 1x4096x14336", op="ffn", rows=1, f=14336, k=4096),
        # a prompt of 4516 tokens through the whole block
        dict(name="ffn 4516x4096x14336", op="ffn", rows=4516, f=14336, k=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "linear", "linear", "gated", "ffn"])
    if op == "norm":
        out = rng.choice(["fp16", "int8", "half", "fp8"])
        # groups of 64 and 128 divide the row; a row of e4m3 codes may end inside its last group
        group = 128 if out == "fp8" else 0 if out == "fp16" else rng.choice([0, 64, 128])
        unit = group if group and out != "fp8" else 16
        dim = unit * max(1, _log(rng, 256, 16384) // unit)
        return dict(op=op, rows=_log(rng, 1, 8.0e7 / dim), dim=dim, out=out, group=group, residual=rng.random() < 0.7)
    k = 16 * _log(rng, 16, 900)
    if op == "linear":
        n = _log(rng, 64, 14336)
        return dict(op=op, rows=_log(rng, 1, max(2, min(16384, 2.0e11 / (n * k)))), n=n, k=k)
    k = min(k, 8192)
    f = 16 * _log(rng, 8, 900)
    rows = _log(rng, 1, max(2, min(8192, 2.0e11 / (f * k))))
    if op == "gated":
        return dict(op=op, rows=rows, f=f, k=k, out=rng.choice(["fp16", "fp8"]))
    return dict(op=op, rows=rows, f=f, k=k)


# --------------------------------------------------------------- inputs ----

def _groups(x):
    """x [rows, k] as [rows, groups, 128], the last group filled up with zeros."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % 128)).unflatten(1, (-1, 128))


def _quantize(x):
    """e4m3 codes and e8m0 scales of 32-bit rows."""
    part = _groups(x)
    top = part.abs().amax(-1)
    # top = m 2^e with m in [0.5, 1); 448 = 0.875 * 2^9
    m, e = torch.frexp(torch.where(top > 0, top, 448.0))
    e = (e - 9 + (m > 0.875).int()).clamp(min=-126)
    # 2^-e by its bits: a power function may miss the power by a last bit, and ties with it
    codes = (part * ((127 - e) << 23).view(torch.float32)[..., None]).to(torch.float8_e4m3fn)
    return codes.flatten(1)[:, :x.shape[1]].contiguous(), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _values(codes, scale):
    """What codes stand for, in 32 bits."""
    return (_groups(codes.float()) * scale.float()[..., None]).flatten(1)[:, :codes.shape[1]]


def _rows(gen, rows, dim):
    """Activations: normal, one in a hundred channels strong, tokens of unlike size."""
    x = torch.randn(rows, dim, generator=gen, device="cuda")
    x *= 1 + 29 * (torch.rand(dim, generator=gen, device="cuda") > 0.99)
    x *= 0.5 + torch.rand(rows, 1, generator=gen, device="cuda")
    return x


def _weights(gen, n, k):
    return _quantize(0.02 * torch.randn(n, k, generator=gen, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = dict(case)
    rows = case["rows"]
    if case["op"] == "norm":
        dim = case["dim"]
        s["x"] = _rows(gen, rows, dim).half()
        s["r"] = (4 * torch.randn(rows, dim, generator=gen, device="cuda")).half() if case["residual"] else None
        s["w"] = (1 + 0.2 * torch.randn(dim, generator=gen, device="cuda")).half()
        return s
    k = case["k"]
    x = _rows(gen, rows, k)
    if case["op"] == "linear":
        s["x"], s["wq"] = x.half(), _weights(gen, case["n"], k)
        s["y"] = torch.empty(rows, case["n"], dtype=torch.float16, device="cuda")
        s["workspace"] = torch.empty(rows * (k + k // 128 + 1) + 2048, dtype=torch.uint8, device="cuda")
        return s
    f = case["f"]
    s["wg"], s["wu"] = _weights(gen, f, k), _weights(gen, f, k)
    if case["op"] == "gated":
        s["xq"] = _quantize(x)
        return s
    s["x"], s["wd"] = x.half(), _weights(gen, k, f)
    s["y"] = torch.empty(rows, k, dtype=torch.float16, device="cuda")
    s["workspace"] = torch.empty(rows * (2 * k + 6 * f) + 4096, dtype=torch.uint8, device="cuda")
    return s


# ----------------------------------------------------------------- runs ----

def _plain_norm(s):
    h = s["x"].float()
    if s["r"] is not None:
        h = (h + s["r"].float()).half().float()
    # squares of 64 bits: long sums
    mean = h.double().square().mean(-1, keepdim=True)
    v = h * torch.rsqrt(mean + 1e-5).float() * s["w"].float()
    res = {} if s["r"] is None else {"r": h.half()}
    if s["out"] == "fp16":
        return {"y": v.half(), **res}
    if s["out"] == "fp8":
        codes, scale = _quantize(v)
        return {"q": codes, "scale": scale, **res}
    part = v.unflatten(1, (-1, s["group"] or v.shape[1]))
    scale = part.abs().amax(-1) / 127
    codes = torch.round(part / torch.where(scale > 0, scale, 1.0)[..., None]).clamp(-127, 127)
    return {"q": codes.flatten(1).half(), "scale": scale, **res}


def _plain_gated(xq, wg, wu):
    x = _values(*xq)
    g = x @ _values(*wg).T
    return g / (1 + torch.exp(-g)) * (x @ _values(*wu).T)


def run(s):
    op = s["op"]
    if not own:
        if op == "norm":
            return _plain_norm(s)
        if op == "linear":
            return (_values(*_quantize(s["x"].float())) @ _values(*s["wq"]).T).half()
        if op == "gated":
            h = _plain_gated(s["xq"], s["wg"], s["wu"])
            return h.half() if s["out"] == "fp16" else _quantize(h)
        h = _quantize(_plain_gated(_quantize(s["x"].float()), s["wg"], s["wu"]))
        return (_values(*h) @ _values(*s["wd"]).T).half()
    import w4a8_int8_quantized_gb300 as w8
    if op == "linear":
        return w8.fp8_linear(s["x"], *s["wq"], workspace=s["workspace"], y=s["y"])
    if op == "gated":
        return w8.fp8_gated_gemm(*s["xq"], *s["wg"], *s["wu"], codes=s["out"] == "fp8")
    if op == "ffn":
        return w8.fp8_feed_forward(s["x"], *s["wg"], *s["wu"], *s["wd"], workspace=s["workspace"], y=s["y"])
    if s["out"] == "fp16":
        got = w8.rms_norm(s["x"], s["w"], residual=s["r"], eps=1e-5)
        return {"y": got} if s["r"] is None else {"y": got[0], "r": got[1]}
    got = w8.rms_norm_quantize(s["x"], s["w"], residual=s["r"], eps=1e-5, codes=s["out"], group_size=s["group"])
    q = got[0].half() if s["out"] == "int8" else got[0]
    return {"q": q, "scale": got[1]} if s["r"] is None else {"q": q, "scale": got[1], "r": got[2]}


# ----------------------------------------------------------------- work ----

def _held(rows, k):
    """Bytes of e4m3 rows with their scales."""
    return rows * (k + -(-k // 128))


def work(case):
    rows = case["rows"]
    if case["op"] == "norm":
        dim = case["dim"]
        streams = 3 if case["residual"] else 1  # x, residual in and out
        each = {"fp16": 2, "half": 2, "int8": 1, "fp8": 1}[case["out"]]
        scales = {"fp16": 0, "fp8": -(-dim // 128)}.get(case["out"], 4 * (dim // case["group"] if case["group"] else 1))
        return {"bytes": rows * (dim * (2 * streams + each) + scales) + 2 * dim, "flops": 6 * rows * dim}
    k = case["k"]
    if case["op"] == "linear":
        n = case["n"]
        return {"bytes": 2 * rows * k + _held(n, k) + 2 * rows * n, "flops": 2 * rows * n * k}
    f = case["f"]
    if case["op"] == "gated":
        out = 2 * rows * f if case["out"] == "fp16" else _held(rows, f)
        return {"bytes": _held(rows, k) + 2 * _held(f, k) + out, "flops": 4 * rows * f * k}
    return {"bytes": 4 * rows * k + 2 * _held(f, k) + _held(k, f), "flops": 6 * rows * f * k}


# ---------------------------------------------------------------- exact ----

def _exact_power(e):
    """2^e in 64 bits, by its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_scale(x):
    """Per element of x [rows, k], the power of two of its group, in 64 bits; and per group."""
    rows, k = x.shape
    at = torch.arange(k, device=x.device) // 128
    top = torch.zeros(rows, int(at[-1]) + 1, dtype=torch.float64, device=x.device)
    top.scatter_reduce_(1, at.expand(rows, k), x.abs(), "amax")
    s = _exact_power(torch.ceil(torch.log2(torch.where(top == 0, torch.full_like(top, 448.0), top) / 448)))
    # the logarithm is rounded: put right what lies beside a power of two
    s = torch.where(top / s > 448, 2 * s, s)
    s = torch.where(torch.logical_and(top > 0, 2 * top / s <= 448), s / 2, s)
    return s[:, at], s


def _exact_codes(x):
    """e4m3 codes of 64-bit rows as numbers, ties to even: three bits behind the leading one, steps of 2^-9 at the bottom."""
    each, s = _exact_scale(x)
    v = x / each
    step = _exact_power(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step, s


def _exact_numbers(codes, scale):
    at = torch.arange(codes.shape[1], device=codes.device) // 128
    return codes.double() * scale.double()[:, at]


def _exact_hidden(x, s):
    g = x @ _exact_numbers(*s["wg"]).T
    return g * torch.sigmoid(g) * (x @ _exact_numbers(*s["wu"]).T)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h, out = s["x"].double(), {}
        if case["residual"]:
            h = (h + s["r"].double()).half().double()
            out["r"] = h
        v = h * s["w"].double() / torch.sqrt((h * h).sum(-1, keepdim=True) / case["dim"] + 1e-5)
        if case["out"] == "fp16":
            out["y"] = v
        elif case["out"] == "fp8":
            out["q"], out["scale"] = _exact_codes(v)
        else:
            size = case["group"] or case["dim"]
            v = v.reshape(case["rows"], -1, size)
            out["scale"] = v.abs().amax(-1) / 127
            out["q"] = torch.round(127 * v / v.abs().amax(-1, keepdim=True)).reshape(case["rows"], -1)
        return out
    if case["op"] == "gated":
        h = _exact_hidden(_exact_numbers(*s["xq"]), s)
        return h if case["out"] == "fp16" else _exact_codes(h)
    codes, scale = _exact_codes(s["x"].double())
    x = _exact_numbers(codes, scale)
    if case["op"] == "linear":
        return x @ _exact_numbers(*s["wq"]).T
    h = _exact_numbers(*_exact_codes(_exact_hidden(x, s)))
    return h @ _exact_numbers(*s["wd"]).T
