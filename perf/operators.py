"""The quantized key/value cache and the attention over it, as cases for measurement.

Three operators: ``write`` quantizes new tokens' keys and values into the paged
cache (and reads them back, so that what it stored is seen), ``read`` gathers
dequantized tokens, ``attend`` is attention of single tokens, chunks or whole
prompts over the cache.  With ``own`` true the framework's entry points run,
otherwise a plain form in elementary torch operations.

Cache: codes [pages, kv heads, page, D] int8 (8 bits) or [pages, kv heads,
page, D / 2] uint8 (4 bits, low nibble = even element, two's complement), one
fp32 scale per token and head [pages, kv heads, page], for K and for V.
"""
import math

import torch

own = False


# ---------------------------------------------------------------- cases ----

def listed():
    return [
        # one user's decoding step: one token's k and v go into the cache
        dict(name="write 1 token 4b", op="write", bits=4, tokens=1, kv_heads=8, q_heads=32, dim=128, page=16),
        # a prompt of 4516 tokens
        dict(name="write 4516 4b", op="write", bits=4, tokens=4516, kv_heads=8, q_heads=32, dim=128, page=64),
        # a batch of long prompts at 8 bits, an odd token count
        dict(name="write 32771 8b", op="write", bits=8, tokens=32771, kv_heads=8, q_heads=32, dim=128, page=16),
        # a short shared prefix, small heads
        dict(name="read 1237 8b d64", op="read", bits=8, tokens=1237, kv_heads=16, q_heads=16, dim=64, page=32),
        # a long document's prefix handed to dense code
        dict(name="read 65536 4b", op="read", bits=4, tokens=65536, kv_heads=8, q_heads=32, dim=128, page=64),
        # the smallest call: one user, a short prompt, one new token
        dict(name="decode b1 len77 4b", op="attend", bits=4, batch=1, len_lo=77, len_hi=77, q_lo=1, q_hi=1,
             kv_heads=8, q_heads=32, dim=128, page=16, window=0),
        # a serving batch of ragged lengths
        dict(name="decode b64 512..8192 4b", op="attend", bits=4, batch=64, len_lo=512, len_hi=8192, q_lo=1, q_hi=1,
             kv_heads=8, q_heads=32, dim=128, page=16, window=0),
        # one user with a long document
        dict(name="decode b1 len131072 4b", op="attend", bits=4, batch=1, len_lo=131072, len_hi=131072, q_lo=1, q_hi=1,
             kv_heads=8, q_heads=32, dim=128, page=64, window=0),
        # every head with its own keys, small heads, 8 bits, 4 tokens a step (draft verification)
        dict(name="verify b16 q4 8b d64", op="attend", bits=8, batch=16, len_lo=900, len_hi=4516, q_lo=4, q_hi=4,
             kv_heads=16, q_heads=16, dim=64, page=32, window=0),
        # a whole prompt of 4516 tokens
        dict(name="prefill 4516 4b", op="attend", bits=4, batch=1, len_lo=4516, len_hi=4516, q_lo=4516, q_hi=4516,
             kv_heads=8, q_heads=32, dim=128, page=64, window=0),
        # ragged prompts behind earlier turns, sliding window, 8 bits
        dict(name="prefill b6 ragged w1024 8b", op="attend", bits=8, batch=6, len_lo=700, len_hi=5003, q_lo=17, q_hi=1500,
             kv_heads=4, q_heads=32, dim=128, page=16, window=1024),
        # one chunk of a long prompt
        dict(name="chunk 512 of 32768 4b", op="attend", bits=4, batch=1, len_lo=32768, len_hi=32768, q_lo=512, q_hi=512,
             kv_heads=8, q_heads=32, dim=128, page=64, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    bits, dim = rng.choice([4, 4, 8]), rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8, 16])
    heads = dict(bits=bits, dim=dim, kv_heads=kv, q_heads=kv * rng.choice([1, 2, 3, 4, 7, 8]), page=rng.choice([16, 32, 64, 128]))
    op = rng.choice(["write", "read", "decode", "decode", "verify", "prefill", "prefill"])
    if op in ("write", "read"):
        most = (32000 if op == "write" else 64000) * 1024 // (kv * dim)
        return dict(op=op, tokens=_log(rng, 1, most), **heads)
    if op == "prefill":
        batch, q_hi = _log(rng, 1, 6), _log(rng, 33, 4000)
        most = 2.4e8 / (batch * heads["q_heads"] * q_hi)  # (row, key) pairs of the plain form's padded scores
        len_hi = max(q_hi, min(_log(rng, q_hi, 8 * q_hi), int(most)))
        if most < q_hi:
            q_hi = len_hi = max(33, int(math.sqrt(2.4e8 / (batch * heads["q_heads"]))))
        q_lo = rng.randint(1, q_hi)
    else:
        batch = _log(rng, 1, 96)
        q_hi = 1 if op == "decode" else rng.randint(2, 8)
        q_lo = q_hi
        len_hi = _log(rng, 16, max(17, min(100000, int(2.0e8 / (batch * kv * dim)))))
        len_hi = max(len_hi, q_hi)
    return dict(op="attend", batch=batch, len_lo=rng.randint(max(1, len_hi // 8), len_hi), len_hi=len_hi, q_lo=q_lo, q_hi=q_hi,
                window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]), **heads)


def _spread(lo, hi, n, step):
    """n whole numbers between lo and hi, the first one hi."""
    return [int(round(hi - (hi - lo) * ((i * step) % 1.0))) for i in range(n)]


def _lengths(case):
    lens = _spread(case["len_lo"], case["len_hi"], case["batch"], 0.6180339887)
    new = _spread(case["q_lo"], case["q_hi"], case["batch"], 0.7548776662)
    return lens, [min(a, b) for a, b in zip(new, lens)]


# --------------------------------------------------------------- inputs ----

def _values(codes, scale):
    """What the codes stand for, in 32 bits."""
    if codes.dtype == torch.uint8:
        x = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
        x = x - 16 * (x > 7)
    else:
        x = codes.float()
    return x * scale[..., None]


def _quantize(x, bits):
    """Codes and scales of fp16 rows."""
    x = torch.nan_to_num(x.float(), nan=0.0, posinf=65504.0, neginf=-65504.0)
    most = 2.0 ** (bits - 1) - 1
    # / tensor, not / number: a number may be turned into a product with its reciprocal
    scale = x.abs().amax(-1) / torch.full((), most, device=x.device)
    q = torch.round(x / torch.where(scale > 0, scale, 1.0)[..., None]).clamp(-most, most)
    q = q.to(torch.int8)
    if bits == 4:
        q = ((q[..., 0::2] & 15) | (q[..., 1::2] << 4)).view(torch.uint8)
    return q, scale


def _rows(gen, *shape):
    """Activations: normal, with a few strong channels and tokens of unlike size."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= 1 + 6 * (torch.rand(shape[-2:], generator=gen, device="cuda") > 0.97)
    x *= 0.5 + torch.rand(shape[:-1], generator=gen, device="cuda")[..., None]
    return x.half()


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    kv, heads, dim, page, bits = case["kv_heads"], case["q_heads"], case["dim"], case["page"], case["bits"]
    s = dict(op=case["op"], bits=bits, kv_heads=kv, page=page)
    if case["op"] == "attend":
        lens, new = _lengths(case)
        counts = [-(-n // page) for n in lens]
        need = sum(counts)
    else:
        need = -(-case["tokens"] // page)
    total = need + 1 + need // 16
    order = torch.randperm(total, generator=gen, device="cuda")[:need]
    s["code_shape"] = (total, kv, page, dim * bits // 8)
    if case["op"] == "write":
        tokens = case["tokens"]
        s["cache"] = [torch.zeros(s["code_shape"], dtype=torch.uint8 if bits == 4 else torch.int8, device="cuda") for _ in "kv"]
        s["cache"] += [torch.zeros(s["code_shape"][:3], device="cuda") for _ in "kv"]
        qkv = _rows(gen, tokens, heads + 2 * kv, dim)  # the fused projection's output
        s["k"], s["v"] = qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    else:
        quantized = [_quantize(_rows(gen, total, page, kv, dim).transpose(1, 2), bits) for _ in "kv"]
        s["cache"] = [c.contiguous() for c, _ in quantized] + [x.contiguous() for _, x in quantized]
    if case["op"] == "attend":
        table = torch.zeros(case["batch"], max(counts), dtype=torch.int64, device="cuda")
        inside = torch.arange(max(counts), device="cuda")[None] < torch.tensor(counts, device="cuda")[:, None]
        table[inside] = order
        s["table"] = table.int()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        s["max_q"], s["window"] = max(new), case["window"]
        s["q"] = _rows(gen, starts[-1], heads, dim)
    else:
        s["slots"] = (order[:, None] * page + torch.arange(page, device="cuda")).flatten()[:case["tokens"]].contiguous()
    if own:
        # what a serving program keeps: the cache's handle and a workspace
        import w4a8_int8_quantized_gb300 as w8
        s["handle"] = w8.KVCache(*s["cache"])
        if case["op"] == "attend":
            need = w8.kv_cache_attention_workspace_bytes(s["q"].shape[0], heads, s["handle"], s["table"], s["max_q"])
            s["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    return s


# ----------------------------------------------------------------- runs ----

def _plain_write(s):
    k_codes, v_codes, k_scale, v_scale = s["cache"]
    page, slot = s["slots"] // s["page"], s["slots"] % s["page"]
    for x, codes, scale in ((s["k"], k_codes, k_scale), (s["v"], v_codes, v_scale)):
        codes[page, :, slot], scale[page, :, slot] = _quantize(x, s["bits"])


def _plain_read(s):
    k_codes, v_codes, k_scale, v_scale = s["cache"]
    page, slot = s["slots"] // s["page"], s["slots"] % s["page"]
    return [_values(codes[page, :, slot], scale[page, :, slot]).half() for codes, scale in ((k_codes, k_scale), (v_codes, v_scale))]


def _plain_attend(s):
    k_codes, v_codes, k_scale, v_scale = s["cache"]
    q, table, starts, lens = s["q"], s["table"].long(), s["starts"].long(), s["lens"].long()
    rows, heads, dim = q.shape
    batch, kv, most = table.shape[0], s["kv_heads"], s["max_q"]
    new = starts[1:] - starts[:-1]
    i = torch.arange(most, device=q.device)
    at = (starts[:-1, None] + i).clamp(max=rows - 1)
    x = q.float()[at].view(batch, most, kv, -1, dim).transpose(1, 2).flatten(2, 3)  # [b, kv, most * group, dim]
    k, v = (_values(c[table], z[table]).transpose(1, 2).flatten(2, 3) for c, z in ((k_codes, k_scale), (v_codes, v_scale)))
    scores = x @ k.transpose(2, 3)
    scores *= dim ** -0.5
    j, pos = torch.arange(k.shape[2], device=q.device), lens[:, None] - new[:, None] + i
    seen = (j <= pos[..., None]) & (j < lens[:, None, None])
    if s["window"]:
        seen &= j > pos[..., None] - s["window"]
    seen = seen.repeat_interleave(heads // kv, 1)[:, None]
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total > 0, total, 1.0)
    lse = top + total.log()
    row = torch.arange(rows, device=q.device)
    b = torch.searchsorted(starts, row, right=True) - 1
    out = out.view(batch, kv, most, -1, dim).transpose(1, 2).flatten(2, 3)[b, row - starts[b]]
    lse = lse.view(batch, kv, most, -1).transpose(1, 2).flatten(2, 3)[b, row - starts[b]]
    return {"out": out.half(), "lse": lse}


def run(s):
    if own:
        import w4a8_int8_quantized_gb300 as w8
    if s["op"] == "attend":
        if not own:
            return _plain_attend(s)
        out, lse = w8.kv_cache_attention(s["q"], s["handle"], s["table"], s["lens"], q_offsets=s["starts"], max_q=s["max_q"],
                                         window=s["window"], return_lse=True, workspace=s["workspace"])
        return {"out": out, "lse": lse}
    if s["op"] == "write":
        w8.kv_cache_write(s["k"], s["v"], s["slots"], s["handle"]) if own else _plain_write(s)
    k, v = w8.kv_cache_read(s["slots"], s["handle"]) if own else _plain_read(s)
    if s["op"] == "read":
        return {"k": k, "v": v}
    return {"k": k, "v": v, "k_scale": s["cache"][2], "v_scale": s["cache"][3]}


# ----------------------------------------------------------------- work ----

def _pairs(n, new, window):
    """Visible (row, key) pairs of one head, and the keys that any row sees."""
    total = 0
    for i in range(new):
        pos = n - new + i
        total += min(pos + 1, window) if window else pos + 1
    first = max(0, n - new - window + 1) if window else 0
    return total, n - first


def work(case):
    kv, heads, dim = case["kv_heads"], case["q_heads"], case["dim"]
    held = 2 * kv * (dim * case["bits"] // 8 + 4)  # bytes of one token's k and v in the cache
    half = 2 * kv * dim * 2
    if case["op"] == "read":
        return {"bytes": case["tokens"] * (8 + held + half), "flops": case["tokens"] * 2 * kv * dim}
    if case["op"] == "write":  # fp16 in, codes out and in again, fp16 out
        return {"bytes": case["tokens"] * (16 + 2 * held + 2 * half), "flops": case["tokens"] * 2 * kv * dim * 5}
    lens, new = _lengths(case)
    each = [_pairs(n, m, case["window"]) for n, m in zip(lens, new)]
    pages = sum(-(-k // case["page"]) for _, k in each)
    rows = sum(new)
    return {"bytes": held * sum(k for _, k in each) + 4 * pages + 8 * len(lens) + rows * heads * (4 * dim + 4),
            "flops": 4 * dim * heads * sum(p for p, _ in each)}


# ---------------------------------------------------------------- exact ----

def _exact_codes(x, bits):
    """(codes, scales) by the definition: scale and quotient are each rounded to 32 bits once."""
    x = x.double()
    top = float((1 << (bits - 1)) - 1)
    scale = (x.abs().max(-1, keepdim=True).values / top).float().double()
    quotient = torch.where(scale == 0, torch.zeros_like(x), x / scale).float().double()
    return quotient.round(), scale


def _exact_tokens(codes, scale, slots, page):
    """Values of the tokens at the slots, [tokens, heads, D] in 64 bits."""
    where = (torch.div(slots, page, rounding_mode="floor"), slice(None), slots % page)
    c = codes[where].to(torch.int64)
    if codes.dtype == torch.uint8:
        c = torch.cat(((c % 16).unsqueeze(-1), torch.div(c, 16, rounding_mode="floor").unsqueeze(-1)), -1).reshape(*c.shape[:-1], -1)
        c = torch.where(c >= 8, c - 16, c)
    return c.double() * scale[where].double().unsqueeze(-1)


def exact(case, seed):
    s = prepare(case, seed)
    page = s["page"]
    if case["op"] == "write":
        out = {}
        for name, x, scale in (("k", s["k"], s["cache"][2]), ("v", s["v"], s["cache"][3])):
            codes, z = _exact_codes(x, case["bits"])
            whole = scale.double().clone()
            for h in range(case["kv_heads"]):
                whole[torch.div(s["slots"], page, rounding_mode="floor"), h, s["slots"] % page] = z[:, h, 0]
            out[name], out[name + "_scale"] = codes * z, whole
        return out
    if case["op"] == "read":
        return {n: _exact_tokens(s["cache"][i], s["cache"][i + 2], s["slots"], page) for i, n in enumerate("kv")}
    lens, new = _lengths(case)
    kv, heads, dim = case["kv_heads"], case["q_heads"], case["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    start = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        t = torch.arange(n, device="cuda")
        slots = s["table"][b].long()[t // page] * page + t % page
        k = _exact_tokens(s["cache"][0], s["cache"][2], slots, page)
        v = _exact_tokens(s["cache"][1], s["cache"][3], slots, page)
        pos = torch.arange(n - m, n, device="cuda")[:, None]
        hidden = t[None] > pos
        if case["window"]:
            hidden = hidden | (pos - t[None] >= case["window"])
        for h in range(heads):
            a = s["q"][start:start + m, h].double() @ k[:, h * kv // heads].T / math.sqrt(dim)
            a = a.masked_fill(hidden, -math.inf)
            lse[start:start + m, h] = torch.logsumexp(a, -1)
            out[start:start + m, h] = torch.softmax(a, -1) @ v[:, h * kv // heads]
        start += m
    return {"out": out, "lse": lse}
