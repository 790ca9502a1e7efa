"""The norm, the 8-bit float rows and their products in plain 64-bit torch, for
the tests: the definitions, with tolerances that follow from the kernels'
arithmetic."""
import torch

GROUP = 128


def bits(e):
    """2^e in 64 bits, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def floor_log2(x):
    """Exponent of positive 64-bit values, exactly."""
    return torch.frexp(x)[1] - 1


def per_element(per_group, k):
    return per_group.repeat_interleave(GROUP, 1)[:, :k]


def group_max(x):
    pad = torch.nn.functional.pad(x.abs(), (0, -x.shape[1] % GROUP))
    return pad.view(x.shape[0], -1, GROUP).amax(-1)


def scale_of(top):
    """Smallest power of two s with top / s <= 448; 1 for 0; at least 2^-126."""
    e = floor_log2(torch.where(top > 0, top, 448.0).double())
    s = bits(e - 8)
    s = torch.where(top > 448 * s, 2 * s, s)
    return torch.where(top > 0, s.clamp(min=2.0 ** -126), 1.0)


def e4m3(x):
    """64-bit values rounded to e4m3, ties to even, saturating."""
    a = x.abs()
    step = bits(floor_log2(a.clamp(min=2.0 ** -6)) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def quantize(x):
    """(codes as numbers, scales) of 64-bit rows."""
    s = scale_of(group_max(x))
    return e4m3(x / per_element(s, x.shape[1])), s


def values(codes, scale):
    return codes.double() * per_element(scale.double(), codes.shape[1])


def half_step(x, s):
    """Most that rounding x / s to e4m3 moves x, per element."""
    return torch.maximum(x.abs() * 2.0 ** -4, s * 2.0 ** -10)


# ---------------------------------------------------------------- norm ----

# Relative error of the norm's fp32 value.  A thread adds at most 64 squares in
# a chain, then come 5 + 16 additions: 85 roundings, each 2^-24, of a sum of
# non-negative terms; half of that through the square root; the division by K,
# eps, the root, the reciprocal and the product: 5 more.  (85 / 2 + 5) 2^-24 <
# 2^-18.
NORM = 2.0 ** -18


def norm(x, w, r=None, eps=1e-5):
    """(v, h) in 64 bits."""
    h = x.double() if r is None else (x.double() + r.double()).half().double()
    mean = h.square().mean(-1, keepdim=True) + eps
    inv = torch.where(mean > 0, mean.rsqrt(), 0.0)
    return h * w.double() * inv, h


def check_values(got, v, rel):
    """fp16 of a value known to rel."""
    assert ((got.double() - v).abs() <= v.abs() * (2.0 ** -11 + 2 * rel) + 2.0 ** -25).all()


def check_int8(codes, scale, v, group, rel):
    """INT8 codes and fp32 scales of values known to rel."""
    part = v.view(v.shape[0], -1, group or v.shape[1])
    want = part.abs().amax(-1) / 127
    scale = scale.view(want.shape).double()
    assert ((scale - want).abs() <= want * (rel + 2.0 ** -23)).all()
    safe = torch.where(want > 0, want, 1.0)
    t = (part / safe[..., None]).flatten(1)
    # v and s are each off by rel and a rounding: 127 (2 rel + 2^-22) of a code
    assert ((codes.double() - t).abs() <= 0.5 + 127 * (2 * rel + 2.0 ** -22)).all()
    assert (codes.double().abs() <= 127).all()


def check_fp8(codes, scale, v, err):
    """e4m3 codes and scales of values known to err (absolute, per element)."""
    scale = scale.double()
    lo, hi = (group_max((v.abs() + d * err).clamp(min=0)) for d in (-1, 1))
    assert ((scale >= scale_of(lo)) | (lo == 0)).all() and (scale <= torch.maximum(scale_of(hi), scale_of(lo))).all()
    s = per_element(scale, v.shape[1])
    got = codes.double() * s
    assert ((got - v).abs() <= half_step(v.abs() + err, s) + err).all()
    # away from a border between two codes the code is the nearest one
    near = e4m3(v / s)
    sure = e4m3((v - err) / s) == e4m3((v + err) / s)
    assert (codes.double()[sure] == near[sure]).all()


# ------------------------------------------------------------ products ----

def product(x, w):
    """(x w^T, error of its fp32 sum) in 64 bits.

    A product of two e4m3 values is exact in fp32.  The sum is made of at most
    K additions, in the tensor core and after it, of which each loses at most
    2^-23 of a partial sum (a truncation); a partial sum is at most A = sum |x w|.
    The chains are shorter than K: an instruction adds 16 products or more at
    once, losing at most 2^-23 A for each of them on the way, then come the groups
    of 128 and the 8 joined warps.  Hence (K / 16 + K / 128 + 16) 2^-23 A."""
    k = x.shape[1]
    return x @ w.T, (k / 16 + k / 128 + 16) * 2.0 ** -23 * (x.abs() @ w.abs().T)


def check_product(got, y, err):
    diff = (got.double() - y).abs()
    assert (diff <= y.abs() * 2.0 ** -11 + 2.0 ** -25 + err * (1 + 2.0 ** -11)).all()
    # on the whole: the rounding's 2^-11 at most, and errors of sums that do not all point one way
    assert diff.norm() <= y.norm() * 2.0 ** -11 + 2.0 ** -25 * y.numel() ** 0.5 + 0.05 * err.norm()


def act(g, gelu):
    if gelu:
        return 0.5 * g * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3)))
    return g * torch.sigmoid(g)


def gated(x, wg, wu, gelu=False):
    """(h, error of its fp32 value).  |act'| <= 1.13 (both forms); the exponential
    and the quotient are good to 2^-20 of act(g) where it counts: the exponent's
    argument is rounded (2^-23 |t|, with |t| e^-|t| small), and each function is off
    by 2^-21 at most."""
    g, eg = product(x, wg)
    u, eu = product(x, wu)
    a = act(g, gelu)
    h = a * u
    return h, 1.13 * eg * (u.abs() + eu) + a.abs() * eu + (2.0 ** -19 * g.abs() + 2.0 ** -20) * (a.abs() + 1e-6) * u.abs()
