"""The key/value cache and its attention in plain 64-bit numpy, for the tests.

Quantization rule: per (token, head) s = fl32(max|x| / qmax), code =
rint(fl32(x / s)) -- both divisions done in 64 bits and rounded to 32, which
for 24-bit operands is the IEEE 32-bit quotient -- NaN taken as 0 and +-Inf as
+-65504.  Attention: the definition, in 64 bits.
"""
import numpy as np


def quantize(x, bits):
    """fp16 [..., D] -> (codes int64 [..., D], scales float64 [...])."""
    x = np.nan_to_num(x.astype(np.float64), nan=0.0, posinf=65504.0, neginf=-65504.0)
    qmax = 2 ** (bits - 1) - 1
    s = (np.abs(x).max(-1) / qmax).astype(np.float32).astype(np.float64)
    safe = np.where(s > 0, s, 1.0)
    q = np.rint((x / safe[..., None]).astype(np.float32).astype(np.float64))
    return np.clip(q, -qmax, qmax).astype(np.int64), s


def pack(codes, bits):
    """Codes as the cache holds them."""
    if bits == 8:
        return codes.astype(np.int8)
    return ((codes[..., 0::2] & 15) | ((codes[..., 1::2] & 15) << 4)).astype(np.uint8)


def unpack(held, bits):
    if bits == 8:
        return held.astype(np.int64)
    n = np.stack([held & 15, held >> 4], -1).reshape(*held.shape[:-1], -1).astype(np.int64)
    return np.where(n > 7, n - 16, n)


def attend(q, kcode, ks, vcode, vs, scale, causal=True, window=0):
    """One sequence: q [n, Hq, D], codes [len, Hkv, D], scales [len, Hkv].

    Returns (out, lse, tol_out, tol_lse) in 64 bits.  The tolerances follow
    from the kernels' arithmetic:
      E   bounds a score's error: D products summed in 32 bits, then a few
          32-bit products: (D + 8) 2^-23 * scale * sum_d |q_d k_d|, and the
          rounding of the exponent's argument, 2^-22 (|S| + |log2 s_v| + 8);
      A   = sum_j P_j |v_j|: each weight is rounded to fp16 once (2^-11), the
          output once more (2^-11), and a weight is off by 2 E relative;
      U   weights that are subnormal in fp16 are off by 2^-25 of the largest
          weighted scale, times the code;
      2^-24: the output's own subnormal rounding."""
    n, Hq, D = q.shape
    L, Hkv = ks.shape
    g = Hq // Hkv
    q = q.astype(np.float64)
    k = kcode * ks[..., None]
    v = vcode * vs[..., None]
    out = np.zeros((n, Hq, D))
    lse = np.full((n, Hq), -np.inf)
    tol = np.full((n, Hq, D), 2.0 ** -24)
    tol_lse = np.zeros((n, Hq))
    cmax = np.abs(vcode).max() if L else 0
    for h in range(Hq):
        kh, vh, sv = k[:, h // g], v[:, h // g], vs[:, h // g]
        for i in range(n):
            pos = L - n + i
            hi = min(pos + 1, L) if causal else L
            lo = max(pos + 1 - window, 0) if window else 0
            if hi <= lo:
                continue
            a = kh[lo:hi] @ q[i, h] * scale
            top = a.max()
            e = np.exp(a - top)
            P = e / e.sum()
            out[i, h] = P @ vh[lo:hi]
            lse[i, h] = top + np.log(e.sum())
            s = sv[lo:hi]
            lg = np.abs(np.log2(np.where(s > 0, s, 1.0))).max()
            E = ((D + 8) * 2.0 ** -23 * abs(scale) * (np.abs(kh[lo:hi]) @ np.abs(q[i, h])).max()
                 + 2.0 ** -22 * (np.abs(a).max() * 2 + lg + 8))
            A = P @ np.abs(vh[lo:hi])
            U = (hi - lo) * 2.0 ** -25 * cmax * (P * s).max()
            tol[i, h] += (2.0 ** -10 + 4 * E) * A + U
            tol_lse[i, h] = 2 * E + (hi - lo + 64) * 2.0 ** -24 + 2.0 ** -22 * abs(lse[i, h])
    return out, lse, tol, tol_lse
