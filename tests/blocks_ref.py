"""Plain float64 references of the 8-bit block format, the gated block and the gradients through
packed weights, for the tests: torch on the CPU, from the definitions in include/awq.h, with no
code of the package. Also the error bounds that the tests hold the kernels to."""
import numpy as np
import torch

U32 = 2.0 ** -24                       # half a step of fp32, relative
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}

# the 127 non-negative e4m3 values by code: exponent field E, mantissa m: E = 0: m 2^-9, otherwise
# (1 + m / 8) 2^(E - 7); code 0x7F is NaN
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def e4m3_codes(v):
    """Codes of |v| <= 448 (numpy float64): the nearest value, ties to the even code; NaN 0x7F."""
    a = np.abs(np.where(np.isfinite(v), v, 0.0))
    hi = np.clip(np.searchsorted(E4M3, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = E4M3[hi] - a, a - E4M3[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(a == E4M3[hi], hi, code).astype(np.uint8)
    code = code | (np.signbit(v).astype(np.uint8) << 7)
    return np.where(np.isfinite(v), code, 0x7F).astype(np.uint8)


def e4m3_values(code):
    v = np.append(E4M3, np.nan)[code & 0x7F]
    return np.where(code & 0x80, -v, v)


def spread(scales, rows, m, k):
    return np.repeat(np.repeat(scales, rows, 0)[:m], 128, 1)[:, :k]


def quantize(x, rows):
    """(codes, scales) of x (numpy, any float type)."""
    x = x.astype(np.float64)
    m, k = x.shape
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    a = np.pad(a, ((0, -m % rows), (0, -k % 128)))
    top = a.reshape(a.shape[0] // rows, rows, -1, 128).max((1, 3))
    scales = np.ones_like(top)
    for i in np.ndindex(top.shape):
        if top[i] > 0:
            e = -126
            while top[i] > 448 * 2.0 ** e:
                e += 1
            scales[i] = 2.0 ** e
    return e4m3_codes(x / spread(scales, rows, m, k)), scales


def within(y, ref, out_dtype, slack):
    """|y - ref| <= half a step of the output type of |ref| + slack, and the largest share of that
    bound that was used. `slack` bounds everything but the final rounding; the rounding is of a
    value within slack of ref."""
    h = HALF_STEP[out_dtype]
    tol = h * (np.abs(ref) + slack) + TINY[out_dtype] + slack
    err = np.abs(y.astype(np.float64) - ref)
    used = float((err / tol).max()) if err.size else 0.0
    return bool((err <= tol).all()), used


def unpack(qweight, scales16, zeros, group):
    """(codes with the zero point taken off, steps), both float64 [N, K]."""
    n = qweight.shape[0]
    w = qweight.astype(np.int64) & 0xFFFFFFFF
    q = (w[:, :, None] >> (4 * np.arange(8))) & 15
    q = q.reshape(n, -1)
    steps = np.repeat(scales16.astype(np.float64), group, 1)
    if zeros is None:
        q = np.where(q > 7, q - 16, q)
    else:
        q = q - np.repeat(zeros.astype(np.int64), group, 1)
    return q.astype(np.float64), steps


def act(g, name):
    """The activation and its derivative in float64."""
    with np.errstate(over="ignore"):
        if name == "silu":
            p = 1 / (1 + np.exp(-g))
            return g * p, p + g * p * (1 - p)
        c = 2 * np.sqrt(2 / np.pi)
        p = 1 / (1 + np.exp(-c * (g + 0.044715 * g ** 3)))
        return g * p, p + g * p * (1 - p) * c * (1 + 3 * 0.044715 * g * g)


# ---- the gated block and the gradients ---------------------------------------------------------
# Bounds. (1) A sum of T exact products in fp32, in any order and grouping, each addition within
# 2^-23 of the sum of magnitudes (fp16 MFMA and dot instructions cut or round at fp32's last bit),
# plus the fma by the step of each group: (T + 2 groups + 16) 2^-23 sum |.|; 16 covers the additions
# of waves and slices. (2) act: p = 1 / (1 + exp2(-z log2 e)) has a relative error of at most
# (4 |z| + 8) 2^-23: the exponent's product and z itself round by 4 2^-24 |z| at most, exp2, the
# addition and the reciprocal by an ulp (2^-23) each.
def sum_slack(terms, groups, magnitudes):
    return (terms + 2 * groups + 16) * 2.0 ** -23 * magnitudes


def act_z(g, name):
    return np.abs(g) if name == "silu" else 1.6 * (np.abs(g) + 0.0448 * np.abs(g) ** 3)


def gated(a, gate, up, group, name):
    """(g, u, their slack, H, its slack) for a (float64) and unpack()ed weights."""
    out = []
    for c, step in (gate, up):
        mag = np.abs(a) @ np.abs(c * step).T
        out += [a @ (c * step).T, sum_slack(a.shape[1], a.shape[1] // group, mag)]
    g, eg, u, eu = out
    f, _ = act(g, name)
    ef = 1.2 * eg + np.abs(f) * (4 * act_z(g, name) + 8) * 2.0 ** -23      # |act'| < 1.2
    return g, eg, u, eu, f * u, ef * (np.abs(u) + eu) + np.abs(f) * eu + 2.0 ** -23 * np.abs(f * u)


def grads(dh, g, u, name):
    """(dg, du, and a bound of their fp32 errors): four products and the activation's errors."""
    f, df = act(g, name)
    dg, du = dh * u * df, dh * f
    rel = (4 * act_z(g, name) + 16) * 2.0 ** -23
    # df = p + q z', |p|, |q z'| < 1.2 each: its error is relative to those, not to their sum
    slope = 1.0 if name == "silu" else 1.6 * (1 + 0.1342 * g * g)
    p = np.where(np.abs(g) > 0, f / np.where(g == 0, 1, g), 0.5)
    parts = np.abs(p) + np.abs(f * (1 - p)) * slope
    return dg, du, np.abs(dh * u) * parts * rel + 2.0 ** -22 * np.abs(dg), np.abs(du) * (rel + 2.0 ** -22)


def backward(pairs, group):
    """sum over (d, error of d, (codes, steps)) of d @ (codes * steps), and its slack: each operand
    fp16(d step) rounds by 2^-11, or by 2^-25 in units of 2^-14 max|d| (the row) times twice the
    largest step of the column's group (subnormals, of the high and of the low part); then the
    fp32 sum."""
    out, slack, mag = 0.0, 0.0, 0.0
    top_d = np.max([np.abs(d).max(1) for d, _, _ in pairs], 0)
    top_s = np.max([s.max(0) for _, _, (_, s) in pairs], 0)
    terms = 0
    for d, ed, (c, s) in pairs:
        w = c * s
        m = np.abs(d) @ np.abs(w)
        out = out + d @ w
        mag = mag + m
        slack = slack + 2.0 ** -11 * m + (1 + 2.0 ** -10) * (ed @ np.abs(w)) + \
            2 * 2.0 ** -38 * np.outer(top_d, top_s * np.abs(c).sum(0))
        terms += d.shape[1]
    return out, slack + sum_slack(terms, 0, mag * (1 + 2.0 ** -10))
