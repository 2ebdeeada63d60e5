"""FP64 NumPy definitions of the operators around the cross entropy: the norm before the
classifier and its gradients, microscaled quantisation, the product of two microscaled
matrices, and sampling.  Independent of the library and of torch."""
from __future__ import annotations

import numpy as np

FORMATS = {"e2m1": (6.0, 0, 1), "e4m3": (448.0, -6, 3)}  # largest value, least exponent, mantissa bits


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------

def rms_norm(h, w, eps):
    """(y, rstd) of h [n, H] (already the rounded sum)."""
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    r = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * r[:, None] * w, r


def rms_norm_backward(dy, h, w, rstd, dh=None):
    """(dx, dw) from y = h r w with r = (mean h^2 + eps)^(-1/2) and the given r."""
    dy, h, w = (np.asarray(a, np.float64) for a in (dy, h, w))
    r = np.asarray(rstd, np.float64)[:, None]
    g = dy * w
    dx = r * (g - h * r ** 2 * (g * h).mean(1, keepdims=True))
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, (dy * h * r).sum(0)


# ---------------------------------------------------------------------------
# microscaled formats
# ---------------------------------------------------------------------------

def mx_values(fmt):
    """Every non-negative value of the format in code order."""
    _, low, bits = FORMATS[fmt]
    out, m, e = [], 0, 0
    for code in range(8 if fmt == "e2m1" else 127):  # E4M3's last code is its NaN
        e, m = code >> bits, code & ((1 << bits) - 1)
        frac = m / (1 << bits)
        out.append(frac * 2.0 ** low if e == 0 else (1 + frac) * 2.0 ** (e - 1 + low))
    return np.array(out)


def mx_quantize(x, fmt):
    """(codes [n, blocks * 32], exponents [n, blocks]) of x [n, c] in FP64; exponent 128: a
    block with an infinity or a NaN.  A code is its index in mx_values, plus the sign bit."""
    x = np.asarray(x, np.float64)
    n, c = x.shape
    most = FORMATS[fmt][0]
    pad = np.zeros((n, -(-c // 32) * 32))
    pad[:, :c] = x
    b = pad.reshape(n, -1, 32)
    bad = ~np.isfinite(b).all(2)
    b = np.where(bad[:, :, None], 0.0, b)
    amax = np.abs(b).max(2)
    frac, exp = np.frexp(amax)               # amax = frac 2^exp, frac in [0.5, 1)
    mfrac, mexp = np.frexp(most)
    e = np.where(amax > 0, exp - mexp + (frac > mfrac), -127)
    e = np.clip(e, -127, 127)
    t = np.abs(b) * 2.0 ** -e[:, :, None].astype(np.float64)
    vals = mx_values(fmt)
    hi = np.clip(np.searchsorted(vals, t), 0, len(vals) - 1)
    lo = np.maximum(hi - 1, 0)
    mid = (vals[lo] + vals[hi]) / 2
    up = (t > mid) | ((t == mid) & (hi % 2 == 0))   # ties to the even code
    code = np.where(vals[hi] <= t, hi, np.where(up, hi, lo))
    sign = np.signbit(b).astype(int) << (3 if fmt == "e2m1" else 7)
    code = np.where(bad[:, :, None], 0, code | sign)
    return code.reshape(n, -1), np.where(bad, 128, e)


def mx_dequantize(codes, e, fmt):
    """FP64 values of codes [n, blocks * 32] and exponents [n, blocks]."""
    half = 8 if fmt == "e2m1" else 128
    vals = mx_values(fmt)
    vals = np.concatenate([vals, [np.nan] * (half - len(vals))])
    q = np.where(codes >= half, -vals[codes % half], vals[codes % half])
    s = np.where(e == 128, np.nan, 2.0 ** e.astype(np.float64))
    n = codes.shape[0]
    return (q.reshape(n, -1, 32) * s[:, :, None]).reshape(n, -1)


def mx_pack(codes, e, cols, fmt):
    """(code bytes, scale tiles) as the library stores them."""
    n, c = codes.shape
    padded = -(-cols // 128) * 128
    full = np.zeros((n, padded), np.uint8)
    full[:, :c] = codes
    packed = full if fmt == "e4m3" else full[:, 0::2] | (full[:, 1::2] << 4)
    tiles = np.zeros((-(-n // 128), padded // 128, 512), np.uint8)
    for r in range(n):
        for b in range(e.shape[1]):
            tiles[r // 128, b // 4, r % 32 * 16 + r % 128 // 32 * 4 + b % 4] = e[r, b] + 127
    return packed, tiles


# ---------------------------------------------------------------------------
# sampling
# ---------------------------------------------------------------------------

def sample_row(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log probability) of one row of FP64 logits; (-1, nan) where nothing can be drawn."""
    z = np.asarray(z, np.float64)
    if np.isnan(z).any() or np.isnan([u, temperature, top_p, min_p]).any() or not np.isfinite(z.max()):
        return -1, np.nan
    order = np.lexsort((np.arange(len(z)), -z))       # logit descending, index ascending
    if temperature <= 0:
        return int(order[0]), 0.0
    with np.errstate(over="ignore", under="ignore"):
        w = np.exp((z[order] - z.max()) / np.float64(np.clip(temperature, 1e-30, 1e30)))
    w = w[:int((w > 0).sum())]
    if 0 < top_k < len(z):
        w = w[:top_k]
    c = np.cumsum(w)
    kept = len(w)
    if top_p < 1:
        kept = max(1, int((c - w < top_p * c[-1]).sum()))
    if min_p > 0:
        kept = min(kept, int((w >= min(min_p, 1.0)).sum()))
    at = min(int((c[:kept] <= max(u, 0.0) * c[kept - 1]).sum()), kept - 1)
    return int(order[at]), float(np.log(w[at] / c[kept - 1]))
