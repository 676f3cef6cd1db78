"""Plain 64-bit implementations of the attention operators, for the tests
(numpy; written from the formulas of include/scaled_attention.h)."""
import math

import numpy as np


def e4m3_values():
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = np.nan if (c & 127) == 127 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v[c] = -x if c & 128 else x
    return v


E4M3 = e4m3_values()
POSITIVE = E4M3[:127]


def e4m3_round(x):
    """Codes of the nearest e4m3 values (ties to even, saturated, NaN stays NaN)."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0, x)), 448.0)
    hi = np.clip(np.searchsorted(POSITIVE, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = POSITIVE[hi] - a, a - POSITIVE[lo]
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 0x7F, code)
    return (code | (np.signbit(x) & ~np.isnan(x)) * 0x80).astype(np.uint8)


def pow2(code):
    return np.where(np.asarray(code) == 255, np.nan, 2.0 ** (np.asarray(code, np.float64) - 127))


def rotate(x, cs, inter):
    """x [n, heads, d] fp32, cs [n, 2, rot/2] fp32: the fp32 steps of the header, one rounding each."""
    y = x.copy()
    h = cs.shape[2]
    lo, hi = (np.arange(0, 2 * h, 2), np.arange(1, 2 * h, 2)) if inter else (np.arange(h), np.arange(h, 2 * h))
    c, s = cs[:, None, 0], cs[:, None, 1]
    with np.errstate(invalid="ignore", over="ignore"):
        y[..., lo] = x[..., lo] * c - x[..., hi] * s
        y[..., hi] = x[..., lo] * s + x[..., hi] * c
    assert y.dtype == np.float32
    return y


def scale_code(amax):
    """e8m0 code of the least 2^e with amax <= 448 2^e, by trying them."""
    if not amax > 0:
        return 0
    amax = min(float(amax), float(np.finfo(np.float32).max))
    e = math.floor(math.log2(amax / 448.0)) - 1
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return min(max(e + 127, 0), 254)


def append(q, k, v, codes, scales, table, ctx, cu, rot, inter):
    """Arrays in fp32; codes / scales (k, v) uint8, updated in place.  Returns rotated q, k."""
    pages, hk, page, d = codes[0].shape
    q, k = q.copy(), k.copy()
    for b in range(len(ctx)):
        t0, n, c0 = cu[b], cu[b + 1] - cu[b], max(int(ctx[b]), 0)
        if rot is not None and n:
            cs = rot[np.minimum(c0 + np.arange(n), len(rot) - 1)]
            q[t0:t0 + n] = rotate(q[t0:t0 + n], cs, inter)
            k[t0:t0 + n] = rotate(k[t0:t0 + n], cs, inter)
        for p0 in range(c0 // 16 * 16, c0 + n, 16):
            lo, hi = max(p0, c0), min(p0 + 16, c0 + n)
            pg = table[b, p0 // page] if p0 // page < table.shape[1] else -1
            if pg < 0 or pg >= pages:
                continue
            s0 = p0 % page
            for x, cod, sca in ((k, codes[0], scales[0]), (v, codes[1], scales[1])):
                for h in range(hk):
                    part = x[t0 + lo - c0:t0 + hi - c0, h].astype(np.float64)
                    a = np.abs(part)
                    code = scale_code(np.max(np.where(np.isnan(a), 0, a), initial=0))
                    if lo > p0:
                        was = min(int(sca[pg, h, s0 // 16]), 254)
                        code = max(code, was)
                        if code > was:
                            held = E4M3[cod[pg, h, s0:s0 + lo - p0]]
                            cod[pg, h, s0:s0 + lo - p0] = e4m3_round(held * 2.0 ** (was - code))
                    sca[pg, h, s0 // 16] = code
                    cod[pg, h, s0 + lo - p0:s0 + hi - p0] = e4m3_round(part * 2.0 ** (127 - code))
    return q, k


def attend(q, k, v, see, scale):
    """q [n, Hq, D], k, v [m, Hk, D] (64 bits), see [n]: keys that row i sees (the first see[i]), or a
    boolean [n, m].  Returns out, lse, and per element sum_j w_j |v_j| and per row max_j scale sum |q k|."""
    n, hq, d = q.shape
    m, hk = k.shape[:2]
    vis = see if getattr(see, "ndim", 1) == 2 else np.arange(m)[None, :] < np.asarray(see)[:, None]
    out, mag = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    lse, big = np.full((n, hq), -np.inf), np.zeros((n, hq))
    for h in range(hq):
        for i in range(n):
            j = np.flatnonzero(vis[i])
            if not len(j):
                continue
            kk, vv = k[j, h // (hq // hk)], v[j, h // (hq // hk)]
            s = kk @ q[i, h] * scale
            big[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
            top = s.max()
            w = np.exp(s - top)
            lse[i, h] = top + np.log(w.sum())
            w /= w.sum()
            out[i, h], mag[i, h] = w @ vv, w @ np.abs(vv)
    return out, lse, mag, big


def cached(codes, scales, pages, hk, page, n):
    """The first n tokens of a sequence, [n, Hk, D] in 64 bits, and whether each has a page."""
    toks, has = [], []
    for j in range(n):
        pg = pages[j // page] if j // page < len(pages) else -1
        ok = 0 <= pg < codes.shape[0]
        has.append(ok)
        s = j % page
        toks.append(E4M3[codes[pg, :, s]] * pow2(scales[pg, :, s // 16])[:, None] if ok else np.zeros((hk, codes.shape[3])))
    return np.array(toks).reshape(n, hk, codes.shape[3]), np.array(has, bool)


# Tolerances.  bf16 output: half a unit in the last place is at most 2^-8 |o|.
# The weights e^(s - m) enter the product with v rounded to `bits` significant bits
# (bf16: 8, so each is off by at most 2^-8 of itself; fp16: 11), which moves o by at most
# that fraction of sum w |v|; fp32 scores, exponentials and sums add at most 2^-13
# of it (scores of up to 2^7 with relative errors of 2^-22, twice).
def out_tolerance(out, mag, bits):
    return 2.0 ** -8 * np.abs(out) + (2.0 ** -bits + 2.0 ** -13) * mag + 1e-30


# A score of D <= 128 products summed in fp32 in any order, each step off by at most 2^-23 of the
# largest partial sum (|q| . |k|), 16 steps deep, twice that for the scaling; the logarithm adds as much again.
def lse_tolerance(lse, big):
    return 2.0 ** -18 * (1 + big + np.abs(np.where(np.isfinite(lse), lse, 0)))
