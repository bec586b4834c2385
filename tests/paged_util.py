"""Plain reference of the paged 8-bit cache operators, on the host in 64 bits.

Written from the definitions in ``include/dsa.h``, one sequence, page and query
after the other; it shares no code with the library.
"""
import math

import numpy as np

LATENT = 512
E_MIN, E_MAX = -110, 119
TOP = {"e4m3": 448.0, "s8": 127.0}


def e4m3_values():
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3
    mantissa bits; exponent 0 subnormal, 0x7f and 0xff NaN, no infinities."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        if (c & 0x7F) == 0x7F:
            x = math.nan
        v[c] = -x if c & 0x80 else x
    return v


_E4M3 = e4m3_values()
_E4M3_POS = _E4M3[:0x7F]                    # 0 .. 448, ascending


def decode(codes, fmt):
    codes = np.asarray(codes, dtype=np.uint8)
    return _E4M3[codes] if fmt == "e4m3" else codes.view(np.int8).astype(np.float64)


def encode(x, fmt):
    """Round to nearest, ties to even, +-top beyond it; NaN as the header says."""
    x = np.asarray(x, dtype=np.float64)
    nan = np.isnan(x)
    a = np.minimum(np.where(nan, 0.0, np.abs(x)), TOP[fmt])
    neg = np.signbit(x)
    if fmt == "s8":
        return np.where(nan, 0, np.where(neg, -1, 1) * np.rint(a)).astype(np.int8).view(np.uint8)
    hi = np.searchsorted(_E4M3_POS, a)      # first code at or above a
    lo = np.maximum(hi - 1, 0)
    d_hi, d_lo = _E4M3_POS[hi] - a, a - _E4M3_POS[lo]
    up = (d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0))
    c = np.where(up, hi, lo)
    c = np.where(nan, 0x7F, c) | (neg.astype(np.int64) << 7)
    return c.astype(np.uint8)


def exponent(amax, fmt):
    if amax == 0.0:
        return E_MIN
    m, k = math.frexp(amax / TOP[fmt])      # exact enough: equality only at amax = top 2^k
    return min(max(k - 1 if m == 0.5 else k, E_MIN), E_MAX)


def parts(width):
    return [(0, LATENT)] + ([(LATENT, width)] if width > LATENT else [])


def widen(codes, scales, fmt):
    """Pool rows as float64 [n_pages, page_rows, W]."""
    out = decode(codes, fmt)
    for i, (a, b) in enumerate(parts(codes.shape[-1])):
        f = np.exp2(scales[:, i].astype(np.float64) - 127)
        f[scales[:, i] == 255] = math.nan
        out[..., a:b] *= f[:, None, None]
    return out


def pages_for(n, page):
    return -(-n // page)


def plan(page, held, kv, q, free, n_free, table, max_new):
    """(table, free, n_free, row_off, q_off, slots, enough) of dsa_page_plan."""
    table, free = table.copy(), free.copy()
    stack = list(free[:n_free])
    n = len(kv)
    row_off, q_off = np.concatenate([[0], np.cumsum(kv)]), np.concatenate([[0], np.cumsum(q)])
    slots = np.full(max_new, -1, dtype=np.int64)
    grow = sum(max(pages_for(kv[s], page) - pages_for(held[s], page), 0) for s in range(n))
    back = sum(max(pages_for(held[s], page) - pages_for(kv[s], page), 0) for s in range(n))
    if grow > n_free + back:
        return table, free, n_free, row_off, q_off, slots, False
    for s in range(n):
        for c in range(pages_for(kv[s], page), pages_for(held[s], page)):
            stack.append(table[s, c])
    for s in range(n):
        for c in range(pages_for(held[s], page), pages_for(kv[s], page)):
            table[s, c] = stack.pop()
    for i in range(n_free, len(stack)):
        free[i] = stack[i]
    for s in range(n):
        for i in range(q[s]):
            pos = kv[s] - q[s] + i
            if q_off[s] + i < max_new:
                slots[q_off[s] + i] = int(table[s, pos // page]) * page + pos % page
    return table, free, len(stack), row_off, q_off, slots, True


def append(page, kv, q, rows, slots, codes, scales, fmt):
    """(codes, scales) after dsa_cache_append; rows float64 [tokens, W]."""
    codes, scales = codes.copy(), scales.copy()
    t0 = 0
    for s in range(len(kv)):
        t = 0
        while t < q[s]:
            off = (kv[s] - q[s] + t) % page
            end = min(q[s], t + page - off)
            slot = int(slots[t0 + t])
            if slot >= 0:
                p = slot // page
                new = rows[t0 + t:t0 + end]
                for i, (a, b) in enumerate(parts(rows.shape[1])):
                    x = np.abs(new[:, a:b])
                    e = exponent(float(np.where(np.isfinite(x), x, 0).max()), fmt)
                    if off > 0:
                        e_old = int(scales[p, i]) - 127
                        e = max(e, e_old)
                        if e > e_old:
                            moved = decode(codes[p, :off, a:b], fmt) * 2.0 ** (e_old - e)
                            codes[p, :off, a:b] = encode(moved, fmt)
                    scales[p, i] = e + 127
                    codes[p, off:off + end - t, a:b] = encode(new[:, a:b] / 2.0 ** e, fmt)
            t = end
        t0 += q[s]
    return codes, scales


def attention(q_abs, rows, at, scale, unit=None):
    """(out [H, 512], lse [H], weight [H, 512], reach, floor [H, 512]) of one query
    over rows[at]: weight = sum_j p_j |row_j|, reach = max_hj scale sum_c |q_hc
    row_jc|, floor = max_j (p_j unit_j) sum_j |row_j| / unit_j with unit the rows'
    latent scales (0 without them)."""
    H = q_abs.shape[0]
    if len(at) == 0:
        z = np.zeros((H, LATENT))
        return z, np.full(H, -np.inf), z, 0.0, z
    r = rows[at]
    z = scale * q_abs @ r.T
    m = z.max(1, keepdims=True)
    p = np.exp(z - m)
    tot = p.sum(1, keepdims=True)
    p /= tot
    floor = np.zeros((H, LATENT))
    if unit is not None:
        u = unit[at]
        floor = (p * u).max(1)[:, None] * (np.abs(r[:, :LATENT]) / u[:, None]).sum(0)
    return (p @ r[:, :LATENT], (m + np.log(tot))[:, 0], p @ np.abs(r[:, :LATENT]),
            float((scale * np.abs(q_abs) @ np.abs(r).T).max()), floor)


def attention_bounds(dtype, width, n_rows, weight, reach, lse, floor):
    """Element-wise bounds of the library's error.

    A logit is a float32 sum of W products, |error| <= W 2^-23 sum|q r| scale
    (half of that with rounding, all of it where the tensor cores truncate);
    the exponential adds 2^-21 and, through the float32 argument, 2^-23 of it.
    With bf16 queries a row's weight w = p 2^e is carried as hi + lo in f16:
    each is off by half a step, 2^-11 * 2^-11 = 2^-22 of w, but by no less than
    half of f16's smallest step, 2^-25, where w is relative to a running maximum
    that is at most the largest w; times the row's codes, |row| / 2^e, that is
    2^-25 of `floor`.  The output's numerator and denominator each take the
    relative error per weight, and the float32 sums over the rows n 2^-23 of the
    sum of magnitudes."""
    logit = width * 2.0 ** -23 * reach
    per_weight = logit + 2.0 ** -21 + 2.0 ** -23 * reach + (2.0 ** -22 if dtype == "bf16" else 0.0)
    rel = 2 * per_weight + (n_rows + 2) * 2.0 ** -23
    finite = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    least = 2.0 ** -25 * floor if dtype == "bf16" else 0.0
    return (rel * weight + least + 1e-37,
            logit + per_weight + n_rows * 2.0 ** -23 + 2.0 ** -22 * (finite + 1))
