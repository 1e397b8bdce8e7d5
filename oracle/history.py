"""fp64 definitions of the paged 4-bit history (CPU, NumPy).

Shares no code with the library or the workloads: the page format, the
quantiser, the tables and the attention are written here from their
definitions, one request and one row at a time.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

PAGE = 64


def bf16_bits(x):
    """Bits of bf16-representable fp32 values."""
    return (np.asarray(x, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)


def bf16_value(bits):
    return (np.asarray(bits, dtype=np.uint32) << 16).view(np.float32).astype(np.float64)


def least_bf16_not_below(x) -> float:
    """The smallest bf16 value >= x (x >= 0; a float or a Fraction)."""
    f = np.float32(x)
    if float(f) < x:
        f = np.nextafter(f, np.float32(np.inf))
    u = int(f.view(np.uint32))
    u = (u + 0xffff) >> 16 << 16
    return float(np.uint32(u).view(np.float32))


def quantize_row(x):
    """(codes, scale, least) of one row of bf16 values given as float64."""
    x = np.asarray(x, dtype=np.float64)
    if not np.isfinite(x).all():
        return np.zeros(len(x), np.uint8), np.nan, np.nan
    lo, hi = x.min(), x.max()
    s = least_bf16_not_below((Fraction(float(hi)) - Fraction(float(lo))) / 15)
    if s == 0:
        return np.zeros(len(x), np.uint8), s, lo
    q = (x - lo) / s
    c = np.rint(q)
    # near the middle between two codes fp64 may not know the side
    for i in np.flatnonzero(np.abs(np.abs(q - c) - 0.5) < 1e-9):
        c[i] = round((Fraction(float(x[i])) - Fraction(float(lo))) / Fraction(float(s)))    # ties to even
    return c.astype(np.uint8), s, lo


def row_values(codes, scale, least):
    return codes.astype(np.float64) * scale + least


def unpack_page(page, d):
    """K and V codes [64, d] and (scale, least) [64, 2] each, of one page of one head (uint8)."""
    half = PAGE * d // 2
    out = []
    for which in range(2):
        raw = page[which * half:(which + 1) * half].reshape(PAGE, d // 2)
        codes = np.empty((PAGE, d), np.uint8)
        codes[:, 0::2], codes[:, 1::2] = raw & 15, raw >> 4
        at = 2 * half + which * PAGE * 4
        meta = bf16_value(page[at:at + PAGE * 4].copy().view(np.uint16).reshape(PAGE, 2))
        out.append((codes, meta))
    return out


def tables(ctx, new, free, table, max_tokens):
    """(table, kv_len, q_off, slot_map, pages_used, bad) after placing the new tokens."""
    table = np.array(table)
    R, width = table.shape
    kv, slots = [], np.full(max_tokens, -1, np.int64)
    off, at, used, bad, taken = [0], 0, 0, False, 0
    for r in range(R):
        c, n = max(int(ctx[r]), 0), max(int(new[r]), 0)
        ok = ctx[r] >= 0 and new[r] >= 0 and -(-(c + n) // PAGE) <= width
        have, need = -(-c // PAGE), -(-(c + n) // PAGE)
        extra = need - have if ok else 0
        fits = ok and (n == 0 or at + n <= max_tokens) and (extra == 0 or taken + extra <= len(free))
        if fits:
            for k in range(extra):
                table[r, have + k] = free[taken + k]
            for t in range(n):
                p = c + t
                slots[at + t] = table[r, p // PAGE] * PAGE + p % PAGE
            if extra:
                used = taken + extra
        else:
            bad = True
        kv.append(c + n if fits else min(c, width * PAGE))
        at += n
        taken += extra
        off.append(min(at, max_tokens))
    return table, np.array(kv), np.array(off), slots, used, bad


def attend_rows(q, k, v, scale):
    """O [d] and lse of each row of q over keys k, values v; 0 and -inf without keys."""
    if len(k) == 0:
        return np.zeros((len(q), v.shape[1])), np.full(len(q), -np.inf), np.zeros((len(q), 0))
    s = q @ k.T * scale
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(1, keepdims=True)
    return p / l @ v, (m + np.log(l))[:, 0], p / l


def summary(rows):
    """8-bit codes, scale and mean of the mean row of `rows` (float64)."""
    d = rows.shape[1]
    if len(rows) == 0:
        return np.zeros(d, np.int8), np.float32(0), np.zeros(d)
    s = np.zeros(d)
    for r in rows:
        s = s + r
    if not np.isfinite(s).all() or np.abs(s).max() == 0:
        return np.zeros(d, np.int8), np.float32(0), s / len(rows)
    top = np.abs(s).max()
    return np.rint(s * 127 / top).astype(np.int8), np.float32(top / (127 * len(rows))), s / len(rows)


def scores(q_codes, q_scale, k_codes, k_scale):
    """fp32 scores [n_k] of one query block: q_codes [G, d], k_codes [n_k, d]."""
    total = None
    with np.errstate(all="ignore"):
        for g in range(len(q_codes)):
            dot = k_codes.astype(np.int64) @ q_codes[g].astype(np.int64)
            part = np.float32(q_scale[g]) * dot.astype(np.float32)
            total = part if total is None else total + part
        return total * k_scale.astype(np.float32)


def choose(score, forced, k):
    """Ascending list: the forced entries, then the best others (ties to the lower index)."""
    n = len(score)
    forced = sorted(j for j in forced if 0 <= j < n)
    need = min(n, max(len(forced), k))
    rest = sorted((j for j in range(n) if j not in set(forced)), key=lambda j: (-float(score[j]), j))
    return sorted(forced + rest[:need - len(forced)])
