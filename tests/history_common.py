"""Helpers of the tests of the 4-bit history and the selected-block operators:
seeded bf16 inputs, caches on the device, and error bounds.

Bounds.  eps = 2^-8 is half a step of bf16.  The kernels round the
probabilities (times the V scale) to bf16 once, so |O - exact| is at most
eps * sum_j P_j |x_j|, x_j being what they multiply (v_j, or v_j - least_j for a
4-bit value), plus eps |O| where O is stored as bf16.  A logit is an fp32 sum of
d exact products and a few more operations: it is at most
(d + 16) 2^-23 scale sum_i |q_i y_i| off, y_i being the key's value (for a 4-bit
key (16 + c_i) s + |least|), and lse by at most the worst of that, a relative
2^-20 of the exponentials and of its own rounding.  The logits' error moves O by
that much relative to sum_j P_j |v_j - O|.
"""
from __future__ import annotations

import numpy as np

from oracle import history as OH

EPS = 2.0 ** -8


def bf16_round(x):
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7fff + ((u >> 16) & 1)) >> 16 << 16
    return u.astype(np.uint32).view(np.float32)


def up(x, device="cuda"):
    """fp32 numpy values that are bf16 -> a bf16 tensor."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).to(device)


def keys_values(rng, T, Hkv, d):
    K = bf16_round(rng.standard_normal((T, Hkv, d)) + 1.5 * rng.standard_normal((1, Hkv, d)))
    return K, bf16_round(rng.standard_normal((T, Hkv, d)))


def logit_bound(q, y, scale, d):
    """Largest possible error of the logits: q [rows, d], y [keys, d] >= 0."""
    if len(y) == 0:
        return 0.0
    return (d + 16) * 2.0 ** -23 * scale * float((np.abs(q) @ y.T).max())


def check(got_o, got_lse, o, lse, P, x, v, dS, bf16_out, what):
    """O [rows, d] and lse [rows] against the exact ones; P [rows, keys]."""
    empty = ~np.isfinite(lse)
    assert (got_lse[empty] == -np.inf).all() and (got_o[empty] == 0).all(), what
    if empty.all():
        return
    P, o, lse, got_o, got_lse = (a[~empty] for a in (P, o, lse, got_o, got_lse))
    assert np.isfinite(got_o).all() and np.isfinite(got_lse).all(), what
    tol = EPS * (P @ np.abs(x)) + 2 * (dS + 2.0 ** -20) * (P @ np.abs(v) + np.abs(o)) + 2.0 ** -20 * (P @ np.abs(v))
    if bf16_out:
        tol = tol + EPS * (np.abs(o) + tol)
    err = np.abs(got_o - o)
    assert (err <= tol).all(), (what, float((err - tol).max()), float(err.max()))
    # far below the bound on the whole: an error of many rows would show here
    # (the roundings are independent: their sum over keys is a random one)
    lerr = np.abs(got_lse - lse)
    assert (lerr <= dS + 2.0 ** -19 * (1 + np.abs(lse))).all(), (what, float(lerr.max()), dS)


class HostPages:
    """Pages filled on the host by the oracle's quantiser."""

    def __init__(self, n_pages, Hkv, d, fill=0):
        self.n_pages, self.Hkv, self.d = n_pages, Hkv, d
        self.data = np.full((n_pages, Hkv, OH.PAGE * (d + 8)), fill, np.uint8)

    def put(self, page, at, h, which, row):
        d, half = self.d, OH.PAGE * self.d // 2
        codes, s, lo = OH.quantize_row(row)
        p = self.data[page, h]
        p[which * half + at * d // 2:which * half + (at + 1) * d // 2] = codes[0::2] | (codes[1::2] << 4)
        off = 2 * half + which * OH.PAGE * 4 + at * 4
        meta = np.array([s, lo], np.float32)
        bits = OH.bf16_bits(meta) if np.isfinite(meta).all() else np.full(2, 0x7fff, np.uint16)
        p[off:off + 4] = bits.view(np.uint8)

    def get(self, page, h):
        """(k, v, ky, vx): values and what the bounds go by."""
        (kc, km), (vc, vm) = OH.unpack_page(self.data[page, h], self.d)
        k = kc * km[:, :1] + km[:, 1:]
        v = vc * vm[:, :1] + vm[:, 1:]
        return k, v, (16.0 + kc) * km[:, :1] + np.abs(km[:, 1:]), vc * vm[:, :1]
