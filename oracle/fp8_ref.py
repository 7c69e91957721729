"""fp64 CPU oracle of the paged 8-bit caches (test infrastructure only, like
lsa_ref: the product never imports it and shares no code with it).

Plain numpy: the e4m3 rounding by a table of the format's 127 non-negative
values, the quantisation rule, the page plan as a loop over requests, and the
indexer and attention of one row over the values that the codes stand for.
"""
from __future__ import annotations

import numpy as np

from . import lsa_ref as R

PAGE, LAT, KEY = 64, 576, 128
LAT_ROW, KEY_PAGE = 592, 8448

# e4m3 (no infinities; 0x7f is NaN): exponent bias 7, three mantissa bits
E4M3 = np.array([m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def e4m3_codes(y: np.ndarray) -> np.ndarray:
    """Codes of |y| <= 448, nearest value, ties to the even code."""
    a = np.abs(y)
    hi = np.clip(np.searchsorted(E4M3, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = E4M3[hi] - a, a - E4M3[lo]
    take_lo = (dl < dh) | ((dl == dh) & (lo % 2 == 0))
    c = np.where(take_lo, lo, hi).astype(np.uint8)
    return c | (np.signbit(y).astype(np.uint8) << 7)


def e4m3_values(codes: np.ndarray) -> np.ndarray:
    v = E4M3[np.minimum(codes & 0x7F, 126)]
    return np.where(codes & 0x80, -v, v)


def quant(x: np.ndarray):
    """(codes uint8 [..., d], scale fp64 [...]) of fp64 vectors along the last axis."""
    with np.errstate(invalid="ignore"):
        a = np.max(np.abs(x), axis=-1)
    fin = np.isfinite(x).all(axis=-1)
    e = np.zeros(a.shape, dtype=np.int64)
    for i in np.ndindex(a.shape):
        if fin[i] and a[i] > 0:
            k = -126
            while a[i] > 448.0 * 2.0 ** k:  # the smallest power of two that covers the largest element
                k += 1
            e[i] = k
    s = 2.0 ** e
    y = np.where(fin[..., None], x, 0.0) / s[..., None]
    return e4m3_codes(y), np.where(fin, s, np.nan)


def dequant(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    return e4m3_values(codes) * scale[..., None]


def page_plan(cached, fresh, free_pages, table, cap):
    """The plan by one loop: (table, seq, pos, slot, totals)."""
    table = np.array(table, dtype=np.int64)
    n_seq, width = table.shape
    seq, pos, slot, taken, rows = [], [], [], 0, 0
    for s in range(n_seq):
        c, f = int(cached[s]), int(fresh[s])
        if c < 0 or f < 0 or c + f > width * PAGE:
            continue
        for col in range(-(-c // PAGE), -(-(c + f) // PAGE)):
            p = int(free_pages[taken]) if taken < len(free_pages) else -1
            table[s, col] = p if 0 <= p < 2 ** 25 - 1 else -1
            taken += 1
        for i in range(f):
            t = c + i
            p = int(table[s, t // PAGE])
            seq.append(s)
            pos.append(t)
            slot.append(p * PAGE + t % PAGE if 0 <= p < 2 ** 25 - 1 else -1)
        rows += f
    pad = [-1] * max(0, cap - rows)
    return table, (seq + pad)[:cap], (pos + pad)[:cap], (slot + pad)[:cap], [rows, taken]


def score_row(q, w, k_val, p, cfg: R.LsaConfig):
    """Scores of columns 0..p of one row: q bf16 values [32, 128], k_val the keys' values."""
    qc, qs = quant(q)
    s = R.score_row(np.nan_to_num(dequant(qc, np.nan_to_num(qs, nan=0.0))), w, k_val[: p + 1])
    return R.mask_and_force(s, p, p + 1, cfg)


def attend(q, c_val, keys, scale):
    """(out [32, 512], lse [32], weights [32, n]) over the listed keys of one row."""
    if len(keys) == 0:
        return np.zeros((q.shape[0], 512)), np.full(q.shape[0], -np.inf), np.zeros((q.shape[0], 0))
    c = c_val[np.asarray(keys)]
    x = scale * (q @ c.T)
    m = x.max(axis=1, keepdims=True)
    e = np.exp(x - m)
    tot = e.sum(axis=1, keepdims=True)
    return (e / tot) @ c[:, :512], (m + np.log(tot))[:, 0], e / tot
