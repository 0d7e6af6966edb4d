"""fp64 CPU oracle of the paged key/value cache calls: the norm and rotation of queries
and keys, 4-bit rows, rows in pages, and one query token over them.

TEST INFRASTRUCTURE ONLY, under the same rule as the rest of ``oracle/``: only
``tests/`` may use it; the HIP library never does.

Everything is written one head and one row at a time, from the definitions:

    n = x w / sqrt(mean(x^2) + eps)
    (n_a, n_b) <- (n_a cos u - n_b sin u, n_b cos u + n_a sin u),  u = t inv_freq[i]

for the pairs (i, i + R / 2), or (2 i, 2 i + 1); row r of a sequence is line r % P of
page table[r // P]; 64 values in 4 bits have a least value m = half(min) and a step
s = half((max - min) / 15), code = round((x - m) / s) and value = code s + m.
"""
from __future__ import annotations

import numpy as np

from .attention import attn

GROUP = 64


def turn(x, weight, eps, position, inv_freq, interleaved):
    """One head x [D], normed (unless weight is None) and rotated.  Returns (result, |n|:
    what the result is a rotation of, for error bounds)."""
    x = np.array(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean() + eps) * np.asarray(weight, dtype=np.float64)
    out, size = x.copy(), np.abs(x)
    half = 0 if inv_freq is None else len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        u = float(position) * float(inv_freq[i])
        out[a] = x[a] * np.cos(u) - x[b] * np.sin(u)
        out[b] = x[b] * np.cos(u) + x[a] * np.sin(u)
        size[a] = size[b] = np.abs(x[a]) + np.abs(x[b])
    return out, size


def turn_rows(x, weight, eps, positions, inv_freq, interleaved):
    """turn() of every head of x [T, H, D]."""
    out, size = np.empty(x.shape), np.empty(x.shape)
    for t in range(x.shape[0]):
        for h in range(x.shape[1]):
            out[t, h], size[t, h] = turn(x[t, h], weight, eps, positions[t] if inv_freq is not None else 0,
                                         inv_freq, interleaved)
    return out, size


def quantise(x):
    """64 values: (codes, step, least)."""
    x = np.asarray(x, dtype=np.float64)
    lo, hi = x.min(), x.max()
    with np.errstate(over="ignore", invalid="ignore"):
        least = float(np.float16(np.clip(lo, -65504, 65504)))
        step = float(np.float16(min((hi - lo) / 15, 65504)))
    code = np.clip(np.rint((x - least) / step), 0, 15) if step > 0 else np.zeros(len(x))   # (0 or NaN: 0)
    return code.astype(np.uint8), step, least


def store4(x):
    """A row [D] in 4 bits: (bytes [D / 2], scales [D / 64, 2] float16)."""
    codes, scales = [], []
    for g in range(0, len(x), GROUP):
        c, s, m = quantise(x[g:g + GROUP])
        codes.append(c)
        scales.append((s, m))
    c = np.concatenate(codes)
    return c[0::2] | (c[1::2] << 4), np.array(scales, dtype=np.float16)


def load4(codes, scales):
    """What bytes [.., D / 2] with scales [.., D / 64, 2] stand for."""
    c = np.empty(codes.shape[:-1] + (2 * codes.shape[-1],))
    c[..., 0::2], c[..., 1::2] = codes & 15, codes >> 4
    s = np.repeat(scales.astype(np.float64), GROUP, axis=-2)
    return c * s[..., 0] + s[..., 1]


def page_line(table, page_size, num_pages, row):
    """(page, line) of a row of a sequence with this table row, or None."""
    if row < 0 or row >= len(table) * page_size:
        return None
    page = int(table[row // page_size])
    return (page, row % page_size) if 0 <= page < num_pages else None


def rows_of(pages, table, first, n):
    """Rows first .. first + n - 1 [n, Hkv, D] of pages [N, Hkv, P, D] and which exist;
    the others are 0."""
    N, H, P, D = pages.shape
    out, there = np.zeros((n, H, D)), np.zeros(n, dtype=bool)
    for r in range(n):
        at = page_line(table, P, N, first + r)
        if at is not None:
            out[r], there[r] = pages[at[0], :, at[1]], True
    return out, there


def decode(q, k_pages, v_pages, table, length, scale):
    """One query token q [Hq, D] over rows 0 .. length.  Returns (o, sum p |v|, largest
    sum |scale q k| of a score), 0 for an unused slot or where no row exists."""
    if length < 0 or length >= len(table) * k_pages.shape[2]:
        return np.zeros(q.shape), np.zeros(q.shape), np.zeros((q.shape[0], 1))
    k, there = rows_of(k_pages, table, 0, length + 1)
    v, _ = rows_of(v_pages, table, 0, length + 1)
    o, ao, big = attn(q[None], k[there], v[there], scale)
    return o[0], ao[0], big[0]
