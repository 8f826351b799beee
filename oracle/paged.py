"""fp64 oracle of rotary positions, the paged KV cache and decode over it.

Plain definitions in numpy, on the same 16-bit inputs widened exactly.  It
shares no code with the CUDA path; only tests import it.
"""
from __future__ import annotations

import numpy as np

from .attention import to_f64 as f64

TAU = np.longdouble("6.283185307179586476925286766559005768")


def angles(positions, freqs):
    """pos * freq reduced to one turn, from 64-bit-mantissa products (an fp64
    product of a position near 2^31 would be off by 2^-22 radians)."""
    a = np.asarray(positions).astype(np.longdouble)[..., None] * np.asarray(freqs, dtype=np.float64).astype(np.longdouble)
    return (a - TAU * np.rint(a / TAU)).astype(np.float64)


def rotate(x, positions, freqs, interleaved=False, amp=1.0, backward=False):
    """x [..., T, D] turned by positions [..., T] (broadcast over what is in front)."""
    x = f64(x)
    R = 2 * len(freqs)
    a = angles(positions, freqs)
    c, s = amp * np.cos(a), amp * np.sin(a) * (-1.0 if backward else 1.0)
    y = x.copy()
    first, second = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    u, w = x[..., first], x[..., second]
    y[..., first] = u * c - w * s
    y[..., second] = w * c + u * s
    return y


def packed_positions(cu, total):
    """Index of each packed row in its own sequence; -1 for rows of none."""
    pos = np.full(total, -1, dtype=np.int64)
    for a, b in zip(cu, cu[1:]):
        pos[a:b] = np.arange(b - a)
    return pos


def rows_of(pages, table_row, n):
    """The first n rows [Hkv, n, D] of the sequence whose pages the table row names."""
    pages = pages if isinstance(pages, np.ndarray) else f64(pages)
    page = pages.shape[2]
    return np.stack([pages[table_row[i // page], :, i % page] for i in range(n)], axis=1) if n else \
        np.zeros((pages.shape[1], 0, pages.shape[3]))


def decode_paged(q, k_pages, v_pages, table, lens, scale):
    """O [B, Hq, D], LSE [B, Hq], and what the comparison needs: the mean of
    |V| under the weights, and the largest sum of |q_i k_i| * scale of a row."""
    q, k_pages, v_pages = f64(q), f64(k_pages), f64(v_pages)
    B, Hq, D = q.shape
    G = Hq // k_pages.shape[1]
    o, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    mean_v, size = np.zeros((B, Hq, D)), np.zeros((B, Hq))
    for b in range(B):
        k, v = (rows_of(x, table[b], int(lens[b])) for x in (k_pages, v_pages))
        if k.shape[1] == 0:
            continue
        for h in range(Hq):
            kk, vv = k[h // G], v[h // G]
            s = kk @ q[b, h] * scale
            m = s.max()
            e = np.exp(s - m)
            o[b, h] = e @ vv / e.sum()
            lse[b, h] = m + np.log(e.sum())
            mean_v[b, h] = e @ np.abs(vv) / e.sum()
            size[b, h] = (np.abs(kk) @ np.abs(q[b, h])).max() * scale
    return o, lse, mean_v, size
