"""FP64 oracle of the paged-cache operators: rotary positions, the append of new
K/V rows, and attention of new tokens by routes or by position.

Plain loops over rows and Python integers for every index, written from the
definitions in ``include/qsa.h`` and sharing no code with the CUDA library.
Attention comes with ``bound``, the elementwise error that the kernels'
roundings allow (see ``attend``).
"""

from __future__ import annotations

import math

import numpy as np

R = 12  # query heads per KV head


def rope(x, positions, inv_freq, *, interleaved=False, mscale=1.0, backward=False):
    """Rotary positions of x [T, heads, D]; backward turns the other way."""
    x = np.array(x, dtype=np.float64)
    y = x.copy()
    n = len(inv_freq)
    for t in range(x.shape[0]):
        for i in range(n):
            a = math.fmod(int(positions[t]) * float(inv_freq[i]), 2.0 * math.pi)
            c, s = math.cos(a) * mscale, math.sin(-a if backward else a) * mscale
            u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
            y[t, :, u] = x[t, :, u] * c - x[t, :, v] * s
            y[t, :, v] = x[t, :, u] * s + x[t, :, v] * c
    return y


def place(t, kv_len, cu_q):
    """(sequence, position) of packed row t, or None for a row of no sequence."""
    for b in range(len(kv_len)):
        if int(cu_q[b]) <= t < int(cu_q[b + 1]):
            return b, int(kv_len[b]) - (int(cu_q[b + 1]) - t)
    return None


def pool_row(j, b, block_table, page_size, n_pages):
    """Pool row of position j of sequence b, or None without one."""
    if j < 0 or j // page_size >= block_table.shape[1]:
        return None
    page = int(block_table[b, j // page_size])
    return page * page_size + j % page_size if 0 <= page < n_pages else None


def append(k_new, v_new, k_pages, v_pages, block_table, kv_len, cu_q):
    """The pools with the new rows written (k_new already rotated)."""
    n_pages, page_size, G, D = k_pages.shape
    k = np.array(k_pages, dtype=np.float64).reshape(-1, G, D)
    v = np.array(v_pages, dtype=np.float64).reshape(-1, G, D)
    for t in range(len(k_new)):
        at = place(t, kv_len, cu_q)
        row = None if at is None else pool_row(at[1], at[0], block_table, page_size, n_pages)
        if row is not None:
            k[row], v[row] = k_new[t], v_new[t]
    return k.reshape(k_pages.shape), v.reshape(v_pages.shape)


def route_set(ids, b, kv_len):
    """Positions that a row of route IDs names."""
    return sorted({int(r) for r in ids if 0 <= int(r) < int(kv_len[b])})


def causal_set(p, window, sinks, limit):
    """Positions below `limit` that a token at position p sees."""
    return [j for j in range(min(p + 1, limit)) if window == 0 or j > p - window or j < sinks]


def attend(q, k_pages, v_pages, block_table, kv_len, cu_q, scale, *, routes=None, window=0, sinks=0):
    """(out, lse, bound_out, bound_lse) [T, H, D] / [T, H]; rows of no sequence are NaN.

    The kernels take exact BF16 products summed in FP32 (an error of at most
    256 * 2^-24 of scale * sum |q||k| per score, and as much again for the
    exponent's argument), round each P to BF16 (2^-8 of it), sum in FP32 (one
    2^-24 per term) and round the output to BF16 once (2^-8).  So
      |out - exact| <= (2^-8 + 2 e + n 2^-23) sum p|v| + 2^-8 |out|,
      |lse - exact| <= e + n 2^-23 + 2^-22 (1 + |lse|),
    e the largest score error of the row."""
    T, H, D = q.shape
    n_pages, page_size, G, _ = k_pages.shape
    k, v = k_pages.reshape(-1, G, D), v_pages.reshape(-1, G, D)
    out, bound = np.full((T, H, D), np.nan), np.zeros((T, H, D))
    lse, bound_lse = np.full((T, H), np.nan), np.zeros((T, H))
    for t in range(T):
        at = place(t, kv_len, cu_q)
        if at is None:
            continue
        b, p = at
        if routes is not None:
            keys = route_set(routes[t], b, kv_len)
        else:
            keys = causal_set(p, window, sinks, block_table.shape[1] * page_size)
        rows = [r for r in (pool_row(j, b, block_table, page_size, n_pages) for j in keys) if r is not None]
        if not rows:
            out[t], lse[t] = 0.0, -np.inf
            continue
        for g in range(G):
            h = slice(g * R, (g + 1) * R)
            kk, vv = k[rows, g], v[rows, g]
            s = scale * (q[t, h] @ kk.T)
            e = 2.0 * 256 * 2.0**-24 * scale * (np.abs(q[t, h]) @ np.abs(kk).T).max(1)
            top = s.max(1, keepdims=True)
            w = np.exp(s - top)
            total = w.sum(1, keepdims=True)
            w = w / total
            out[t, h], lse[t, h] = w @ vv, (top + np.log(total))[:, 0]
            n = len(rows)
            bound[t, h] = (2.0**-8 + 2 * e[:, None] + n * 2.0**-23) * (w @ np.abs(vv)) + 2.0**-8 * np.abs(out[t, h])
            bound_lse[t, h] = e + n * 2.0**-23 + 2.0**-22 * (1 + np.abs(lse[t, h]))
    return out, lse, bound, bound_lse
