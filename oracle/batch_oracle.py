"""Independent fp64 NumPy model of the batched-request calls: block tables and
slot map from request lengths, the rotated cache write, and attention over a
shared prefix and each request's own keys.  Plain loops over requests, written
from the definitions in include/wf.h; test infrastructure only.
"""
from __future__ import annotations

import numpy as np


def tables(cached, fresh, prefix_len, page, free_pages, free_head, block_table, held=None):
    """(block_table, token_start, slot_map, positions, free_head_out, held_out) of one step."""
    table = [list(map(int, row)) for row in block_table]
    start, slots, positions, held_out = [0], [], [], []
    at = int(free_head)
    for b, (c, f) in enumerate(zip(cached, fresh)):
        have = -(-c // page) if held is None else held[b]
        need = max(have, -(-(c + f) // page))
        for i in range(have, need):
            table[b][i] = int(free_pages[at])
            at += 1
        held_out.append(need)
        for x in range(c, c + f):
            slots.append(table[b][x // page] * page + x % page)
            positions.append(prefix_len + x)
        start.append(start[-1] + f)
    return np.array(table), np.array(start), np.array(slots, dtype=np.int64), np.array(positions, dtype=np.int64), at, \
        np.array(held_out)


def rotate(x, cos_sin):
    """Rows x [T, H, D] turned by cos_sin [T, D/2, 2], interleaved pairs."""
    x = np.asarray(x, dtype=np.float64)
    c, s = (np.asarray(cos_sin, dtype=np.float64)[:, None, :, i] for i in (0, 1))
    out = np.empty_like(x)
    out[..., 0::2] = x[..., 0::2] * c - x[..., 1::2] * s
    out[..., 1::2] = x[..., 0::2] * s + x[..., 1::2] * c
    return out


def page_tokens(pages, n, page):
    return np.array([int(pages[i // page]) * page + i % page for i in range(n)], dtype=np.int64)


def attention(q, k_pool, v_pool, cached, fresh, prefix_len, block_table, prefix_table, page, block, scale=None):
    """dict of O, LSE and, for error bounds, per row: A = sum p |v| / sum p and
    Z = max over visible keys of scale * sum |q| |k|."""
    q, k_pool, v_pool = (np.asarray(a, dtype=np.float64) for a in (q, k_pool, v_pool))
    T, H, D = q.shape
    group = H // k_pool.shape[1]
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    out, mean_abs = np.zeros((T, H, D)), np.zeros((T, H, D))
    lse, size = np.zeros((H, T)), np.zeros((H, T))
    pre = page_tokens(prefix_table, prefix_len, page)
    t0 = 0
    for b, (c, f) in enumerate(zip(cached, fresh)):
        keys = np.concatenate([pre, page_tokens(block_table[b], c + f, page)])
        x = c + np.arange(f)
        seen = prefix_len + np.minimum(c + f, (x // block + 1) * block)
        hidden = np.arange(len(keys))[None, :] >= seen[:, None]
        for h in range(H):
            k, v = k_pool[keys, h // group], v_pool[keys, h // group]
            rows = q[t0:t0 + f, h]
            s = rows @ k.T * scale
            s[hidden] = -np.inf
            if f == 0:
                continue
            z = np.abs(rows) @ np.abs(k).T * scale
            z[hidden] = 0
            m = s.max(axis=1, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(axis=1, keepdims=True)
            out[t0:t0 + f, h] = p @ v / l
            mean_abs[t0:t0 + f, h] = p @ np.abs(v) / l
            lse[h, t0:t0 + f] = (m + np.log(l))[:, 0]
            size[h, t0:t0 + f] = z.max(axis=1)
        t0 += f
    return dict(O=out, LSE=lse, A=mean_abs, Z=size)
