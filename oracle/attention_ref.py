"""Plain fp64 reference of the attention operators: rotary positions with
several axes, the paged key-value cache and attention of one new token.

TEST INFRASTRUCTURE ONLY. Written from the definitions, token by token and
head by head, with explicit loops over contexts and pages.
"""

import numpy as np

from .fp8 import bf16_round, e4m3_decode
from .moe_ref import quant_rows_ref


def rotary_ref(x, positions, inv_freq, pair_axis, neighbours=False, inverse=False):
    """x [T, H, D] (values) rotated in fp64: pair i turns by
    positions[pair_axis[i], t] * inv_freq[i]."""
    x = np.asarray(x, np.float64)
    inv_freq = np.asarray(inv_freq, np.float64)
    pos = np.asarray(positions, np.float64)[np.asarray(pair_axis)]     # [pairs, T]
    angle = (pos * inv_freq[:, None]).T[:, None, :]                    # [T, 1, pairs]
    c, s = np.cos(angle), np.sin(angle) * (-1.0 if inverse else 1.0)
    n = len(inv_freq)
    first = np.arange(0, 2 * n, 2) if neighbours else np.arange(n)
    second = first + 1 if neighbours else first + n
    y = x.copy()
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    return y


def kv_write_ref(k_pages, scales, x, slots):
    """Store rows x [T, H, D] fp32 at `slots` into pages [P, H, page, D]: e4m3
    codes with `scales` [P, H, page], or bf16 values when scales is None. In
    place; slots outside the cache are skipped."""
    pages, heads, size, _ = k_pages.shape
    for t, slot in enumerate(np.asarray(slots).tolist()):
        if not 0 <= slot < pages * size:
            continue
        p, o = divmod(slot, size)
        if scales is None:
            k_pages[p, :, o] = bf16_round(x[t])
        else:
            k_pages[p, :, o], scales[p, :, o] = quant_rows_ref(x[t].astype(np.float32))


def cache_rows_ref(pages, scales, table, tokens):
    """Values [n, H, D] fp64 of a context's `tokens`, and which of them lie on
    a page of the cache (rows of the others are zero)."""
    count, heads, size, dim = pages.shape
    out = np.zeros((len(tokens), heads, dim))
    there = np.zeros(len(tokens), bool)
    for i, t in enumerate(tokens):
        entry = int(table[t // size]) if t // size < len(table) else -1
        if not 0 <= entry < count:
            continue
        there[i] = True
        row = pages[entry, :, t % size]
        if scales is None:
            out[i] = row
        else:
            out[i] = e4m3_decode(row) * scales[entry, :, t % size].astype(np.float64)[:, None]
    return out, there


def paged_attention_ref(q, k_pages, v_pages, k_scale, v_scale, table, lengths, scale, window=0):
    """(out [B, Hq, D], lse [B, Hq], spread [B, Hq, D], reach [B, Hq]) in fp64.
    spread = sum_j p_j |v_j| and reach = max_j scale sum_d |q_d k_jd| are what
    error bounds are relative to."""
    q = np.asarray(q, np.float64)
    B, hq, d = q.shape
    heads = k_pages.shape[1]
    group = hq // heads
    out, spread = np.zeros((B, hq, d)), np.zeros((B, hq, d))
    lse, reach = np.full((B, hq), -np.inf), np.zeros((B, hq))
    for b in range(B):
        n = int(lengths[b])
        tokens = range(max(0, n - window) if window > 0 else 0, max(n, 0))
        k, there = cache_rows_ref(k_pages, k_scale, table[b], tokens)
        v, _ = cache_rows_ref(v_pages, v_scale, table[b], tokens)
        k, v = k[there], v[there]
        if not len(k):
            continue
        for h in range(hq):
            kh, vh = k[:, h // group], v[:, h // group]
            s = scale * (kh @ q[b, h])
            m = s.max()
            e = np.exp(s - m)
            p = e / e.sum()
            out[b, h], spread[b, h] = p @ vh, p @ np.abs(vh)
            lse[b, h] = m + np.log(e.sum())
            reach[b, h] = abs(scale) * (np.abs(kh) @ np.abs(q[b, h])).max()
    return out, lse, spread, reach
