"""Plain fp64 reference of the attention operators: rotary positions with
several axes, the paged key-value cache, attention of one or many new tokens, and
the block tables and slot maps of a step.

TEST INFRASTRUCTURE ONLY. Written from the definitions, token by token and
head by head, with explicit loops over contexts and pages.
"""

import numpy as np

from .fp8 import bf16_round, e4m3_decode, e4m3_encode
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
            scale = scales[entry] if scales.ndim == 2 else scales[entry, :, t % size]
            out[i] = e4m3_decode(row) * scale.astype(np.float64)[:, None]
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


def page_scale_ref(amax):
    """The least power of two from 2^-48 on whose 448-fold is not below amax."""
    e = -48
    while 448.0 * 2.0 ** e < amax:
        e += 1
    return 2.0 ** e


def kv_write_page_ref(pages, scales, x, slots):
    """Store rows x [T, H, D] (values) at `slots` into codes [P, H, page, D] with one
    scale per page and head, scales [P, H]. In place; slots outside the cache are
    skipped."""
    count, heads, size, _ = pages.shape
    by_page = {}
    for t, slot in enumerate(np.asarray(slots).tolist()):
        if 0 <= slot < count * size:
            by_page.setdefault(slot // size, []).append((t, slot % size))
    for p, tokens in by_page.items():
        for h in range(heads):
            rows = x[[t for t, _ in tokens], h].astype(np.float64)
            scale = page_scale_ref(np.abs(rows).max())
            if all(o != 0 for _, o in tokens):
                was = float(scales[p, h])
                if scale > was:
                    pages[p, h] = e4m3_encode((e4m3_decode(pages[p, h]) * (was / scale))
                                              .astype(np.float32))
                scale = max(scale, was)
            scales[p, h] = scale
            for (_, o), row in zip(tokens, rows):
                pages[p, h, o] = e4m3_encode((row / scale).astype(np.float32))


def prompt_attention_ref(q, k_pages, v_pages, k_scale, v_scale, table, lengths, offsets, scale,
                         window=0):
    """(out, lse, spread, reach, mass): as of paged_attention_ref for the rows
    offsets[b]..offsets[b + 1] of q [rows, Hq, D], the last tokens of context b, and
    mass [rows, Hq, D] = max_j p_j sum_j |v_j|; rows behind the last are zeros."""
    q = np.asarray(q, np.float64)
    rows, hq, d = q.shape
    group = hq // k_pages.shape[1]
    out, spread, mass = (np.zeros((rows, hq, d)) for _ in range(3))
    lse, reach = np.full((rows, hq), -np.inf), np.zeros((rows, hq))
    for b, n in enumerate(lengths):
        s, e = int(offsets[b]), int(offsets[b + 1])
        if s == e or n <= 0:
            continue
        k, there = cache_rows_ref(k_pages, k_scale, table[b], range(n))
        v, _ = cache_rows_ref(v_pages, v_scale, table[b], range(n))
        at = n - (e - np.arange(s, e))[:, None]
        token = np.arange(n)
        seen = there & (token <= at)
        if window > 0:
            seen &= token > at - window
        for h in range(hq):
            kh, vh = k[:, h // group], v[:, h // group]
            x = np.where(seen, scale * (q[s:e, h] @ kh.T), -np.inf)
            m = x.max(-1)
            some = np.isfinite(m)
            w = np.exp(x[some] - m[some, None])
            p = w / w.sum(-1, keepdims=True)
            at_rows = np.arange(s, e)[some]
            out[at_rows, h], spread[at_rows, h] = p @ vh, p @ np.abs(vh)
            mass[at_rows, h] = p.max(-1, keepdims=True) * (seen[some] @ np.abs(vh))
            lse[at_rows, h] = m[some] + np.log(w.sum(-1))
            r = np.abs(scale) * (np.abs(q[s:e, h]) @ np.abs(kh).T)
            reach[s:e, h] = np.where(seen, r, 0.0).max(-1)
    return out, lse, spread, reach, mass


def kv_plan_ref(state, new, table, stack, page_size, rows):
    """One request after the other: (offsets, slots, positions, state, refused), with
    table and stack (lists) changed in place."""
    *held, count = state
    pages, wide = len(stack), len(table[0])
    free, after = list(stack[:count]), list(held)

    def pages_of(n):
        return -(-n // page_size)

    for b, n in enumerate(new):
        if n < 0:
            free += [p for p in table[b][:pages_of(held[b])] if 0 <= p < pages]
            after[b] = 0
    stack[:len(free)] = free
    offsets, slots, positions, refused, full = [0], [], [], 0, False
    for b, n in enumerate(new):
        fits = n >= 0 and held[b] >= 0 and held[b] + n <= wide * page_size
        if fits:
            need = pages_of(held[b] + n) - pages_of(held[b])
            full = full or need > len(free) or len(slots) + n > rows
        if fits and not full:
            for i in range(need):
                table[b][pages_of(held[b]) + i] = free.pop()
            for t in range(held[b], held[b] + n):
                p = table[b][t // page_size]
                slots.append(p * page_size + t % page_size if 0 <= p < pages else -1)
                positions.append(t)
            after[b] = held[b] + n
        elif n > 0:
            refused += 1
        offsets.append(len(slots))
    pad = rows - len(slots)
    return offsets, slots + [-1] * pad, positions + [0] * pad, after + [len(free)], refused
