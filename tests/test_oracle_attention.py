"""Pins of the attention oracle, and of the host-side parts of the attention
operators (frequencies as 64-bit turns, pair axes), without a GPU."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from expert_layer_ptpc_gb300 import attention


# ---------------------------------------------------------------------------
# rotation
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("neighbours", [False, True])
def test_rotary_is_complex_multiplication(neighbours):
    rng = np.random.default_rng(3)
    T, H, D, n = 5, 3, 32, 8
    x = rng.standard_normal((T, H, D))
    pos = rng.integers(0, 1000, size=(3, T))
    axis = [0, 1, 2, 0, 1, 2, 0, 0]
    freq = 10000.0 ** (-np.arange(n) / n)
    y = oracle.rotary_ref(x, pos, freq, axis, neighbours)
    for i in range(n):
        lo, hi = (2 * i, 2 * i + 1) if neighbours else (i, i + n)
        z = (x[..., lo] + 1j * x[..., hi]) * np.exp(1j * pos[axis[i]] * freq[i])[:, None]
        np.testing.assert_allclose(y[..., lo], z.real, atol=1e-13)
        np.testing.assert_allclose(y[..., hi], z.imag, atol=1e-13)
    assert np.array_equal(y[..., 2 * n:], x[..., 2 * n:])
    back = oracle.rotary_ref(y, pos, freq, axis, neighbours, inverse=True)
    np.testing.assert_allclose(back, x, atol=1e-13)


def test_rotary_inverse_is_the_gradient():
    """The gradient of <g, rotate(x)> is the inverse rotation of g: against
    central differences, which are exact up to rounding for a linear map."""
    rng = np.random.default_rng(4)
    x, g = rng.standard_normal((2, 2, 1, 16))
    pos = np.array([[3, 70]])
    freq, axis = 100.0 ** (-np.arange(8) / 8), [0] * 8
    grad = oracle.rotary_ref(g, pos, freq, axis, inverse=True)
    h = 0.5
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        diff = ((g * oracle.rotary_ref(up, pos, freq, axis)).sum() -
                (g * oracle.rotary_ref(down, pos, freq, axis)).sum()) / (2 * h)
        assert abs(diff - grad[i]) < 1e-12


def _turns(freq):
    """attention.Rotary's fixed-point frequencies, on the CPU."""
    return attention.Rotary(torch.tensor(freq, dtype=torch.float64), device="cpu").turns


@pytest.mark.parametrize("base", [10000.0, 1000000.0, 5.0])
def test_turns_reduce_any_position_exactly(base):
    """position * turns modulo 2^64 is the angle modulo a turn, to 2^-31 turns,
    for positions up to 2^31 and for negative ones."""
    freq = attention.frequencies(32, base).tolist()
    turns = _turns(freq).tolist()
    # 2 pi to 70 digits, so that the check's own error is far below the bound
    two_pi = 2 * Fraction(
        "3.1415926535897932384626433832795028841971693993751058209749445923078164")
    for f, n in zip(freq, turns):
        for p in (0, 1, 12345, 1000003, 2 ** 31 - 1, -1, -2 ** 31):
            fixed = (p * n) % 2 ** 64
            exact = Fraction(p) * Fraction(f) / two_pi
            off = (Fraction(fixed, 2 ** 64) - exact) % 1
            off = min(off, 1 - off)
            # 2^31 positions times half a step of 2^-64, and the double
            # quotient's 2^-53 relative error
            assert off <= Fraction(1, 2 ** 31) * max(1, abs(exact) / 2 ** 21), (p, f)


def test_pair_axes():
    assert attention.pair_axes([2, 1, 1]) == [0, 0, 1, 2]
    assert attention.pair_axes([4, 2, 2], woven=True) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert attention.pair_axes([0, 3]) == [1, 1, 1]
    with pytest.raises(ValueError):
        attention.pair_axes([2, -1])


def test_rotary_plan_refusals():
    eight = torch.ones(8)
    for bad in (dict(inv_freq=torch.ones(7)), dict(inv_freq=torch.ones(0)),
                dict(inv_freq=torch.ones(2, 8)),
                dict(inv_freq=eight, pair_axis=[0] * 7),
                dict(inv_freq=eight, pair_axis=[0] * 7 + [3], axes=3),
                dict(inv_freq=eight, pair_axis=[-1] + [0] * 7),
                dict(inv_freq=eight, axes=9),
                dict(inv_freq=torch.full((8,), math.inf))):
        with pytest.raises(ValueError):
            attention.Rotary(device="cpu", **bad)


# ---------------------------------------------------------------------------
# cache and attention
# ---------------------------------------------------------------------------
def test_write_then_rows_gives_the_rows_back():
    rng = np.random.default_rng(5)
    pages = np.zeros((4, 2, 8, 16), np.uint8)
    scales = np.zeros((4, 2, 8), np.float32)
    x = rng.standard_normal((11, 2, 16)).astype(np.float32)
    order = rng.permutation(4)[:2]
    slots = np.array([order[t // 8] * 8 + t % 8 for t in range(11)])
    slots[3] = -1
    slots[7] = 4 * 8
    oracle.kv_write_ref(pages, scales, x, slots)
    back, there = oracle.cache_rows_ref(pages, scales, order, range(20))
    assert list(there) == [t < 16 for t in range(20)]
    for t in range(11):
        if t in (3, 7):
            assert np.all(back[t] == 0)
        else:   # e4m3: half a step of 3 mantissa bits, or of the smallest step
            step = np.maximum(np.abs(x[t]) / 16, scales[order[t // 8], :, t % 8][:, None] / 1024)
            assert np.all(np.abs(back[t] - x[t]) <= 1.001 * step)


@pytest.mark.parametrize("window", [0, 5])
def test_attention_matches_torch_dense(window):
    rng = np.random.default_rng(6)
    B, hq, hk, d, size = 3, 6, 2, 8, 4
    k = rng.standard_normal((10, hk, size, d))
    v = rng.standard_normal((10, hk, size, d))
    q = rng.standard_normal((B, hq, d))
    table = np.array([[3, 1, 7], [5, -1, 2], [0, 4, 6]])
    lengths = [9, 12, 0]
    out, lse, spread, _ = oracle.paged_attention_ref(q, k, v, None, None, table, lengths, 0.3,
                                                     window)
    for b in range(B):
        rows = [(table[b][t // size], t % size) for t in range(lengths[b])
                if table[b][t // size] >= 0 and (not window or t >= lengths[b] - window)]
        if not rows:
            assert np.all(out[b] == 0) and np.all(np.isneginf(lse[b]))
            continue
        kk = torch.tensor(np.stack([k[p, :, o] for p, o in rows])).repeat_interleave(3, 1)
        vv = torch.tensor(np.stack([v[p, :, o] for p, o in rows])).repeat_interleave(3, 1)
        s = torch.einsum("hd,nhd->hn", torch.tensor(q[b]), kk) * 0.3
        want = torch.einsum("hn,nhd->hd", torch.softmax(s, -1), vv)
        np.testing.assert_allclose(out[b], want.numpy(), atol=1e-13)
        np.testing.assert_allclose(lse[b], torch.logsumexp(s, -1).numpy(), atol=1e-13)
        assert np.all(spread[b] >= np.abs(out[b]) - 1e-13)
