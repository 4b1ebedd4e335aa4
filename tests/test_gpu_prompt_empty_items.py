"""Rows of prompt attention whose items have no tiles at all: the warp that hands out the work
writes them, and everything else runs on beside it."""

import numpy as np
import pytest
import torch

import oracle
from expert_layer_ptpc_gb300 import attention, binding
from tests.gpu_helpers import ensure_library, require_gpu
from tests.test_gpu_attention import assert_rotated, host, values, wide_heads
from tests.test_gpu_prompt_attention import KINDS, check_prompt, ints, page_cache, prompt_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    require_gpu()
    ensure_library()
    yield
    assert binding.moe_device_status() == (0, 0)     # no wait of any test ran out


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_runs_of_empty_contexts(kind, d):
    """More contexts of no tokens in a row than the ring holds segments, with rows of their own,
    at the start, in the middle and at the end."""
    lengths = [0] * 20 + [300, 5] + [0] * 50 + [700, 129] + [0] * 33 + [1, 64] + [0] * 18
    news = [1, 9, 3, 40] * 5 + [40, 5] + [2, 7] * 25 + [3, 129] + [1, 4, 90] * 11 + [1, 64] + [30] * 18
    cache, q, table = prompt_case(d, lengths, news, 6, 3, d, 16, kind, pad=2)
    check_prompt(cache, q, table, lengths, news, kind=kind)
    lengths = [-5 if n == 0 else n for n in lengths]
    check_prompt(cache, q, table, lengths, news, kind=kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_first_items_of_a_context_without_tiles(kind, d):
    """Far more new rows than tokens: the first items of every head have no tiles, one has rows of
    both kinds, and the last ones have tiles."""
    for lengths, news in (([40], [900]), ([40, 1, 300], [900, 700, 1000]), ([1], [600])):
        cache, q, table = prompt_case(d, lengths, news, 4, 2, d, 16, kind, pad=3)
        check_prompt(cache, q, table, lengths, news, kind=kind)
        check_prompt(cache, q, table, lengths, news, window=7, kind=kind)


def test_hundreds_of_empty_contexts_between_long_ones():
    rng = np.random.default_rng(1)
    lengths = sum(([int(rng.integers(1, 400))] + [0] * int(rng.integers(0, 90)) for _ in range(30)), [])
    news = [min(n, 20) if n else int(rng.integers(0, 30)) for n in lengths]
    assert len(lengths) > 640
    cache, q, table = prompt_case(2, lengths, news, 8, 2, 64, 16, "e4m3_page")
    check_prompt(cache, q, table, lengths, news, kind="e4m3_page")


# ---------------------------------------------------------------------------
# plan and write in the order of their stream
# ---------------------------------------------------------------------------
def test_another_stream_for_plan_and_write():
    """The plan and the pages that it leads to, written on a stream of the caller's, against
    the oracle."""
    rng = np.random.default_rng(2)
    stream = torch.cuda.Stream()
    pool = attention.PagePool.empty(9, 16, 2, 5)
    table, stack = pool.table.tolist(), pool.stack.tolist()
    cache = page_cache(rng, 9, 2, 16, 64)
    want = [t.copy() for t in host(cache)]
    k, v = wide_heads(rng, 30, 2, 2, d=64)
    new = ints([20, 9])
    torch.cuda.synchronize()
    plan = pool.plan(new, 30, stream=stream)
    cache.write(k, v, plan.slots, stream=stream)
    pool.commit(plan, stream=stream)
    stream.synchronize()
    offsets, slots, positions, after, refused = oracle.kv_plan_ref([0, 0, 9], [20, 9], table, stack,
                                                                   16, 30)
    assert plan.offsets.tolist() == offsets and plan.slots.tolist() == slots
    assert plan.positions.tolist() == [positions] and plan.refused.tolist() == [refused]
    assert pool.state.tolist() == after and pool.table.tolist() == table
    assert pool.stack.tolist() == stack
    for x, i in ((k, 0), (v, 1)):
        oracle.kv_write_page_ref(want[i], want[2 + i], values(x), np.array(slots, np.int32))
    for got, ref in zip(host(cache), want):
        assert np.array_equal(got, ref)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("rows", [7, 300])
def test_rotation_right_behind_its_positions(kind, captured, rows):
    """q, k and v rotated and written right behind the plan that makes their positions, step after
    step over the same memory: q and the values against the oracle."""
    rng = np.random.default_rng(rows)
    hq, hk, d, page, batch = 16, 2, 128, 16, 4
    pool = attention.PagePool.empty(400, page, batch, 200)
    cache = attention.PagedKVCache.empty(400, hk, page, d, dtype=kind)
    freq = attention.frequencies(d, 10000.0)
    axis = [i % 3 for i in range(d // 2)]
    rotary = attention.Rotary(freq, axis, axes=3)
    new = ints([0] * batch)
    q, k, v = wide_heads(rng, rows, hq, hk, hk, d=d)

    def step():
        plan = pool.plan(new, rows, axes=3)
        turned = cache.write_rotary(rotary, plan.positions, q, k, v, plan.slots)
        pool.commit(plan)
        return plan, turned

    step()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            made = step()
    held = [0] * batch
    for i in range(12):
        news = [int(n) for n in rng.multinomial(rows - 1, [1 / batch] * batch)]
        news = [-1 if i and (i + b) % 7 == 0 else n for b, n in enumerate(news)]
        new.copy_(ints(news))
        if captured:
            graph.replay()
            plan, turned = made
        else:
            plan, turned = step()
        at, positions = 0, np.zeros((3, rows), np.int64)
        for b, n in enumerate(news):
            m = max(n, 0)
            positions[:, at:at + m] = held[b] + np.arange(m)
            at, held[b] = at + m, 0 if n < 0 else held[b] + n
        assert np.array_equal(plan.positions.cpu().numpy(), positions)
        x = values(q)
        assert_rotated(turned, x, oracle.rotary_ref(x, positions, freq.numpy(), axis), d, False)
        _, vc = cache.read(pool.table, ints(np.concatenate([[0], np.cumsum(held)]).tolist()),
                           sum(held))
        ends = np.cumsum(held)
        at = 0
        for b, n in enumerate(news):     # the values that this step wrote
            m = max(n, 0)
            got, want = values(vc[ends[b] - m:ends[b]]), values(v)[at:at + m]
            tol = 0.0 if kind == "bf16" else 2.0 ** -3 * np.abs(want) + 2.0 ** -9 * np.abs(want).max(
                initial=0.0)
            assert np.all(np.abs(got - want) <= tol)
            at += m
