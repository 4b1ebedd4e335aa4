"""Paths of the operators around a step's attention that sizes alone do not reach:
captured graphs, streams, threads, workspaces, many contexts, rows that see nothing, and
offsets and lengths that a caller got wrong."""

import threading

import numpy as np
import pytest
import torch

from expert_layer_ptpc_gb300 import attention, binding
from tests.gpu_helpers import ensure_library, require_gpu
from tests.test_gpu_attention import scattered_table, wide_heads
from tests.test_gpu_prompt_attention import (KINDS, any_cache, check_prompt, ints, page_cache,
                                             prompt_case)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    require_gpu()
    ensure_library()
    yield
    assert binding.moe_device_status() == (0, 0)     # no wait of any test ran out


@pytest.mark.parametrize("kind", KINDS)
def test_many_contexts(kind):
    """More contexts than a CTA keeps at hand (256), and than it has threads (640)."""
    for batch, longest in ((300, 70), (900, 20)):
        rng = np.random.default_rng(batch)
        lengths = rng.integers(0, longest, size=batch).tolist()
        news = [int(rng.integers(0, n + 1)) for n in lengths]
        cache, q, table = prompt_case(batch, lengths, news, 4, 2, 64, 8, kind, pad=1)
        check_prompt(cache, q, table, lengths, news, kind=kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_runs_of_contexts_without_tokens(kind, d):
    """Long runs of rows that see nothing, between contexts of one tile and of many."""
    lengths = [5, 300, 1] + [9] * 120 + [200] + [3] * 40 + [129]
    news = [5, 40, 1] + [9] * 120 + [130] + [3] * 40 + [129]
    cache, q, table = prompt_case(d, lengths, news, 6, 3, d, 16, kind)
    table[3:123] = -1
    table[124:164] = cache.pages
    check_prompt(cache, q, table, lengths, news, kind=kind)


@pytest.mark.parametrize("group", [127, 128, 129, 300])
def test_large_groups(group):
    cache, q, table = prompt_case(group, [40, 9], [4, 9], group, 1, 64, 16, "e4m3_page")
    check_prompt(cache, q, table, [40, 9], [4, 9], kind="e4m3_page")


@pytest.mark.parametrize("kind", KINDS)
def test_one_row_over_a_long_context(kind):
    """A context cut over every CTA, against attention of one new token."""
    cache, q, table = prompt_case(5, [70001], [1], 4, 1, 128, 64, kind)
    t = torch.from_numpy(table).cuda()
    a = cache.attend(q, t, ints([70001]), return_lse=True)
    b = cache.attend_prompt(q, ints([0, 1]), t, ints([70001]), return_lse=True)
    # both within 2^-8 of the output's rounding and 2^-8 of a weight (bf16) of the same sums
    assert torch.allclose(a[0].float(), b[0].float(), rtol=2.0 ** -6, atol=2.0 ** -6 *
                          float(a[0].float().abs().max()))
    assert torch.allclose(a[1], b[1], rtol=1e-5, atol=1e-4)
    assert torch.equal(b[0], cache.attend_prompt(q, ints([0, 1]), t, ints([70001])))


@pytest.mark.parametrize("kind", KINDS)
def test_a_captured_step_follows_its_lengths(kind):
    """Plan, write, attention and the pool's new state in one graph: every replay hands out
    pages and attends to what came before, like the same calls without a graph."""
    batch, hq, hk, d, page, rows = 3, 4, 2, 64, 16, 12
    rng = np.random.default_rng(3)
    pools = [attention.PagePool.empty(40, page, batch, 12) for _ in range(2)]
    caches = [attention.PagedKVCache.empty(40, hk, page, d, dtype=kind) for _ in range(2)]
    rotary = attention.Rotary(attention.frequencies(d))
    new = ints([0, 0, 0])
    q, k, v = wide_heads(rng, rows, hq, hk, hk, d=d)

    def step(i):
        plan = pools[i].plan(new, rows)
        qo = caches[i].write_rotary(rotary, plan.positions, q, k, v, plan.slots)
        out = torch.zeros((rows, hq, d), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((rows, hq), device="cuda")
        caches[i].attend_prompt(qo, plan.offsets, pools[i].table, plan.lengths, out=out, lse=lse)
        pools[i].commit(plan)
        return out, lse, plan

    step(0)
    step(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse, plan = step(0)
    for counts in ([7, 1, 4], [1, 1, 1], [-1, 9, 1], [5, 0, -1], [1, 1, 10]):
        new.copy_(ints(counts))
        q.copy_(torch.randn(q.shape, device="cuda"))
        k.copy_(torch.randn(k.shape, device="cuda"))
        graph.replay()
        want = step(1)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        assert torch.equal(pools[0].state, pools[1].state)
        assert torch.equal(pools[0].table, pools[1].table)
        assert torch.equal(plan.slots, want[2].slots)


def test_two_graphs_on_two_streams():
    """Each captured call has a workspace of its own."""
    made = []
    for seed in (1, 2):
        cache, q, table = prompt_case(seed, [9000], [40], 8, 1, 128, 64, "e4m3_page")
        t, n, o = torch.from_numpy(table).cuda(), ints([9000]), ints([0, 40])
        want = cache.attend_prompt(q, o, t, n).clone()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph):
            out = cache.attend_prompt(q, o, t, n)
        made.append((graph, stream, out, want, cache, q, t, n, o))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream, *_ in made:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, out, want, *_ in made:
        assert torch.equal(out, want)


def test_streams_and_threads():
    cache, q, table = prompt_case(8, [5000, 700], [30, 90], 8, 2, 128, 32, "bf16")
    t, n, o = torch.from_numpy(table).cuda(), ints([5000, 700]), ints([0, 30, 120])
    want = cache.attend_prompt(q, o, t, n)
    torch.cuda.synchronize()
    outs, errors = [], []

    def work(stream):
        try:
            for _ in range(10):
                outs.append(cache.attend_prompt(q, o, t, n, stream=stream))
        except Exception as e:   # noqa: BLE001 (shown below)
            errors.append(e)

    shared = torch.cuda.Stream()
    threads = [threading.Thread(target=work, args=(s,))
               for s in (shared, shared, torch.cuda.Stream(), torch.cuda.Stream())]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    torch.cuda.synchronize()
    assert not errors and len(outs) == 40
    for x in outs:
        assert torch.equal(x, want)


def test_another_stream_for_plan_write_and_commit():
    rng = np.random.default_rng(2)
    stream = torch.cuda.Stream()
    pool = attention.PagePool.empty(9, 16, 2, 5)
    cache = page_cache(rng, 9, 2, 16, 64)
    before = [x.clone() for x in (cache.k, cache.k_scale)]
    k, v = wide_heads(rng, 30, 2, 2, d=64)
    new = ints([20, 9])
    torch.cuda.synchronize()
    plan = pool.plan(new, 30, stream=stream)
    cache.write(k, v, plan.slots, stream=stream)
    pool.commit(plan, stream=stream)
    stream.synchronize()
    assert pool.state.tolist() == [20, 9, 6]
    cache.k.copy_(before[0])
    cache.k_scale.copy_(before[1])
    got = cache.k.clone()
    cache.write(k, v, plan.slots)
    assert not torch.equal(cache.k, got)


def test_workspaces():
    cache, q, table = prompt_case(9, [9000, 30], [50, 30], 4, 1, 64, 64, "e4m3")
    t, n, o = torch.from_numpy(table).cuda(), ints([9000, 30]), ints([0, 50, 80])
    want = cache.attend_prompt(q, o, t, n, return_lse=True)
    need = binding.moe_prompt_attention_workspace_size(cache.struct, 4)
    for fill in (0, 0x7f, 0xff):
        wide = torch.full((need + 512,), fill, dtype=torch.uint8, device="cuda")
        got = cache.attend_prompt(q, o, t, n, return_lse=True, ws=wide[256:256 + need])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.all(wide[:256] == fill) and torch.all(wide[256 + need:] == fill)
    with pytest.raises(binding.MoeError):
        cache.attend_prompt(q, o, t, n, ws=wide[:need - 1])
    with pytest.raises(ValueError):
        cache.attend_prompt(q, o, t, n, ws=wide[::2])


@pytest.mark.parametrize("offsets", [
    [0, 100, 50, 120], [-5, 60, 80, 120], [0, 60, 80, 5000], [7, 7, 7, 7], [120, 60, 0, -9],
    [2 ** 31 - 1, -2 ** 31, 0, 5], [3, 50, 90, 110],
])
@pytest.mark.parametrize("kind,d", [("e4m3_page", 128), ("bf16", 256)])
def test_wrong_offsets_stay_inside_the_outputs(offsets, kind, d):
    """Contexts whose rows run backwards or past the tensors have none."""
    lengths = [200, 80, 40]
    cache, q, table = prompt_case(4, lengths, [60, 20, 40], 4, 2, d, 16, kind)
    guard = torch.full((3 * 120, 4, d), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3, 120, 4), 3.0, device="cuda")
    cache.attend_prompt(q, ints(offsets), torch.from_numpy(table).cuda(), ints(lengths),
                        out=guard[120:240], lse=lse[1])
    assert torch.all(guard[:120] == 3.0) and torch.all(guard[240:] == 3.0)
    assert torch.all(lse[0] == 3.0) and torch.all(lse[2] == 3.0)


@pytest.mark.parametrize("lengths", [[-1, -2 ** 31, 5], [2 ** 31 - 1, 100, 100], [0, 0, 0]])
def test_wrong_lengths(lengths):
    """Negative lengths are none; what a length has past its table is absent."""
    cache, q, table = prompt_case(4, [100, 100, 100], [20, 30, 40], 4, 2, 64, 16, "e4m3_page")
    out, lse = cache.attend_prompt(q, ints([0, 20, 50, 90]), torch.from_numpy(table).cuda(),
                                   ints(lengths), return_lse=True)
    assert torch.isfinite(out.float()).all()
    for b, (s, e) in enumerate(((0, 20), (20, 50), (50, 90))):
        if lengths[b] <= 0:
            assert torch.all(out[s:e] == 0) and torch.all(torch.isneginf(lse[s:e]))
        elif lengths[b] > 10 ** 6:        # the rows lie far past the table: all of it is seen
            assert torch.all(torch.isfinite(lse[s:e]))


def test_pages_shared_by_contexts():
    """A prefix that two requests share, in the same pages."""
    rng = np.random.default_rng(6)
    cache = any_cache(rng, 20, 2, 16, 128, "e4m3_page")
    table = scattered_table(rng, 3, 6, 20)
    table[1, :3] = table[0, :3]
    table[2] = table[0]
    lengths, news = [90, 70, 90], [10, 22, 90]
    q = torch.from_numpy(rng.standard_normal((sum(news), 8, 128)).astype(np.float32))
    check_prompt(cache, q.to(torch.bfloat16).cuda(), table, lengths, news, kind="e4m3_page")


def test_tensors_elsewhere_refused():
    cache, q, table = prompt_case(4, [70], [70], 6, 3, 64, 8, "bf16")
    t, n, o = torch.from_numpy(table).cuda(), ints([70]), ints([0, 70])
    good = dict(q=q, offsets=o, block_table=t, lengths=n)
    for bad in (dict(q=q.float()), dict(q=q[:, :5]), dict(q=q.cpu()), dict(offsets=o.long()),
                dict(offsets=o.cpu()), dict(offsets=ints([0, 1, 2])), dict(block_table=t.cpu()),
                dict(block_table=t.t()), dict(lengths=n.float()), dict(window=2 ** 31),
                dict(out=q[:5]), dict(out=q.float()), dict(out=q), dict(lse=torch.zeros(70, 6)),
                dict(lse=torch.zeros((70, 5), device="cuda"))):
        with pytest.raises((ValueError, binding.MoeError)):
            cache.attend_prompt(**{**good, **bad})
    with pytest.raises(binding.MoeError):
        cache.attend_prompt(**good, window=-1)
    pool = attention.PagePool.empty(4, 16, 2, 3)
    for bad in (dict(new_tokens=ints([1])), dict(new_tokens=ints([1, 1]).long()),
                dict(new_tokens=ints([1, 1]).cpu()), dict(rows=-1), dict(axes=0), dict(axes=9)):
        with pytest.raises(ValueError):
            pool.plan(**{**dict(new_tokens=ints([1, 1]), rows=4), **bad})


def test_decoder_example_with_page_scales():
    import importlib.util
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location(
        "decoder_step", os.path.join(root, "examples", "decoder_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # both sides round to bf16 (half a step is 2^-8 of the value); the contexts
    # read back are rounded to bf16 too
    worst = example.main(["--steps", "3", "--batch", "6", "--prompt", "333", "--cache",
                          "e4m3_page"])
    assert worst <= 2 * 2.0 ** -8


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,lengths,news,window", [
    (16, [5000, 700, 0, 3333], [5, 8, 0, 1], 0), (1, [5121], [128], 0), (3, [6000, 64], [43, 1], 0),
    (64, [4000], [2], 1500), (20, [9000, 2500], [6, 6], 2000),
])
def test_few_rows_over_long_contexts(kind, d, group, lengths, news, window):
    """Items of up to 128 rows that are cut: the halves of a CTA take every other tile, and
    their pieces are joined; pages absent in the middle and at an end, rows that see nothing."""
    cache, q, table = prompt_case(group, lengths, news, 2 * group, 2, d, 32, kind)
    check_prompt(cache, q, table, lengths, news, window=window, kind=kind)
    table[0, 20:60] = -1
    table[-1, :9] = cache.pages
    check_prompt(cache, q, table, lengths, news, window=window, kind=kind)
    table[0] = -1
    check_prompt(cache, q, table, lengths, news, window=window, kind=kind)
