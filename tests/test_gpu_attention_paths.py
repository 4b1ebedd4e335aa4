"""Paths of the attention operators that the sizes of test_gpu_attention.py do not
reach, with the same oracle, and calls from threads, streams and graphs.

The bounds are those of test_gpu_attention.py and, for an e4m3 cache, one more: the
weights go to the tensor cores in fp16 with the largest at 2^7 at least, so that a
weight's rounding is also off by up to half of fp16's smallest step, 2^-25, which is
2^-32 of the largest. (A weight is p_j times the value row's scale a_j.) It counts in an
element whose codes are zero in all tokens but such faint ones."""

import threading

import numpy as np
import pytest
import torch

import oracle
from expert_layer_ptpc_gb300 import binding
from tests import test_gpu_attention as base
from tests.gpu_helpers import U32, ensure_library, require_gpu
from tests.test_gpu_attention import (HALF_BF16, assert_rotated, attention_case,
                                      check_attention, fresh_cache, host, make_rotary,
                                      rotary_slack, values, wide_heads)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    require_gpu()
    ensure_library()


def on_gpu(lengths):
    return torch.tensor(lengths, dtype=torch.int32, device="cuda")


def faint(cache, q, table, lengths, window):
    """2^-32 max_j (p_j a_j) sum_j |c_j| of every output element of an e4m3 cache."""
    kc, vc, ks, vs = host(cache)
    if ks is None:
        return 0.0
    k, codes = (oracle.e4m3_decode(x) for x in (kc, vc))
    k *= ks.astype(np.float64)[..., None]
    x, size = values(q), kc.shape[2]
    group, out = x.shape[1] // kc.shape[1], np.zeros(x.shape)
    for b, n in enumerate(lengths):
        t = np.arange(max(0, n - window) if window else 0, n)
        entry = table[b, t // size]
        t, entry = t[(entry >= 0) & (entry < len(kc))] % size, entry[(entry >= 0) &
                                                                     (entry < len(kc))]
        for kv in range(kc.shape[1] if len(t) else 0):
            s = x[b, kv * group:(kv + 1) * group] @ k[entry, kv, t].T * x.shape[2] ** -0.5
            p = np.exp(s - s.max(1, keepdims=True))
            top = (p / p.sum(1, keepdims=True) * vs[entry, kv, t]).max(1)
            out[b, kv * group:(kv + 1) * group] = np.outer(
                top, np.abs(codes[entry, kv, t]).sum(0))
    return 2.0 ** -32 * out


def check(cache, q, table, lengths, window=0):
    """check_attention with the faint weights' rounding."""
    out, lse = cache.attend(q, torch.from_numpy(table).cuda(), on_gpu(lengths), window=window,
                            return_lse=True)
    d = q.shape[-1]
    kc, vc, ks, vs = host(cache)
    ref, ref_lse, spread, reach = oracle.paged_attention_ref(
        values(q), kc, vc, ks, vs, table, lengths, np.float32(d ** -0.5).astype(np.float64),
        window)
    n = np.minimum(np.array(lengths), window if window else 2 ** 31 - 1)[:, None]
    e = (2 * (d + 8) + 4) * U32 * reach
    rel = 2 * e + 2.0 ** -11 + 2 * n * U32
    got, got_lse = values(out), lse.cpu().numpy().astype(np.float64)
    tol = HALF_BF16 * np.abs(ref) + rel[..., None] * spread
    tol += faint(cache, q, table, lengths, window)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4], tol[bad][:4])
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(got_lse), empty) and np.all(got[empty] == 0)
    tol = (e + 2 * n * U32 + 4 * U32 * (1 + np.abs(np.where(empty, 0, ref_lse))))[~empty]
    assert np.all(np.abs(got_lse[~empty] - ref_lse[~empty]) <= tol)
    return out, lse


# ---------------------------------------------------------------------------
# the cut of the work
# ---------------------------------------------------------------------------
def cut_of(lengths, items, unit, workers, window=0):
    """The kernel's cut of a batch: how many items are shared by workers, and the most
    contexts (empty ones included) that one worker's run goes on past its first."""
    places, at, units_of = [], 0, []
    for n in lengths:
        begin = max(0, n - window) // 16 * 16 if window else 0
        units = -(-(n - begin) // unit) if n > 0 else 0
        units_of.append(units)
        places.append(at)
        at += (units + 2) * items if units else 0
    workers, places = min(workers, at), np.array(places + [at])
    ends = [at * w // workers for w in range(workers + 1)]
    cut = 0
    for e in ends[1:-1]:
        b = int(np.searchsorted(places, e, side="right")) - 1
        cut += (e - places[b]) % (units_of[b] + 2) > 2
    run = max(int(np.searchsorted(places, hi - 1, side="right")) -
              int(np.searchsorted(places, lo, side="right"))
              for lo, hi in zip(ends, ends[1:]))
    return cut, run


@pytest.mark.parametrize("hq,hk,d,kind,unit,workers", [
    (16, 4, 128, "e4m3", 128, 304), (16, 4, 64, "bf16", 128, 304), (32, 8, 64, "e4m3", 128, 456),
    (8, 4, 256, "bf16", 64, 152), (4, 4, 256, "e4m3", 64, 304), (80, 4, 128, "e4m3", 128, 304),
    (40, 2, 128, "bf16", 64, 304),
])
@pytest.mark.parametrize("window", [0, 700])
def test_attention_more_items_than_workers(hq, hk, d, kind, unit, workers, window):
    """Partial results by worker: more items than CTAs, many of them shared by two."""
    count = workers // hk * 5 // 4
    rng = np.random.default_rng(d + hq)
    lengths = [int(n) for n in rng.integers(0, 1500, size=count)]
    lengths[:6] = [0, 1, 1500, 0, unit, unit + 1]
    cut, _ = cut_of(lengths, hk, unit, workers, window)
    assert count * hk > workers and cut > 50
    cache, q, table = attention_case(hq + window, lengths, hq, hk, d, 16, kind)
    for b, n in enumerate(lengths):            # pages before the window are gone
        table[b, :max(0, n - window) // 16 if window else 0] = -1
    check(cache, q, table, lengths, window)


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
def test_attention_long_runs_of_empty_contexts(kind):
    """A worker's run that goes on past more contexts than it keeps the lengths of."""
    lengths = []
    for i in range(56):
        lengths += [1 + (7 * i + 3 * j) % 140 for j in range(40)] + [0] * 300
    _, run = cut_of(lengths, 1, 128, 456 if kind == "e4m3" else 304)
    assert run > 256
    cache, q, table = attention_case(91, lengths, 2, 1, 64, 16, kind)
    check(cache, q, table, lengths)


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
def test_attention_bad_contexts_that_share_workers_with_others(kind):
    """NaN in contexts of several units, cut and joined: in their rows alone."""
    lengths = [100 + 37 * b % 500 for b in range(400)]
    cut, _ = cut_of(lengths, 1, 128 if kind == "e4m3" else 64, 304)
    assert cut > 50
    cache, q, table = attention_case(92, lengths, 4, 1, 128, 16, kind)
    t, n = torch.from_numpy(table).cuda(), on_gpu(lengths)
    out, lse = check(cache, q, table, lengths)
    hurt = np.arange(0, 400, 7)
    pages = {int(table[b, 2]): b for b in hurt}
    for page in pages:
        for i, t_ in enumerate((cache.k, cache.v) if kind == "bf16" else
                               (cache.k_scale, cache.v_scale)):
            if page % 2 == i:
                t_[page, 0, 3] = float("nan")
    uses = np.isin(table, list(pages)) & (np.arange(table.shape[1]) * 16 + 3 <
                                         np.array(lengths)[:, None])
    hit = torch.from_numpy(uses.any(1)).cuda()
    assert 0 < int(hit.sum()) < 400
    o, l = cache.attend(q, t, n, return_lse=True)
    assert torch.equal(o[~hit], out[~hit]) and torch.equal(l[~hit], lse[~hit])
    assert bool(torch.isnan(o[hit].float()).any(-1).all())


# ---------------------------------------------------------------------------
# q's range
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("low", [-16, -18, -20])
def test_attention_q_of_many_sizes(low):
    """Elements of q down to 2^low of the head's largest, against an e4m3 cache whose
    keys make them count. They go to fp16 with the head's largest in [1, 2): below
    2^-17 of its power of two they are off by up to half of fp16's smallest step,
    2^-25 of that power."""
    rng = np.random.default_rng(-low)
    lengths = [300, 41]
    cache, q, table = attention_case(93, lengths, 8, 2, 128, 16, "e4m3")
    cache.k[..., 0] = 0                                # the largest element meets zeros
    small = np.exp2(rng.integers(low, low + 4, size=(2, 8, 127)).astype(np.float64))
    small *= rng.uniform(1, 1.99, small.shape) * rng.choice((-1, 1), small.shape)
    x = np.concatenate([np.full((2, 8, 1), 1.5), small], -1)
    top = np.exp2(rng.integers(-20, 20, size=(2, 8, 1)).astype(np.float64))
    q = torch.from_numpy(x * top).to(torch.bfloat16).cuda()
    kc, vc, ks, vs = host(cache)
    for scale in np.unique(top):       # heads of larger q are beyond any bound here
        s = 2.0 ** -low / scale / 32
        got, lse = cache.attend(q, torch.from_numpy(table).cuda(), on_gpu(lengths), scale=s,
                                return_lse=True)
        ref, ref_lse, spread, reach = oracle.paged_attention_ref(
            values(q), kc, vc, ks, vs, table, lengths, np.float32(s).astype(np.float64))
        most = np.abs(oracle.e4m3_decode(kc) * ks.astype(np.float64)[..., None]).sum(-1).max()
        lost = s * 2.0 ** -25 * top[..., 0] * most if low < -17 else 0.0
        n = np.array(lengths)[:, None]
        fine = top[..., 0] <= scale
        e = np.where(fine, (2 * (128 + 8) + 4) * U32 * reach + lost, 0.0)
        rel = 2 * e * np.exp(2 * e) + 2.0 ** -11 + 2 * n * U32
        tol = HALF_BF16 * np.abs(ref) + rel[..., None] * spread
        tol += 2.0 ** -32 * n[..., None] * np.abs(vs).max() * 448     # faint weights, see above
        assert np.all((np.abs(values(got) - ref) <= tol)[fine])
        tol = e + 2 * n * U32 + 4 * U32 * (1 + np.abs(ref_lse))
        assert np.all((np.abs(lse.cpu().numpy() - ref_lse) <= tol)[fine])


# ---------------------------------------------------------------------------
# rotation and cache write: warps that take several steps
# ---------------------------------------------------------------------------
def steps_of(T, heads, d):
    """Steps (of 512 elements) of a warp in the launcher's rule."""
    at_once = 32 // (d // 16)
    steps = -(-heads // at_once)
    most = min(steps, max(1, T * steps // (3 * 152 * 32), min(8, T * steps // (152 * 32))))
    parts = -(-steps // most)
    return -(-steps // parts)


def sample(rng, T):
    return np.unique(np.concatenate([[0, 1, T - 2, T - 1], rng.integers(0, T, size=400)]))


@pytest.mark.parametrize("T,hq,hk,d,rot,neighbours,inverse,steps", [
    (4099, 16, 2, 256, 64, True, True, 5), (2000, 64, 4, 128, 128, False, False, 6),
    (8192, 64, 4, 128, 96, False, True, 9), (16500, 64, 4, 64, 64, True, False, 9),
    (3001, 21, 5, 80, 48, False, False, 3), (700, 33, 3, 512, 256, True, False, 5),
])
def test_rotary_warps_of_several_steps(T, hq, hk, d, rot, neighbours, inverse, steps):
    assert steps_of(T, hq + hk, d) == steps
    rng = np.random.default_rng(T)
    q, k, _ = wide_heads(rng, T, hq, hk, 1, d=d)
    r, freq, axis, pos = make_rotary(rng, rot, 3, T, neighbours)
    p, at = torch.from_numpy(pos).cuda(), sample(rng, T)
    fresh = r.apply(p, q, k, inverse=inverse)
    for x, y in ((q, fresh[0]), (k, fresh[1])):
        want = oracle.rotary_ref(values(x[at]), pos[:, at], freq, axis, neighbours, inverse)
        assert_rotated(y[at], values(x[at]), want, rot, neighbours)
    r.apply(p, q, k, inverse=inverse, q_out=q, k_out=k)          # in place
    assert torch.equal(fresh[0], q) and torch.equal(fresh[1], k)


@pytest.mark.parametrize("T,hq,hk,d,rot,axes,neighbours,size,kind,steps", [
    (3000, 64, 4, 128, 128, 3, False, 64, "e4m3", 6), (2500, 40, 8, 64, 32, 2, True, 16, "e4m3", 3),
    (2100, 24, 3, 256, 256, 3, False, 8, "bf16", 5), (9000, 5, 1, 128, 64, 1, False, 32, "bf16", 2),
    (1100, 61, 2, 128, 128, 3, True, 16, "e4m3", 3),
])
def test_write_rotary_warps_of_several_steps(T, hq, hk, d, rot, axes, neighbours, size, kind,
                                             steps):
    assert steps_of(T, hq + 2 * hk, d) == steps
    base.test_write_rotary(T, hq, hk, d, rot, axes, neighbours, size, kind)


@pytest.mark.parametrize("T,heads,d,size,kind,steps", [
    (5000, 8, 128, 16, "e4m3", 4), (3000, 16, 64, 64, "bf16", 2), (3000, 7, 256, 8, "e4m3", 4),
])
def test_write_warps_of_several_steps(T, heads, d, size, kind, steps):
    assert steps_of(T, 2 * heads, d) == steps
    base.test_write_is_bit_exact(T, heads, d, size, kind)


# ---------------------------------------------------------------------------
# threads, streams, graphs
# ---------------------------------------------------------------------------
def test_threads_on_one_stream():
    """Threads that attend over one cache on one stream, each with contexts that are cut
    over many CTAs and joined: every call gives its own results."""
    cases = [attention_case(71, [5000, 300], 16, 2, 128, 16, "e4m3"),
             attention_case(72, [900, 0, 4100, 33, 2500], 32, 2, 128, 16, "e4m3")]
    cache = cases[0][0]
    cases[1][2][:] %= cache.pages
    lengths = ([5000, 300], [900, 0, 4100, 33, 2500])
    inputs = [(q, torch.from_numpy(table).cuda(), on_gpu(n))
              for (_, q, table), n in zip(cases, lengths)]
    want = [check_attention(cache, q, table, n) for (_, q, table), n in zip(cases, lengths)]
    stream = torch.cuda.current_stream()
    wrong, start = [], threading.Barrier(4)

    def serve(i):
        with torch.cuda.stream(stream):
            start.wait()
            for _ in range(300):
                out, lse = cache.attend(*inputs[i % 2], return_lse=True)
                if not (torch.equal(out, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])):
                    wrong.append(i)

    threads = [threading.Thread(target=serve, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("explicit", [False, True])
def test_a_captured_call_has_a_workspace_of_its_own(explicit):
    """A graph captured with the cache's own workspace, from the current stream or from
    one that the call names, replayed between and next to eager calls."""
    lengths = [3000, 0, 700]
    cache, q, table = attention_case(73, lengths, 16, 2, 128, 16, "e4m3")
    want = check_attention(cache, q, table, lengths)
    args = (q, torch.from_numpy(table).cuda(), on_gpu(lengths))
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    side = torch.cuda.Stream()
    kept = cache.workspace(3, 16, side)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    if explicit:
        with torch.cuda.stream(side):
            graph.capture_begin()
        assert cache.workspace(3, 16, side).data_ptr() != kept.data_ptr()
        cache.attend(*args, out=out, lse=lse, stream=side)
        with torch.cuda.stream(side):
            graph.capture_end()
    else:
        with torch.cuda.graph(graph, stream=side):
            cache.attend(*args, out=out, lse=lse)
    torch.cuda.synchronize()
    assert cache.workspace(3, 16, side) is kept
    for _ in range(20):
        out.zero_()
        lse.zero_()
        torch.cuda.synchronize()
        graph.replay()
        got = [cache.attend(*args, return_lse=True, stream=side) for _ in range(3)]
        torch.cuda.synchronize()
        for o, l in got + [(out, lse)]:
            assert torch.equal(o, want[0]) and torch.equal(l, want[1])


def test_caches_share_a_workspace_that_growing_batches_keep():
    """One buffer serves caches of other shapes and every batch size, with the results of
    a buffer of their own."""
    shapes = [([3000, 100], 16, 2, 128, "e4m3"), ([2000, 0, 900], 8, 2, 256, "bf16"),
              ([700] * 30, 40, 2, 64, "e4m3"), ([1500], 4, 4, 128, "bf16")]
    cases = [(attention_case(80 + i, n, hq, hk, d, 16, kind), n)
             for i, (n, hq, hk, d, kind) in enumerate(shapes)]
    want = [check_attention(*case, n) for case, n in cases]
    buffers = {(c.workspace(1, q.shape[1]).data_ptr()) for (c, q, _), _ in cases}
    assert len(buffers) == 1
    before = torch.cuda.memory_allocated()
    for (cache, q, _), _ in cases:
        for batch in range(1, 200, 7):
            cache.workspace(batch, q.shape[1])
    assert torch.cuda.memory_allocated() == before
    # one after the other on one stream, without a wait between them
    got = [c.attend(q, torch.from_numpy(t).cuda(), on_gpu(n), return_lse=True)
           for _ in range(3) for (c, q, t), n in cases]
    for (out, lse), (o, l) in zip(got, want * 3):
        assert torch.equal(out, o) and torch.equal(lse, l)


def test_lengths_that_change_under_a_call():
    """What a call then gives is not defined, but it stays in its buffers (joints that
    nobody wrote hold what the workspace held), and the next call is right."""
    lengths = [4000, 0, 2500, 700]
    cache, q, table = attention_case(97, lengths, 16, 2, 128, 16, "e4m3")
    want = check_attention(cache, q, table, lengths)
    t, n, full = torch.from_numpy(table).cuda(), on_gpu(lengths), on_gpu(lengths)
    need = binding.moe_paged_attention_workspace_size(cache.struct, 4, 16)
    ws = torch.full((need + 512,), 0x01, dtype=torch.uint8, device="cuda")
    outs = torch.full((3, 4, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    for _ in range(200):
        torch.cuda.synchronize()
        ws[256:256 + need] = 0x01
        n.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(4):
                n.copy_(full)
                n.zero_()
            n.copy_(full)
        cache.attend(q, t, n, out=outs[1], ws=ws[256:256 + need])
    torch.cuda.synchronize()
    assert bool((ws[:256] == 0x01).all()) and bool((ws[256 + need:] == 0x01).all())
    assert bool((outs[0] == 7).all()) and bool((outs[2] == 7).all())
    out, lse = cache.attend(q, t, n, return_lse=True, ws=ws[256:256 + need])
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_streams_that_overlap():
    """Calls of one cache in flight on two streams at once, of many CTAs each."""
    cases = [attention_case(95, [6000, 5000, 4000], 16, 2, 128, 16, "e4m3"),
             attention_case(96, [3000, 10, 7000], 32, 2, 128, 16, "e4m3")]
    lengths = ([6000, 5000, 4000], [3000, 10, 7000])
    cache = cases[0][0]
    cases[1][2][:] %= cache.pages
    want = [check_attention(cache, q, table, n) for (_, q, table), n in zip(cases, lengths)]
    inputs = [(q, torch.from_numpy(table).cuda(), on_gpu(n))
              for (_, q, table), n in zip(cases, lengths)]
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(100):
        for i, side in enumerate(sides):
            got[i].append(cache.attend(*inputs[i], return_lse=True, stream=side))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


@pytest.mark.parametrize("most", [24, 45])
def test_attention_value_scales_far_apart(most):
    """Scales of value rows from 2^-most to 2^most of the usual: each row's scale goes into
    its weight's exponent and out of the sum again."""
    lengths = [777, 60, 0, 1]
    cache, q, table = attention_case(98, lengths, 16, 2, 128, 16, "e4m3", 1.0, spread=0.3)
    cache.v_scale.mul_(torch.exp2(torch.randint(-most, most + 1, cache.v_scale.shape,
                                                device="cuda").float()))
    check(cache, q, table, lengths)
    # rows of zeros among them, as the cache write leaves them: the smallest scale
    zeros = torch.rand(cache.v_scale.shape, device="cuda") < 0.3
    cache.v[zeros] = 0
    cache.v_scale[zeros] = float(np.float32(1e-12) / np.float32(448))
    check(cache, q, table, lengths)
