"""Parity of the operators around a step's attention with the fp64 oracle, through
the public classes: block tables and slot maps, the cache with one scale per page and
head (written, read, attended to by one token), and attention of many new tokens.

Bounds, with u = 2^-24 (fp32) and half a bf16 step = 2^-8 of the value:
* plans, and writes of unrotated rows: bit for bit.
* attention of many tokens: a score errs by at most e = (D + 8) 2 u scale sum|q k| (the
  tensor cores' fp32 sums may truncate: 2 u a step) plus 4 u |s| (scalings,
  exponential); an e4m3 cache's q is off by up to 2^-25 of its head's largest element,
  times sum |k|: within 2^-25 D of reach's largest when keys' elements are of like size,
  counted as 2^-18 reach; a weight by 2 e in the ratio of the sums. The weights'
  rounding to fp16 (e4m3 caches) is off by 2^-11, to bf16 (bf16 caches) by 2^-8; a value's
  to fp16 by 2^-11 where its scale is no power of two; the sum over n tokens by 2 n u.
  All these are relative to sum_j p_j |v_j|; then the output's rounding. fp16 weights below
  its normal numbers are off by up to half of 2^-24, where the row's largest weight is at
  least 2^7 (the bound is set 7 below a tile's largest, and moves when a later one
  passes it by 15): 2^-32 of the largest, of each token's value."""

import numpy as np
import pytest
import torch

import oracle
from expert_layer_ptpc_gb300 import attention
from tests.gpu_helpers import U32, ensure_library, require_gpu
from tests.test_gpu_attention import (HALF_BF16, assert_rotated, check_attention, host, make_rotary,
                                      rotary_slack, scattered_table, values, wide_heads)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    require_gpu()
    ensure_library()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# block tables and slot maps
# ---------------------------------------------------------------------------
def random_pool(rng, batch, longest, page, spare):
    held = rng.integers(0, longest + 1, size=batch).tolist()
    wide = -(-longest // page) + 2
    count = [-(-h // page) for h in held]
    pages = sum(count) + spare
    order = rng.permutation(pages).tolist()
    table, at = [], 0
    for c in count:
        table.append(order[at:at + c] + [-1] * (wide - c))
        at += c
    free = order[at:]
    return table, free + [-7] * (pages - len(free)), held + [len(free)]


def check_plan(table, stack, state, new, page, rows, axes=1):
    t, s = ints(table), ints(stack)
    pool = attention.PagePool.from_tensors(t, s, ints(state), page)
    plans = [pool.plan(ints(new), rows, axes=axes) for _ in range(2)]   # (it can be repeated)
    want_table, want_stack = [list(r) for r in table], list(stack)
    offsets, slots, positions, after, refused = oracle.kv_plan_ref(state, new, want_table,
                                                                   want_stack, page, rows)
    for p in plans:
        assert p.offsets.tolist() == offsets
        assert p.slots.tolist() == slots
        assert p.positions.tolist() == [positions] * axes
        assert p.state.tolist() == after and p.lengths.tolist() == after[:-1]
        assert p.refused.tolist() == [refused]
    assert t.tolist() == want_table and s.tolist() == want_stack
    return pool, plans[0]


@pytest.mark.parametrize("batch,longest,page,new,rows,spare,axes", [
    (1, 0, 16, [1], 1, 1, 1), (1, 5, 1, [3], 3, 3, 1), (3, 40, 16, [1, 1, 1], 4, 3, 3),
    (5, 100, 8, [0, -1, 30, -1, 2], 32, 9, 1), (4, 64, 64, [64, 0, 1, 63], 128, 4, 8),
    (40, 200, 16, None, 40, 40, 1), (300, 300, 16, None, 300, 7, 3), (33, 50, 32, None, 0, 5, 1),
    (600, 20, 8, None, 900, 2000, 1), (4096, 9, 4, None, 4096, 4096, 1),
])
def test_plan(batch, longest, page, new, rows, spare, axes):
    rng = np.random.default_rng(batch + longest)
    table, stack, state = random_pool(rng, batch, longest, page, spare)
    if new is None:
        new = rng.choice([-1, 0, 1, 1, 2, 5], size=batch).tolist()
    check_plan(table, stack, state, new, page, rows, axes)


def test_plan_long_prompts_and_refusals():
    rng = np.random.default_rng(5)
    table, stack, state = random_pool(rng, 6, 3000, 16, 700)
    for row in table:
        row += [-1] * 400
    check_plan(table, stack, state, [4000, -1, 700, 1, 2000, 16], 16, 9000, 2)
    check_plan(table, stack, state, [4000, -1, 700, 1, 2000, 16], 16, 4701, 2)    # rows run out
    check_plan(table, stack, state, [4000, 0, 0, 9000, 2000, 1], 16, 20000)       # pages run out
    check_plan(table, stack, state, [1, 2 ** 31 - 1, 3, 10 ** 6, 0, 1], 16, 64)   # past the table


def test_plan_keeps_to_the_cache_when_the_pool_is_damaged():
    """Entries that are no pages, on the stack and in tables, counts past the stack."""
    table = [[3, -1, 9, 2], [1, 5, -1, -1], [-1, 70000, 0, -1]]
    check_plan(table, [4, -3, 6, 99, 0, 0, 0, 0], [10, 5, 9, 4], [-1, 9, 1], 4, 16)
    check_plan(table, [4, 7, 6, 1, 0, 0, 0, 0], [16, -5, 0, 4], [-1, 1, 13], 4, 16)
    t, s = ints(table), ints([4, 7, 6, 1, 0, 0, 0, 0])
    pool = attention.PagePool.from_tensors(t, s, ints([16, 8, 0, 900]), 4)
    p = pool.plan(ints([-1, 1, 13]), 16)
    assert p.state.tolist()[-1] <= 8 and p.slots.max().item() < 32 and p.slots.min().item() >= -1
    pool = attention.PagePool.from_tensors(t, s, ints([16, 8, 0, -4]), 4)
    p = pool.plan(ints([0, 1, 13]), 16)
    assert p.refused.tolist() == [2] and p.slots.tolist() == [-1] * 16


def test_pool_over_many_steps():
    """Requests come, grow and leave; no page has two owners and none is lost."""
    rng = np.random.default_rng(9)
    pool = attention.PagePool.empty(50, 8, 7, 20)
    for step in range(60):
        held = pool.state.tolist()[:-1]
        new = [int(rng.choice([-1, 0, 1, 3, 17])) if h else int(rng.integers(0, 40))
               for h in held]
        plan = pool.plan(ints(new), 200)
        pool.commit(plan)
        *held, free = pool.state.tolist()
        used = [p for row, h in zip(pool.table.tolist(), held) for p in row[:-(-h // 8)]]
        assert sorted(used + pool.stack.tolist()[:free]) == list(range(50))


# ---------------------------------------------------------------------------
# the cache with one scale per page and head
# ---------------------------------------------------------------------------
def page_cache(rng, pages, heads, size, d, spread=1.0):
    """A cache of codes over the whole range, every page with a scale of its own."""
    c = attention.PagedKVCache.empty(pages, heads, size, d, dtype="e4m3_page")
    for name in ("k", "v"):
        x = torch.from_numpy(rng.standard_normal((pages, heads, size, d)).astype(np.float32))
        x = x * torch.from_numpy(np.exp(spread * rng.standard_normal((pages, heads, size, 1)))
                                 .astype(np.float32))
        amax = x.abs().amax((-1, -2)).double().numpy()
        s = torch.from_numpy(np.vectorize(oracle.page_scale_ref)(amax).astype(np.float32))
        t = getattr(c, name)
        t.copy_((x / s[..., None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
                .view(torch.uint8))
        getattr(c, name + "_scale").copy_(s)
    return c


def run_slots(rng, pages, size, runs):
    """Slots of runs (first offset, tokens) on pages of their own, in shuffled order
    inside a run when it is short, with skipped tokens behind some runs."""
    slots, order = [], rng.permutation(pages)
    at = 0
    for i, (first, n) in enumerate(runs):
        while n > 0:
            m = min(n, size - first)
            run = (order[at] * size + first + np.arange(m)).tolist()
            if m < 5:
                rng.shuffle(run)
            slots += run
            at, n, first = at + 1, n - m, 0
        if i % 3 == 1:
            slots += [-1, pages * size]
    return np.array(slots, np.int32)


RUNS = [
    (1, 128, 64, [(0, 1)]), (4, 64, 16, [(3, 1), (0, 40), (15, 2)]),
    (3, 256, 8, [(0, 8), (7, 1), (1, 30), (0, 2), (4, 4)]), (2, 128, 1, [(0, 5), (0, 3)]),
    (8, 128, 64, [(0, 200), (63, 66), (5, 1), (10, 54)]), (5, 64, 1024, [(0, 700), (1000, 300)]),
    (1, 256, 128, [(1, 127), (0, 128), (64, 64)]), (2, 128, 16, [(i % 16, 3) for i in range(90)]),
]


@pytest.mark.parametrize("heads,d,size,runs", RUNS)
def test_page_write_is_bit_exact(heads, d, size, runs):
    rng = np.random.default_rng(d + size)
    pages = sum(-(-(f + n) // size) for f, n in runs) + 2
    cache = page_cache(rng, pages, heads, size, d)
    slots = run_slots(rng, pages, size, runs)
    want = [t.copy() for t in host(cache)]
    for step in range(2):          # the second call brings larger values to pages in use
        k, v = wide_heads(rng, len(slots), heads, heads, d=d)
        k *= torch.exp(3 * torch.randn((len(slots), heads, 1), device="cuda")).to(torch.bfloat16)
        v *= 2.0 ** (5 * step)
        v[0, 0] = 0
        cache.write(k, v, torch.from_numpy(slots).cuda())
        for x, i in ((k, 0), (v, 1)):
            oracle.kv_write_page_ref(want[i], want[2 + i], values(x), slots)
        for got, ref in zip(host(cache), want):
            assert np.array_equal(got, ref)
        last = slots[slots >= 0][-1]                       # one more token behind the last
        slots = np.array([last + 1 if (last + 1) % size else last], np.int32)


def test_page_write_at_the_borders_of_scales():
    """Maxima at and next to 448 times a power of two, tiny and huge ones, zeros."""
    tops = [448.0, 446.0, 450.0, 1.75, 1.7421875, 1.7578125, 2.0 ** -40, 2.0 ** -46, 2.0 ** -60,
            2.0 ** -126, 0.0, 2.0 ** 100, 1.75 * 2.0 ** 120, 2.0 ** 127, 3.0e38]
    n, d, size = len(tops), 64, 4
    cache = attention.PagedKVCache.empty(n, 1, size, d, dtype="e4m3_page")
    x = torch.linspace(-1, 1, d).repeat(n, 1) * torch.tensor(tops)[:, None]
    k = x.to(torch.bfloat16).view(n, 1, d).cuda()
    slots = np.arange(0, n * size, size, dtype=np.int32)
    want = [t.copy() for t in host(cache)]
    cache.write(k, -k, torch.from_numpy(slots).cuda())
    for y, i in ((k, 0), (-k, 1)):
        oracle.kv_write_page_ref(want[i], want[2 + i], values(y), slots)
    for got, ref in zip(host(cache)[2:], want[2:]):
        assert np.array_equal(got, ref)
    for got, ref in zip(host(cache)[:2], want[:2]):
        assert np.array_equal(got[:, :, 0], ref[:, :, 0])


@pytest.mark.parametrize("hq,hk,d,rot,axes,neighbours,size,runs", [
    (64, 4, 128, 128, 3, False, 64, [(5, 1), (63, 2), (0, 1)]),
    (5, 1, 256, 64, 3, True, 8, [(0, 21), (3, 5)]), (12, 3, 64, 64, 2, False, 16, [(9, 40)]),
    (8, 4, 64, 32, 1, False, 16, [(0, 16), (1, 20)]), (16, 2, 128, 128, 3, True, 32, [(31, 80)]),
])
def test_page_write_rotary(hq, hk, d, rot, axes, neighbours, size, runs):
    rng = np.random.default_rng(hq + d)
    pages = sum(-(-(f + n) // size) for f, n in runs) + 2
    cache = page_cache(rng, pages, hk, size, d)
    slots = run_slots(rng, pages, size, runs)
    T = len(slots)
    q, k, v = wide_heads(rng, T, hq, hk, hk, d=d)
    r, freq, axis, pos = make_rotary(rng, rot, axes, T, neighbours)
    before = [t.copy() for t in host(cache)]
    qo = cache.write_rotary(r, torch.from_numpy(pos).cuda(), q, k, v,
                            torch.from_numpy(slots).cuda())
    assert_rotated(qo, values(q), oracle.rotary_ref(values(q), pos, freq, axis, neighbours), rot,
                   neighbours)
    kc, vc, ks, vs = host(cache)
    oracle.kv_write_page_ref(before[1], before[3], values(v), slots)
    assert np.array_equal(vc, before[1]) and np.array_equal(vs, before[3])
    # keys: rows that were rotated in fp64, under the scales that the maxima ask for
    y = oracle.rotary_ref(values(k), pos, freq, axis, neighbours)
    oracle.kv_write_page_ref(before[0], before[2], y, slots)
    assert np.array_equal(ks, before[2])
    slack = 2.0 ** -20 * rotary_slack(values(k), rot, neighbours).max()
    live = {int(s): t for t, s in enumerate(slots) if 0 <= s < pages * size}
    for s, t in live.items():
        p, o = divmod(s, size)
        scale = ks[p].astype(np.float64)[:, None]
        got = oracle.e4m3_decode(kc[p, :, o]) * scale
        tol = np.maximum(2.0 ** -4 * np.abs(y[t]), 2.0 ** -10 * scale)
        assert np.all(np.abs(got - y[t]) <= 1.001 * tol + 2 * slack)
    rest = np.ones(pages * size, bool)
    rest[list(live)] = False
    rest = rest.reshape(pages, size)
    assert np.array_equal(kc.transpose(0, 2, 1, 3)[rest], before[0].transpose(0, 2, 1, 3)[rest])


@pytest.mark.parametrize("lengths,hq,hk,d,size", [
    ([1], 1, 1, 64, 16), ([300, 0, 17], 64, 4, 128, 64), ([127, 128, 129, 257], 6, 2, 64, 4),
    ([1000, 3, 0, 77], 20, 1, 256, 128), ([9000], 16, 2, 128, 64), ([700] * 9, 20, 1, 128, 16),
])
@pytest.mark.parametrize("window", [0, 33])
def test_attention_of_one_token_over_page_scales(lengths, hq, hk, d, size, window):
    rng = np.random.default_rng(sum(lengths) + d)
    wide = -(-max(lengths) // size)
    cache = page_cache(rng, len(lengths) * wide + 2, hk, size, d)
    q = torch.from_numpy((1.5 * rng.standard_normal((len(lengths), hq, d))).astype(np.float32))
    table = scattered_table(rng, len(lengths), wide, cache.pages)
    check_attention(cache, q.to(torch.bfloat16).cuda(), table, lengths, window=window)


def test_read_of_page_scales():
    rng = np.random.default_rng(4)
    lengths, size = [40, 0, 17, 1], 8
    cache = page_cache(rng, 25, 3, size, 128)
    table = scattered_table(rng, 4, 5, 25)
    offsets = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    got = cache.read(torch.from_numpy(table).cuda(), torch.from_numpy(offsets).cuda(), 60)
    kc, vc, ks, vs = host(cache)
    for y, codes, scales in zip(got, (kc, vc), (ks, vs)):
        want = np.zeros((60, 3, 128))
        for b, n in enumerate(lengths):
            want[offsets[b]:offsets[b + 1]], _ = oracle.cache_rows_ref(codes, scales, table[b],
                                                                      range(n))
        assert np.array_equal(values(y), oracle.bf16_round(want))


# ---------------------------------------------------------------------------
# attention of many new tokens
# ---------------------------------------------------------------------------
def any_cache(rng, pages, heads, size, d, kind, spread=1.0):
    if kind == "e4m3_page":
        return page_cache(rng, pages, heads, size, d, spread)
    from tests.test_gpu_attention import filled_cache
    return filled_cache(rng, pages, heads, size, d, kind, spread)


def check_prompt(cache, q, table, lengths, news, scale=None, window=0, pad=0, kind="e4m3",
                 ranges=None, **kw):
    offsets = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    rows, hq, d = q.shape
    out = torch.full((rows, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, hq), 7.0, device="cuda")
    got = cache.attend_prompt(q, torch.from_numpy(offsets).cuda(), torch.from_numpy(table).cuda(),
                              ints(lengths), scale=scale, window=window, out=out, lse=lse, **kw)
    assert got[0] is out and got[1] is lse
    scale = d ** -0.5 if scale is None else scale
    kc, vc, ks, vs = host(cache)
    ref, ref_lse, spread, reach, mass = oracle.prompt_attention_ref(
        values(q), kc, vc, ks, vs, table, lengths, offsets, np.float32(scale).astype(np.float64),
        window)
    end = offsets[-1]
    assert torch.all(out[end:] == 7.0) and torch.all(lse[end:] == 7.0)
    n = max(max(lengths), 1)
    e = (2 * (d + 8) + 4) * U32 * reach + (2.0 ** -18 * reach if kind != "bf16" else 0)
    rel = 2 * e + 2 * n * U32 + {"bf16": 2.0 ** -8, "e4m3": 2.0 ** -10,
                                 "e4m3_page": 2.0 ** -11}[kind]
    y, z = values(out)[:end], lse.cpu().numpy().astype(np.float64)[:end]
    ref, ref_lse, spread, e, rel, mass = (x[:end] for x in (ref, ref_lse, spread, e, rel, mass))
    tol = HALF_BF16 * np.abs(ref) + rel[..., None] * spread
    tol = tol + (2.0 ** -32 * mass if kind != "bf16" else 0)
    bad = np.abs(y - ref) > tol
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], y[bad][:4], ref[bad][:4], tol[bad][:4])
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(z), empty)
    assert np.all(y[empty] == 0)
    tol = (e + 2 * n * U32 + 4 * U32 * (1 + np.abs(np.where(empty, 0, ref_lse))))[~empty]
    assert np.all(np.abs(z[~empty] - ref_lse[~empty]) <= tol)
    return out, lse


def prompt_case(seed, lengths, news, hq, hk, d, size, kind, sharp=1.5, spread=1.0, pad=0):
    rng = np.random.default_rng(seed)
    wide = max(1, -(-max(lengths) // size))
    pages = len(lengths) * wide + 2
    cache = any_cache(rng, pages, hk, size, d, kind, spread)
    q = torch.from_numpy((sharp * rng.standard_normal((sum(news) + pad, hq, d)))
                         .astype(np.float32))
    return cache, q.to(torch.bfloat16).cuda(), scattered_table(rng, len(lengths), wide, pages)


KINDS = ["e4m3_page", "e4m3", "bf16"]
CASES = [
    # lengths, news, q heads, kv heads, head_dim, page size
    ([1], [1], 1, 1, 64, 16), ([5], [3], 4, 4, 128, 8), ([200], [200], 2, 2, 128, 64),
    ([129, 1, 64], [129, 1, 5], 8, 2, 64, 16), ([300, 257], [31, 257], 16, 1, 128, 32),
    ([127, 128, 129], [127, 128, 129], 3, 3, 64, 128), ([700], [9], 20, 1, 128, 64),
    ([513], [400], 5, 1, 256, 16), ([260, 70, 0, 33], [17, 70, 0, 1], 12, 2, 256, 64),
    ([1500], [3], 7, 1, 64, 1), ([640, 640], [2, 128], 71, 1, 128, 1024),
    ([90] * 20, [1, 2, 3, 4, 5] * 4, 16, 4, 128, 8), ([1000], [300], 16, 2, 128, 64),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lengths,news,hq,hk,d,size", CASES)
def test_prompt(lengths, news, hq, hk, d, size, kind):
    cache, q, table = prompt_case(sum(lengths) + d, lengths, news, hq, hk, d, size, kind, pad=3)
    check_prompt(cache, q, table, lengths, news, kind=kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 2, 63, 128, 200, 5000])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_windows(window, kind, d):
    lengths, news = [600, 90, 300], [300, 90, 2]
    cache, q, table = prompt_case(window, lengths, news, 6, 2, d, 16, kind)
    for b, (n, m) in enumerate(zip(lengths, news)):       # pages before the window: given back
        table[b, :max(0, n - m + 1 - window) // 16] = -1
    check_prompt(cache, q, table, lengths, news, window=window, kind=kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 2.5])
def test_prompt_scales(kind, scale):
    lengths, news = [300, 40], [150, 40]
    cache, q, table = prompt_case(3, lengths, news, 8, 2, 128, 16, kind, sharp=1.0)
    check_prompt(cache, q, table, lengths, news, scale=scale, kind=kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_rows_that_see_nothing(kind, d):
    """Absent pages (all of a context's, or those of some rows' windows), more new
    tokens than the context has, tables too short for the length."""
    lengths, news = [40, 300, 10, 200], [40, 300, 30, 5]
    cache, q, table = prompt_case(d, lengths, news, 4, 2, d, 16, kind)
    table[0, :] = -1
    table[1, 3:9] = cache.pages
    check_prompt(cache, q, table, lengths, news, kind=kind)
    check_prompt(cache, q, table, lengths, news, window=20, kind=kind)
    short = np.ascontiguousarray(table[:, :7])
    check_prompt(cache, q, short, lengths, news, kind=kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_ignores_what_no_context_covers(kind, d):
    lengths, news, size = [130, 77], [130, 20], 32
    cache, q, table = prompt_case(d, lengths, news, 4, 2, d, size, kind)
    out = check_prompt(cache, q, table, lengths, news, window=60, kind=kind)
    covered = np.zeros((cache.pages, size), bool)
    for b, (n, m) in enumerate(zip(lengths, news)):
        for t in range(max(0, n - m + 1 - 60), n):
            covered[table[b, t // size], t % size] = True
    hide = torch.from_numpy(~covered).cuda()[:, None, :].expand(-1, 2, -1)
    for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        if kind == "bf16":
            t[hide] = float("nan")
        else:
            t[hide] = 0x7f
            if kind == "e4m3":
                s[hide] = float("nan")
            else:
                s[torch.from_numpy(~covered.any(1)).cuda()] = float("nan")
    again = cache.attend_prompt(q, ints([0, 130, 150]), torch.from_numpy(table).cuda(),
                                ints(lengths), window=60, return_lse=True)
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])


@pytest.mark.parametrize("kind", KINDS)
def test_prompt_maxima_that_move(kind):
    """Scores that grow along the context, that fall, and that reach far: the running
    maximum moves in every tile, or never."""
    lengths, news, d = [900, 900], [200, 130], 128
    for slope in (0.02, -0.02, 0.3):
        cache, q, table = prompt_case(7, lengths, news, 4, 1, d, 64, "bf16", sharp=0.1)
        along = slope * torch.arange(960, device="cuda")
        for b in range(2):
            for i, p in enumerate(table[b].tolist()):
                cache.k[p, 0, :, 0] = along[64 * i:64 * i + 64]
        q[..., 0] = d ** 0.5
        if kind != "bf16":
            k, v = cache.k, cache.v
            cache = any_cache(np.random.default_rng(0), cache.pages, 1, 64, d, kind)
            slots = torch.arange(cache.pages * 64, dtype=torch.int32, device="cuda")
            cache.write(k.transpose(1, 2).reshape(-1, 1, d), v.transpose(1, 2).reshape(-1, 1, d),
                        slots)
        check_prompt(cache, q, table, lengths, news, kind=kind)


@pytest.mark.parametrize("kind", ["e4m3_page", "e4m3"])
def test_prompt_scales_far_apart(kind):
    """Keys and values whose scales lie up to 2^40 apart, from page to page and from
    token to token, q heads of any size."""
    lengths, news, d = [700], [200], 128
    cache, q, table = prompt_case(11, lengths, news, 4, 1, d, 16, kind)
    for s in (cache.k_scale, cache.v_scale):
        e = torch.randint(-20, 21, s.shape, device="cuda").float()
        s.copy_(torch.exp2(e) * (1.0 if kind == "e4m3_page" else 1.37) / (2.0 ** 20))
    q *= torch.exp2(torch.randint(-30, 3, (200, 4, 1), device="cuda").float()).to(torch.bfloat16)
    check_prompt(cache, q, table, lengths, news, kind=kind)


def test_prompt_faint_tokens_of_a_long_context():
    """A first token that takes most of the weight, and 60000 that share the rest."""
    lengths, news, d, kind = [60000], [2], 64, "e4m3_page"
    cache, q, table = prompt_case(2, lengths, news, 2, 1, d, 64, kind)
    cache.k.zero_()
    cache.k_scale.fill_(1.0)
    cache.v.fill_(0x38)                                   # 1.0
    cache.v_scale.fill_(1.0)
    p = int(table[0, 0])
    cache.k[p, 0, 0, 0] = 0x38
    cache.v[p, 0, 0] = 0                                  # the first token brings nothing
    q.zero_()
    q[..., 0] = 15.0                                      # its weight: e^15 = 3.3e6 of 6e4
    check_prompt(cache, q, table, lengths, news, scale=1.0, kind=kind)


def test_prompt_agrees_with_one_token():
    """A step of one token a request is the attention of one new token."""
    rng = np.random.default_rng(12)
    lengths = [1, 400, 77, 0, 128]
    for kind in KINDS:
        cache, q, table = prompt_case(21, lengths, [1] * 5, 16, 2, 128, 16, kind)
        t, n = torch.from_numpy(table).cuda(), ints(lengths)
        a = cache.attend(q, t, n, return_lse=True)
        b = cache.attend_prompt(q, ints([0, 1, 2, 3, 4, 5]), t, n, return_lse=True)
        assert torch.allclose(a[0].float(), b[0].float(), rtol=2.0 ** -6, atol=2.0 ** -7)
        assert torch.allclose(a[1], b[1], rtol=1e-5, atol=1e-5)
    assert rng is not None


def test_prompt_strided_and_without_lse():
    lengths, news = [70, 40], [70, 9]
    cache, q, table = prompt_case(4, lengths, news, 6, 3, 64, 8, "e4m3_page")
    t, n, o = torch.from_numpy(table).cuda(), ints(lengths), ints([0, 70, 79])
    want = cache.attend_prompt(q, o, t, n)
    wide = torch.zeros((79, 12, 64), dtype=torch.bfloat16, device="cuda")
    wide[:, :6] = q
    into = torch.full((79, 10, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    big = torch.full((2, 99), -5, dtype=torch.int32, device="cuda")
    big[:, 3:3 + t.shape[1]] = t
    got = cache.attend_prompt(wide[:, :6], o, big[:, 3:3 + t.shape[1]], n, out=into[:, 2:8])
    assert torch.equal(got, want)
    assert torch.all(into[:, :2] == 3.0) and torch.all(into[:, 8:] == 3.0)


def test_prompt_empty_calls():
    cache, q, table = prompt_case(4, [70], [70], 6, 3, 64, 8, "bf16")
    t = torch.from_numpy(table).cuda()
    assert cache.attend_prompt(q[:0], ints([0, 0]), t, ints([70])).shape == (0, 6, 64)
    assert cache.attend_prompt(q, ints([0]), t[:0], ints([])).shape == q.shape


# ---------------------------------------------------------------------------
# a run of them together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", KINDS)
def test_steps_of_a_serving_loop(kind):
    """Plans, writes behind the rotation and attention, step after step, requests
    coming and leaving; every step's attention against a dense evaluation of what the
    cache holds, and the contexts read back against the tokens that were written."""
    rng = np.random.default_rng(31)
    batch, hq, hk, d, page = 5, 8, 2, 128, 16
    pool = attention.PagePool.empty(60, page, batch, 20)
    cache = attention.PagedKVCache.empty(60, hk, page, d, dtype=kind)
    r = attention.Rotary(attention.frequencies(d, 1e6))
    written = [[] for _ in range(batch)]
    for new in ([37, 0, 5, 100, 0], [1, 64, 1, 1, 0], [-1, 1, 3, 1, 17], [20, 1, -1, 1, 1],
                [1, 1, 40, 1, 1]):
        rows = max(0, sum(n for n in new if n > 0)) + 2
        plan = pool.plan(ints(new), rows)
        q, k, v = wide_heads(rng, rows, hq, hk, hk, d=d)
        qo = cache.write_rotary(r, plan.positions, q, k, v, plan.slots)
        out = cache.attend_prompt(qo, plan.offsets, pool.table, plan.lengths)
        pool.commit(plan)
        offsets, lengths = plan.offsets.tolist(), plan.lengths.tolist()
        assert plan.refused.tolist() == [0]
        for b, n in enumerate(new):
            written[b] = [] if n < 0 else written[b] + list(values(v)[offsets[b]:offsets[b + 1]])
            assert lengths[b] == len(written[b])
        check_prompt(cache, qo[:offsets[-1]], pool.table.cpu().numpy(), lengths,
                     np.diff(offsets).tolist(), kind=kind)
        assert torch.isfinite(out[:offsets[-1]].float()).all()
        total = sum(lengths)
        _, vb = cache.read(pool.table, ints(np.concatenate([[0], np.cumsum(lengths)]).tolist()),
                           total)
        want = np.concatenate([np.array(w).reshape(-1, hk, d) for w in written])
        # e4m3: half a step of a code (2^-4), and as much again where a page's scale grew;
        # below the normal codes 2^-10 of the scale, at most 2^-9 of the page's largest
        tol = 0.0 if kind == "bf16" else 2.0 ** -3 * np.abs(want) + 2.0 ** -9 * np.abs(want).max()
        assert np.all(np.abs(values(vb) - want) <= tol)
