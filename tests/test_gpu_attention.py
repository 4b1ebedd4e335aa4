"""Parity of the attention operators' kernels with the fp64 oracle, through the
public classes: rotary positions, the paged cache's write and read, and
attention of one new token.

Bounds, with u = 2^-24 (fp32) and half a bf16 step = 2^-8 of the value:
* rotation: the angle is exact to 2^-31 turns and rounded once to fp32 (at most
  half a turn, 2^-25 of it), sincospi errs by at most 2 steps, and the two
  products and their sum by 3 roundings: below 2^-20 (|x1| + |x2|), then the
  output's rounding.
* cache write of unrotated rows, and reading back: bit for bit.
* attention: a score errs by at most e = (D + 8) 2 u scale sum|q k| (products
  summed by the tensor cores, whose fp32 sums may truncate: 2 u a step) plus
  4 u |s| (scalings, exponential); a weight by 2 e in the ratio of the sums; the
  weights' rounding to 11 bits by 2^-11, and the sum over n tokens by 2 n u.
  All these are relative to sum_j p_j |v_j|; then the output's rounding."""

import numpy as np
import pytest
import torch

import oracle
from expert_layer_ptpc_gb300 import attention
from tests.gpu_helpers import U32, ensure_library, require_gpu

pytestmark = pytest.mark.gpu

HALF_BF16 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    require_gpu()
    ensure_library()


def wide_heads(rng, T, *heads, d):
    """q, k, ... as slices of one [T, sum(heads) * d] bf16 projection."""
    x = torch.from_numpy(rng.standard_normal((T, sum(heads) * d)).astype(np.float32))
    x = x.to(torch.bfloat16).cuda()
    out, at = [], 0
    for h in heads:
        out.append(x[:, at:at + h * d].unflatten(1, (h, d)))
        at += h * d
    return out


def values(t):
    return t.float().cpu().numpy().astype(np.float64)


def rotary_slack(x, rot, neighbours):
    """|x1| + |x2| of each element's pair, zero past rot."""
    a = np.abs(x)
    out = np.zeros_like(a)
    if neighbours:
        s = a[..., 0:rot:2] + a[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = s, s
    else:
        s = a[..., :rot // 2] + a[..., rot // 2:rot]
        out[..., :rot // 2], out[..., rot // 2:rot] = s, s
    return out


def assert_rotated(got, x, want, rot, neighbours):
    tol = HALF_BF16 * np.abs(want) + 2.0 ** -20 * rotary_slack(x, rot, neighbours)
    assert np.all(np.abs(values(got) - want) <= tol)
    assert np.array_equal(values(got)[..., rot:], x[..., rot:])


def make_rotary(rng, rot, axes, T, neighbours, far=100000):
    freq = attention.frequencies(rot, 1000000.0)
    n = rot // 2
    axis = attention.pair_axes([n - 2 * (n // axes) if axes == 3 and a == 0 else n // axes
                                for a in range(axes)], woven=True)
    axis = (axis + [0] * n)[:n]
    pos = rng.integers(0, far, size=(axes, T)).astype(np.int32)
    return (attention.Rotary(freq, axis, axes=axes, neighbours=neighbours), freq.numpy(), axis,
            pos)


# ---------------------------------------------------------------------------
# rotation
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,hq,hk,d,rot,axes,neighbours,far", [
    (1, 1, 0, 16, 16, 1, False, 100), (1, 64, 4, 128, 128, 3, False, 40000),
    (7, 5, 3, 128, 128, 3, True, 1000), (33, 16, 2, 256, 64, 3, True, 1000000),
    (5, 3, 1, 80, 32, 2, False, 2 ** 31 - 1), (3, 9, 3, 512, 512, 3, False, 5000),
    (300, 20, 4, 64, 32, 3, False, 5000), (2, 7, 7, 112, 112, 4, True, 65536),
])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary(T, hq, hk, d, rot, axes, neighbours, far, inverse):
    rng = np.random.default_rng(T * 31 + d)
    q, *k = wide_heads(rng, T, *([hq, hk] if hk else [hq]), d=d)
    r, freq, axis, pos = make_rotary(rng, rot, axes, T, neighbours, far)
    k = k[0] if k else None
    qo, ko = r.apply(torch.from_numpy(pos).cuda(), q, k, inverse=inverse)
    for x, y in ((q, qo), (k, ko)):
        if x is not None:
            want = oracle.rotary_ref(values(x), pos, freq, axis, neighbours, inverse)
            assert_rotated(y, values(x), want, rot, neighbours)
    assert (ko is None) == (k is None)


def test_rotary_in_place_negative_positions_and_strides():
    rng = np.random.default_rng(8)
    q, k, _ = wide_heads(rng, 19, 6, 2, 2, d=128)
    r, freq, axis, pos = make_rotary(rng, 96, 3, 19, False)
    pos[:, ::3] *= -1
    p = torch.from_numpy(pos).cuda()
    x, y = values(q), values(k)
    fresh = r.apply(p, q, k)
    r.apply(p, q, k, q_out=q, k_out=k)
    assert torch.equal(fresh[0], q) and torch.equal(fresh[1], k)
    assert_rotated(q, x, oracle.rotary_ref(x, pos, freq, axis), 96, False)
    assert_rotated(k, y, oracle.rotary_ref(y, pos, freq, axis), 96, False)


def test_rotary_empty_and_refused():
    r = attention.Rotary(attention.frequencies(64))
    q = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert r.apply(torch.zeros((1, 0), dtype=torch.int32, device="cuda"), q)[0].shape == q.shape
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    p = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    for bad in (dict(positions=p.long(), q=q), dict(positions=p[:, :1].contiguous(), q=q),
                dict(positions=p, q=q.float()), dict(positions=p, q=q.transpose(1, 2)),
                dict(positions=p, q=q, k=q[:1]), dict(positions=p, q=q, k_out=q)):
        with pytest.raises(ValueError):
            r.apply(**bad)


# ---------------------------------------------------------------------------
# the cache: write and read
# ---------------------------------------------------------------------------
def scattered_slots(rng, T, pages, size):
    slots = rng.permutation(pages * size)[:T].astype(np.int32)
    if T > 4:
        slots[1], slots[3] = -1, pages * size          # no slot: skipped
    return slots


def host(cache):
    return [None if t is None else
            (t.cpu().numpy() if t.dtype != torch.bfloat16 else values(t))
            for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]


def fresh_cache(pages, heads, size, d, kind):
    c = attention.PagedKVCache.empty(pages, heads, size, d, dtype=kind)
    for t in (c.k, c.v, c.k_scale, c.v_scale):
        if t is not None:
            t.zero_()
    return c


@pytest.mark.parametrize("T,heads,d,size,kind", [
    (1, 4, 128, 64, "e4m3"), (1, 1, 64, 1, "e4m3"), (37, 3, 256, 8, "e4m3"),
    (130, 8, 64, 16, "e4m3"), (61, 5, 128, 1024, "e4m3"), (37, 3, 128, 16, "bf16"),
    (9, 2, 256, 32, "bf16"), (5, 1, 64, 2, "bf16"),
])
def test_write_is_bit_exact(T, heads, d, size, kind):
    rng = np.random.default_rng(T + d)
    pages = -(-(T + 3) // size) + 2
    cache = fresh_cache(pages, heads, size, d, kind)
    k, v = wide_heads(rng, T, heads, heads, d=d)
    k *= torch.exp(8 * torch.randn((T, heads, 1), device="cuda")).to(torch.bfloat16)
    v[0, 0] = 0                                         # a row of zeros: the floor's scale
    slots = scattered_slots(rng, T, pages, size)
    want = [t.copy() if t is not None else None for t in host(cache)]
    cache.write(k, v, torch.from_numpy(slots).cuda())
    for x, i in ((k, 0), (v, 1)):
        oracle.kv_write_ref(want[i], want[2 + i], values(x).astype(np.float32), slots)
    for got, ref in zip(host(cache), want):
        assert (got is None and ref is None) or np.array_equal(got, ref)


@pytest.mark.parametrize("T,hq,hk,d,rot,axes,neighbours,size,kind", [
    (1, 64, 4, 128, 128, 3, False, 64, "e4m3"), (21, 5, 1, 256, 64, 3, True, 8, "e4m3"),
    (40, 12, 3, 64, 64, 2, False, 16, "e4m3"), (40, 8, 4, 64, 32, 1, False, 16, "bf16"),
    (13, 16, 2, 128, 128, 3, True, 32, "bf16"),
])
def test_write_rotary(T, hq, hk, d, rot, axes, neighbours, size, kind):
    rng = np.random.default_rng(T * 5 + d)
    pages = -(-(T + 3) // size) + 2
    cache = fresh_cache(pages, hk, size, d, kind)
    q, k, v = wide_heads(rng, T, hq, hk, hk, d=d)
    r, freq, axis, pos = make_rotary(rng, rot, axes, T, neighbours)
    slots = scattered_slots(rng, T, pages, size)
    before = host(cache)
    qo = cache.write_rotary(r, torch.from_numpy(pos).cuda(), q, k, v,
                            torch.from_numpy(slots).cuda())
    assert_rotated(qo, values(q), oracle.rotary_ref(values(q), pos, freq, axis, neighbours), rot,
                   neighbours)
    kc, vc, ks, vs = host(cache)
    oracle.kv_write_ref(before[1], before[3], values(v).astype(np.float32), slots)
    assert np.array_equal(vc, before[1]) and (vs is None or np.array_equal(vs, before[3]))
    y = oracle.rotary_ref(values(k), pos, freq, axis, neighbours)
    slack = 2.0 ** -20 * rotary_slack(values(k), rot, neighbours)
    written = np.zeros(pages * size, bool)
    for t, s in enumerate(slots.tolist()):
        if not 0 <= s < pages * size:
            continue
        written[s] = True
        p, o = divmod(s, size)
        if kind == "bf16":
            assert np.all(np.abs(kc[p, :, o] - y[t]) <= HALF_BF16 * np.abs(y[t]) + slack[t])
            continue
        scale = ks[p, :, o].astype(np.float64)
        top = np.abs(y[t]).max(-1)
        assert np.all(np.abs(scale * 448 - top) <= 4 * U32 * top + slack[t].max(-1))
        got = oracle.e4m3_decode(kc[p, :, o]) * scale[:, None]
        # half a step: 2^-4 of a normal code, 2^-10 of the scale below those
        tol = np.maximum(2.0 ** -4 * np.abs(y[t]), 2.0 ** -10 * scale[:, None])
        assert np.all(np.abs(got - y[t]) <= 1.001 * tol + 2 * slack[t].max())
    untouched = ~written.reshape(pages, size)
    assert np.all(kc.transpose(0, 2, 1, 3)[untouched] == 0)


def filled_cache(rng, pages, heads, size, d, kind, spread=1.0):
    """Codes over the whole e4m3 range with scales of many sizes, or bf16."""
    c = attention.PagedKVCache.empty(pages, heads, size, d, dtype=kind)
    for name in ("k", "v"):
        x = torch.from_numpy(rng.standard_normal((pages, heads, size, d)).astype(np.float32))
        x = x * torch.from_numpy(np.exp(spread * rng.standard_normal((pages, heads, size, 1)))
                                 .astype(np.float32))
        t = getattr(c, name)
        if kind == "bf16":
            t.copy_(x.to(torch.bfloat16))
        else:
            s = x.abs().amax(-1) / 448.0
            t.copy_((x / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
                    .view(torch.uint8))
            getattr(c, name + "_scale").copy_(s)
    return c


def scattered_table(rng, batch, max_pages, pages):
    """Distinct pages in random order (where there are enough)."""
    n = batch * max_pages
    ids = rng.permutation(pages)[:n] if n <= pages else rng.integers(0, pages, size=n)
    return np.ascontiguousarray(ids.reshape(batch, max_pages).astype(np.int32))


@pytest.mark.parametrize("lengths,heads,d,size,kind", [
    ([1], 1, 64, 16, "e4m3"), ([0, 5, 0, 33, 1], 3, 128, 16, "e4m3"),
    ([130, 64, 63], 2, 256, 64, "e4m3"), ([17, 0, 8], 8, 64, 1, "bf16"),
    ([40] * 9, 1, 128, 8, "bf16"), (list(range(70)), 2, 64, 4, "e4m3"),
])
def test_read(lengths, heads, d, size, kind):
    rng = np.random.default_rng(sum(lengths) + d)
    max_pages = -(-max(lengths) // size) + 1
    pages = len(lengths) * max_pages + 1
    cache = filled_cache(rng, pages, heads, size, d, kind)
    table = scattered_table(rng, len(lengths), max_pages, pages)
    table[-1, 0] = -1 if lengths[-1] != 1 else table[-1, 0]       # an absent page: zeros
    if len(lengths) > 2:
        table[1, 0] = pages                                       # past the cache: zeros
    offsets = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    rows = int(offsets[-1]) + 3                                   # rows past the end: zeros
    k, v = cache.read(torch.from_numpy(table).cuda(), torch.from_numpy(offsets).cuda(), rows)
    kc, vc, ks, vs = host(cache)
    for got, codes, scales in ((k, kc, ks), (v, vc, vs)):
        want = np.zeros((rows, heads, d))
        for b, n in enumerate(lengths):
            want[offsets[b]:offsets[b + 1]], _ = oracle.cache_rows_ref(codes, scales, table[b],
                                                                      range(n))
        # fp32 product, then bf16: the same two roundings
        want = oracle.bf16_round(want.astype(np.float32).astype(np.float64))
        assert np.array_equal(values(got), want.astype(np.float64))


# ---------------------------------------------------------------------------
# attention of one new token
# ---------------------------------------------------------------------------
def check_attention(cache, q, table, lengths, scale=None, window=0, **kw):
    out, lse = cache.attend(q, torch.from_numpy(table).cuda(),
                            torch.tensor(lengths, dtype=torch.int32, device="cuda"), scale=scale,
                            window=window, return_lse=True, **kw)
    d = q.shape[-1]
    scale = d ** -0.5 if scale is None else scale
    kc, vc, ks, vs = host(cache)
    ref, ref_lse, spread, reach = oracle.paged_attention_ref(
        values(q), kc, vc, ks, vs, table, lengths, np.float32(scale).astype(np.float64), window)
    n = np.minimum(np.array(lengths), window if window else 2 ** 31 - 1)[:, None]
    e = (2 * (d + 8) + 4) * U32 * reach
    rel = 2 * e + 2.0 ** -11 + 2 * n * U32
    got, got_lse = values(out), lse.cpu().numpy().astype(np.float64)
    tol = HALF_BF16 * np.abs(ref) + rel[..., None] * spread
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4], tol[bad][:4])
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(got_lse), empty)
    assert np.all(got[empty] == 0)
    fine = ~empty
    tol = (e + 2 * n * U32 + 4 * U32 * (1 + np.abs(np.where(fine, ref_lse, 0))))[fine]
    assert np.all(np.abs(got_lse[fine] - ref_lse[fine]) <= tol)
    return out, lse


def attention_case(seed, lengths, hq, hk, d, size, kind, sharp=1.5, spread=1.0):
    rng = np.random.default_rng(seed)
    max_pages = max(1, -(-max(lengths) // size))
    pages = min(len(lengths) * max_pages + 2, 4000)
    cache = filled_cache(rng, pages, hk, size, d, kind, spread)
    q = torch.from_numpy((sharp * rng.standard_normal((len(lengths), hq, d))).astype(np.float32))
    return cache, q.to(torch.bfloat16).cuda(), scattered_table(rng, len(lengths), max_pages, pages)


@pytest.mark.parametrize("lengths,hq,hk,d,size,kind", [
    ([1], 1, 1, 64, 16, "e4m3"), ([1], 64, 4, 128, 64, "e4m3"), ([2, 0, 1], 8, 2, 256, 8, "e4m3"),
    ([15, 16, 17, 31, 32, 33, 63, 64, 65], 16, 1, 128, 16, "e4m3"),
    ([127, 128, 129, 255, 257], 6, 2, 64, 4, "e4m3"), ([300], 64, 4, 128, 64, "e4m3"),
    ([1000, 3, 0, 77], 40, 8, 64, 16, "bf16"), ([500, 501], 20, 1, 128, 32, "e4m3"),
    ([333, 90], 34, 2, 256, 64, "bf16"), ([4100], 5, 1, 128, 128, "bf16"),
    ([9000], 16, 2, 128, 64, "e4m3"), ([700] * 40, 4, 4, 64, 16, "e4m3"),
    ([129] * 3, 33, 1, 256, 1, "e4m3"), ([64, 5000, 1, 640], 7, 7, 128, 1024, "bf16"),
    (list(range(0, 200, 3)), 12, 4, 128, 8, "e4m3"),
])
def test_attention(lengths, hq, hk, d, size, kind):
    cache, q, table = attention_case(sum(lengths) + d, lengths, hq, hk, d, size, kind)
    check_attention(cache, q, table, lengths)


@pytest.mark.parametrize("group", [17, 24, 32, 33, 71])
@pytest.mark.parametrize("d,kind", [(64, "e4m3"), (128, "e4m3"), (64, "bf16"), (128, "bf16")])
def test_attention_many_heads_a_kv_head(group, d, kind):
    """Groups that fill two tensor core tiles, end inside the second or need more:
    one CTA an item, and in wide tables, whose items have two tiles, cut and joined."""
    for lengths, hk, size in (([1, 0, 63, 64, 65, 127, 128, 129, 200], 2, 16),
                              ([6000, 17], 1, 64)):
        cache, q, table = attention_case(group, lengths, hk * group, hk, d, size, kind)
        check_attention(cache, q, table, lengths)
        wide = np.full((len(lengths), 5000), -1, np.int32)
        wide[:, :table.shape[1]] = table
        check_attention(cache, q, wide, lengths)


@pytest.mark.parametrize("d,kind", [(64, "e4m3"), (128, "e4m3"), (64, "bf16"), (128, "bf16")])
def test_attention_many_heads_in_a_window(d, kind):
    lengths = [4000, 3001, 3000, 2999, 0] + [17 + b for b in range(45)]
    cache, q, table = attention_case(d, lengths, 40, 2, d, 16, kind)
    table[0, :1000 // 16] = -1
    table[1, 5:9] = cache.pages
    check_attention(cache, q, table, lengths, window=3000)


def test_attention_many_heads_in_a_workspace_of_any_content():
    """The largest workspace a call can ask for, between guard bands that stay, and the
    same results from call to call."""
    lengths = [40000, 0, 20000, 5]
    cache, q, table = attention_case(61, lengths, 48, 2, 128, 64, "e4m3")
    wide = np.full((4, 2000), -1, np.int32)
    wide[:, :table.shape[1]] = table
    want = check_attention(cache, q, wide, lengths)
    from expert_layer_ptpc_gb300 import binding
    need = binding.moe_paged_attention_workspace_size(cache.struct, 4, 48)
    space = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    t = torch.from_numpy(wide).cuda()
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    for fill in (0xFF, 0):
        space[256:256 + need] = fill
        out, lse = cache.attend(q, t, n, return_lse=True, ws=space[256:256 + need])
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert bool((space[:256] == 0xA5).all()) and bool((space[256 + need:] == 0xA5).all())


@pytest.mark.parametrize("window", [1, 15, 64, 100, 5000])
@pytest.mark.parametrize("kind,d", [("e4m3", 128), ("bf16", 64)])
def test_attention_window(window, kind, d):
    lengths = [1, 0, 64, 99, 100, 101, 1500]
    cache, q, table = attention_case(window, lengths, 8, 2, d, 16, kind)
    # pages wholly before the window are gone, as a cache that recycles them
    for b, n in enumerate(lengths):
        table[b, :max(0, n - window) // 16] = -1
    check_attention(cache, q, table, lengths, window=window)


def test_attention_of_one_sequence_of_many_heads_and_scales():
    """Token scales that differ by many orders of magnitude: tokens of great
    weight with tiny values next to tokens of little weight with huge ones."""
    for kind in ("e4m3", "bf16"):
        lengths = [777, 60]
        cache, q, table = attention_case(17, lengths, 16, 2, 128, 16, kind, 1.0, spread=0.3)
        factor = torch.exp2(torch.randint(-12, 13, cache.v.shape[:3], device="cuda").float())
        if kind == "e4m3":
            cache.v_scale.mul_(factor)
        else:
            cache.v.mul_(factor[..., None].to(torch.bfloat16))
        check_attention(cache, q, table, lengths)


def test_attention_sharp_scores():
    """One token takes nearly all of the weight, early and late in the context;
    scores from far below zero."""
    lengths = [2000, 2000, 40]
    cache, q, table = attention_case(23, lengths, 4, 2, 128, 64, "e4m3", sharp=12.0)
    check_attention(cache, q, table, lengths)
    check_attention(cache, q, table, lengths, scale=-0.11)
    check_attention(cache, q, table, lengths, scale=0.0)


def test_attention_absent_pages_and_short_tables():
    """Entries outside the cache take their tokens out, a row can lose all of
    them, and a length past the table ends with the table."""
    lengths = [200, 200, 90, 500]
    cache, q, table = attention_case(29, [200] * 4, 16, 2, 128, 16, "e4m3")
    table[0, ::3] = -1
    table[1, :] = -5
    table[2, 1:5] = cache.pages + 3
    table[3, 4] = 2 ** 31 - 1
    clipped = [200, 200, 90, table.shape[1] * 16]
    out, lse = check_attention(cache, q, table, clipped)
    again = cache.attend(q, torch.from_numpy(table).cuda(),
                         torch.tensor(lengths, dtype=torch.int32, device="cuda"), return_lse=True)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    wild = torch.tensor([-7, 0, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    o, l = cache.attend(q, torch.from_numpy(table).cuda(), wild, return_lse=True)
    assert torch.all(o[:3] == 0) and torch.all(torch.isneginf(l[:3]))
    assert torch.equal(o[3], out[3]) and torch.equal(l[3], lse[3])


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
def test_attention_ignores_what_other_slots_hold(kind):
    """NaN and infinities in slots that take no part change nothing."""
    lengths = [37, 0, 90, 16]
    cache, q, table = attention_case(31, lengths, 8, 2, 128, 32, kind)
    out, lse = check_attention(cache, q, table, lengths, window=50)
    keep = torch.zeros(cache.k.shape[0], cache.page_size, dtype=torch.bool)
    for b, n in enumerate(lengths):
        for t in range(max(0, n - 50), n):
            keep[table[b, t // 32], t % 32] = True
    drop = (~keep).cuda()[:, None].expand(cache.k.shape[:3])
    for t in (cache.k, cache.v):
        t[drop] = 0x7F if kind == "e4m3" else float("nan")
    if kind == "e4m3":
        cache.k_scale[drop] = float("inf")
        cache.v_scale[drop] = float("nan")
    o, l = cache.attend(q, torch.from_numpy(table).cuda(),
                        torch.tensor(lengths, dtype=torch.int32, device="cuda"), window=50,
                        return_lse=True)
    assert torch.equal(o, out) and torch.equal(l, lse)


def test_attention_strided_inputs_streams_and_repeats():
    """q and the table as slices of wider tensors; the same bits on another
    stream, with a workspace of any content, and from a graph."""
    lengths = [300, 17, 0, 4000]
    cache, q, table = attention_case(37, lengths, 16, 2, 128, 16, "e4m3")
    out, lse = check_attention(cache, q, table, lengths)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    wide_q = torch.full((4, 30, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    wide_q[:, 3:19] = q
    wide_t = torch.full((4, table.shape[1] + 5), 123456, dtype=torch.int32, device="cuda")
    wide_t[:, 2:2 + table.shape[1]] = torch.from_numpy(table).cuda()
    args = (wide_q[:, 3:19], wide_t[:, 2:2 + table.shape[1]], n)
    ws = torch.full_like(cache.workspace(4, 16), 0xFF)
    for _ in range(3):
        o, l = cache.attend(*args, return_lse=True, ws=ws)
        assert torch.equal(o, out) and torch.equal(l, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, l = cache.attend(*args, return_lse=True, stream=side)
    side.synchronize()
    assert torch.equal(o, out) and torch.equal(l, lse)
    graph = torch.cuda.CUDAGraph()
    o, l = torch.empty_like(out), torch.empty_like(lse)
    with torch.cuda.graph(graph):
        cache.attend(*args, out=o, lse=l, ws=ws)
    for shift in (0, -100):
        n.copy_(torch.tensor([max(0, x + shift) for x in lengths], dtype=torch.int32))
        graph.replay()
        want = cache.attend(*args, return_lse=True)
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


def test_attention_far_rows_of_a_large_cache():
    """Rows whose byte offsets pass 32 bits: the last pages of a cache of 2^33
    bytes a side."""
    heads, size, d = 4, 64, 256
    pages = (1 << 33) // (heads * size * d) + 3
    cache = attention.PagedKVCache.empty(pages, heads, size, d)
    rng = np.random.default_rng(41)
    small = filled_cache(rng, 6, heads, size, d, "e4m3")
    for name in ("k", "v", "k_scale", "v_scale"):
        getattr(cache, name)[-6:] = getattr(small, name)
    q = torch.from_numpy(rng.standard_normal((2, 8, d)).astype(np.float32))
    q = q.to(torch.bfloat16).cuda()
    lengths = [130, 100]
    table = np.array([[0, 3, 5], [4, 1, 2]], np.int32)
    out, lse = check_attention(small, q, table, lengths)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    far = torch.from_numpy(table + pages - 6).cuda()
    o, l = cache.attend(q, far, n, return_lse=True)
    assert torch.equal(o, out) and torch.equal(l, lse)
    # and written and read there
    k = torch.from_numpy(rng.standard_normal((3, heads, d)).astype(np.float32))
    k = k.to(torch.bfloat16).cuda()
    slots = torch.tensor([0, 70, 383], dtype=torch.int32, device="cuda")
    small.write(k, -k, slots)
    cache.write(k, -k, slots + (pages - 6) * size)
    assert torch.equal(cache.k[-6:], small.k) and torch.equal(cache.v[-6:], small.v)
    offsets = torch.tensor([0, 130, 230], dtype=torch.int32, device="cuda")
    for got, want in zip(cache.read(far, offsets, 230),
                         small.read(torch.from_numpy(table).cuda(), offsets, 230)):
        assert torch.equal(got, want)


def test_attention_tensor_refusals():
    cache, q, table = attention_case(43, [20, 20], 8, 2, 64, 16, "e4m3")
    t = torch.from_numpy(table).cuda()
    n = torch.tensor([20, 20], dtype=torch.int32, device="cuda")
    for bad in (dict(q=q.float()), dict(q=q[..., :32]), dict(block_table=t.long()),
                dict(block_table=t[:1]), dict(lengths=n.long()), dict(lengths=n[:1]),
                dict(block_table=t.t().contiguous().t()), dict(lengths=n.cpu()),
                dict(out=q.float()), dict(lse=torch.empty(2, 7, device="cuda"))):
        kw = dict(q=q, block_table=t, lengths=n)
        kw.update(bad)
        with pytest.raises(ValueError):
            cache.attend(**kw)
    from expert_layer_ptpc_gb300.binding import MoeError
    with pytest.raises(MoeError) as e:
        cache.attend(q[:, :7], t, n)
    assert e.value.status == -1
    with pytest.raises(MoeError) as e:
        cache.attend(q, t, n, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -4


def test_write_divides_like_ieee_for_every_pair_of_mantissas():
    """Every bf16 mantissa against every mantissa of the row's largest element,
    over the 19 binades that reach a code: the codes equal those of an IEEE
    division (the oracle's), for small and large rows."""
    top = (128 + np.arange(128)) / 128.0                               # [1, 2)
    small = ((128 + np.arange(128))[:, None] / 128.0 * 2.0 ** -np.arange(19.0)).reshape(-1)
    for shift in (0, 60, -40):
        rows = []
        for m in top:
            v = small[small <= m]
            v = np.concatenate([v, np.zeros(-len(v) % 63)]).reshape(-1, 63)
            rows.append(np.concatenate([np.full((len(v), 1), m), v], 1))
        x = (np.concatenate(rows) * 2.0 ** shift).astype(np.float32)
        x[::2] *= -1
        t = torch.from_numpy(x)[:, None].to(torch.bfloat16).cuda()
        assert np.array_equal(values(t)[:, 0], x)                      # bf16 values
        T = len(x)
        cache = fresh_cache(-(-T // 64), 1, 64, 64, "e4m3")
        cache.write(t, t, torch.arange(T, dtype=torch.int32, device="cuda"))
        codes, scales = oracle.quant_rows_ref(x)
        kc, vc, ks, _ = host(cache)
        assert np.array_equal(kc.reshape(-1, 64)[:T], codes)
        assert np.array_equal(vc, kc) and np.array_equal(ks.reshape(-1)[:T], scales)


@pytest.mark.parametrize("lengths,hq,hk,d,kind", [
    ([70001], 16, 1, 128, "e4m3"),            # one item on every CTA
    ([40000, 1, 0, 300], 8, 2, 64, "bf16"), ([3000] * 5, 6, 6, 128, "e4m3"),
    ([20000, 20000], 2, 1, 256, "e4m3"), ([0, 200], 40, 2, 128, "e4m3"),
])
def test_attention_workspace_of_any_content_is_not_passed(lengths, hq, hk, d, kind):
    """A workspace of any content, between guard bands that stay."""
    cache, q, table = attention_case(47, lengths, hq, hk, d, 16, kind)
    want = check_attention(cache, q, table, lengths)
    from expert_layer_ptpc_gb300 import binding
    need = binding.moe_paged_attention_workspace_size(cache.struct, len(lengths), hq)
    wide = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    t = torch.from_numpy(table).cuda()
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    for fill in (0xA5, 0xFF, 0):
        wide[256:256 + need] = fill
        out, lse = cache.attend(q, t, n, return_lse=True, ws=wide[256:256 + need])
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert bool((wide[:256] == 0xA5).all()) and bool((wide[256 + need:] == 0xA5).all())


def test_attention_whole_contexts_and_cut_ones_agree():
    """Short tables run without the cut; a wider table of the same contexts runs
    with it, with the same results up to the order of the sums."""
    lengths = [1, 0, 200, 256, 77]
    cache, q, table = attention_case(53, lengths, 24, 2, 128, 16, "e4m3")
    check_attention(cache, q, table, lengths)
    wide = np.full((5, 4000), -1, np.int32)
    wide[:, :table.shape[1]] = table
    check_attention(cache, q, wide, lengths)
    check_attention(cache, q, wide, lengths, window=100)
    check_attention(cache, q, table, lengths, window=100)


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
@pytest.mark.parametrize("gap", [12.0, 18.0, 21.0])
def test_attention_sink_and_a_long_faint_tail(kind, gap):
    """One token of great weight and very many of e^-gap of it, whose values agree in
    elements where the first's are zero: what the tail adds there must not be
    rounded away. Weights are exact powers apart, so the bound is the weights'
    and the sums' rounding; a weight of e^-21 = 2^-30.3 of the largest keeps at
    least 2 bits of fp16's subnormals (2^-32 of it is half a step)."""
    n, d, size = 20000, 128, 64
    pages = -(-n // size)
    cache = fresh_cache(pages, 1, size, d, kind)
    k = torch.zeros((n, 1, d), device="cuda")
    v = torch.zeros((n, 1, d), device="cuda")
    k[7, 0, 0] = 1.0                       # the sink
    v[7, 0, :64] = 1.0
    v[:7, 0, 64:] = 1.0
    v[8:, 0, 64:] = 1.0
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    cache.write(k.to(torch.bfloat16), v.to(torch.bfloat16), slots)
    q = torch.zeros((1, 16, d), device="cuda")
    q[..., 0] = gap
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    lengths = torch.tensor([n], dtype=torch.int32, device="cuda")
    out = cache.attend(q.to(torch.bfloat16), table, lengths, scale=1.0)
    tail = (n - 1) * np.exp(-gap)
    want = np.concatenate([np.full(64, 1 / (1 + tail)), np.full(64, tail / (1 + tail))])
    got = values(out)[0]
    # half a step of a weight: 2^-11 of it, or 2^-32 of the largest
    rel = HALF_BF16 + max(2.0 ** -11, 2.0 ** -32 * np.exp(gap)) + 4 * n * U32
    assert np.all(np.abs(got - want) <= rel * want), (got[0, [0, 64]], want[[0, 64]])


def test_attention_a_bad_context_does_not_reach_others():
    """NaN in the keys, values or scales of some contexts stays in their rows."""
    for kind in ("e4m3", "bf16"):
        lengths = [40 + b % 30 for b in range(700)]
        cache, q, table = attention_case(59, lengths, 4, 1, 128, 16, kind)
        wide = np.full((700, 100), -1, np.int32)       # cut and joined, not one CTA an item
        wide[:, :table.shape[1]] = table
        t = torch.from_numpy(wide).cuda()
        n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        want = cache.attend(q, t, n, return_lse=True)
        bad = range(0, 700, 7)
        for i, b in enumerate(bad):
            page, at = int(table[b, (lengths[b] - 1) // 16]), (lengths[b] - 1) % 16
            if kind == "bf16":
                (cache.k if i % 2 else cache.v)[page, 0, at, 5] = float("nan")
            elif i % 3 == 0:
                (cache.k if i % 2 else cache.v)[page, 0, at, 5] = 0x7F
            else:
                (cache.k_scale if i % 2 else cache.v_scale)[page, 0, at] = float("nan")
        got = cache.attend(q, t, n, return_lse=True)
        good = torch.tensor([b not in set(bad) for b in range(700)], device="cuda")
        assert torch.equal(got[0][good], want[0][good])
        assert torch.equal(got[1][good], want[1][good])
