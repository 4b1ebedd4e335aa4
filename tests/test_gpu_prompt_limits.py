"""Attention of many new tokens at the ends of its range: NaN, scales of every size, long
segments of work, and rows of padding."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from expert_layer_ptpc_gb300 import attention, binding
from tests.gpu_helpers import U32, ensure_library, require_gpu
from tests.test_gpu_attention import HALF_BF16, host, values
from tests.test_gpu_prompt_attention import KINDS, check_prompt, ints, prompt_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    require_gpu()
    ensure_library()
    yield
    assert binding.moe_device_status() == (0, 0)     # no wait of any test ran out


# ---------------------------------------------------------------------------
# NaN stays in the rows that it reaches, whole items and cut ones alike
# ---------------------------------------------------------------------------
LONG_AND_SHORT = ([9000, 60, 300], [40, 60, 2])     # cut over many CTAs, and whole


class WithNan:
    """A cache whose attend_prompt gets NaN in some rows of q, and gives back what those
    rows are without."""

    def __init__(self, cache, hurt):
        self.cache, self.hurt = cache, hurt
        self.k, self.v, self.k_scale, self.v_scale = cache.k, cache.v, cache.k_scale, cache.v_scale

    def attend_prompt(self, q, *call, out, lse, **kw):
        clean = self.cache.attend_prompt(q, *call, return_lse=True, **kw)
        q = q.clone()
        q[self.hurt] = float("nan")
        self.cache.attend_prompt(q, *call, out=out, lse=lse, **kw)
        assert torch.isnan(out[self.hurt].float()).all() and torch.isnan(lse[self.hurt]).all()
        out[self.hurt], lse[self.hurt] = clean[0][self.hurt], clean[1][self.hurt]
        return out, lse


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [2, 5])           # items of up to 128 rows, and of more
def test_nan_of_q_stays_in_its_rows(kind, d, group):
    """(A row's neighbours need not be the same bit for bit: the 32 rows of a warp move the
    bounds of their weights together, by what is no power of two, and a row of NaN moves none.)"""
    lengths, news = LONG_AND_SHORT
    cache, q, table = prompt_case(d, lengths, news, 2 * group, 2, d, 32, kind)
    hurt = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    for row, head in ((0, 0), (17, group), (39, 2 * group - 1), (40, 1), (77, group), (101, 0)):
        hurt[row, head] = True
    check_prompt(WithNan(cache, hurt), q, table, lengths, news, kind=kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("which", ["k", "v"])
def test_nan_of_the_cache_reaches_every_row_that_sees_it(kind, which):
    """A NaN in a token that all rows of a context see, and in no other context."""
    lengths, news = LONG_AND_SHORT
    cache, q, table = prompt_case(3, lengths, news, 6, 2, 128, 32, kind)
    call = ints(np.concatenate([[0], np.cumsum(news)]).tolist()), torch.from_numpy(table).cuda(), \
        ints(lengths)
    clean = cache.attend_prompt(q, *call, return_lse=True)
    for context, rows in ((0, slice(0, 40)), (2, slice(100, 102))):
        t = getattr(cache, which)
        page, offset = int(table[context, 5]), 3
        kept = t[page, :, offset].clone()
        t[page, :, offset, 9] = float("nan") if kind == "bf16" else 0x7f
        out, lse = cache.attend_prompt(q, *call, return_lse=True)
        t[page, :, offset] = kept
        seen = out[rows] if which == "k" else out[rows][..., 9]
        assert torch.isnan(seen.float()).all()
        if which == "k":
            assert torch.isnan(lse[rows]).all()
        else:
            assert torch.equal(lse[rows], clean[1][rows])
        others = torch.ones(102, dtype=torch.bool, device="cuda")
        others[rows] = False
        assert torch.equal(out[others], clean[0][others])
        assert torch.equal(lse[others], clean[1][others])


# ---------------------------------------------------------------------------
# page scales that are no powers of two
# ---------------------------------------------------------------------------
def bounds(cache, q, table, lengths, news, score=0.0, value=0.0, weight=2.0 ** -11, window=0,
           more=0.0):
    """The oracle's out and lse, with what attention of many tokens may be off from them
    over an e4m3 cache: as in test_gpu_prompt_attention, with every product of q and a key off by
    `score` of it more and every score by `more`, and every value by `value` of it."""
    offsets = np.concatenate([[0], np.cumsum(news)])
    kc, vc, ks, vs = host(cache)
    d, n = cache.head_dim, max(max(lengths), 1)
    ref, lse, spread, reach, mass = oracle.prompt_attention_ref(
        values(q), kc, vc, ks, vs, table, lengths, offsets,
        np.float32(d ** -0.5).astype(np.float64), window)
    e = ((2 * (d + 8) + 4) * U32 + 2.0 ** -18 + score) * reach + more
    rel = np.expm1(np.minimum(2 * e, 50.0)) + 2 * n * U32 + weight + value
    tol = HALF_BF16 * np.abs(ref) + rel[..., None] * spread + 2.0 ** -32 * mass
    lse_tol = e + 2 * n * U32 + 4 * U32 * (1 + np.abs(np.where(np.isneginf(lse), 0, lse)))
    return ref, lse, tol, lse_tol


@pytest.mark.parametrize("d", [64, 128, 256])
def test_page_scales_that_are_no_powers_of_two(d):
    """A caller's own scales: every operator takes them as they are. In the prompt's attention a
    scale is rounded to fp16 and its product with a code once more: 2^-11 twice."""
    lengths, news = [300, 70, 2000], [120, 70, 9]
    cache, q, table = prompt_case(d, lengths, news, 6, 2, d, 32, "e4m3_page")
    for s in (cache.k_scale, cache.v_scale):
        s *= 1 + torch.rand(s.shape, device="cuda")
    t, n = torch.from_numpy(table).cuda(), ints(lengths)
    ends = np.concatenate([[0], np.cumsum(news)])
    out, lse = cache.attend_prompt(q, ints(ends.tolist()), t, n, return_lse=True)
    twice = 2.0 ** -10 + 2.0 ** -22
    ref, ref_lse, tol, lse_tol = bounds(cache, q, table, lengths, news, twice, twice)
    assert np.all(np.abs(values(out) - ref) <= tol)
    assert np.all(np.abs(lse.cpu().numpy() - ref_lse) <= lse_tol)
    # one token a request: the last row of each
    last = torch.from_numpy(ends[1:] - 1).cuda()
    one, one_lse = cache.attend(q[last], t, n, return_lse=True)
    at = ends[1:] - 1
    assert np.all(np.abs(values(one) - ref[at]) <= tol[at])
    assert np.all(np.abs(one_lse.cpu().numpy() - ref_lse[at]) <= lse_tol[at])
    k, _ = cache.read(t, ints([0, 300, 370, 2370]), 2370)
    kc, _, ks, _ = host(cache)
    want, _ = oracle.cache_rows_ref(kc, ks, table[0], range(300))
    assert np.array_equal(values(k)[:300], oracle.bf16_round(want))


@pytest.mark.parametrize("kind", KINDS)
def test_large_keys_and_small_queries(kind):
    """Keys near the end of bf16's range, and queries as far below one: scores like any others."""
    lengths, news, d, size = [300, 40], [90, 40], 128, 16
    cache, q, table = prompt_case(8, lengths, news, 4, 2, d, size, "bf16")
    far = 2.0 ** 112
    cache.k *= far
    assert torch.isfinite(cache.k.float()).all()
    q /= far
    if kind != "bf16":
        coded = attention.PagedKVCache.empty(cache.pages, 2, size, d, dtype=kind)
        coded.write(cache.k.transpose(1, 2).reshape(-1, 2, d),
                    cache.v.transpose(1, 2).reshape(-1, 2, d),
                    torch.arange(cache.pages * size, dtype=torch.int32, device="cuda"))
        cache = coded
    check_prompt(cache, q, table, lengths, news, kind=kind)


# ---------------------------------------------------------------------------
# segments that take long
# ---------------------------------------------------------------------------
def test_a_role_waits_as_long_as_the_others_work():
    """Items of one row over 20 million tokens each, and behind eight of them on every CTA items of
    more than 128 rows: the second half of the softmax warps waits for those from the start on, for
    over a second."""
    ctas, heads, d, size, pages = 152, 8, 64, 1024, 20000
    lengths, news = [pages * size, 129] * ctas, [1, 129] * ctas
    cache, q, _ = prompt_case(4, [2 * size], news, heads, heads, d, size, "e4m3_page")
    table = torch.zeros((2 * ctas, pages), dtype=torch.int32, device="cuda")
    offsets = ints(np.concatenate([[0], np.cumsum(news)]).tolist())
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    cache.attend_prompt(q, offsets, table, ints(lengths), out=out, lse=lse)
    end.record()
    assert binding.moe_device_status() == (0, 0)
    assert start.elapsed_time(end) > 1100
    # every page is the same one: the attention over it, and its sum that many times
    first = offsets[:-1].long()[::2]
    once, once_lse = cache.attend(q[first], table[::2, :1].contiguous(), ints([size] * ctas),
                                  return_lse=True)
    tiles = pages * size // 128
    # fp32 sums of a tile at a time, and of 16 tokens at a time (truncated): 2 u a step
    assert np.all(np.abs((lse[first] - once_lse).cpu().numpy() - np.log(pages)) <=
                  4 * tiles * U32 + 1e-4)
    kc, vc, ks, vs = host(cache)
    spread = np.abs(oracle.e4m3_decode(vc[0])).max(1) * vs[0][:, None]
    assert np.all(np.abs(values(out[first]) - values(once)) <=
                  (2 * 8 * tiles * U32 + 2.0 ** -10) * spread + 2 * HALF_BF16 * np.abs(values(once)))
    for b in range(0, ctas, 37):
        at = slice(int(offsets[2 * b + 1]), int(offsets[2 * b + 2]))
        check_prompt(Given(cache, out[at], lse[at]), q[at], np.zeros((1, 1), np.int32), [129], [129],
                     kind="e4m3_page")


class Given:
    """A cache with results that are there already."""

    def __init__(self, cache, out, lse):
        self.k, self.v, self.k_scale, self.v_scale = cache.k, cache.v, cache.k_scale, cache.v_scale
        self.out, self.lse = out, lse

    def attend_prompt(self, q, *call, out, lse, **kw):
        out.copy_(self.out)
        lse.copy_(self.lse)
        return out, lse


# ---------------------------------------------------------------------------
# rows of padding
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("streamed", [False, True])
def test_padding_of_new_outputs(kind, d, streamed):
    """Rows behind the last context's are zeros, with log-sums of -inf, in tensors that the call
    makes, whatever their memory held; in the caller's they stay."""
    lengths, news, pad = [4000, 60, 300], [70, 60, 2], 200
    cache, q, table = prompt_case(d, lengths, news, 6, 2, d, 32, kind, pad=pad)
    call = ints([0, 70, 130, 132]), torch.from_numpy(table).cuda(), ints(lengths)
    rows = len(q)
    out, lse = check_prompt(cache, q, table, lengths, news, kind=kind)
    stream = torch.cuda.Stream() if streamed else None
    torch.cuda.synchronize()

    def poison():       # what the next new tensors of these sizes are made of
        with torch.cuda.stream(stream):
            for _ in range(3):
                held = [torch.full((rows, 6, d), float("nan"), dtype=torch.bfloat16,
                                   device="cuda"),
                        torch.full((rows, 6), float("nan"), device="cuda")]
                del held

    def check(new, of, want, behind):
        torch.cuda.synchronize()
        if new:
            assert torch.equal(of[:132], want[:132]) and torch.all(of[132:] == behind)
        else:
            assert torch.equal(of, want)

    zero, none = 0.0, float("-inf")
    poison()
    check(True, cache.attend_prompt(q, *call, stream=stream), out, zero)
    poison()
    got = cache.attend_prompt(q, *call, return_lse=True, stream=stream)
    check(True, got[0], out, zero)
    check(True, got[1], lse, none)
    poison()
    given = torch.full_like(lse, 7.0)
    torch.cuda.synchronize()
    got = cache.attend_prompt(q, *call, lse=given, stream=stream)
    check(True, got[0], out, zero)
    check(False, got[1], lse, none)
    poison()
    given = torch.full_like(out, 7.0)
    torch.cuda.synchronize()
    got = cache.attend_prompt(q, *call, out=given, return_lse=True, stream=stream)
    check(False, got[0], out, zero)
    check(True, got[1], lse, none)


def test_padding_alone_and_wrong_ends():
    cache, q, table = prompt_case(2, [40], [40], 4, 2, 64, 16, "bf16")
    t, n = torch.from_numpy(table).cuda(), ints([40])
    out, lse = cache.attend_prompt(q, ints([0]), t[:0], ints([]), return_lse=True)
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))
    wide = torch.full((3, 40, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    need = binding.moe_prompt_attention_workspace_size(cache.struct, 4)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for end in (2 ** 31 - 1, -2 ** 31, -1, 41, 40, 0):
        wide.fill_(3.0)
        offsets = ints([0, end])
        assert binding.load_library().moe_prompt_attention_padded(
            ctypes.byref(cache.struct), q.data_ptr(), 256, 40, 4, offsets.data_ptr(), t.data_ptr(),
            t.shape[1], t.shape[1], n.data_ptr(), 1, 0.125, 0, wide[1].data_ptr(), 256, None,
            ws.data_ptr(), need, None) == 0
        torch.cuda.synchronize()
        assert torch.all(wide[0] == 3.0) and torch.all(wide[2] == 3.0)
        if end <= 0:
            assert torch.all(wide[1] == 0)
        if end > 40:
            assert torch.all(wide[1] == 3.0)


def test_padding_follows_the_lengths_of_a_captured_step():
    """A step of fixed size without outputs of the caller's, replayed with other lengths."""
    cache, q, table = prompt_case(6, [200, 300], [24, 40], 4, 2, 128, 16, "e4m3_page")
    t, n, o = torch.from_numpy(table).cuda(), ints([200, 300]), ints([0, 24, 64])
    cache.attend_prompt(q, o, t, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = cache.attend_prompt(q, o, t, n, return_lse=True)
    for news, lengths in (([24, 40], [200, 300]), ([1, 1], [9, 300]), ([0, 0], [9, 0]),
                          ([5, 0], [5, 77]), ([30, 34], [200, 34])):
        o.copy_(ints([0, news[0], sum(news)]))
        n.copy_(ints(lengths))
        graph.replay()
        end = sum(news)
        want = [torch.zeros_like(out), torch.full_like(lse, float("-inf"))]
        cache.attend_prompt(q, o, t, n, out=want[0], lse=want[1])
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        assert torch.all(out[end:] == 0) and torch.all(torch.isneginf(lse[end:]))


# ---------------------------------------------------------------------------
# scales far above a row's own, in tokens that it does not see
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("window", [0, 12])
@pytest.mark.parametrize("gap", [10, 21, 22, 24, 27, 30, 31, 34])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_scales_far_above_a_rows_own(d, gap, window):
    """Tokens from the 48th on (without a window: later ones; with one: the rows behind come to see
    them alone) with page scales 2^gap above those before, in one tile: rows that see the small
    ones only are within what the header states, exact up to 2^21, and see zeros from 2^31 on."""
    lengths, news, size = [60], [60], 16
    cache, q, table = prompt_case(gap, lengths, news, 4, 2, d, size, "e4m3_page", spread=0.0)
    for s in (cache.k_scale, cache.v_scale):
        s.fill_(2.0 ** -6)
        s[torch.from_numpy(table[0, 3:]).long().cuda()] = 2.0 ** (gap - 6)
    out, lse = cache.attend_prompt(q, ints([0, 60]), torch.from_numpy(table).cuda(), ints(lengths),
                                   window=window, return_lse=True)
    # a rounding of fp16 numbers down to 2^-24 that stand for scales 2^-6 of theirs
    off = 2.0 ** -25 * 2.0 ** (gap - 6 - 6) if gap > 21 else 0.0
    # (elements of 2^-31 of the largest scale and below: codes up to 448 times that)
    off = 448 * 2.0 ** -6 if gap >= 31 else off
    most = np.abs(values(q)).sum(-1) * d ** -0.5 * off
    ref, ref_lse, tol, lse_tol = bounds(cache, q, table, lengths, news, window=window, more=most)
    small = np.arange(60) < 48
    y, z = values(out)[small], lse.cpu().numpy()[small]
    if gap >= 31:
        assert np.all(y == 0)
        return
    assert np.all(np.abs(y - ref[small]) <= tol[small] + 1.01 * off)
    assert np.all(np.abs(z - ref_lse[small]) <= lse_tol[small])
