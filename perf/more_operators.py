"""Cases for the operators around a serving step's attention: block tables and
slot maps built on the GPU from request lengths, the paged cache in e4m3 with one
scale per page and head (written, and attended to by one new token a request),
and attention of many new tokens a request over the paged cache. `listed` and
`draw` give the cases, `prepare` the inputs, `run` one pass (in plain torch, or
through the package where `own` is set), `work` the bytes and operations a pass
cannot do without, and `exact` the results in 64 bits.
"""

import math

import torch

own = False

DEVICE = "cuda"
LEAST = -48      # the exponent of the smallest scale of a page


def listed():
    return [
        # one decode step of a serving batch: a token a request, some leave
        dict(name="plan step", op="plan", batch=128, longest=16384, new=1, page=64, rows=128,
             axes=1, leaving=9, idle=0, tight=False),
        # a prefill step that packs many prompts, with positions of three axes; the
        # pool runs out, so that the last requests wait
        dict(name="plan prompts", op="plan", batch=301, longest=2000, new=110, page=16,
             rows=16384, axes=3, leaving=7, idle=5, tight=True),
        # one decode step: q rotated, k rotated and both quantised into their pages
        dict(name="write step", op="write", batch=16, new=1, longest=40000, q_heads=64,
             kv_heads=4, dim=128, rot=128, page=64, padding=0),
        # a prompt's chunk
        dict(name="write prompt", op="write", batch=3, new=2731, longest=500, q_heads=64,
             kv_heads=4, dim=128, rot=128, page=64, padding=0),
        # keys and values that come rotated, chunks that begin inside a page, and
        # padding tokens without a slot behind each
        dict(name="write rotated", op="write", batch=37, new=433, longest=9000, q_heads=0,
             kv_heads=8, dim=128, rot=0, page=16, padding=3),
        # one new token a request: a serving batch from an empty slot to a long context
        dict(name="attend batch", op="attend", batch=128, longest=16384, ragged=True, q_heads=64,
             kv_heads=4, dim=128, page=64, window=0),
        # the same early in the answers, an odd group, a window: latency
        dict(name="attend short", op="attend", batch=9, longest=501, ragged=True, q_heads=10,
             kv_heads=2, dim=256, page=16, window=200),
        # a few drafted tokens of every request, checked against long contexts
        dict(name="prompt drafts", op="prompt", batch=32, longest=16384, new=5, q_heads=64,
             kv_heads=4, dim=128, page=64, cache="blocks", window=0, padding=0),
        # a whole prompt, compute bound
        dict(name="prompt whole", op="prompt", batch=1, longest=8192, new=8192, q_heads=64,
             kv_heads=4, dim=128, page=64, cache="blocks", window=0, padding=0),
        # a chunk of a long document's prompt, scales per token
        dict(name="prompt chunk", op="prompt", batch=1, longest=40001, new=2048, q_heads=64,
             kv_heads=4, dim=128, page=64, cache="tokens", window=0, padding=0),
        # many prompts packed into one step, a bf16 cache, small heads, a window
        dict(name="prompt packed", op="prompt", batch=48, longest=1500, new=300, q_heads=40,
             kv_heads=8, dim=64, page=16, cache="bf16", window=512, padding=11),
        # a few short prompts with wide heads
        dict(name="prompt short", op="prompt", batch=9, longest=700, new=170, q_heads=10,
             kv_heads=2, dim=256, page=16, cache="blocks", window=0, padding=0),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("plan", "write", "attend", "prompt", "prompt", "prompt"))
    page = rng.choice((8, 16, 32, 64, 128))
    if op == "plan":
        batch = _log(rng, 1, 512)
        longest = _log(rng, 20, 16384)
        new = rng.choice((1, 1, _log(rng, 1, max(1, 16384 // batch))))
        rows = batch * new + rng.choice((0, 0, 37))
        return dict(op=op, batch=batch, longest=longest, new=new, page=page, rows=rows,
                    axes=rng.choice((1, 1, 3)), leaving=rng.choice((0, 3, 10)),
                    idle=rng.choice((0, 4)), tight=rng.random() < 0.3)
    dim = rng.choice((64, 128, 128, 256))
    kv_heads = rng.choice((1, 2, 3, 4, 8))
    group = rng.choice((1, 4, 5, 7, 8, 12, 16, 20))
    if op == "write":
        most = max(1, min(16384, (8192 * 68 * 128) // (kv_heads * (group + 2) * dim)))
        tokens = _log(rng, 1, most)
        batch = _log(rng, 1, min(tokens, 128))
        fused = rng.random() < 0.6
        return dict(op=op, batch=batch, new=max(1, tokens // batch),
                    longest=_log(rng, 20, 10000), q_heads=group * kv_heads if fused else 0,
                    kv_heads=kv_heads, dim=dim, rot=rng.choice((dim, dim // 2)) if fused else 0,
                    page=page, padding=rng.choice((0, 0, 5)))
    if op == "attend":
        batch = _log(rng, 1, 128)
        longest = _log(rng, 1, max(1, min(131072, (1 << 29) // (kv_heads * dim * batch))))
        return dict(op=op, batch=batch, longest=longest, ragged=rng.random() < 0.7,
                    q_heads=group * kv_heads, kv_heads=kv_heads, dim=dim, page=page,
                    window=rng.choice((0, 0, 0, _log(rng, 1, longest))))
    # pairs of (row, token): at most an eighth of the whole prompt's, 2^25 of each of
    # 64 heads of 128 elements
    batch = _log(rng, 1, 32)
    q_heads = group * kv_heads
    pairs = (1 << 28) * 128 // (q_heads * dim * batch)
    new = _log(rng, 1, max(1, min(4096 // batch, int(math.sqrt(pairs)))))
    longest = max(new, _log(rng, 20, max(20, min(65536 // batch, pairs // new))))
    return dict(op=op, batch=batch, longest=longest, new=new, q_heads=q_heads,
                kv_heads=kv_heads, dim=dim, page=page,
                cache=rng.choice(("blocks", "blocks", "tokens", "bf16")),
                window=rng.choice((0, 0, 0, _log(rng, 1, longest))),
                padding=rng.choice((0, 0, 9)))


def _spread(top, n, least=0):
    """n numbers spread evenly from `least` to `top` (one: top)."""
    return [top] if n == 1 else [least + (top - least) * i // (n - 1) for i in range(n)]


def _lengths(case):
    """Context lengths, the new tokens counted."""
    n, top = case["batch"], case["longest"]
    if case["op"] == "prompt":
        return [max(a, b) for a, b in zip(_spread(top, n), _news(case))]
    if case["op"] == "write":   # held before the step
        return [x + y for x, y in zip(_spread(top, n), _news(case))]
    return _spread(top, n) if case["ragged"] else [top] * n


def _news(case):
    """New tokens of each request: the first has half, the last all of `new`."""
    return _spread(case["new"], case["batch"], least=(case["new"] + 1) // 2)


def _pages_of(tokens, page):
    return -(-tokens // page)


def _kinds(case):
    """A plan's requests: held tokens, and new ones (-1: the request leaves)."""
    held, new = _spread(case["longest"], case["batch"]), _news(case)
    for b in range(case["batch"]):
        if case["leaving"] and b % case["leaving"] == case["leaving"] // 2:
            new[b] = -1
        elif case["idle"] and b % case["idle"] == 0:
            new[b] = 0
    return held, new


def _taken(case):
    held, new = _kinds(case)
    p = case["page"]
    return [_pages_of(h + n, p) - _pages_of(h, p) if n > 0 else 0 for h, n in zip(held, new)]


def work(case):
    if case["op"] == "plan":
        n, taken = case["batch"], sum(_taken(case))
        held, new = _kinds(case)
        freed = sum(_pages_of(h, case["page"]) for h, m in zip(held, new) if m < 0)
        return {"bytes": 16 * n + case["rows"] * 4 * (1 + case["axes"]) + 8 * (taken + freed),
                "flops": 0}
    d, hk, hq = case["dim"], case["kv_heads"], case["q_heads"]
    page = case["page"]
    if case["op"] == "write":
        t = sum(_news(case))
        rows = t + case["batch"] * case["padding"]
        pages = sum(_pages_of(n, page) - (n - m) // page
                    for n, m in zip(_lengths(case), _news(case)))
        place = 4 * rows if case["rot"] else 0
        return {"bytes": 4 * rows * hq * d + t * hk * 6 * d + 8 * pages * hk + 4 * rows + place,
                "flops": 3 * t * (hq + hk) * case["rot"] + 3 * t * hk * d}
    lengths, w = _lengths(case), case["window"]
    news = _news(case) if case["op"] == "prompt" else [min(n, 1) for n in lengths]
    seen = pairs = 0
    for n, m in zip(lengths, news):
        reach = min(n, w + m - 1) if w > 0 else n
        seen += reach if m else 0
        # row i of m sees the tokens up to n - m + i, at most w of them
        first = n - m + 1
        if w == 0 or w >= n:
            pairs += m * (first + n) // 2
        else:
            under = max(0, min(m, w - first))   # rows that see fewer than w
            pairs += under * (2 * first + under - 1) // 2 + (m - under) * w
    kind = case.get("cache", "blocks")
    row = 4 * d if kind == "bf16" else 2 * d + (8 if kind == "tokens" else 0)
    scales = 8 * hk * _pages_of(seen, page) if kind == "blocks" else 0
    rows = sum(news) if case["op"] == "prompt" else case["batch"]
    return {"bytes": seen * hk * row + scales + 4 * _pages_of(seen, page) + 8 * case["batch"] +
            rows * hq * (4 * d + 4),
            "flops": 4 * d * pairs * hq}


def _exponent(amax):
    """The least e >= LEAST with amax <= 448 * 2^e (448 = 0.875 * 2^9)."""
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(amax > 0, e, LEAST).clamp(min=LEAST)


def _power(e):
    """2^e in fp32, from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _coded(x, scale):
    return (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _filled(case, pages, g):
    """A cache of `pages` pages that earlier steps have filled. Keys have a
    few strong channels and tokens differ in size, as projections' do."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    channel = torch.ones(case["dim"], device=DEVICE)
    channel[::13] = 3.0
    made, kind = {}, case.get("cache", "blocks")
    for n, weight in (("k", channel), ("v", None)):
        x = torch.randn(shape, generator=g, device=DEVICE)
        x *= torch.exp(0.5 * torch.randn(shape[:3] + (1,), generator=g, device=DEVICE))
        if weight is not None:
            x *= weight
        if kind == "bf16":
            made[n] = x.to(torch.bfloat16)
            continue
        if kind == "blocks":
            scale = _power(_exponent(x.abs().amax((-1, -2))))
            made[n] = _coded(x, scale[..., None, None])
        else:
            scale = x.abs().amax(-1) / 448.0
            made[n] = _coded(x, scale[..., None])
        made[n], made[n + "_scale"] = made[n].view(torch.uint8), scale
    return made


def _paged(lengths, page, spare, g, least=0):
    """A block table for contexts of these lengths on shuffled pages, and the
    number of pages; entries past a context's pages are -1, and so are those of
    pages before token `least[b]`, which have been given back."""
    count = [_pages_of(n, page) for n in lengths]
    wide = max(1, max(count))
    pages = sum(count) + spare
    count = torch.tensor(count, device=DEVICE)
    column = torch.arange(wide, device=DEVICE)
    held = column < count[:, None]
    ids = (torch.cumsum(held.reshape(-1), 0) - 1).reshape(held.shape).clamp(min=0)
    shuffled = torch.randperm(pages, generator=g, device=DEVICE)
    table = torch.where(held, shuffled[ids], -1)
    if least:
        table[column < torch.tensor(least, device=DEVICE)[:, None] // page] = -1
    return table.to(torch.int32), pages, shuffled[int(count.sum()):].to(torch.int32)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEVICE)


def _offsets(news):
    out = [0]
    for n in news:
        out.append(out[-1] + n)
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    state = {"case": case, "kept": {}}
    if case["op"] == "plan":
        held, new = _kinds(case)
        # requests arrive in any order
        order = torch.randperm(case["batch"], generator=g, device=DEVICE)
        taken = sum(_taken(case))
        wide = [h + max(0, n) + 3 * case["page"] for h, n in zip(held, new)]
        table, pages, free = _paged(held, case["page"], taken + 5, g)
        room = _pages_of(max(wide), case["page"])
        state["table"] = torch.full((case["batch"], room), -1, dtype=torch.int32, device=DEVICE)
        state["table"][:, :table.shape[1]] = table
        state["table"] = state["table"][order].contiguous()
        state["held"], state["new"] = _ints(held)[order], _ints(new)[order]
        state["pages"] = pages
        state["stack"] = torch.zeros(pages, dtype=torch.int32, device=DEVICE)
        # a tight pool has half the pages that the step asks for, and those that leave
        count = taken // 2 if case["tight"] else len(free)
        state["stack"][:count] = free[:count]
        state["state"] = torch.cat((state["held"], _ints([count])))
        return state
    d, hk, hq = case["dim"], case["kv_heads"], case["q_heads"]
    lengths, page = _lengths(case), case["page"]
    if case["op"] == "write":
        news = _news(case)
        table, pages, _ = _paged(lengths, page, 3, g)
        for n, x in _filled(case, pages, g).items():
            state["cache_" + n] = x
        # tokens request by request, each followed by its padding
        b, at = [], []
        for i, (n, m) in enumerate(zip(lengths, news)):
            b += [i] * (m + case["padding"])
            at += list(range(n - m, n)) + [-1] * case["padding"]
        b, at = torch.tensor(b, device=DEVICE), torch.tensor(at, device=DEVICE)
        slots = table[b, at.clamp(min=0) // page] * page + at.clamp(min=0) % page
        state["slots"] = torch.where(at >= 0, slots, -1).to(torch.int32)
        # q, k and v as a projection leaves them: side by side in a row
        wide = torch.randn((len(b), (hq + 2 * hk) * d), generator=g, device=DEVICE)
        wide *= torch.exp(0.5 * torch.randn((len(b), 1), generator=g, device=DEVICE))
        wide = wide.to(torch.bfloat16)
        state["q"] = wide[:, :hq * d].unflatten(1, (hq, d)) if hq else None
        state["k"] = wide[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        state["v"] = wide[:, (hq + hk) * d:].unflatten(1, (hk, d))
        if case["rot"]:
            i = torch.arange(0, case["rot"], 2, dtype=torch.float64, device=DEVICE)
            state["inv_freq"] = 1000000.0 ** (-i / case["rot"])
            state["positions"] = at.clamp(min=0).to(torch.int32)[None].contiguous()
        return state
    w = case["window"]
    news = _news(case) if case["op"] == "prompt" else [min(n, 1) for n in lengths]
    least = [max(0, n - m + 1 - w) for n, m in zip(lengths, news)] if w else 0
    state["table"], pages, _ = _paged(lengths, page, 2, g, least)
    for n, x in _filled(case, pages, g).items():
        state["cache_" + n] = x
    state["lengths"] = _ints(lengths)
    rows = case["batch"]
    if case["op"] == "prompt":
        state["ends"] = _offsets(news)
        state["offsets"] = _ints(state["ends"])
        state["contexts"] = lengths
        rows = state["ends"][-1] + case["padding"]
        # (a step of fixed size keeps its output buffers; rows of padding stay)
        state["out"] = torch.zeros((rows, hq, d), dtype=torch.bfloat16, device=DEVICE)
        state["lse"] = torch.zeros((rows, hq), device=DEVICE)
    q = torch.randn((rows, hq, d), generator=g, device=DEVICE)
    state["q"] = (1.5 * q).to(torch.bfloat16)
    return state


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_plan(state):
    case, table, stack = state["case"], state["table"], state["stack"]
    page, rows, pages = case["page"], case["rows"], state["pages"]
    held, new = state["state"][:-1].long(), state["new"].long()
    count = state["state"][-1].long()
    batch, wide = table.shape
    have = (held + page - 1) // page
    column = torch.arange(wide, device=DEVICE)
    # pages of requests that leave go onto the stack
    back = (new < 0)[:, None] & (column < have[:, None]) & (table >= 0) & (table < pages)
    to = count + torch.cumsum(back.reshape(-1), 0) - 1
    to = torch.where(back.reshape(-1), to, pages).clamp(max=pages)
    longer = torch.cat((stack, stack[:1]))
    longer[to] = table.reshape(-1)
    stack.copy_(longer[:pages])
    free = count + back.sum()
    # requests are served in order while pages and rows last
    fits = (new >= 0) & (held + new <= wide * page)
    need = torch.where(fits, (held + new + page - 1) // page - have, 0)
    asked, tokens = torch.cumsum(need, 0), torch.cumsum(torch.where(fits, new, 0), 0)
    served = fits & (asked <= free) & (tokens <= rows)
    grown = torch.where(served, new, 0)
    offsets = torch.zeros(batch + 1, dtype=torch.int64, device=DEVICE)
    offsets[1:] = torch.cumsum(grown, 0)
    # the k-th page taken is the k-th from the stack's top
    rank = column - have[:, None]
    takes = served[:, None] & (rank >= 0) & (rank < need[:, None])
    k = (asked - need)[:, None] + rank
    got = stack[(free - 1 - k).clamp(min=0, max=pages - 1)]
    table.copy_(torch.where(takes, got, table))
    row = torch.arange(rows, device=DEVICE)
    b = torch.searchsorted(offsets[1:].contiguous(), row, right=True).clamp(max=batch - 1)
    live = row < offsets[-1]
    at = torch.where(live, held[b] + row - offsets[b], 0)
    slots = table[b, (at // page).clamp(max=wide - 1)].long() * page + at % page
    left = free - torch.where(served, need, 0).sum()
    after = torch.where(new < 0, 0, held + grown)
    refused = ((new > 0) & ~served).sum()
    return {"table": table, "stack": stack, "offsets": offsets.to(torch.int32),
            "slots": torch.where(live, slots, -1).to(torch.int32),
            "positions": at.to(torch.int32).expand(case["axes"], rows).contiguous(),
            "state": torch.cat((after, left[None])).to(torch.int32),
            "refused": refused[None].to(torch.int32)}


def _turn(x, cos, sin, rot):
    """The rotated dimensions of x [T, H, D] in fp32, the others as they are."""
    x = x.float()
    a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    cos, sin = cos[:, None], sin[:, None]
    return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., rot:]), -1)


def _plain_write(state):
    case, out = state["case"], {}
    slots, page = state["slots"].long(), case["page"]
    k, v = state["k"].float(), state["v"].float()
    if case["rot"]:
        angle = state["positions"][0].double()[:, None] * state["inv_freq"]
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
        out["q"] = _turn(state["q"], cos, sin, case["rot"]).to(torch.bfloat16)
        k = _turn(k, cos, sin, case["rot"])
    pages = state["cache_k"].shape[0]
    # (tokens without a slot go to a page behind the cache's)
    at = torch.where(slots >= 0, slots, pages * page)
    for n, x in (("k", k), ("v", v)):
        codes, scale = state["cache_" + n], state["cache_" + n + "_scale"]
        index = (at // page)[:, None].expand(x.shape[:2])
        amax = torch.full((pages + 1, case["kv_heads"]), -1.0, device=DEVICE)
        amax.scatter_reduce_(0, index, x.abs().amax(-1), "amax")
        begun = torch.zeros(pages * page + page, dtype=torch.bool, device=DEVICE)
        begun[at] = True
        begun = begun.view(-1, page)[:pages, 0, None]
        touched, amax = amax[:pages] >= 0, amax[:pages]
        mine = _power(_exponent(amax))
        new = torch.where(begun, mine, torch.maximum(scale, mine))
        new = torch.where(touched, new, scale)
        # codes that stay, under the new scale
        factor = (scale / new)[..., None, None]
        old = codes.view(torch.float8_e4m3fn).float() * factor
        stays = (touched & ~begun & (new > scale))[..., None, None]
        codes.copy_(torch.where(stays, old.to(torch.float8_e4m3fn).view(torch.uint8), codes))
        row = _coded(x, torch.cat((new, new[:1]))[at // page][..., None]).view(torch.uint8)
        longer = torch.cat((codes, codes[:1]))
        longer[at // page, :, at % page] = row
        codes.copy_(longer[:pages])
        scale.copy_(new)
    return {**out, **_cache_values(state)}


def _cache_values(state):
    """The cache after a write: codes as the e4m3 values they are, and scales."""
    return {"k": state["cache_k"].view(torch.float8_e4m3fn),
            "v": state["cache_v"].view(torch.float8_e4m3fn),
            "k_scale": state["cache_k_scale"], "v_scale": state["cache_v_scale"]}


def _fetch(state, name, page, at):
    """fp32 rows [..., H, D] of the cache at (page, at)."""
    x = state["cache_" + name]
    if x.dtype == torch.bfloat16:
        return x[page, :, at].float()
    scale = state["cache_" + name + "_scale"]
    scale = scale[page] if scale.dim() == 2 else scale[page, :, at]
    return x.view(torch.float8_e4m3fn)[page, :, at].float() * scale[..., None]


def _plain_attend(state):
    case, page = state["case"], state["case"]["page"]
    b, hq, d = state["q"].shape
    hk = case["kv_heads"]
    token = torch.arange(case["longest"], device=DEVICE)
    entry = state["table"].long()[:, token // page]                       # [B, L]
    length = state["lengths"].long()[:, None]
    here = (token < length) & (entry >= 0)
    if case["window"] > 0:
        here = here & (token >= length - case["window"])
    at = (token % page).expand_as(entry)
    entry = entry.clamp(min=0)
    k = _fetch(state, "k", entry, at).permute(0, 2, 3, 1)                  # [B, H, D, L]
    q = state["q"].float().reshape(b, hk, hq // hk, d)
    s = torch.matmul(q, k) * (1.0 / math.sqrt(d))
    del k
    s = s.masked_fill(~here[:, None, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top.isinf(), 0.0, top))
    total = p.sum(-1, keepdim=True)
    v = _fetch(state, "v", entry, at)
    v = torch.where(here[..., None, None], v, 0.0).permute(0, 2, 1, 3)     # [B, H, L, D]
    out = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = torch.log(total) + torch.where(top.isinf(), 0.0, top)
    return out.reshape(b, hq, d).to(torch.bfloat16), lse.reshape(b, hq)


MOST_SCORES = 1 << 28    # scores that the plain form holds at a time


def _plain_prompt(state):
    case, page, w = state["case"], state["case"]["page"], state["case"]["window"]
    d, hk = case["dim"], case["kv_heads"]
    group = case["q_heads"] // hk
    ends = state["ends"]
    for b, n in enumerate(state["contexts"]):
        s, e = ends[b], ends[b + 1]
        first = n - (e - s)                       # the first new token
        least = max(0, first + 1 - w) if w else 0
        token = torch.arange(least, n, device=DEVICE)
        entry = state["table"][b].long()[token // page]
        k = _fetch(state, "k", entry, token % page).permute(1, 2, 0)      # [H, D, n]
        v = _fetch(state, "v", entry, token % page).permute(1, 0, 2)
        step = max(1, MOST_SCORES // (group * (n - least)))
        for h in range(hk):
            heads = slice(h * group, (h + 1) * group)
            for r in range(s, e, step):
                z = min(e, r + step)
                q = state["q"][r:z, heads].float().reshape(-1, d)
                x = torch.matmul(q, k[h]) * (1.0 / math.sqrt(d))
                x = x.view(z - r, group, n - least)
                own_at = first + torch.arange(r - s, z - s, device=DEVICE)[:, None]
                seen = token <= own_at
                if w:
                    seen = seen & (token > own_at - w)
                x.masked_fill_(~seen[:, None], float("-inf"))
                top = x.amax(-1, keepdim=True)
                p = torch.exp(x - top)
                total = p.sum(-1, keepdim=True)
                y = torch.matmul(p.view(-1, n - least), v[h]).view(z - r, group, d) / total
                state["out"][r:z, heads] = y.to(torch.bfloat16)
                state["lse"][r:z, heads] = (torch.log(total) + top)[..., 0]
    return state["out"], state["lse"]


# ---------------------------------------------------------------------------
# the package's operators
# ---------------------------------------------------------------------------
def _cache(state):
    if "cache" not in state["kept"]:
        from expert_layer_ptpc_gb300.attention import PagedKVCache
        state["kept"]["cache"] = PagedKVCache.from_tensors(
            state["cache_k"], state["cache_v"], state.get("cache_k_scale"),
            state.get("cache_v_scale"))
    return state["kept"]["cache"]


def _own_plan(state):
    case = state["case"]
    if "pool" not in state["kept"]:
        from expert_layer_ptpc_gb300.attention import PagePool
        state["kept"]["pool"] = PagePool.from_tensors(state["table"], state["stack"],
                                                      state["state"], case["page"])
    plan = state["kept"]["pool"].plan(state["new"], case["rows"], axes=case["axes"])
    return {"table": state["table"], "stack": state["stack"], "offsets": plan.offsets,
            "slots": plan.slots, "positions": plan.positions, "state": plan.state,
            "refused": plan.refused}


def _own_write(state):
    cache, out = _cache(state), {}
    if state["case"]["rot"]:
        if "rotary" not in state["kept"]:
            from expert_layer_ptpc_gb300.attention import Rotary
            state["kept"]["rotary"] = Rotary(state["inv_freq"])
        out["q"] = cache.write_rotary(state["kept"]["rotary"], state["positions"], state["q"],
                                      state["k"], state["v"], state["slots"])
    else:
        cache.write(state["k"], state["v"], state["slots"])
    return {**out, **_cache_values(state)}


def _own_attend(state):
    return _cache(state).attend(state["q"], state["table"], state["lengths"],
                                window=state["case"]["window"], return_lse=True)


def _own_prompt(state):
    return _cache(state).attend_prompt(state["q"], state["offsets"], state["table"],
                                       state["lengths"], window=state["case"]["window"],
                                       out=state["out"], lse=state["lse"])


def run(state):
    if own:
        return {"plan": _own_plan, "write": _own_write, "attend": _own_attend,
                "prompt": _own_prompt}[state["case"]["op"]](state)
    return {"plan": _plain_plan, "write": _plain_write, "attend": _plain_attend,
            "prompt": _plain_prompt}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------
def _exact_plan(state):
    """Request by request, on the host."""
    case, page = state["case"], state["case"]["page"]
    table, stack = state["table"].tolist(), state["stack"].tolist()
    *held, count = state["state"].tolist()
    new, pages, wide = state["new"].tolist(), state["pages"], state["table"].shape[1]
    free, after = stack[:count], list(held)
    for b, n in enumerate(new):
        if n < 0:
            free += [p for p in table[b][:_pages_of(held[b], page)] if 0 <= p < pages]
            after[b] = 0
    stack[:len(free)] = free
    slots, at, offsets, refused, full = [], [], [0], 0, False
    for b, n in enumerate(new):
        if n >= 0 and held[b] + n <= wide * page:
            need = _pages_of(held[b] + n, page) - _pages_of(held[b], page)
            full = full or need > len(free) or len(slots) + n > case["rows"]
            if not full:
                for i in range(need):
                    table[b][_pages_of(held[b], page) + i] = free.pop()
                for t in range(held[b], held[b] + n):
                    slots.append(table[b][t // page] * page + t % page)
                    at.append(t)
                after[b] = held[b] + n
            refused += full and n > 0
        elif n > 0:
            refused += 1
        offsets.append(len(slots))
    slots += [-1] * (case["rows"] - len(slots))
    at += [0] * (case["rows"] - len(at))
    return {"table": _ints(table), "stack": _ints(stack), "offsets": _ints(offsets),
            "slots": _ints(slots), "positions": _ints([at] * case["axes"]),
            "state": _ints(after + [len(free)]), "refused": _ints([refused])}


def _exact_turn(state, name):
    """Each rotated pair as a complex number times e^(i angle)."""
    rot = state["case"]["rot"]
    x = state[name].double().clone()
    angle = state["positions"][0].double()[:, None] * state["inv_freq"]
    z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot])
    z = z * torch.polar(torch.ones_like(angle), angle)[:, None]
    x[..., :rot // 2], x[..., rot // 2:rot] = z.real, z.imag
    return x


def _least_power(x):
    """The least power of two from 2^LEAST on that is not below x."""
    m, e = math.frexp(max(x, 2.0 ** LEAST))
    return 2.0 ** (e - 1 if m == 0.5 else e)


def _exact_write(state):
    """Page by page: what the call's tokens bring to each, and what was there."""
    case, out, size = state["case"], {}, state["case"]["page"]
    if case["rot"]:
        out["q"] = _exact_turn(state, "q")
    slots = state["slots"].tolist()
    by_page = {}
    for t, s in enumerate(slots):
        if s >= 0:
            by_page.setdefault(s // size, []).append((t, s % size))
    for n in ("k", "v"):
        x = _exact_turn(state, n) if n == "k" and case["rot"] else state[n].double()
        scale = state["cache_" + n + "_scale"].double().clone()
        whole = state["cache_" + n].view(torch.float8_e4m3fn).double()
        for p, tokens in by_page.items():
            rows = x[[t for t, _ in tokens]]                              # [n, H, D]
            ratio = rows.abs().amax((0, 2)).tolist()
            least = torch.tensor([_least_power(r / 448.0) for r in ratio], device=DEVICE,
                                 dtype=torch.float64)
            if all(at != 0 for _, at in tokens):
                new = torch.maximum(scale[p], least)
                whole[p] *= (scale[p] / new)[:, None, None]
            else:
                new = least
            scale[p] = new
            whole[p][:, [at for _, at in tokens]] = (rows / new[:, None]).transpose(0, 1)
        out[n], out[n + "_scale"] = whole, scale
    return out


def _exact_context(state, b, first, last):
    """Keys and values [n, H, D] of tokens first..last-1 of context b."""
    size, got = state["case"]["page"], []
    for n in ("k", "v"):
        x = state["cache_" + n]
        pages = state["table"][b, first // size:-(-last // size)].long()
        if x.dtype == torch.uint8:
            scale = state["cache_" + n + "_scale"][pages].double()
            scale = scale[..., None] if scale.dim() == 2 else scale
            rows = x.view(torch.float8_e4m3fn)[pages].double() * scale[..., None]
        else:
            rows = x[pages].double()
        rows = rows.transpose(1, 2).flatten(0, 1)
        got.append(rows[first % size:first % size + last - first])
    return got


def _exact_attend(state):
    case = state["case"]
    hq, d, hk, w = case["q_heads"], case["dim"], case["kv_heads"], case["window"]
    out = torch.zeros((case["batch"], hq, d), dtype=torch.float64, device=DEVICE)
    lse = torch.full((case["batch"], hq), float("-inf"), dtype=torch.float64, device=DEVICE)
    for b, n in enumerate(state["lengths"].tolist()):
        if n == 0:
            continue
        k, v = _exact_context(state, b, max(0, n - w) if w else 0, n)
        for h in range(hq):
            s = k[:, h // (hq // hk)] @ state["q"][b, h].double() / math.sqrt(d)
            lse[b, h] = torch.logsumexp(s, 0)
            out[b, h] = torch.softmax(s, 0) @ v[:, h // (hq // hk)]
    return out, lse


def _exact_prompt(state):
    """Head by head and in blocks of queries, each over the tokens up to its last."""
    case = state["case"]
    hq, d, hk, w = case["q_heads"], case["dim"], case["kv_heads"], case["window"]
    out, lse = state["out"].double(), state["lse"].double()
    ends, block = state["ends"], 1024
    for b, n in enumerate(state["contexts"]):
        first = n - (ends[b + 1] - ends[b])
        for r in range(ends[b], ends[b + 1], block):
            z = min(r + block, ends[b + 1])
            at = first + torch.arange(r - ends[b], z - ends[b], device=DEVICE)
            last = first + z - ends[b]
            start = max(0, first + r - ends[b] + 1 - w) if w else 0
            k, v = _exact_context(state, b, start, last)
            token = torch.arange(start, last, device=DEVICE)
            hide = token > at[:, None]
            if w:
                hide |= token <= at[:, None] - w
            for h in range(hq):
                s = state["q"][r:z, h].double() @ k[:, h // (hq // hk)].t() / math.sqrt(d)
                s.masked_fill_(hide, float("-inf"))
                lse[r:z, h] = torch.logsumexp(s, -1)
                out[r:z, h] = torch.softmax(s, -1) @ v[:, h // (hq // hk)]
    return out, lse


def exact(case, seed):
    state = prepare(case, seed)
    return {"plan": _exact_plan, "write": _exact_write, "attend": _exact_attend,
            "prompt": _exact_prompt}[case["op"]](state)
