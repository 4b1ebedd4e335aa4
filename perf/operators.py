"""Cases for the attention operators that stand next to the MoE layer in a
decoder block: rotary positions with several axes, the paged key-value cache
(quantised as it is written, and read back), and attention of one new token
over that cache. `listed` and `draw` give the cases, `prepare` the inputs,
`run` one pass (in plain torch, or through the package where `own` is set),
`work` the bytes and operations a pass cannot do without, and `exact` the
results in 64 bits.
"""

import math

import torch

own = False

DEVICE = "cuda"


def listed():
    return [
        # one decode step of a small batch: the rotation is latency
        dict(name="rotary step", op="rotary", tokens=16, q_heads=64, kv_heads=4, dim=128,
             rot=128, axes=3, woven=True, neighbours=False, inverse=False, far=40000),
        # a prefill chunk with images: three axes in blocks, memory bound
        dict(name="rotary prompt", op="rotary", tokens=8192, q_heads=64, kv_heads=4, dim=128,
             rot=128, axes=3, woven=False, neighbours=False, inverse=False, far=9000),
        # gradients of q and k through a partial rotation, an odd token count,
        # positions far out in a long document
        dict(name="rotary gradient", op="rotary", tokens=4099, q_heads=16, kv_heads=2, dim=256,
             rot=64, axes=3, woven=True, neighbours=True, inverse=True, far=1000000),
        # one decode step: q rotated, k rotated and quantised, v quantised
        dict(name="write step", op="write", tokens=16, q_heads=64, kv_heads=4, dim=128, rot=128,
             axes=3, woven=True, neighbours=False, far=40000, page=64, cache="e4m3", skipped=0),
        # the same for a prefill chunk
        dict(name="write prompt", op="write", tokens=8192, q_heads=64, kv_heads=4, dim=128,
             rot=128, axes=3, woven=True, neighbours=False, far=9000, page=64, cache="e4m3",
             skipped=0),
        # keys and values that come rotated, with padding tokens that have no slot
        dict(name="write rotated", op="write", tokens=16001, q_heads=0, kv_heads=8, dim=128,
             rot=0, axes=1, woven=False, neighbours=False, far=1, page=16, cache="e4m3",
             skipped=9),
        # a cached prefix of a few requests, read back for a prefill chunk
        dict(name="read prefixes", op="read", batch=9, longest=700, ragged=True, kv_heads=2,
             dim=256, page=16, cache="e4m3"),
        # a long document read back
        dict(name="read long", op="read", batch=2, longest=60001, ragged=False, kv_heads=4,
             dim=128, page=64, cache="e4m3"),
        # one request early in its answer: latency
        dict(name="attend one", op="attend", batch=1, longest=300, ragged=False, q_heads=64,
             kv_heads=4, dim=128, page=64, cache="e4m3", window=0),
        # one request over a very long document: the length is split
        dict(name="attend long", op="attend", batch=1, longest=262143, ragged=False, q_heads=64,
             kv_heads=4, dim=128, page=64, cache="e4m3", window=0),
        # a serving batch, from an empty slot to a long context
        dict(name="attend batch", op="attend", batch=128, longest=16384, ragged=True, q_heads=64,
             kv_heads=4, dim=128, page=64, cache="e4m3", window=0),
        # a bf16 cache, small heads, an odd group, a sliding window
        dict(name="attend window", op="attend", batch=48, longest=6000, ragged=True, q_heads=40,
             kv_heads=8, dim=64, page=16, cache="bf16", window=2048),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("rotary", "write", "read", "attend", "attend"))
    dim = rng.choice((64, 128, 128, 256))
    kv_heads = rng.choice((1, 2, 3, 4, 8))
    group = rng.choice((1, 4, 5, 7, 8, 12, 16, 20))
    page = rng.choice((8, 16, 32, 64, 128))
    cache = rng.choice(("e4m3", "e4m3", "bf16"))
    turn = dict(axes=rng.choice((1, 2, 3, 3)), woven=rng.random() < 0.5,
                neighbours=rng.random() < 0.3, far=_log(rng, 100, 1000000))
    rot = rng.choice((dim, dim, dim // 2, 32))
    if op in ("rotary", "write"):
        most = max(1, min(16384, (8192 * 68 * 128) // (kv_heads * (group + 2) * dim)))
        tokens = _log(rng, 1, most)
        if op == "rotary":
            return dict(op=op, tokens=tokens, q_heads=group * kv_heads, kv_heads=kv_heads,
                        dim=dim, rot=rot, inverse=rng.random() < 0.5, **turn)
        fused = rng.random() < 0.6
        return dict(op=op, tokens=tokens, q_heads=group * kv_heads if fused else 0,
                    kv_heads=kv_heads, dim=dim, rot=rot if fused else 0, page=page, cache=cache,
                    skipped=rng.choice((0, 0, 5)), **turn)
    batch = _log(rng, 1, 128)
    row = kv_heads * dim * (2 if cache == "bf16" else 1)
    most = (1 << 26) if op == "read" else (1 << 29)
    longest = _log(rng, 1, max(1, min(131072, most // (row * batch))))
    case = dict(op=op, batch=batch, longest=longest, ragged=rng.random() < 0.7,
                kv_heads=kv_heads, dim=dim, page=page, cache=cache)
    if op == "attend":
        case.update(q_heads=group * kv_heads,
                    window=rng.choice((0, 0, 0, _log(rng, 1, longest))))
    return case


def _lengths(case):
    """Context lengths: all the longest, or spread evenly from 0 to it."""
    n, top = case["batch"], case["longest"]
    if not case["ragged"] or n == 1:
        return [top] * n
    return [top * i // (n - 1) for i in range(n)]


def _seen(case):
    """Tokens of each context that take part (those inside the window)."""
    w = case.get("window", 0)
    return [min(n, w) if w > 0 else n for n in _lengths(case)]


def _pair_axis(case):
    """The axis of each rotated pair: blocks of pairs, or axes in turn."""
    pairs, axes = case["rot"] // 2, case["axes"]
    if case["woven"]:
        return [i % axes for i in range(pairs)]
    size = -(-pairs // axes)
    return [i // size for i in range(pairs)]


def work(case):
    d = case["dim"]
    if case["op"] in ("rotary", "write"):
        t, hq, hk = case["tokens"], case["q_heads"], case["kv_heads"]
        place = 4 * case["axes"] * t if case["rot"] else 0
        turned = t * (hq + hk) * case["rot"]
        if case["op"] == "rotary":
            return {"bytes": 4 * t * (hq + hk) * d + place, "flops": 3 * turned}
        kept = t - (-(-t // case["skipped"]) if case["skipped"] else 0)
        out = kept * hk * (2 * d + 8 if case["cache"] == "e4m3" else 4 * d)
        read = t * hq * d * 2 + kept * hk * d * 4
        return {"bytes": read + 2 * t * hq * d + out + place + 4 * t,
                "flops": 3 * turned + 3 * kept * hk * d}
    row = 2 * d + 8 if case["cache"] == "e4m3" else 4 * d
    n = sum(_seen(case))
    table = 4 * sum(-(-x // case["page"]) for x in _seen(case)) + 4 * case["batch"]
    if case["op"] == "read":
        return {"bytes": n * case["kv_heads"] * (row + 4 * d) + table,
                "flops": 2 * n * case["kv_heads"] * d}
    q = case["batch"] * case["q_heads"]
    return {"bytes": n * case["kv_heads"] * row + table + q * (4 * d + 4),
            "flops": n * case["q_heads"] * (4 * d + 4)}


def _coded(x):
    """e4m3 codes and scales of the rows of x, as the cache holds them."""
    scale = x.abs().amax(-1).clamp(min=1e-12) / 448.0
    codes = (x / scale[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), scale


def _filled(case, pages, g):
    """A cache of `pages` pages that earlier steps have filled. Keys have a
    few strong channels and tokens differ in size, as projections' do."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    channel = torch.ones(case["dim"], device=DEVICE)
    channel[::13] = 3.0
    made = {}
    for n, weight in (("k", channel), ("v", None)):
        x = torch.randn(shape, generator=g, device=DEVICE)
        x *= torch.exp(0.5 * torch.randn(shape[:3] + (1,), generator=g, device=DEVICE))
        if weight is not None:
            x *= weight
        if case["cache"] == "e4m3":
            made[n], made[n + "_scale"] = _coded(x)
        else:
            made[n] = x.to(torch.bfloat16)
    return made


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    d, hk = case["dim"], case["kv_heads"]
    state = {"case": case, "kept": {}}
    if case["op"] in ("rotary", "write"):
        t, hq = case["tokens"], case["q_heads"]
        # q, k and v as a projection leaves them: side by side in a row
        wide = torch.randn((t, (hq + 2 * hk) * d), generator=g, device=DEVICE)
        wide = wide.to(torch.bfloat16)
        state["q"] = wide[:, :hq * d].unflatten(1, (hq, d)) if hq else None
        state["k"] = wide[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        state["v"] = wide[:, (hq + hk) * d:].unflatten(1, (hk, d))
        if case["rot"]:
            i = torch.arange(0, case["rot"], 2, dtype=torch.float64, device=DEVICE)
            state["inv_freq"] = 1000000.0 ** (-i / case["rot"])
            state["pair_axis"] = torch.tensor(_pair_axis(case), dtype=torch.uint8, device=DEVICE)
            state["positions"] = torch.randint(0, case["far"], (case["axes"], t), generator=g,
                                               device=DEVICE, dtype=torch.int32)
        if case["op"] == "write":
            # page 0 is nobody's: tokens get slots in the other pages
            pages = -(-t // case["page"]) + 3
            slots = torch.randperm((pages - 1) * case["page"], generator=g, device=DEVICE)[:t]
            slots = (slots + case["page"]).to(torch.int32)
            if case["skipped"]:
                slots[::case["skipped"]] = -1
            state["slots"] = slots
            kind = torch.uint8 if case["cache"] == "e4m3" else torch.bfloat16
            for n in ("k", "v"):
                state["cache_" + n] = torch.zeros((pages, hk, case["page"], d), dtype=kind,
                                                  device=DEVICE)
                if case["cache"] == "e4m3":
                    state["cache_" + n + "_scale"] = torch.ones((pages, hk, case["page"]),
                                                                device=DEVICE)
        return state
    lengths, page = _lengths(case), case["page"]
    order = torch.randperm(len(lengths), generator=g, device=DEVICE)
    lengths = torch.tensor(lengths, dtype=torch.int32, device=DEVICE)[order]
    # pages of a context wholly before its window have been given back
    first = (lengths - case["window"]).clamp(min=0) // page if case.get("window") else 0 * lengths
    count = -(-lengths // page)
    wide = max(1, -(-case["longest"] // page))
    column = torch.arange(wide, device=DEVICE, dtype=torch.int32)
    held = (column >= first[:, None]) & (column < count[:, None])
    pages = sum(-(-n // page) for n in _lengths(case)) + 2
    ids = (torch.cumsum(held.reshape(-1), 0) - 1).reshape(held.shape).clamp(min=0)
    shuffled = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
    state["table"] = torch.where(held, shuffled[ids], -1).to(torch.int32)
    for n, x in _filled(case, pages, g).items():
        state["cache_" + n] = x
    if case["op"] == "read":
        state["offsets"] = torch.zeros(len(lengths) + 1, dtype=torch.int32, device=DEVICE)
        state["offsets"][1:] = torch.cumsum(lengths, 0)
        state["rows"] = sum(_lengths(case))
        state["longest"] = case["longest"]
    else:
        state["lengths"] = lengths
        q = torch.randn((case["batch"], case["q_heads"], d), generator=g, device=DEVICE)
        state["q"] = (1.5 * q).to(torch.bfloat16)
    return state


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _turn(x, cos, sin, case):
    """The rotated dimensions of x [T, H, D] in fp32, the others as they are."""
    rot = case["rot"]
    x = x.float()
    y, rest = x[..., :rot], x[..., rot:]
    cos, sin = cos[:, None], sin[:, None]
    if case["neighbours"]:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, rest), -1)


def _angles(state, inverse=False):
    where = state["positions"][state["pair_axis"].long()].double()      # [pairs, T]
    angle = (where * state["inv_freq"][:, None]).t()
    sin = torch.sin(angle).float()
    return torch.cos(angle).float(), -sin if inverse else sin


def _plain_rotary(state):
    case = state["case"]
    cos, sin = _angles(state, case["inverse"])
    return tuple(_turn(state[n], cos, sin, case).to(torch.bfloat16) for n in ("q", "k"))


def _put(pages, slots, rows):
    """rows [T, H, ...] into the slots of pages [P, H, page, ...]; rows of
    slot -1 leave the cache as it is (they rewrite slot 0, nobody's)."""
    size = pages.shape[2]
    to = slots.long().clamp(min=0)
    page, at = to // size, to % size
    keep = (slots >= 0).reshape([-1] + [1] * (rows.dim() - 1))
    pages[page, :, at] = torch.where(keep, rows, pages[0, :, 0])


def _plain_write(state):
    case, out = state["case"], {}
    k, v = state["k"].float(), state["v"].float()
    if case["rot"]:
        cos, sin = _angles(state)
        out["q"] = _turn(state["q"], cos, sin, case).to(torch.bfloat16)
        k = _turn(state["k"], cos, sin, case)
    for n, x in (("k", k), ("v", v)):
        if case["cache"] == "e4m3":
            codes, scale = _coded(x)
            _put(state["cache_" + n], state["slots"], codes)
            _put(state["cache_" + n + "_scale"], state["slots"], scale)
        else:
            _put(state["cache_" + n], state["slots"], x.to(torch.bfloat16))
    return {**out, **_cache_values(state)}


def _cache_values(state):
    """The cache after a write: codes as the e4m3 values they are, and scales."""
    if state["case"]["cache"] == "bf16":
        return {"k": state["cache_k"], "v": state["cache_v"]}
    return {"k": state["cache_k"].view(torch.float8_e4m3fn),
            "v": state["cache_v"].view(torch.float8_e4m3fn),
            "k_scale": state["cache_k_scale"], "v_scale": state["cache_v_scale"]}


def _fetch(state, name, page, at):
    """fp32 rows [..., H, D] of the cache at (page, at)."""
    x = state["cache_" + name]
    if x.dtype == torch.bfloat16:
        return x[page, :, at].float()
    scale = state["cache_" + name + "_scale"]
    return x.view(torch.float8_e4m3fn)[page, :, at].float() * scale[page, :, at][..., None]


def _plain_read(state):
    case, page = state["case"], state["case"]["page"]
    row = torch.arange(state["rows"], device=DEVICE)
    b = torch.searchsorted(state["offsets"][1:].long(), row, right=True)
    token = row - state["offsets"].long()[b]
    page, at = state["table"].long()[b, token // page], token % page
    return tuple(_fetch(state, n, page, at).to(torch.bfloat16) for n in ("k", "v"))


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


# ---------------------------------------------------------------------------
# the package's operators
# ---------------------------------------------------------------------------
def _rotary(state):
    if "rotary" not in state["kept"]:
        from expert_layer_ptpc_gb300.attention import Rotary
        state["kept"]["rotary"] = Rotary(state["inv_freq"], state["pair_axis"],
                                         axes=state["case"]["axes"],
                                         neighbours=state["case"]["neighbours"])
    return state["kept"]["rotary"]


def _cache(state):
    if "cache" not in state["kept"]:
        from expert_layer_ptpc_gb300.attention import PagedKVCache
        state["kept"]["cache"] = PagedKVCache.from_tensors(
            state["cache_k"], state["cache_v"], state.get("cache_k_scale"),
            state.get("cache_v_scale"))
    return state["kept"]["cache"]


def _own_rotary(state):
    return _rotary(state).apply(state["positions"], state["q"], state["k"],
                                inverse=state["case"]["inverse"])


def _own_write(state):
    cache, out = _cache(state), {}
    if state["case"]["rot"]:
        out["q"] = cache.write_rotary(_rotary(state), state["positions"], state["q"], state["k"],
                                      state["v"], state["slots"])
    else:
        cache.write(state["k"], state["v"], state["slots"])
    return {**out, **_cache_values(state)}


def _own_read(state):
    return _cache(state).read(state["table"], state["offsets"], state["rows"])


def _own_attend(state):
    return _cache(state).attend(state["q"], state["table"], state["lengths"],
                                window=state["case"]["window"], return_lse=True)


def run(state):
    if own:
        return {"rotary": _own_rotary, "write": _own_write, "read": _own_read,
                "attend": _own_attend}[state["case"]["op"]](state)
    return {"rotary": _plain_rotary, "write": _plain_write, "read": _plain_read,
            "attend": _plain_attend}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------
def _exact_turn(state, name, back):
    """Each rotated pair as a complex number times e^(i angle)."""
    case = state["case"]
    x = state[name].double().clone()
    t, h, _ = x.shape
    rot, where = case["rot"], state["positions"].double()
    for i, axis in enumerate(state["pair_axis"].tolist()):
        lo, hi = (2 * i, 2 * i + 1) if case["neighbours"] else (i, i + rot // 2)
        angle = where[axis] * state["inv_freq"][i] * (-1.0 if back else 1.0)
        z = torch.complex(x[..., lo], x[..., hi])
        z = z * torch.polar(torch.ones_like(angle), angle)[:, None]
        x[..., lo], x[..., hi] = z.real, z.imag
    return x


def _exact_write(state):
    case, out = state["case"], {}
    size = case["page"]
    if case["rot"]:
        out["q"] = _exact_turn(state, "q", False)
    slots = state["slots"].tolist()
    rows = torch.tensor([i for i, s in enumerate(slots) if s >= 0], device=DEVICE)
    to = torch.tensor([s for s in slots if s >= 0], device=DEVICE)
    for n in ("k", "v"):
        x = _exact_turn(state, n, False) if n == "k" and case["rot"] else state[n].double()
        pages, h, _, d = state["cache_" + n].shape
        whole = torch.zeros((pages * size, h, d), dtype=torch.float64, device=DEVICE)
        if case["cache"] == "e4m3":
            scale = torch.ones((pages * size, h), dtype=torch.float64, device=DEVICE)
            scale[to] = x[rows].abs().amax(-1).clamp(min=1e-12) / 448.0
            x = x / (x.abs().amax(-1, keepdim=True).clamp(min=1e-12) / 448.0)
            out[n + "_scale"] = scale.reshape(pages, size, h).transpose(1, 2).contiguous()
        whole[to] = x[rows]
        out[n] = whole.reshape(pages, size, h, d).transpose(1, 2).contiguous()
    return out


def _exact_context(state, b, first, last):
    """Keys and values [n, H, D] of tokens first..last-1 of context b."""
    size, got = state["case"]["page"], []
    for n in ("k", "v"):
        x = state["cache_" + n]
        pages = state["table"][b, first // size:-(-last // size)].long()
        if x.dtype == torch.uint8:
            rows = x.view(torch.float8_e4m3fn)[pages].double()
            rows = rows * state["cache_" + n + "_scale"][pages].double()[..., None]
        else:
            rows = x[pages].double()
        rows = rows.transpose(1, 2).flatten(0, 1)
        got.append(rows[first % size:first % size + last - first])
    return got


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "rotary":
        return tuple(_exact_turn(state, n, case["inverse"]) for n in ("q", "k"))
    if case["op"] == "write":
        return _exact_write(state)
    if case["op"] == "read":
        ends = state["offsets"].tolist()
        parts = [_exact_context(state, b, 0, e - s)
                 for b, (s, e) in enumerate(zip(ends, ends[1:])) if e > s]
        return tuple(torch.cat([p[i] for p in parts]) for i in (0, 1))
    hq, d, hk = case["q_heads"], case["dim"], case["kv_heads"]
    out = torch.zeros((case["batch"], hq, d), dtype=torch.float64, device=DEVICE)
    lse = torch.full((case["batch"], hq), float("-inf"), dtype=torch.float64, device=DEVICE)
    for b, n in enumerate(state["lengths"].tolist()):
        if n == 0:
            continue
        k, v = _exact_context(state, b, max(0, n - case["window"]) if case["window"] else 0, n)
        for h in range(hq):
            s = k[:, h // (hq // hk)] @ state["q"][b, h].double() / math.sqrt(d)
            lse[b, h] = torch.logsumexp(s, 0)
            out[b, h] = torch.softmax(s, 0) @ v[:, h // (hq // hk)]
    return out, lse
