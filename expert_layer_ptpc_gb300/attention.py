"""The attention half of a decoder step next to the MoE layer: rotary
positions with several axes, a paged key-value cache, attention of one or of many
new tokens over it, and the block tables and slot maps of a step.

`Rotary`, `PagedKVCache` and `PagePool` hold what a serving loop keeps between
steps (the frequencies, the cache's tensors, the requests' pages) and call the
library entry points of `binding`; all arithmetic runs in the library's kernels.
"""

import math
import threading
from fractions import Fraction

import torch

from . import binding


_PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494")
_RADIAN = round(2 ** 256 / (2 * _PI))   # in units of 2^-256 turns, to some 200 bits


def pair_axes(sections, woven=False):
    """The axis of each rotated pair. `sections[a]` pairs belong to axis a: in
    blocks (all of axis 0, then axis 1, ...), or `woven` (the axes in turn,
    each as long as it has pairs left)."""
    if any(n < 0 for n in sections):
        raise ValueError(f"sections must not be negative, got {sections}")
    if not woven:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, order = list(sections), []
    while any(left):
        for a, n in enumerate(left):
            if n:
                order.append(a)
                left[a] -= 1
    return order


def frequencies(rot_dim, base=10000.0, device=None):
    """inv_freq[i] = base^(-2i / rot_dim) in fp64."""
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device)
    return base ** (-i / rot_dim)


class Rotary:
    """A rotation of q and k heads by positions on one or more axes.

    inv_freq: [rot_dim / 2] angles per position (any float dtype; taken in
    fp64); pair_axis: the axis of each pair (a list or an integer tensor; None:
    one axis); axes: the number of axes (default: the largest named + 1);
    neighbours: pairs (2i, 2i + 1) instead of (i, i + rot_dim / 2). The plan
    lives on `device` (default: inv_freq's if that is a GPU, else the current
    GPU); making one copies to and from the host.
    """

    def __init__(self, inv_freq, pair_axis=None, axes=None, neighbours=False, device=None):
        freq = torch.as_tensor(inv_freq, dtype=torch.float64)
        if freq.dim() != 1 or freq.numel() == 0 or freq.numel() % 8 != 0:
            raise ValueError("inv_freq must hold a positive multiple of 8 frequencies")
        if device is None:
            device = freq.device if freq.is_cuda else torch.device("cuda")
        axis = torch.zeros(freq.numel(), dtype=torch.int64) if pair_axis is None else \
            torch.as_tensor(pair_axis).to("cpu", torch.int64)
        if tuple(axis.shape) != tuple(freq.shape):
            raise ValueError("pair_axis must name an axis for every frequency")
        if axes is None:
            axes = int(axis.max()) + 1
        if not 1 <= axes <= 8:
            raise ValueError(f"1 to 8 axes are supported, got {axes}")
        if int(axis.min()) < 0 or int(axis.max()) >= axes:
            raise ValueError(f"pair_axis must lie in [0, {axes})")
        turns = []
        for f in freq.tolist():
            if not math.isfinite(f):
                raise ValueError("inv_freq must be finite")
            # a fraction of a turn per position in units of 2^-64, rounded once
            # (a double's quotient would be 2^-24 turns off after 2^31 positions)
            top, below = f.as_integer_ratio()
            shift = below.bit_length() - 1 + 256 - 64          # below = 2^(bits - 1)
            n = (((top * _RADIAN >> (shift - 1)) + 1) >> 1) % (1 << 64)
            turns.append(n - (1 << 64) if n >= 1 << 63 else n)
        self.turns = torch.tensor(turns, dtype=torch.int64).to(device)
        self.pair_axis = axis.to(torch.uint8).to(device)
        self.rot_dim, self.axes = 2 * freq.numel(), axes
        self.plan = binding.moe_rotary_plan(self.turns.data_ptr(), self.pair_axis.data_ptr(),
                                            axes, self.rot_dim, int(bool(neighbours)))
        self.plan.device = self.turns.get_device()

    def apply(self, positions, q, k=None, inverse=False, q_out=None, k_out=None, stream=None):
        """q [T, heads, head_dim] bf16, and k, rotated by positions [axes, T]
        int32 (`inverse`: back, which is also the gradient). Returns
        (q_out, k_out); an output may be its input."""
        return binding.moe_rotary(self.plan, positions, q, k, inverse, q_out, k_out, stream)


_kept = threading.local()   # workspaces: this host thread's, by GPU and stream


class PagedKVCache:
    """Pages of keys and values, [pages, heads, page_size, head_dim] each, as
    e4m3 codes with one fp32 scale per token and head (scales [pages, heads,
    page_size]) or per page and head (scales [pages, heads]: powers of two as the writes
    make them; attend_prompt rounds others to 11 bits), or in bf16."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v must be [pages, heads, page_size, head_dim], alike")
        dtypes = {torch.uint8: binding.MOE_DTYPE_E4M3, torch.bfloat16: binding.MOE_DTYPE_BF16}
        if k.dtype not in dtypes:
            raise ValueError(f"the cache must be uint8 (e4m3 codes) or bf16, got {k.dtype}")
        coded = k.dtype == torch.uint8
        if coded != (k_scale is not None) or coded != (v_scale is not None):
            raise ValueError("an e4m3 cache has scales for k and v, a bf16 cache has none")
        binding._need(k, k.dtype, "k")
        index = k.get_device()
        for t, n in ((k, "k"), (v, "v")):
            binding._need_on(t, k.dtype, n, index)
        dtype = dtypes[k.dtype]
        if coded:
            by_page = k_scale.dim() == 2
            dtype = binding.MOE_DTYPE_E4M3_PAGE if by_page else dtype
            shape = k.shape[:2 if by_page else 3]
            for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                binding._need_on(t, torch.float32, n, index)
                if t.shape != shape:
                    raise ValueError(f"{n} must be {tuple(shape)}, got {tuple(t.shape)}")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.heads, self.page_size, self.head_dim = k.shape
        self.struct = binding.moe_kv_cache(
            k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if coded else None,
            v_scale.data_ptr() if coded else None, self.pages, self.heads, self.page_size,
            self.head_dim, dtype)
        self.struct.device = index
        self._ws_bytes = {}       # by query heads
        self._prompt_ws_bytes = {}
        self._scale = 1.0 / math.sqrt(self.head_dim)

    @classmethod
    def empty(cls, pages, heads, page_size, head_dim, dtype="e4m3", device="cuda"):
        """A new cache; dtype "e4m3" (a scale per token and head), "e4m3_page" (per page
        and head) or "bf16". Slots hold nothing until written (no operator reads a
        slot that no context covers)."""
        shape = (pages, heads, page_size, head_dim)
        if dtype == "bf16":
            return cls(*(torch.empty(shape, dtype=torch.bfloat16, device=device)
                         for _ in range(2)))
        if dtype == "e4m3_page":   # (scales of 0: whatever a page's first call brings is more)
            return cls(*(torch.empty(shape, dtype=torch.uint8, device=device) for _ in range(2)),
                       *(torch.zeros(shape[:2], dtype=torch.float32, device=device)
                         for _ in range(2)))
        if dtype != "e4m3":
            raise ValueError(f'dtype must be "e4m3", "e4m3_page" or "bf16", got {dtype!r}')
        return cls(*(torch.empty(shape, dtype=torch.uint8, device=device) for _ in range(2)),
                   *(torch.empty(shape[:3], dtype=torch.float32, device=device)
                     for _ in range(2)))

    @classmethod
    def from_tensors(cls, k, v, k_scale=None, v_scale=None):
        """A cache over the caller's tensors (shared, not copied)."""
        return cls(k, v, k_scale, v_scale)

    def write(self, k, v, slots, stream=None):
        """Store k, v [T, heads, head_dim] bf16 at slots [T] int32 (slot =
        page * page_size + offset; a slot outside the cache skips its token). With a
        scale per page, a page's tokens follow one another in the call."""
        binding.moe_kv_write(self.struct, k, v, slots, stream)

    def write_rotary(self, rotary, positions, q, k, v, slots, q_out=None, stream=None):
        """Rotate q and k by `rotary` and store the rotated k and v; returns the
        rotated q."""
        return binding.moe_rotary_kv_write(rotary.plan, positions, self.struct, q, k, v, slots,
                                           q_out, stream)

    def read(self, block_table, offsets, rows, k_out=None, v_out=None, stream=None):
        """Contexts back in bf16: (k, v) [rows, heads, head_dim], context b in
        rows offsets[b] .. offsets[b + 1]; rows = offsets[-1] on the host."""
        return binding.moe_kv_read(self.struct, block_table, offsets, rows, k_out, v_out, stream)

    def workspace(self, batch, q_heads, stream=None):
        """The attention workspace of one stream and host thread, kept for the
        next call, also of another cache. Calls on different streams may overlap, so
        each stream has its own. A call is two launches, between which another
        thread may enqueue its own on the same stream, so each thread has its own
        too. A captured call's belongs to its graph."""
        need = self._ws_bytes.get(q_heads)
        if need is None:          # (the same for every batch)
            need = binding.moe_paged_attention_workspace_size(self.struct, 1, q_heads)
            self._ws_bytes[q_heads] = need
        return self._workspace(need, stream)

    def prompt_workspace(self, q_heads, stream=None):
        """The same for attend_prompt."""
        need = self._prompt_ws_bytes.get(q_heads)
        if need is None:
            need = binding.moe_prompt_attention_workspace_size(self.struct, q_heads)
            self._prompt_ws_bytes[q_heads] = need
        return self._workspace(need, stream)

    def _workspace(self, need, stream):
        index = self.struct.device
        on = binding._raw_stream(stream, index)
        if binding._capturing(stream, index):
            return self._new_workspace(need, stream)
        kept, key = _kept.__dict__, (index, on)
        ws = kept.get(key)
        if ws is None or ws.numel() < need:
            ws = kept[key] = self._new_workspace(need, stream)
        return ws

    def _new_workspace(self, need, stream):
        return binding._empty(max(need, 1), torch.uint8, self.k.device, stream)

    def attend(self, q, block_table, lengths, scale=None, window=0, out=None, lse=None,
               return_lse=False, ws=None, stream=None):
        """Attention of one new token per context: q [batch, q_heads, head_dim]
        bf16 over the first lengths[b] tokens of block_table[b] (the last
        `window` of them when window > 0). Row b is context b's, whatever it gets: the
        rows of a StepPlan are those only where every request got one token, as
        requests without new tokens have no rows there (attend_prompt takes its offsets).
        scale: default 1 / sqrt(head_dim). Returns out, or (out, lse) with `return_lse` or
        `lse`."""
        if scale is None:
            scale = self._scale
        if ws is None:
            ws = self.workspace(q.shape[0], q.shape[1], stream)
        return binding.moe_paged_attention(self.struct, q, block_table, lengths, scale, window,
                                           out, lse, ws, stream, return_lse or lse is not None)

    def attend_prompt(self, q, offsets, block_table, lengths, scale=None, window=0, out=None,
                      lse=None, return_lse=False, ws=None, stream=None):
        """Attention of many new tokens per context: q [rows, q_heads, head_dim] bf16,
        context b's in rows offsets[b] .. offsets[b + 1], which are the last of its
        lengths[b] tokens (keys and values already written). Each sees the tokens
        of its context up to its own (the last `window` of them when window > 0). Rows
        from offsets[-1] on are left as they are in `out` and `lse`, and are 0 and -inf in
        tensors that the call makes. scale: default 1 / sqrt(head_dim).
        Returns out, or (out, lse) with `return_lse` or `lse`."""
        if scale is None:
            scale = self._scale
        if ws is None:
            ws = self.prompt_workspace(q.shape[1], stream)
        return binding.moe_prompt_attention(self.struct, q, offsets, block_table, lengths, scale,
                                            window, out, lse, ws, stream,
                                            return_lse or lse is not None)


class StepPlan:
    """What one step needs to know, all int32 on the GPU: `offsets` [batch + 1] of the
    requests' rows (none for a request that leaves, waits or has no new tokens: the rows of
    those behind it move up), `lengths` [batch] of their contexts with the new tokens, `slots`
    [rows] and `positions` [axes, rows] of the rows (-1 and 0 for rows behind the
    last), `refused` [1], the number of requests that wait for pages or rows, and
    `state`, the pool's after the step."""

    __slots__ = ("offsets", "slots", "positions", "state", "refused")

    def __init__(self, offsets, slots, positions, state, refused):
        self.offsets, self.slots, self.positions = offsets, slots, positions
        self.state, self.refused = state, refused

    @property
    def lengths(self):
        return self.state[:-1]


class PagePool:
    """The pages of a batch of requests: `table` [batch, max_pages] int32, request b's
    pages in order; `stack` [pages] int32, the free pages, the next to be handed out
    last; `state` [batch + 1] int32: the tokens that each request holds, then the
    number of free pages. All of it lives on the GPU, and so a captured step can go
    on handing out pages.

    A page has one owner: the stack, or one entry of one request's ceil(tokens / page_size)
    first. A page in two of them (a prefix that requests share) would come back twice, and
    then have two owners; such pages belong to the caller, in tables of its own. Pages come
    back when their request leaves. A caller who gives some back before (those behind a
    window, or of drafted tokens that are rejected) changes all three tensors together: the
    page goes to stack[state[-1]], state[-1] grows by one, and the entry becomes -1, or lies
    behind the tokens that are left in state[b]. Lowering state[b] alone loses the pages
    behind."""

    def __init__(self, table, stack, state, page_size):
        if table.dim() != 2 or stack.dim() != 1 or state.dim() != 1:
            raise ValueError("table must be [batch, max_pages], stack [pages], state [batch + 1]")
        if page_size < 1 or page_size > 1024 or page_size & (page_size - 1):
            raise ValueError(f"page_size must be a power of two up to 1024, got {page_size}")
        if state.numel() != table.shape[0] + 1:
            raise ValueError(f"state must have {table.shape[0] + 1} entries, got {state.numel()}")
        self.table, self.stack, self.state, self.page_size = table, stack, state, page_size

    @classmethod
    def empty(cls, pages, page_size, batch, max_pages, device="cuda"):
        """A pool whose pages are all free, for up to `batch` requests at a time."""
        state = torch.zeros(batch + 1, dtype=torch.int32, device=device)
        state[-1] = pages
        return cls(torch.full((batch, max_pages), -1, dtype=torch.int32, device=device),
                   torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=device), state,
                   page_size)

    @classmethod
    def from_tensors(cls, table, stack, state, page_size):
        """A pool over the caller's tensors (shared, not copied)."""
        return cls(table, stack, state, page_size)

    def plan(self, new_tokens, rows, axes=1, stream=None):
        """The StepPlan of new_tokens [batch] int32 more tokens for each request; a
        negative number: the request leaves, and its pages are free for this
        step already. The requests are served in order, until one would need more pages than
        are free or more than `rows` rows in all; that one and those behind it, and a
        request that outgrows its table, wait (their lengths stay). Updates table and
        stack; state stays until `commit`, and planning again starts from there."""
        return StepPlan(*binding.moe_kv_plan(self.state, new_tokens, self.table, self.stack,
                                             self.page_size, rows, axes, stream))

    def commit(self, plan, stream=None):
        """Make the plan's state the pool's."""
        if stream is None:
            self.state.copy_(plan.state)
        else:
            with torch.cuda.stream(stream):
                self.state.copy_(plan.state)
