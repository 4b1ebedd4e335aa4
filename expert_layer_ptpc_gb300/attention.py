"""The attention half of a decoder step next to the MoE layer: rotary
positions with several axes, a paged key-value cache and attention of one new
token over it.

`Rotary` and `PagedKVCache` hold what a serving loop keeps between steps (the
frequencies, the cache's tensors) and call the library entry points of
`binding`; all arithmetic runs in the library's kernels.
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
    e4m3 codes with one fp32 scale per token and head, or in bf16."""

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
        if coded:
            for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                binding._need_on(t, torch.float32, n, index)
                if t.shape != k.shape[:3]:
                    raise ValueError(f"{n} must be {tuple(k.shape[:3])}, got {tuple(t.shape)}")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.heads, self.page_size, self.head_dim = k.shape
        self.struct = binding.moe_kv_cache(
            k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if coded else None,
            v_scale.data_ptr() if coded else None, self.pages, self.heads, self.page_size,
            self.head_dim, dtypes[k.dtype])
        self.struct.device = index
        self._ws_bytes = {}       # by query heads
        self._scale = 1.0 / math.sqrt(self.head_dim)

    @classmethod
    def empty(cls, pages, heads, page_size, head_dim, dtype="e4m3", device="cuda"):
        """A new cache; dtype "e4m3" or "bf16". Slots hold nothing until
        written (no operator reads a slot that no context covers)."""
        shape = (pages, heads, page_size, head_dim)
        if dtype == "bf16":
            return cls(*(torch.empty(shape, dtype=torch.bfloat16, device=device)
                         for _ in range(2)))
        if dtype != "e4m3":
            raise ValueError(f'dtype must be "e4m3" or "bf16", got {dtype!r}')
        return cls(*(torch.empty(shape, dtype=torch.uint8, device=device) for _ in range(2)),
                   *(torch.empty(shape[:3], dtype=torch.float32, device=device)
                     for _ in range(2)))

    @classmethod
    def from_tensors(cls, k, v, k_scale=None, v_scale=None):
        """A cache over the caller's tensors (shared, not copied)."""
        return cls(k, v, k_scale, v_scale)

    def write(self, k, v, slots, stream=None):
        """Store k, v [T, heads, head_dim] bf16 at slots [T] int32 (slot =
        page * page_size + offset; a slot outside the cache skips its token)."""
        binding.moe_kv_write(self.struct, k, v, slots, stream)

    def write_rotary(self, rotary, positions, q, k, v, slots, q_out=None, stream=None):
        """Rotate q and k by `rotary` and store the rotated k and v, in one
        launch; returns the rotated q."""
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
        index = self.struct.device
        on = binding._raw_stream(stream, index)
        need = self._ws_bytes.get(q_heads)
        if need is None:          # (the same for every batch)
            need = binding.moe_paged_attention_workspace_size(self.struct, 1, q_heads)
            self._ws_bytes[q_heads] = need
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
        `window` of them when window > 0). scale: default 1 / sqrt(head_dim).
        Returns out, or (out, lse) with `return_lse` or `lse`."""
        if scale is None:
            scale = self._scale
        if ws is None:
            ws = self.workspace(q.shape[0], q.shape[1], stream)
        return binding.moe_paged_attention(self.struct, q, block_table, lengths, scale, window,
                                           out, lse, ws, stream, return_lse or lse is not None)
