"""Host side of the attention classes and their binding, on stand-ins for GPU
tensors: what is refused before the library is called, and which workspace a
call gets. No call here reaches a kernel."""

import contextlib
import math
import threading
from fractions import Fraction

import pytest
import torch

from expert_layer_ptpc_gb300 import attention, binding, build


class OnGpu:
    """A CPU tensor that says it lies on a GPU."""

    is_cuda = True

    def __init__(self, t, index=0):
        self.t, self.index = t, index

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.index


class Calls:
    """A library that takes every call and writes down its arguments."""

    def __init__(self):
        self.made = []

    def __getattr__(self, name):
        def call(*args):
            self.made.append((name, args))
            return 0
        return call


@pytest.fixture
def calls(monkeypatch):
    """The binding over such a library, on a machine whose current GPU is 0."""
    made = Calls()
    monkeypatch.setattr(binding, "_lib", made)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return made


def bf16(*shape, index=0):
    return OnGpu(torch.zeros(shape, dtype=torch.bfloat16), index)


def int32(*shape, index=0):
    return OnGpu(torch.zeros(shape, dtype=torch.int32), index)


def cache_struct(pages=4, heads=2, size=16, d=64):
    p = 0x10000
    return binding.moe_kv_cache(p, p, p, p, pages, heads, size, d, binding.MOE_DTYPE_E4M3)


def attend(**kw):
    args = dict(cache=cache_struct(), q=bf16(3, 8, 64), block_table=int32(3, 4),
                lengths=int32(3), scale=0.125, out=bf16(3, 8, 64),
                ws=OnGpu(torch.zeros(64, dtype=torch.uint8)))
    args.update(kw)
    return binding.moe_paged_attention(**args)


# ---------------------------------------------------------------------------
# the caller's workspace
# ---------------------------------------------------------------------------
def test_a_workspace_on_the_host_is_refused(calls):
    with pytest.raises(ValueError, match="ws"):
        attend(ws=torch.zeros(64, dtype=torch.uint8))
    assert not calls.made


def test_a_strided_workspace_is_refused(calls):
    with pytest.raises(ValueError, match="ws"):
        attend(ws=OnGpu(torch.zeros(128, dtype=torch.uint8)[::2]))
    assert not calls.made


@pytest.mark.parametrize("dtype,size", [(torch.uint8, 64), (torch.float32, 256)])
def test_a_workspace_counts_in_bytes(calls, dtype, size):
    attend(ws=OnGpu(torch.zeros(64, dtype=dtype)))
    (name, args), = calls.made
    assert name == "moe_paged_attention" and args[-2] == size


# ---------------------------------------------------------------------------
# devices
# ---------------------------------------------------------------------------
def plan_struct(axes=1, rot=64):
    return binding.moe_rotary_plan(0x10000, 0x10000, axes, rot, 0)


def rotate(**kw):
    args = dict(plan=plan_struct(), positions=int32(1, 3), q=bf16(3, 8, 64), k=bf16(3, 2, 64),
                q_out=bf16(3, 8, 64), k_out=bf16(3, 2, 64))
    args.update(kw)
    return binding.moe_rotary(**args)


def write(**kw):
    args = dict(cache=cache_struct(), k=bf16(3, 2, 64), v=bf16(3, 2, 64), slots=int32(3))
    args.update(kw)
    return binding.moe_kv_write(**args)


def write_rotary(**kw):
    args = dict(plan=plan_struct(), positions=int32(1, 3), cache=cache_struct(),
                q=bf16(3, 8, 64), k=bf16(3, 2, 64), v=bf16(3, 2, 64), slots=int32(3),
                q_out=bf16(3, 8, 64))
    args.update(kw)
    return binding.moe_rotary_kv_write(**args)


def read(**kw):
    args = dict(cache=cache_struct(), block_table=int32(3, 4), offsets=int32(4), rows=9,
                k_out=bf16(9, 2, 64), v_out=bf16(9, 2, 64))
    args.update(kw)
    return binding.moe_kv_read(**args)


EVERY_CALL = [rotate, write, write_rotary, read, attend]


def tensors_of(call):
    """The names of a call's tensor arguments, with stand-ins on GPU 1."""
    other = dict(positions=int32(1, 3, index=1), q=bf16(3, 8, 64, index=1),
                 k=bf16(3, 2, 64, index=1), v=bf16(3, 2, 64, index=1),
                 q_out=bf16(3, 8, 64, index=1), slots=int32(3, index=1),
                 block_table=int32(3, 4, index=1))
    own = {rotate: dict(k_out=bf16(3, 2, 64, index=1)),
           read: dict(offsets=int32(4, index=1), k_out=bf16(9, 2, 64, index=1),
                      v_out=bf16(9, 2, 64, index=1)),
           attend: dict(lengths=int32(3, index=1), out=bf16(3, 8, 64, index=1),
                        lse=OnGpu(torch.zeros(3, 8), 1),
                        ws=OnGpu(torch.zeros(64, dtype=torch.uint8), 1))}
    shared = {rotate: ("positions", "q", "k", "q_out"), write: ("k", "v", "slots"),
              write_rotary: ("positions", "q", "k", "v", "slots", "q_out"),
              read: ("block_table",), attend: ("q", "block_table")}
    return {**{n: other[n] for n in shared[call]}, **own.get(call, {})}


@pytest.mark.parametrize("call", EVERY_CALL, ids=lambda f: f.__name__)
def test_tensors_of_two_gpus_are_refused(calls, call):
    call()
    assert len(calls.made) == 1
    for name, t in tensors_of(call).items():
        with pytest.raises(ValueError, match="GPU"):
            call(**{name: t})
    assert len(calls.made) == 1


@pytest.mark.parametrize("call", EVERY_CALL, ids=lambda f: f.__name__)
def test_tensors_of_a_gpu_that_is_not_current_are_refused(calls, call, monkeypatch):
    """The library launches on the current GPU."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    with pytest.raises(ValueError, match="current"):
        call()
    with pytest.raises(ValueError, match="current"):
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
        call(**tensors_of(call))
    assert not calls.made


@pytest.mark.parametrize("call", [write, write_rotary, read, attend], ids=lambda f: f.__name__)
def test_a_cache_on_another_gpu_is_refused(calls, call):
    cache = cache_struct()
    cache.device = 1
    with pytest.raises(ValueError, match="cache"):
        call(cache=cache)
    assert not calls.made


@pytest.mark.parametrize("call", [rotate, write_rotary], ids=lambda f: f.__name__)
def test_a_plan_on_another_gpu_is_refused(calls, call):
    plan = plan_struct()
    plan.device = 1
    with pytest.raises(ValueError, match="plan"):
        call(plan=plan)
    assert not calls.made


@pytest.mark.parametrize("call", EVERY_CALL, ids=lambda f: f.__name__)
def test_a_stream_of_another_gpu_is_refused(calls, call):
    class Stream:
        cuda_stream, device_index = 77, 0
    call(stream=Stream())
    assert calls.made.pop()[1][-1] == 77
    Stream.device_index = 1
    with pytest.raises(ValueError, match="stream"):
        call(stream=Stream())
    assert not calls.made


def test_a_plan_on_the_host_is_refused(calls):
    r = attention.Rotary(attention.frequencies(64), device="cpu")
    with pytest.raises(ValueError, match="plan"):
        r.apply(int32(1, 3), bf16(3, 8, 64), q_out=bf16(3, 8, 64))
    assert not calls.made


# ---------------------------------------------------------------------------
# the workspace a cache keeps
# ---------------------------------------------------------------------------
@pytest.fixture
def streams(monkeypatch):
    """The real library (its sizes), no stream capturing, current stream 5."""
    build.build()
    binding.load_library()
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 5, raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)


def cache_of(heads=4, d=128, index=0):
    pages = torch.zeros((2, heads, 16, d), dtype=torch.uint8)
    scales = torch.ones((2, heads, 16))
    return attention.PagedKVCache(OnGpu(pages, index), OnGpu(pages.clone(), index),
                                  OnGpu(scales, index), OnGpu(scales.clone(), index))


def test_threads_have_workspaces_of_their_own(streams):
    """A call is two launches, and two threads' calls on one stream may be enqueued one
    between the other's: they must not share the partial results."""
    cache = cache_of()
    mine = cache.workspace(8, 64)
    assert cache.workspace(8, 64) is mine
    other = []
    thread = threading.Thread(target=lambda: other.extend(
        (cache.workspace(8, 64), cache.workspace(8, 64))))
    thread.start()
    thread.join()
    assert other[0] is other[1]
    assert other[0].data_ptr() != mine.data_ptr()


class CurrentStream:
    """torch.cuda's current stream, and which streams are being captured."""

    def __init__(self, monkeypatch):
        self.current, self.capturing = None, set()
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream",
                            lambda index: self.current.cuda_stream if self.current else 5)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentStream",
                            lambda index: (self.current.stream_id if self.current else 0, 0, 1))
        monkeypatch.setattr(torch._C, "_cuda_setStream", self.switch)
        monkeypatch.setattr(torch.cuda, "stream", self.switched)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing",
                            lambda: self.current in self.capturing)

    def switch(self, stream_id, device_index, device_type):
        assert (device_index, device_type) == (0, 1)
        self.current = {Side.stream_id: Side, 0: None}[stream_id]

    @contextlib.contextmanager
    def switched(self, stream):
        before, self.current = self.current, stream
        yield
        self.current = before


class Side:
    cuda_stream, stream_id, device_index, device_type = 77, 9, 0, 1


def test_a_captured_call_does_not_use_the_kept_workspace(streams, monkeypatch):
    """A graph that holds the kept workspace would write to it at any later time. The
    stream that counts is the call's, not the current one."""
    on, side, cache = CurrentStream(monkeypatch), Side, cache_of()
    kept = cache.workspace(8, 64, side)
    assert cache.workspace(8, 64, side) is kept
    on.capturing = {side}
    captured = cache.workspace(8, 64, side)
    assert captured.data_ptr() != kept.data_ptr()
    assert cache.workspace(4, 64, side).data_ptr() != kept.data_ptr()
    on.capturing = set()
    assert cache.workspace(8, 64, side) is kept
    # the current stream captures, the call's does not
    on.current, on.capturing = None, {None}
    assert cache.workspace(8, 64, side) is kept
    assert cache.workspace(8, 64) is not kept
    assert on.current is None


def test_growing_batches_keep_one_workspace(streams):
    """Not one of each size, for each cache and as long as it lives."""
    caches = [cache_of(), cache_of(heads=8), cache_of()]
    kept = {id(c.workspace(batch, 64)) for batch in (1, 2, 3, 16, 100, 128, 1000, 65535)
            for c in caches}
    assert len(kept) == 1


def test_a_larger_workspace_takes_the_place_of_a_smaller(streams, monkeypatch):
    cache, wide = cache_of(), cache_of(d=256)
    first = cache.workspace(4, 64)
    larger = wide.workspace(4, 64)
    size = binding.moe_paged_attention_workspace_size
    assert larger.numel() >= size(wide.struct, 4, 64) > first.numel() >= size(cache.struct, 4, 64)
    assert cache.workspace(4, 64) is larger and wide.workspace(9, 32) is larger
    CurrentStream(monkeypatch)
    assert cache.workspace(4, 64, Side) is not larger


def test_the_workspace_size_is_the_same_for_every_batch(streams):
    for d in (64, 128, 256):
        for q_heads in (4, 64, 128):
            sizes = {binding.moe_paged_attention_workspace_size(cache_of(d=d).struct, b, q_heads)
                     for b in (0, 1, 5, 100, 65535)}
            assert len(sizes) == 1 and sizes.pop() > 0
    assert binding.moe_paged_attention_workspace_size(cache_of().struct, 65536, 64) == 0


# ---------------------------------------------------------------------------
# numbers that the library's 32-bit arguments do not hold
# ---------------------------------------------------------------------------
def vast(t, *shape):
    """t with a shape (contiguous) that no host memory would hold."""
    class Vast(OnGpu):
        def numel(self):
            return math.prod(shape)

        def stride(self):
            return tuple(math.prod(shape[i + 1:]) for i in range(len(shape)))
    made = Vast(t.t)
    made.shape = torch.Size(shape)
    return made


def test_a_window_past_32_bits_is_refused(calls):
    attend(window=2 ** 31 - 1)
    for window in (2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 32 + 1):   # ctypes would take 0, 5, 1
        with pytest.raises(ValueError, match="window"):
            attend(window=window)
    assert len(calls.made) == 1


def test_a_table_past_32_bits_is_refused(calls):
    for pages in (2 ** 31, 2 ** 32 + 4):
        with pytest.raises(ValueError, match="block_table"):
            attend(block_table=vast(int32(1), 3, pages))
        with pytest.raises(ValueError, match="block_table"):
            read(block_table=vast(int32(1), 3, pages))
    assert not calls.made


@pytest.mark.parametrize("T", [2 ** 31, 2 ** 32 + 3])
def test_more_tokens_than_32_bits_are_refused(calls, T):
    q, k, s = (vast(bf16(1), T, h, 64) for h in (8, 2, 2))
    p, slots = vast(int32(1), 1, T), vast(int32(1), T)
    for call in (lambda: rotate(q=q, q_out=q, k=None, k_out=None, positions=p),
                 lambda: write(k=k, v=s, slots=slots),
                 lambda: write_rotary(q=q, k=k, v=s, q_out=q, positions=p, slots=slots)):
        with pytest.raises(ValueError, match="tokens"):
            call()
    assert not calls.made


def test_more_contexts_to_read_than_32_bits_are_refused(calls):
    n = 2 ** 32 + 3
    with pytest.raises(ValueError, match="block_table|contexts"):
        read(offsets=vast(int32(1), n + 1), block_table=vast(int32(1), n, 4))
    assert not calls.made


# ---------------------------------------------------------------------------
# frequencies as fractions of a turn
# ---------------------------------------------------------------------------
def two_pi(bits=400):
    """2 pi by Machin's formula, 8 (4 atan(1/5) - atan(1/239))."""
    def atan_inverse(n):
        power, total, i = (1 << bits) // n, 0, 0
        while power:
            total += (-1) ** i * (power // (2 * i + 1))
            power //= n * n
            i += 1
        return total
    return Fraction(8 * (4 * atan_inverse(5) - atan_inverse(239)), 1 << bits)


@pytest.mark.parametrize("base", [10000.0, 1000000.0, 5.0, 0.01])
def test_a_turn_is_exact_to_2_31_for_every_position(base):
    """The nearest multiple of 2^-64 turns to the frequency as it is given, so that 2^31
    positions are off by at most 2^31 halves of that."""
    freq = attention.frequencies(64, base)
    turns = attention.Rotary(freq, device="cpu").turns.tolist()
    circle = two_pi()
    for f, n in zip(freq.tolist(), turns):
        for p in (1, 1000003, 2 ** 31 - 1, -2 ** 31):
            off = (Fraction(p * n, 2 ** 64) - p * Fraction(f) / circle) % 1
            assert min(off, 1 - off) <= abs(p) * Fraction(1, 2 ** 65), (p, f)
