"""Host side of the attention classes and their binding, on stand-ins for GPU
tensors: what is refused before the library is called, and which workspace a
call gets. No call here reaches a kernel."""

import pytest
import torch

from expert_layer_ptpc_gb300 import binding


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
