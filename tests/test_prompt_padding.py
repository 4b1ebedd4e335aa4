"""Which entry point attention of many tokens takes, and what the padded one refuses, on the
host: no call here reaches a kernel."""

import ctypes

import pytest
import torch

from expert_layer_ptpc_gb300 import binding
from tests.test_attention_host import OnGpu, bf16, cache_struct, calls, int32  # noqa: F401
from tests.test_attention_refusals import (A, BAD_CACHES, INVALID, MIS, P, UNSUPPORTED,  # noqa: F401
                                           WORKSPACE, cache, lib)


def padded(lib, c=None, q=A, qs=1024, rows=4, hq=8, offsets=A, table=A, stride=4,  # noqa: F811
           wide=4, lengths=A, batch=2, scale=1.0, window=0, out=A, outs=1024, lse=None, ws=A,
           ws_bytes=1 << 40):
    return lib.moe_prompt_attention_padded(
        ctypes.byref(c if c is not None else cache()), P(q), qs, rows, hq, P(offsets), P(table),
        stride, wide, P(lengths), batch, scale, window, P(out), outs, P(lse), P(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), 0), (dict(rows=0, batch=0), 0), (dict(rows=-1), INVALID),
    (dict(batch=-1), INVALID), (dict(hq=7), INVALID), (dict(window=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(q=None), INVALID), (dict(qs=1016), INVALID),
    (dict(offsets=None), INVALID), (dict(lengths=A + 2), INVALID), (dict(table=None), INVALID),
    (dict(out=MIS), INVALID), (dict(outs=1016), INVALID), (dict(lse=A + 2), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=0), WORKSPACE), (dict(batch=65536), UNSUPPORTED),
    # without a context, but with rows to fill: their place is needed, lengths and tables are not
    (dict(batch=0, out=None), INVALID), (dict(batch=0, offsets=None), INVALID),
    (dict(batch=0, lengths=None, table=None, ws=None), WORKSPACE),
])
def test_padded_refusals(lib, kw, want):  # noqa: F811
    assert padded(lib, **kw) == want


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_caches_refused(lib, kw, want):  # noqa: F811
    assert padded(lib, cache(**kw), rows=0) == want


@pytest.mark.parametrize("out", [False, True])
@pytest.mark.parametrize("lse", ["none", "given", "asked"])
def test_the_entry_point(calls, monkeypatch, out, lse):  # noqa: F811
    """Only where every output is the call's own do the kernels fill the padding; a new tensor
    beside one of the caller's is filled before."""
    class New(OnGpu):
        def fill_(self, value):
            filled.append(value)
            return self

    filled = []
    monkeypatch.setattr(binding, "_empty", lambda shape, dtype, device, stream: New(
        torch.empty(shape, dtype=dtype)))
    kw = dict(out=bf16(5, 8, 64)) if out else {}
    if lse == "given":
        kw["lse"] = OnGpu(torch.zeros((5, 8)))
    binding.moe_prompt_attention(cache_struct(), bf16(5, 8, 64), int32(4), int32(3, 4), int32(3),
                                 0.125, return_lse=lse != "none",
                                 ws=OnGpu(torch.zeros(64, dtype=torch.uint8)), **kw)
    (name, _), = calls.made
    every = not out and lse != "given"
    assert name == ("moe_prompt_attention_padded" if every else "moe_prompt_attention")
    assert filled == ([] if every else [0.0] if not out else
                      [float("-inf")] if lse == "asked" else [])
