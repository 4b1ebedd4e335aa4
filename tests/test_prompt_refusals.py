"""What the entry points of a step's plan, of attention of many tokens and of caches with
one scale per page refuse, checked on the host: no call here reaches a kernel."""

import ctypes

import pytest
import torch

from expert_layer_ptpc_gb300 import attention, binding
from tests.test_attention_refusals import (A, BAD_CACHES, INVALID, MIS, P, UNSUPPORTED, WORKSPACE,
                                           cache, lib, write)  # noqa: F401

PAGE = binding.MOE_DTYPE_E4M3_PAGE


def plan(lib, state=A, new=A, batch=4, table=A, stride=8, wide=8, stack=A, pages=32,  # noqa: F811
         size=16, rows=4, axes=1, offsets=A, slots=A, positions=A, out=A, refused=A):
    return lib.moe_kv_plan(P(state), P(new), batch, P(table), stride, wide, P(stack), pages, size,
                           rows, axes, P(offsets), P(slots), P(positions), P(out), P(refused),
                           None)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=0), INVALID), (dict(batch=4097), UNSUPPORTED), (dict(state=None), INVALID),
    (dict(new=A + 2), INVALID), (dict(table=None), INVALID), (dict(stride=7), INVALID),
    (dict(wide=0), INVALID), (dict(stack=None), INVALID), (dict(pages=0), INVALID),
    (dict(size=0), INVALID), (dict(size=24), UNSUPPORTED), (dict(size=2048), UNSUPPORTED),
    (dict(pages=1 << 27), UNSUPPORTED), (dict(rows=-1), INVALID), (dict(axes=0), INVALID),
    (dict(axes=9), INVALID), (dict(offsets=None), INVALID), (dict(slots=None), INVALID),
    (dict(positions=A + 1), INVALID), (dict(out=None), INVALID), (dict(refused=None), INVALID),
])
def test_plan_refusals(lib, kw, want):  # noqa: F811
    assert plan(lib, **kw) == want


def prompt(lib, c=None, q=A, qs=1024, rows=4, hq=8, offsets=A, table=A, stride=4,  # noqa: F811
           wide=4, lengths=A, batch=2, scale=1.0, window=0, out=A, outs=1024, lse=None, ws=A,
           ws_bytes=1 << 40):
    return lib.moe_prompt_attention(ctypes.byref(c if c is not None else cache()), P(q), qs, rows,
                                    hq, P(offsets), P(table), stride, wide, P(lengths), batch,
                                    scale, window, P(out), outs, P(lse), P(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), 0), (dict(batch=0), 0), (dict(rows=-1), INVALID), (dict(batch=-1), INVALID),
    (dict(hq=0), INVALID), (dict(hq=7), INVALID), (dict(window=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(q=None), INVALID), (dict(q=MIS), INVALID), (dict(qs=1016), INVALID),
    (dict(qs=1020), INVALID), (dict(offsets=None), INVALID), (dict(lengths=A + 2), INVALID),
    (dict(table=None), INVALID), (dict(stride=3), INVALID), (dict(wide=-1), INVALID),
    (dict(out=MIS), INVALID), (dict(outs=1016), INVALID), (dict(lse=A + 2), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=MIS), WORKSPACE), (dict(ws_bytes=0), WORKSPACE),
    (dict(batch=65536), UNSUPPORTED), (dict(hq=65536, qs=65536 * 128), UNSUPPORTED),
    (dict(rows=1 << 28), UNSUPPORTED),
    # (a table's room of 2^31 tokens, 2^24 rows of 8 heads on 2)
    (dict(rows=1 << 24, c=cache(page_size=1024), wide=1 << 21, stride=1 << 21), UNSUPPORTED),
])
def test_prompt_refusals(lib, kw, want):  # noqa: F811
    assert prompt(lib, **kw) == want


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_caches_refused_for_prompts_and_with_page_scales(lib, kw, want):  # noqa: F811
    assert prompt(lib, cache(**kw), rows=0) == want
    assert lib.moe_prompt_attention_workspace_size(ctypes.byref(cache(**kw)), 8) == 0
    if "dtype" in kw:
        return
    c = cache(**{"dtype": PAGE, **kw})
    assert write(lib, c, T=0) == want
    assert prompt(lib, c, rows=0) == want
    assert lib.moe_paged_attention_workspace_size(ctypes.byref(c), 1, 8) == 0


def test_workspaces_of_page_caches(lib):  # noqa: F811
    c = cache(dtype=PAGE)
    assert write(lib, c, T=0) == 0
    assert lib.moe_paged_attention_workspace_size(ctypes.byref(c), 1, 8) == \
        lib.moe_paged_attention_workspace_size(ctypes.byref(cache()), 1, 8) > 0
    assert lib.moe_prompt_attention_workspace_size(ctypes.byref(c), 8) > 0
    assert lib.moe_prompt_attention_workspace_size(ctypes.byref(c), 7) == 0
    assert lib.moe_prompt_attention_workspace_size(None, 8) == 0


def test_pool_arguments():
    table, stack = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    state = torch.zeros(3, dtype=torch.int32)
    for bad in (dict(page_size=0), dict(page_size=24), dict(page_size=2048),
                dict(state=state[:2]), dict(table=table[0]), dict(stack=table),
                dict(state=table)):
        kw = dict(table=table, stack=stack, state=state, page_size=16)
        kw.update(bad)
        with pytest.raises(ValueError):
            attention.PagePool(**kw)
    pool = attention.PagePool(table, stack, state, 16)
    with pytest.raises(ValueError):                     # host tensors
        pool.plan(torch.zeros(2, dtype=torch.int32), 4)


def test_host_tensors_refused():
    q = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.moe_prompt_attention(cache(), q, torch.zeros(2, dtype=torch.int32),
                                     torch.zeros((1, 1), dtype=torch.int32),
                                     torch.zeros(1, dtype=torch.int32), 1.0)
    k = torch.zeros((3, 2, 16, 64), dtype=torch.uint8)
    with pytest.raises(ValueError):
        attention.PagedKVCache(k, k, torch.zeros((3, 2)), torch.zeros((3, 2)))
