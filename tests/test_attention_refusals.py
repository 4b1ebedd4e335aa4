"""What the attention entry points refuse, checked on the host: no call here
reaches a kernel."""

import ctypes

import pytest
import torch

from expert_layer_ptpc_gb300 import attention, binding, build

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -4


def P(v):
    return ctypes.c_void_p(v)


A, MIS = 0x10000, 0x10008     # aligned and misaligned fake pointers


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def cache(**kw):
    f = dict(k=A, v=A, k_scale=A, v_scale=A, pages=8, heads=2, page_size=16, head_dim=128,
             dtype=binding.MOE_DTYPE_E4M3)
    f.update(kw)
    return binding.moe_kv_cache(*(f[n] for n, _ in binding.moe_kv_cache._fields_))


def plan(**kw):
    f = dict(turns=A, pair_axis=A, axes=3, rot_dim=128, neighbours=0)
    f.update(kw)
    return binding.moe_rotary_plan(*(f[n] for n, _ in binding.moe_rotary_plan._fields_))


BAD_CACHES = [
    (dict(k=None), INVALID), (dict(v=MIS), INVALID), (dict(k_scale=None), INVALID),
    (dict(v_scale=MIS), INVALID), (dict(pages=0), INVALID), (dict(heads=-1), INVALID),
    (dict(page_size=0), INVALID), (dict(head_dim=0), INVALID),
    (dict(dtype=binding.MOE_DTYPE_F32), INVALID),
    (dict(dtype=binding.MOE_DTYPE_BF16), INVALID),               # bf16 with scales
    (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=512), UNSUPPORTED),
    (dict(page_size=24), UNSUPPORTED), (dict(page_size=2048), UNSUPPORTED),
    (dict(pages=1 << 27), UNSUPPORTED),                          # 2^31 slots
    (dict(pages=1 << 26, heads=4), UNSUPPORTED),                 # 2^32 rows
    (dict(heads=1 << 20), UNSUPPORTED),
]


def rotary(lib, p=None, positions=A, T=4, d=128, q=A, qs=1024, hq=8, qo=A, qos=1024, k=None,
           ks=0, hk=0, ko=None, kos=0):
    return lib.moe_rotary(ctypes.byref(p if p is not None else plan()), P(positions), T, d, P(q),
                          qs, hq, P(qo), qos, P(k), ks, hk, P(ko), kos, 0, None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(T=0), 0), (dict(hq=0), INVALID), (dict(d=0), INVALID),
    (dict(d=120), UNSUPPORTED), (dict(d=528), UNSUPPORTED),
    (dict(hq=513, qs=65664, qos=65664), UNSUPPORTED),            # more than 65536 elements
    (dict(q=None), INVALID), (dict(q=MIS), INVALID), (dict(qo=None), INVALID),
    (dict(qs=1020), INVALID), (dict(qs=1016), INVALID), (dict(qos=1016), INVALID),
    (dict(positions=None), INVALID), (dict(positions=A + 2), INVALID),
    (dict(k=A, ks=256, hk=2, ko=None), INVALID), (dict(k=A, ks=248, hk=2, ko=A, kos=256), INVALID),
    (dict(k=A, ks=256, hk=0, ko=A, kos=256), INVALID),
    (dict(p=plan(axes=0)), INVALID), (dict(p=plan(axes=9)), INVALID),
    (dict(p=plan(turns=None)), INVALID), (dict(p=plan(turns=A + 4)), INVALID),
    (dict(p=plan(pair_axis=None)), INVALID), (dict(p=plan(rot_dim=0)), INVALID),
    (dict(p=plan(rot_dim=24)), INVALID), (dict(p=plan(rot_dim=144)), INVALID),
    (dict(p=plan(neighbours=2)), INVALID),
])
def test_rotary_refusals(lib, kw, want):
    assert rotary(lib, **kw) == want


def write(lib, c=None, slots=A, T=4, k=A, ks=256, v=A, vs=256):
    return lib.moe_kv_write(ctypes.byref(c if c is not None else cache()), P(slots), T, P(k), ks,
                            P(v), vs, None)


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_caches_refused_everywhere(lib, kw, want):
    c = cache(**kw)
    assert write(lib, c, T=0) == want
    assert lib.moe_kv_read(ctypes.byref(c), P(A), 4, 4, P(A), 1, 0, P(A), P(A), None) == want
    assert lib.moe_paged_attention(ctypes.byref(c), P(A), 1024, 0, 8, P(A), 4, 4, P(A), 1.0, 0,
                                   P(A), None, P(A), 1 << 30, None) == want
    assert lib.moe_rotary_kv_write(ctypes.byref(plan()), P(A), ctypes.byref(c), P(A), 0, P(A),
                                   1024, 8, P(A), 1024, P(A), 256, P(A), 256, None) == want
    assert lib.moe_paged_attention_workspace_size(ctypes.byref(c), 1, 8) == 0


def test_null_cache_refused(lib):
    assert lib.moe_kv_write(None, P(A), 1, P(A), 256, P(A), 256, None) == INVALID
    assert lib.moe_paged_attention_workspace_size(None, 1, 8) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(T=0), 0), (dict(slots=None), INVALID),
    (dict(slots=A + 2), INVALID), (dict(k=None), INVALID), (dict(v=MIS), INVALID),
    (dict(ks=248), INVALID), (dict(vs=260), INVALID),
    (dict(c=cache(heads=512), ks=65536, vs=65536), UNSUPPORTED),
])
def test_write_refusals(lib, kw, want):
    assert write(lib, **kw) == want


def test_fused_write_refusals(lib):
    def call(p=plan(), positions=A, T=4, q=A, qs=1024, hq=8, qo=A, ks=256):
        return lib.moe_rotary_kv_write(ctypes.byref(p), P(positions), ctypes.byref(cache()), P(A),
                                       T, P(q), qs, hq, P(qo), 1024, P(A), ks, P(A), 256, None)
    assert call(T=0) == 0
    for kw in (dict(T=-1), dict(hq=0), dict(q=None), dict(qo=MIS), dict(qs=1016), dict(ks=128),
               dict(positions=None), dict(p=plan(rot_dim=256))):
        assert call(**kw) == INVALID, kw
    assert call(hq=512, qs=65536) == UNSUPPORTED


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), 0), (dict(rows=-1), INVALID), (dict(batch=0), INVALID),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(table=None), INVALID), (dict(table=A + 2), INVALID),
    (dict(stride=3), INVALID), (dict(pages=-1, stride=0), INVALID), (dict(offsets=None), INVALID),
    (dict(ko=None), INVALID), (dict(vo=MIS), INVALID),
])
def test_read_refusals(lib, kw, want):
    f = dict(table=A, stride=4, pages=4, offsets=A, batch=1, rows=7, ko=A, vo=A)
    f.update(kw)
    assert lib.moe_kv_read(ctypes.byref(cache()), P(f["table"]), f["stride"], f["pages"],
                           P(f["offsets"]), f["batch"], f["rows"], P(f["ko"]), P(f["vo"]),
                           None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(batch=0), 0), (dict(batch=-1), INVALID), (dict(hq=0), INVALID), (dict(hq=7), INVALID),
    (dict(batch=65536), UNSUPPORTED), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(window=-1), INVALID), (dict(q=None), INVALID),
    (dict(q=MIS), INVALID), (dict(qs=1016), INVALID), (dict(table=None), INVALID),
    (dict(stride=3), INVALID), (dict(pages=-1, stride=0), INVALID), (dict(lengths=None), INVALID),
    (dict(out=None), INVALID), (dict(out=MIS), INVALID), (dict(lse=A + 2), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=MIS), WORKSPACE), (dict(ws_bytes=16), WORKSPACE),
    # 2 x 65535 items of 2^24 tokens: more units than the cut can number
    (dict(batch=65535, stride=1 << 20, pages=1 << 20), UNSUPPORTED),
])
def test_attention_refusals(lib, kw, want):
    f = dict(q=A, qs=1024, batch=2, hq=8, table=A, stride=4, pages=4, lengths=A, scale=0.1,
             window=0, out=A, lse=None, ws=A, ws_bytes=1 << 30)
    f.update(kw)
    assert lib.moe_paged_attention(
        ctypes.byref(cache()), P(f["q"]), f["qs"], f["batch"], f["hq"], P(f["table"]), f["stride"],
        f["pages"], P(f["lengths"]), f["scale"], f["window"], P(f["out"]), P(f["lse"]),
        P(f["ws"]), f["ws_bytes"], None) == want


def test_workspace_size(lib):
    c = cache()
    n = lib.moe_paged_attention_workspace_size(ctypes.byref(c), 4, 8)
    assert n > 16
    assert lib.moe_paged_attention_workspace_size(ctypes.byref(c), 4, 7) == 0
    assert lib.moe_paged_attention_workspace_size(ctypes.byref(c), -1, 8) == 0


def test_tensor_checks_raise():
    """The classes and the binding name what is wrong with a tensor."""
    pages = torch.zeros((2, 1, 16, 64), dtype=torch.uint8)
    scales = torch.ones((2, 1, 16))
    with pytest.raises(ValueError, match="scales"):
        attention.PagedKVCache(pages, pages)
    with pytest.raises(ValueError, match="alike"):
        attention.PagedKVCache(pages, pages[:1], scales, scales)
    with pytest.raises(ValueError, match="uint8"):
        attention.PagedKVCache(pages.float(), pages.float())
    with pytest.raises(ValueError, match="CUDA"):
        attention.PagedKVCache(pages, pages, scales, scales)
    with pytest.raises(ValueError, match="dtype"):
        attention.PagedKVCache.empty(1, 1, 16, 64, dtype="int8", device="cpu")
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        binding.moe_rotary(plan(), torch.zeros((3, 2), dtype=torch.int32), q)
