"""Outputs of attention of many tokens that lie over q, in one buffer with it in every way, on the
host: no call here reaches a kernel."""

import pytest
import torch

from expert_layer_ptpc_gb300 import binding
from tests.test_attention_host import OnGpu, cache_struct, calls, int32  # noqa: F401


def overlaps(a, a_stride, b, b_stride, rows, width):
    cells = [set(), set()]
    for at, stride, c in ((a, a_stride, cells[0]), (b, b_stride, cells[1])):
        for r in range(rows):
            c.update(range(at // 2 + r * stride, at // 2 + r * stride + width))
    return bool(cells[0] & cells[1])


@pytest.mark.parametrize("rows", [0, 1, 2, 3, 5])
@pytest.mark.parametrize("stride", [8, 9, 13, 16, 24])
def test_equal_strides(rows, stride):
    width, a = 8, 4096
    for ahead in range(-6 * stride, 6 * stride + 1):
        b = a + 2 * ahead
        assert binding._tokens_overlap(a, stride, b, stride, rows, width) == \
            overlaps(a, stride, b, stride, rows, width), ahead


@pytest.mark.parametrize("rows", [1, 2, 4])
def test_other_strides_are_refused_only_where_they_share_elements(rows):
    width, a = 8, 4096
    for a_stride, b_stride in ((8, 16), (16, 24), (24, 8)):
        for ahead in range(-100, 101):
            b = a + 2 * ahead
            if binding._tokens_overlap(a, a_stride, b, b_stride, rows, width):
                assert overlaps(a, a_stride, b, b_stride, rows, width)
        assert binding._tokens_overlap(a, a_stride, a, b_stride, rows, width)


def test_slices_of_one_buffer(calls):  # noqa: F811
    """A token on or a head on is refused, the heads beside q's are taken."""
    wide = torch.zeros((9, 24, 64), dtype=torch.bfloat16)
    args = (int32(4), int32(3, 4), int32(3), 0.125)
    ws = OnGpu(torch.zeros(64, dtype=torch.uint8))
    q = OnGpu(wide[:5, :8])
    for out in (wide[:5, :8], wide[1:6, :8], wide[4:9, :8], wide[:5, 4:12], wide[1:6, 7:15]):
        with pytest.raises(ValueError, match="overlap"):
            binding.moe_prompt_attention(cache_struct(), q, *args, out=OnGpu(out), ws=ws)
    assert not calls.made
    for out in (wide[:5, 8:16], wide[2:7, 16:24], wide[:5, 8:16].clone()):
        binding.moe_prompt_attention(cache_struct(), q, *args, out=OnGpu(out), ws=ws)
    assert len(calls.made) == 3
