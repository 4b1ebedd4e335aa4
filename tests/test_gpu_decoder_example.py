"""The decoder-layer example: attention and MoE block together, step by step."""

import pytest

from tests.gpu_helpers import ensure_library, require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
def test_decoder_step_example(cache):
    require_gpu()
    ensure_library()
    import importlib.util
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location(
        "decoder_step", os.path.join(root, "examples", "decoder_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # both sides round to bf16 (half a step is 2^-8 of the value); the contexts
    # read back from an e4m3 cache are rounded to bf16 too
    worst = example.main(["--steps", "3", "--batch", "5", "--prompt", "150", "--cache", cache])
    assert worst <= 2 * 2.0 ** -8
