"""The serving loop of the README, run as it stands there."""

import os
import re

import numpy as np
import pytest
import torch

from tests.gpu_helpers import ensure_library, require_gpu
from tests.test_gpu_attention import values, wide_heads
from tests.test_gpu_prompt_attention import ints
from tests.test_gpu_prompt_limits import bounds

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_serving_loop_with_requests_that_leave_and_wait():
    """Prompts, and then steps in which requests in the middle leave, have nothing to do or
    outgrow their tables: every row is attended with its own request's context."""
    require_gpu()
    ensure_library()
    text = open(os.path.join(ROOT, "README.md")).read()
    code = next(c for c in re.findall(r"```python\n(.*?)```", text, re.S) if "PagePool" in c)
    loop = {}
    exec(compile(code, "README.md", "exec"), loop)
    pool, cache, rotary = loop["pool"], loop["cache"], loop["rotary"]
    batch, hq, hk, d = pool.table.shape[0], 8, cache.heads, cache.head_dim
    rng = np.random.default_rng(17)
    steps = [[50, 0, 130, 7, 64, 1, 0, 3], [1, 1, 1, 1, 1, 1, 1, 1], [1, 1, -1, 1, 0, 1, 20000, 1],
             [1, -1, 5, 20000, 1, 1, 1, 1]]
    held = [0] * batch
    for news in steps:
        news = news + [0] * (batch - len(news))
        got = [n if 0 < n < 20000 else 0 for n in news]
        rows = sum(got) + 3
        plan = pool.plan(ints(news), rows=rows, axes=3)
        held = [0 if n < 0 else h + g for h, n, g in zip(held, news, got)]
        assert plan.offsets.tolist() == np.concatenate([[0], np.cumsum(got)]).tolist()
        assert plan.lengths.tolist() == held
        assert plan.refused.tolist() == [sum(n == 20000 for n in news)]
        q, k, v = wide_heads(rng, rows, hq, hk, hk, d=d)
        out = loop["step"](plan, q, k, v)
        turned, _ = rotary.apply(plan.positions, q)
        # token scales: half a step of fp16 for a value too
        ref, _, tol, _ = bounds(cache, turned, pool.table.cpu().numpy(), held, got,
                                value=2.0 ** -11)
        assert np.all(np.abs(values(out) - ref) <= tol)
        assert torch.all(out[sum(got):] == 0)
        assert pool.state.tolist()[:-1] == held
