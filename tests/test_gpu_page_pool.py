"""The page pool between its plans: pages that a caller gives back, one owner for each."""

import numpy as np
import pytest
import torch

from expert_layer_ptpc_gb300 import attention
from tests.gpu_helpers import ensure_library, require_gpu
from tests.test_gpu_prompt_attention import KINDS, any_cache, check_prompt, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    require_gpu()
    ensure_library()


def owned(pool):
    """Every page once: of the requests' entries, and of the stack."""
    *held, free = pool.state.tolist()
    size, pages = pool.page_size, pool.stack.numel()
    used = [p for row, h in zip(pool.table.tolist(), held) for p in row[:-(-h // size)]
            if 0 <= p < pages]
    return sorted(used + pool.stack.tolist()[:free]) == list(range(pages))


def give_back(pool, b, columns):
    free = int(pool.state[-1])
    pages = pool.table[b, columns].clone()
    pool.stack[free:free + len(pages)] = pages
    pool.state[-1] += len(pages)
    pool.table[b, columns] = -1


def test_rejected_drafts_go_back():
    """Tokens taken back over page borders, by a page or by several, and all of a request's."""
    rng = np.random.default_rng(3)
    pool = attention.PagePool.empty(60, 4, 5, 20)
    for step in range(40):
        held = pool.state.tolist()[:-1]
        new = [int(rng.choice([0, 1, 6, 9])) if h < 50 else -1 for h in held]
        plan = pool.plan(ints(new), 64)
        pool.commit(plan)
        assert owned(pool)
        held = pool.state.tolist()[:-1]
        for b, h in enumerate(held):
            keep = max(0, h - int(rng.choice([0, 1, 5, 9])))
            give_back(pool, b, slice(-(-keep // 4), -(-h // 4)))
            pool.state[b] = keep
        assert owned(pool)


@pytest.mark.parametrize("kind", KINDS)
def test_pages_behind_a_window_go_back(kind):
    """Requests that see a window only: pages behind it given back as they go, and taken by others;
    attention against the oracle all along."""
    rng = np.random.default_rng(5)
    batch, size, window, hq, hk, d = 3, 8, 20, 4, 2, 64
    pool = attention.PagePool.empty(16, size, batch, 30)
    cache = any_cache(rng, 16, hk, size, d, kind)
    for step in range(12):
        held = pool.state.tolist()[:-1]
        new = [-1 if h > 90 else 9 for h in held]
        plan = pool.plan(ints(new), 27)
        assert plan.refused.tolist() == [0]
        k, v, q = (torch.from_numpy(rng.standard_normal((27, h, d)).astype(np.float32))
                   .to(torch.bfloat16).cuda() for h in (hk, hk, hq))
        cache.write(k, v, plan.slots)
        lengths = plan.lengths.tolist()
        check_prompt(cache, q[:plan.offsets[-1]], pool.table.cpu().numpy(), lengths,
                     np.diff(plan.offsets.tolist()).tolist(), window=window, kind=kind)
        pool.commit(plan)
        for b, n in enumerate(lengths):      # what the next step's first row no longer sees
            behind = max(0, n + 1 - window) // size
            columns = [c for c in range(behind) if int(pool.table[b, c]) >= 0]
            if columns:
                give_back(pool, b, columns)
        assert owned(pool)
