"""Paths of the attention operators that the sizes of test_gpu_attention.py do not
reach, with the same oracle and bounds, and calls from threads, streams and graphs."""

import threading

import pytest
import torch

from tests.gpu_helpers import ensure_library, require_gpu
from tests.test_gpu_attention import attention_case, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    require_gpu()
    ensure_library()


def on_gpu(lengths):
    return torch.tensor(lengths, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# threads, streams, graphs
# ---------------------------------------------------------------------------
def test_threads_on_one_stream():
    """Threads that attend over one cache on one stream, each with contexts that are cut
    over many CTAs and joined: every call gives its own results."""
    cases = [attention_case(71, [5000, 300], 16, 2, 128, 16, "e4m3"),
             attention_case(72, [900, 0, 4100, 33, 2500], 32, 2, 128, 16, "e4m3")]
    cache = cases[0][0]
    cases[1][2][:] %= cache.pages
    lengths = ([5000, 300], [900, 0, 4100, 33, 2500])
    inputs = [(q, torch.from_numpy(table).cuda(), on_gpu(n))
              for (_, q, table), n in zip(cases, lengths)]
    want = [check_attention(cache, q, table, n) for (_, q, table), n in zip(cases, lengths)]
    stream = torch.cuda.current_stream()
    wrong, start = [], threading.Barrier(4)

    def serve(i):
        with torch.cuda.stream(stream):
            start.wait()
            for _ in range(300):
                out, lse = cache.attend(*inputs[i % 2], return_lse=True)
                if not (torch.equal(out, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])):
                    wrong.append(i)

    threads = [threading.Thread(target=serve, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
