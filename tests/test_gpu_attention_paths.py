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


@pytest.mark.parametrize("explicit", [False, True])
def test_a_captured_call_has_a_workspace_of_its_own(explicit):
    """A graph captured with the cache's own workspace, from the current stream or from
    one that the call names, replayed between and next to eager calls."""
    lengths = [3000, 0, 700]
    cache, q, table = attention_case(73, lengths, 16, 2, 128, 16, "e4m3")
    want = check_attention(cache, q, table, lengths)
    args = (q, torch.from_numpy(table).cuda(), on_gpu(lengths))
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    side = torch.cuda.Stream()
    kept = cache.workspace(3, 16, side)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    if explicit:
        with torch.cuda.stream(side):
            graph.capture_begin()
        assert cache.workspace(3, 16, side).data_ptr() != kept.data_ptr()
        cache.attend(*args, out=out, lse=lse, stream=side)
        with torch.cuda.stream(side):
            graph.capture_end()
    else:
        with torch.cuda.graph(graph, stream=side):
            cache.attend(*args, out=out, lse=lse)
    torch.cuda.synchronize()
    assert cache.workspace(3, 16, side) is kept
    for _ in range(20):
        out.zero_()
        lse.zero_()
        torch.cuda.synchronize()
        graph.replay()
        got = [cache.attend(*args, return_lse=True, stream=side) for _ in range(3)]
        torch.cuda.synchronize()
        for o, l in got + [(out, lse)]:
            assert torch.equal(o, want[0]) and torch.equal(l, want[1])


def test_caches_share_a_workspace_that_growing_batches_keep():
    """One buffer serves caches of other shapes and every batch size, with the results of
    a buffer of their own."""
    shapes = [([3000, 100], 16, 2, 128, "e4m3"), ([2000, 0, 900], 8, 2, 256, "bf16"),
              ([700] * 30, 40, 2, 64, "e4m3"), ([1500], 4, 4, 128, "bf16")]
    cases = [(attention_case(80 + i, n, hq, hk, d, 16, kind), n)
             for i, (n, hq, hk, d, kind) in enumerate(shapes)]
    want = [check_attention(*case, n) for case, n in cases]
    buffers = {(c.workspace(1, q.shape[1]).data_ptr()) for (c, q, _), _ in cases}
    assert len(buffers) == 1
    before = torch.cuda.memory_allocated()
    for (cache, q, _), _ in cases:
        for batch in range(1, 200, 7):
            cache.workspace(batch, q.shape[1])
    assert torch.cuda.memory_allocated() == before
    # one after the other on one stream, without a wait between them
    got = [c.attend(q, torch.from_numpy(t).cuda(), on_gpu(n), return_lse=True)
           for _ in range(3) for (c, q, t), n in cases]
    for (out, lse), (o, l) in zip(got, want * 3):
        assert torch.equal(out, o) and torch.equal(lse, l)
