"""Captured calls of the 8-bit cache's attention that run at the same time: every graph has scratch
of its own."""
import pytest

from tests.test_q8_cache_gpu import A, _gpu, bf16, dev_cache, ints, make_attend  # noqa: F401

pytestmark = pytest.mark.gpu


def test_graphs_replayed_at_once():
    """Four graphs of several calls each (one row, several, a chunk), replayed on four streams while
    the current stream runs the same calls."""
    import torch

    import flash_attention_gb300 as fa

    c = A("graphs", 4, 8, 2, 1, 128, 16, 16, [3000, 700, 1, 250])
    rng, table, P, cache, _ = make_attend(c)
    got, tb, lens = dev_cache(*cache), ints(table), ints(c["lengths"])
    qs = [bf16(rng.standard_normal((4, 8, n, 128)))[0] for n in (1, 1, 4, 20)]

    def calls(q):
        return [fa.q8_paged_attention(q, *got, tb, lens, scale=0.1) for _ in range(4)]

    want = [calls(q)[0] for q in qs]
    graphs, outs = [], []
    torch.cuda.synchronize()
    for q in qs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(calls(q))
    streams = [torch.cuda.Stream() for _ in qs]
    for i in range(20):
        for x in outs:
            for o, lse in x:
                o.fill_(7)
                lse.fill_(7)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        eager = calls(qs[i % 4])
        torch.cuda.synchronize()
        for x, (o, lse) in zip([*outs, eager], [*want, want[i % 4]]):
            assert all(torch.equal(a, o) and torch.equal(b, lse) for a, b in x)
    assert fa.fa_device_status(True) == fa.FA_OK
