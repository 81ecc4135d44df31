"""Attention over a paged cache in captured graphs that share their workspaces, replayed in turn with other lengths and other keys, against the
definition."""
import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from attention_testlib import Cache, attention_bound, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.build()


class Step:
    def __init__(self, c, tokens):
        self.c, self.g, self.q = c, c.gpu(), c.q.cuda()
        self.how = dict(tokens_per_seq=tokens) if tokens else dict(cu_seqlens=c.cu.cuda())
        self.out = torch.full_like(self.q, 7.0)

    def call(self):
        gdn.paged_attention(self.q, **self.g, **self.how, output=self.out)

    def shorten(self, by):
        """Sequences end earlier (as if their last tokens had been dropped); the keys before that are new ones."""
        c = self.c
        for s, n in zip(c.seqs.tolist(), c.lens):
            c.lengths[s] = max(n, int(c.lengths[s]) - by)
        c.k, c.v = (torch.where(torch.isnan(t), t, torch.randn(t.shape, generator=torch.Generator().manual_seed(by)).to(t.dtype)) for t in (c.k, c.v))
        self.g["lengths"].copy_(c.lengths)
        self.g["k_cache"].copy_(c.k)
        self.g["v_cache"].copy_(c.v)

    def check(self, name):
        out, _, size, products, count = self.c.want()
        close(name, self.out, out, attention_bound(out, size, products, count, self.c.D, self.c.dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_graphs_of_one_pool(dtype):
    steps = [Step(Cache([1] * 6, [300, 10, 0, 77, 900, 64], 8, 2, 128, 16, dtype), 1),
             Step(Cache([90, 1, 40], [400, 700, 0], 8, 2, 128, 16, dtype, seed=2), 0)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for x in steps:
            x.call()
    s.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in steps]
    for x, graph in zip(steps, graphs):
        with torch.cuda.graph(graph, pool=graphs[0].pool() if graph is not graphs[0] else None):
            x.call()
    for by in (0, 30, 250):
        for x in steps:
            x.shorten(by)
            x.out.fill_(7.0)
        for _ in range(2):
            for graph in graphs:
                graph.replay()
        torch.cuda.synchronize()
        for i, x in enumerate(steps):
            x.check(f"graph {i}, lengths less {by}")
