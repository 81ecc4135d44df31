"""Rotary positions and cache writes: where their results may lie."""
import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from attention_testlib import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.build()


def inputs():
    g = torch.Generator().manual_seed(0)
    whole = torch.randn(70, 8, 64, generator=g).bfloat16().cuda()
    return (whole, *whole.split([4, 2, 2], dim=1))


def test_slices_of_one_tensor_and_in_place():
    whole, q, k, v = inputs()
    f = gdn.rotary_frequencies(64)
    want = gdn.rotary_embedding(q, k, f)
    out = torch.full_like(whole, 7.0)
    gdn.rotary_embedding(q, k, f, q_out=out[:, 3:7], k_out=out[:, 1:3])
    assert torch.equal(out[:, 3:7], want[0]) and torch.equal(out[:, 1:3], want[1]) and bool((out[:, [0, 7]] == 7.0).all())
    other = whole.clone()  # q in place, k into v's heads of the same tensor
    gdn.rotary_embedding(other[:, :4], other[:, 4:6], f, q_out=other[:, :4], k_out=other[:, 6:])
    assert torch.equal(other[:, :4], want[0]) and torch.equal(other[:, 4:6], k) and torch.equal(other[:, 6:], want[1])
    c = Cache([70], [0], 4, 2, 64, 16, "bf16", fill=0.0)
    g = c.gpu()
    got = gdn.cache_append(k, v, **g, q=q, frequencies=f, output=q)
    assert got is q and torch.equal(q, want[0])
    page = c.table[c.seqs[0]].long()[:5].cuda()
    assert torch.equal(g["k_cache"][page].flatten(0, 1)[:70], want[1])


def test_overlaps_are_refused():
    whole, q, k, v = inputs()
    f = gdn.rotary_frequencies(64)
    g = Cache([70], [0], 4, 2, 64, 16, "bf16", fill=0.0).gpu()
    before, cached = whole.clone(), g["k_cache"].clone()
    for kw in (dict(q_out=whole[:, 1:5]), dict(q_out=whole[:, 3:7]), dict(k_out=whole[:, 3:5]), dict(k_out=whole[:, 5:7]),
               dict(k_out=whole[:, :2]), dict(q_out=q, k_out=whole[:, 2:4])):
        with pytest.raises(gdn.GdnError):
            gdn.rotary_embedding(q, k, f, **kw)
    for output in (whole[:, 1:5], whole[:, 2:6], whole[:, 4:]):
        with pytest.raises(gdn.GdnError):
            gdn.cache_append(k, v, **g, q=q, frequencies=f, output=output)
    torch.cuda.synchronize()
    assert torch.equal(whole, before) and torch.equal(g["k_cache"], cached)
