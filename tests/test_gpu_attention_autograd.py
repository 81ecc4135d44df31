"""Cache writes and attention over pages have no gradient, and rotary positions none with respect to their frequencies: a backward pass
that comes to them says so; what is called as a step of serving runs as before."""
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


@pytest.fixture
def step():
    c = Cache([6, 1], [10, 40], 4, 2, 64, 16, "bf16")
    g = c.gpu()
    g["cu_seqlens"] = c.cu.cuda()
    return c.q.cuda(), g


@pytest.mark.parametrize("which", ["q", "k_cache", "v_cache"])
def test_attention(step, which):
    q, g = step
    want = gdn.paged_attention(q, **g)
    assert want.grad_fn is None
    t = q if which == "q" else g[which]
    t.requires_grad_()
    got = gdn.paged_attention(q, **g)
    assert got.requires_grad and torch.equal(got, want)
    with pytest.raises(RuntimeError, match="no gradient"):
        (2 * got).sum().backward()
    got = gdn.paged_attention(q, **g)
    got.mul_(2)  # an output like any other
    with pytest.raises(RuntimeError, match="no gradient"):
        got.sum().backward()
    out = torch.empty_like(want)
    assert gdn.paged_attention(q, **g, output=out) is out and out.grad_fn is None and torch.equal(out, want)
    with torch.no_grad():
        assert gdn.paged_attention(q, **g).grad_fn is None
    assert gdn.paged_attention(q.detach(), **{k: v.detach() for k, v in g.items()}).grad_fn is None


def test_append(step):
    q, g = step
    f = gdn.rotary_frequencies(64)
    k, v = (torch.randn(7, 2, 64, device="cuda").bfloat16() for _ in range(2))
    want = gdn.cache_append(k, v, **g, q=q, frequencies=f)
    assert want.grad_fn is None
    for t in (q, f):
        t.requires_grad_()
        got = gdn.cache_append(k, v, **g, q=q, frequencies=f)
        assert torch.equal(got, want)
        with pytest.raises(RuntimeError, match="no gradient"):
            got.sum().backward()
        t.requires_grad_(False)
    q.requires_grad_()
    out = torch.empty_like(want)
    assert gdn.cache_append(k, v, **g, q=q, frequencies=f, output=out) is out and out.grad_fn is None
    k.requires_grad_()
    assert gdn.cache_append(k, v, **g) is None and not g["k_cache"].requires_grad


def test_a_chain_from_the_rotary_positions(step):
    q, g = step
    q.requires_grad_()
    turned, _ = gdn.rotary_embedding(q, None, gdn.rotary_frequencies(64))
    with pytest.raises(RuntimeError, match="no gradient"):
        gdn.paged_attention(turned, **g).sum().backward()


def test_frequencies(step):
    q, _ = step
    f = gdn.rotary_frequencies(64)
    want, _ = gdn.rotary_embedding(q, None, f)
    f.requires_grad_()
    for grad in (False, True):
        x = q.clone().requires_grad_(grad)
        got, _ = gdn.rotary_embedding(x, None, f)
        assert torch.equal(got, want)
        with pytest.raises(RuntimeError, match="frequencies"):
            got.sum().backward()
    out = torch.empty_like(q)
    assert gdn.rotary_embedding(q, None, f, q_out=out)[0] is out and torch.equal(out, want)
    x = q.clone().requires_grad_()
    gdn.rotary_embedding(x, None, f.detach())[0].sum().backward()
    assert x.grad is not None
