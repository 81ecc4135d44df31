"""Attention over a paged cache at the ends of its types' ranges."""
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


@pytest.mark.parametrize("dtype,value", [("bf16", 1e36), ("f16", 60000.0), ("f32", 1e36)])
@pytest.mark.parametrize("heads,tokens", [(1, 1), (40, 1), (8, 40)])
def test_large_values(dtype, value, heads, tokens):
    """The second tile's scores are 5.5 above the first one's, which is less than what raises a row's maximum: the sum of weights times
    values stays within what the keys' number times the values is, 256 times 1e36, below fp32's largest 3.4e38."""
    n = 400 if tokens == 1 else 30  # several units a block, each whole
    c = Cache([tokens] * n, [256 - tokens] * n, heads, 1, 64, 64, dtype, seed=1)
    c.q = torch.zeros_like(c.q)
    c.q[..., 0] = 1.0
    c.v = torch.full_like(c.v, value)
    c.k = torch.zeros_like(c.k)
    for s in c.seqs.tolist():
        c.k[c.table[s, 2:4].long(), :, :, 0] = 5.5
    c.check(scale=1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, 1e-40, -1e-38, 1e-37])
@pytest.mark.parametrize("tokens", [1, 150])
def test_small_scales_of_large_scores(dtype, scale, tokens):
    """Scores of up to 64e36 under scales that leave nothing of them, or some units: with a scale of zero every key counts the same."""
    c = Cache([tokens] * 3, [300 - tokens, 40, 500], 4, 2, 64, 16, dtype, seed=3)
    c.q = torch.full_like(c.q, 1e18)
    c.k = (c.k.float().sign() * 1e18).to(c.dtype)
    c.check(scale=scale)
