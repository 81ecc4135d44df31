"""Attention over a paged cache on CUDA cores: head sizes around where one or two blocks fit an SM, and what the launch counts on."""
import ctypes

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


@pytest.mark.parametrize("D", [60, 65, 68, 72, 97, 101, 104, 107, 112, 116, 120, 121, 124, 125, 127, 128, 129, 132])
def test_head_sizes(D):
    c = Cache([70, 1, 9], [130, 300, 0], 6, 2, D, 16, "f32", seed=D)
    c.check()
    c.check(window=50)


@pytest.mark.parametrize("D", [64, 100, 112, 124, 125, 128, 256])
def test_as_many_blocks_as_fit_at_once(D):
    """The workspace has two slots of 64 rows for each block of the launch, and the launch as many blocks as are resident: two an SM where
    two times three tiles of 64 rows of an odd multiple of 4 floats, the weights, and 2.5 KB fit 228 KB."""
    row = 4 * ((D + 3) // 4 | 1)
    fit = 2 if 2 * (4 * (3 * 64 * row + 64 * 68) + 64 * 16 + 1536) <= 228 * 1024 else 1
    blocks = fit * torch.cuda.get_device_properties(0).multi_processor_count
    q = torch.zeros(8, 2, D, device="cuda")
    cache, word = torch.zeros(4, 16, 2, D, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    kv = gdn.KvCache(cache.data_ptr(), cache.data_ptr(), *cache.stride()[:3], *cache.stride()[:3], 2, D, gdn.DTYPE_F32)
    batch = gdn.KvBatch(None, None, word.data_ptr(), word.data_ptr(), 8, 1, 8, 0, 1, 1, 4, 16, None)
    args = gdn.AttentionArgs(q.data_ptr(), torch.empty_like(q).data_ptr(), None, 0, 0, 2, 1.0, 1, 0)
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    want = up(2 * blocks * 16) + up(2 * blocks * 64 * 8) + up(2 * blocks * 64 * D * 4)
    assert gdn.lib().gdn_attention_workspace(ctypes.byref(batch), ctypes.byref(kv), ctypes.byref(args)) == want


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [60, 62, 70, 84, 102, 122, 126, 130])
def test_few_rows_in_narrow_pieces(dtype, D):
    """Rows that are multiples of 4 or 8 bytes, on either side of what goes to the CUDA cores."""
    Cache([1] * 5, [0, 45, 130, 700, 1000], 16, 2, D, 64, dtype, seed=D).check(tokens=1)
    Cache([3] * 4, [0, 45, 130, 700], 4, 2, D, 20, dtype, seed=D).check(tokens=3, window=90)
