"""Attention over a paged cache: sequences without keys (inactive entries of a padded batch) between others, in layouts that tiled
copies can fetch and in those that they cannot."""
import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from attention_testlib import DEV, Cache

pytestmark = pytest.mark.gpu

LAYOUTS = [(64, 20), (128, 20), (100, 64), (60, 20), (256, 20), (250, 16), (128, 64)]  # head size, tokens a page


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.build()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page_tokens", LAYOUTS)
@pytest.mark.parametrize("tokens", [1, 3])
def test_every_second_sequence_is_empty(dtype, D, page_tokens, tokens):
    """Eight units without tiles follow each unit with some; a block has both kinds."""
    past = [600 - tokens if i % 2 == 0 else -tokens for i in range(64)]
    Cache([tokens] * 64, past, 16, 8, D, page_tokens, dtype, seed=D).check(tokens=tokens)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page_tokens", LAYOUTS)
def test_inactive_entries(dtype, D, page_tokens):
    """Entries of -1, between active ones, and one at the end of the batch."""
    for inactive in ([5, 6, 20, 41], [63]):
        c = Cache([1] * 64, [600] * 64, 16, 8, D, page_tokens, dtype, seed=D)
        c.seqs[inactive] = -1
        c.check(tokens=1, status=DEV["SEQ"])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page_tokens", LAYOUTS)
def test_chunks_beside_empty_sequences(dtype, D, page_tokens):
    """Units of many rows, and chunks whose tokens all stand before the first position."""
    lens, past = [200, 30, 200, 1, 150, 40], [300, -30, 100, -1, 0, -40]
    Cache(lens * 4, past * 4, 16, 8, D, page_tokens, dtype, seed=D).check()
