"""The angles of rotary positions: far positions times frequencies of any size, against the definition in extended precision."""
import numpy as np
import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from attention_testlib import close_rotary, f64
from oracle import attention as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.build()


@pytest.mark.parametrize("scale", [1.0, 7.0, 1000.5, 123456.789, -3.25, 1e-3])
def test_frequencies_above_and_below_a_turn(scale):
    """The angle is off by 2^-33 of a turn, which is 2^-6.3 of a rounding of 2^-24: the bound of the turn's own roundings holds."""
    pos = [0, 1, -1, 5, 1000003, 2 ** 24 + 1, 2 ** 31 - 1, 2 ** 31 - 2, -2 ** 31, 1234567891]
    x = torch.randn(len(pos), 3, 64, generator=torch.Generator().manual_seed(1)).cuda()
    f = gdn.rotary_frequencies(64) * scale
    got, _ = gdn.rotary_embedding(x, None, f, positions=torch.tensor(pos, device="cuda"))
    want, size = ref.rotary(f64(x), pos, f64(f))
    close_rotary("q", got, want, size, torch.float32)


def test_whole_turns_are_nothing():
    """A frequency next to whole turns: what it lacks to them, a rounding of a double, counts at far positions."""
    f = torch.tensor([2 * np.pi, 4 * np.pi, 200 * np.pi, 2 ** 17 * np.pi], dtype=torch.float64)
    pos = [1, 2 ** 20, 2 ** 31 - 1]
    x = torch.randn(len(pos), 1, 8, generator=torch.Generator().manual_seed(2)).cuda()
    got, _ = gdn.rotary_embedding(x, None, f.cuda(), positions=torch.tensor(pos, device="cuda"))
    want, size = ref.rotary(f64(x), pos, f64(f))
    close_rotary("q", got, want, size, torch.float32)
