"""The gated linear recurrence as a part of autograd's graph."""
import numpy as np
import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from linear_testlib import f64, make, within
from oracle import linear as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.build()


def test_the_status_may_be_cleared_before_the_backward_pass():
    """A caller reads the status word after the forward pass and clears it; the backward pass writes its own bits to it."""
    i = make([100, 30], 2, 16, "f32", seed=31)
    a = i["a"].clone().requires_grad_()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = gdn.gated_linear_recurrence(i["x"], a, i["b"], cu_seqlens=i["cu"], device_status=status)
    assert int(status) == 0
    status.zero_()
    y.sum().backward()
    want = ref.backward(np.ones(y.shape), f64(i["x"]), f64(i["a"]), f64(i["b"]), i["cul"])
    within("da", a.grad, want[0]["da"], want[1]["da"])
    cu = i["cu"].clone()
    cu[1] = 131  # past the next entry
    y = gdn.gated_linear_recurrence(i["x"], a, i["b"], cu_seqlens=cu, device_status=status)
    assert int(status) & gdn.DEVICE_ERR["CU_SEQLENS"]
    status.zero_()
    y.sum().backward()
    assert int(status) & gdn.DEVICE_ERR["CU_SEQLENS"]
