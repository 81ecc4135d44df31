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


WRITES = {
    "output": lambda i, t: gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], cu_seqlens=i["cu"], output=i["x"]),
    "output_state": lambda i, t: gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], initial_state=i["h0"], output_state=i["h0"],
                                                             output_final_state=True, cu_seqlens=i["cu"]),
    "tile_states": lambda i, t: gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], cu_seqlens=i["cu"], tile_states=t),
    "decode_output": lambda i, t: gdn.gated_linear_recurrence_decode(i["x"], i["a"], i["b"], output=i["x"]),
    "decode_state": lambda i, t: gdn.gated_linear_recurrence_decode(
        i["x"][:2], i["a"][:2], i["b"][:2], initial_state=i["h0"], state_indices=torch.tensor([1, 0], dtype=torch.int32, device="cuda")),
    "decode_output_state": lambda i, t: gdn.gated_linear_recurrence_decode(i["x"][:2], i["a"][:2], i["b"][:2], output_state=i["h0"]),
}


@pytest.mark.parametrize("how", list(WRITES))
def test_overwriting_a_saved_tensor_is_noticed(how):
    """What a call writes into a caller's tensor counts as a change in place: a backward pass that saved the tensor refuses to
    compute gradients from the new values.  Reading it changes nothing."""
    i = make([64, 6], 2, 16, "f32", seed=32)
    t = torch.ones(2, 2, 16, device="cuda", requires_grad=True)
    saved = {"output": "x", "decode_output": "x", "tile_states": None}.get(how, "h0")
    kept = i["x"] if saved == "x" else i["h0"] if saved == "h0" else t.detach()
    w = torch.ones_like(kept, requires_grad=True)
    loss = (w * kept).sum()  # saves `kept` for w's gradient
    gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], initial_state=i["h0"], cu_seqlens=i["cu"])  # reads
    loss.backward(retain_graph=True)
    with torch.no_grad():
        WRITES[how](i, kept)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()


def test_a_recurrence_notices_that_its_initial_state_was_overwritten():
    i = make([64, 6], 2, 16, "f32", seed=33)
    a = i["a"].clone().requires_grad_()
    y = gdn.gated_linear_recurrence(i["x"], a, i["b"], initial_state=i["h0"], cu_seqlens=i["cu"])
    with torch.no_grad():
        gdn.gated_linear_recurrence_decode(i["x"][:2], i["a"][:2], i["b"][:2], initial_state=i["h0"],
                                           state_indices=torch.tensor([1, 0], dtype=torch.int32, device="cuda"))
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()


def test_inference_mode():
    """Tensors without a version: the calls work on them as on others."""
    i = make([64, 6], 2, 16, "f32", seed=34)
    want = gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], initial_state=i["h0"], cu_seqlens=i["cu"], output_final_state=True)
    with torch.inference_mode():
        pool, out, tiles = i["h0"].clone(), torch.empty_like(i["x"]), torch.empty(2, 2, 16, device="cuda")
        gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], initial_state=pool, output_state=pool, output_final_state=True,
                                    cu_seqlens=i["cu"], output=out, tile_states=tiles)
        assert torch.equal(out, want[0]) and torch.equal(pool, want[1])
        y, _ = gdn.gated_linear_recurrence_decode(i["x"][:2], i["a"][:2], i["b"][:2], initial_state=pool, output_state=pool)
        torch.testing.assert_close(y, i["a"][:2] * want[1] + i["b"][:2] * i["x"][:2], rtol=0, atol=2 ** -18)  # terms below 16, four roundings


@pytest.mark.parametrize("uses", ["y", "final", "both"])
def test_what_the_loss_does_not_use_has_no_gradient(uses, monkeypatch):
    """An unused final state is not made up as zeros for the backward pass to read; gradients through either output alone."""
    i = make([70, 0, 9], 2, 16, "f32", seed=35)
    seen = []
    backward = gdn.linear.gated_linear_recurrence_backward
    monkeypatch.setattr(gdn.linear, "gated_linear_recurrence_backward",
                        lambda *args, **kw: seen.append(kw["d_final_state"] is None) or backward(*args, **kw))
    leaf = {k: i[k].clone().requires_grad_() for k in ("x", "a", "b", "h0")}
    y, final = gdn.gated_linear_recurrence(leaf["x"], leaf["a"], leaf["b"], initial_state=leaf["h0"], output_final_state=True,
                                           cu_seqlens=i["cu"])
    loss = ((y * i["dy"]).sum() if uses != "final" else 0) + ((final * i["df"]).sum() if uses != "y" else 0)
    loss.backward()
    assert seen == [uses == "y"]
    dy = np.zeros(y.shape) if uses == "final" else f64(i["dy"])
    val, err = ref.backward(dy, *(f64(i[k]) for k in ("x", "a", "b")), i["cul"], f64(i["h0"]), None if uses == "y" else f64(i["df"]))
    for name, e in (("x", "dx"), ("a", "da"), ("b", "db"), ("h0", "d0")):
        within(name, leaf[name].grad, val[e], err[e])
