"""The gated linear recurrence without a GPU: the oracle's gradients against differences, and what the entry points refuse."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from oracle import linear as ref


@pytest.fixture(scope="module", autouse=True)
def _built():
    gdn.build()


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("has_b", [False, True])
def test_oracle_gradients_against_differences(per_head, has_b):
    rng = np.random.default_rng(3)
    cu, H, D = [0, 5, 5, 6, 13], 2, 3
    T, N = cu[-1], len(cu) - 1
    gs = (T, H) if per_head else (T, H, D)
    v = {"x": rng.normal(size=(T, H, D)), "a": rng.uniform(0.5, 1.0, gs), "b": rng.uniform(0, 1, gs) if has_b else None,
         "h0": rng.normal(size=(N, H, D))}
    dy, df = rng.normal(size=(T, H, D)), rng.normal(size=(N, H, D))

    def loss(w):
        y, final = ref.forward(w["x"], w["a"], w["b"], cu, w["h0"])[:2]
        return (y * dy).sum() + (final * df).sum()

    val, _ = ref.backward(dy, v["x"], v["a"], v["b"], cu, v["h0"], df)
    for name, grad in (("x", val["dx"]), ("a", val["da"]), ("b", val["db"]), ("h0", val["d0"])):
        if grad is None:
            continue
        for at in np.ndindex(grad.shape):
            hi, lo = v[name].copy(), v[name].copy()
            hi[at] += 1e-4
            lo[at] -= 1e-4
            # the loss is at most cubic in one entry, a polynomial of degree 1: the difference is exact but for rounding
            assert abs((loss({**v, name: hi}) - loss({**v, name: lo})) / 2e-4 - grad[at]) < 1e-8


def desc(**kw):
    d = dict(num_heads=2, head_dim=8, x_dtype=1, gate_dtype=1, state_dtype=0, max_total_tokens=256, max_num_seqs=4, flags=0)
    d.update(kw)
    return gdn.LinearDesc(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(num_heads=0), 1), (dict(head_dim=0), 1), (dict(head_dim=-1), 1), (dict(max_total_tokens=-1), 1),
    (dict(max_num_seqs=-1), 1), (dict(flags=1 << 7), 1), (dict(x_dtype=3), 2), (dict(gate_dtype=2), 2),
    (dict(x_dtype=0, gate_dtype=1), 2), (dict(state_dtype=5), 2), (dict(num_heads=1 << 20, head_dim=2), 2),
    (dict(max_total_tokens=1 << 31), 2), (dict(num_heads=0x7fffffff, head_dim=0x7fffffff), 2), (dict(), 0),
    (dict(gate_dtype=0, state_dtype=4), 0)])
def test_plan_validation(kw, status):
    st, plan, nbytes = gdn.gdn_linear_plan(desc(**kw))
    assert st == status
    if st == 0:
        assert nbytes > 0
        gdn.gdn_linear_plan_destroy(plan)
    else:
        assert not plan.value


def test_null_arguments_are_refused():
    L = gdn.lib()
    assert L.gdn_linear_plan(None, None, None) == 1
    for fn in (L.gdn_linear_forward_run, L.gdn_linear_backward_run):
        assert fn(None, None, None, 0, None) == 1
    assert L.gdn_linear_decode_run(None, None, 1, None) == 1
    L.gdn_linear_plan_destroy(None)


GOOD = dict(x=4096, a=8192, cu_seqlens=64, num_seqs=2, total_tokens=100, y=16384, tile_states=1 << 20, dy=1 << 16, dx=1 << 17,
            da=1 << 18)


@pytest.mark.parametrize("op", ["forward", "backward"])
@pytest.mark.parametrize("kw", [
    dict(x=None), dict(a=None), dict(x=4097), dict(x_stride=15), dict(x_stride=-16), dict(a_stride=3), dict(num_seqs=-1),
    dict(num_seqs=5), dict(total_tokens=-1), dict(total_tokens=257), dict(num_seqs=0), dict(cu_seqlens=None),
    dict(cu_seqlens=66), dict(device_status=2), dict(tile_states=2)])
def test_runs_refuse_before_launching(op, kw):
    """Every host-checkable condition is refused; nothing is launched (there is no GPU here to launch on)."""
    st, plan, nbytes = gdn.gdn_linear_plan(desc())
    assert st == 0
    fn = getattr(gdn, f"gdn_linear_{op}_run")
    assert fn(plan, gdn.LinearArgs(**{**GOOD, **kw}), 1 << 22, nbytes, None) == 1
    gdn.gdn_linear_plan_destroy(plan)


@pytest.mark.parametrize("op,kw", [("forward", dict(y=None)), ("forward", dict(y_stride=8)), ("backward", dict(dy=None)),
                                   ("backward", dict(dx=None)), ("backward", dict(da=None)), ("backward", dict(tile_states=None)),
                                   ("backward", dict(da_stride=15))])
def test_runs_refuse_missing_outputs(op, kw):
    st, plan, nbytes = gdn.gdn_linear_plan(desc())
    assert getattr(gdn, f"gdn_linear_{op}_run")(plan, gdn.LinearArgs(**{**GOOD, **kw}), 1 << 22, nbytes, None) == 1
    gdn.gdn_linear_plan_destroy(plan)


def test_workspace_is_checked():
    """Runs that hand something on from block to block need a workspace: 16 channels of 200 tokens at an odd address."""
    st, plan, nbytes = gdn.gdn_linear_plan(desc())
    args = gdn.LinearArgs(**{**GOOD, "x": 4098, "total_tokens": 200})
    for back, run in ((False, gdn.gdn_linear_forward_run), (True, gdn.gdn_linear_backward_run)):
        n = gdn.gdn_linear_run_workspace(plan, args, back)
        assert 0 < n <= nbytes
        for ws, size in ((None, n), (1 << 22, n - 1), ((1 << 22) + 8, n)):
            assert run(plan, args, ws, size, None) == 1
    assert gdn.gdn_linear_run_workspace(plan, gdn.LinearArgs(**{**GOOD, "x": None}), False) == 0  # refused
    gdn.gdn_linear_plan_destroy(plan)


@pytest.mark.parametrize("T,H,D", [(1, 1, 1), (64, 1, 1), (65, 3, 7), (5000, 2, 128), (70000, 1, 16), (4096, 1, 4100), (999, 40, 96),
                                   (4096, 64, 16), (1000, 4, 80), (512, 8, 48)])
@pytest.mark.parametrize("per_head", [False, True])
def test_a_runs_workspace_is_within_the_plans(T, H, D, per_head):
    flags = gdn.LINEAR_FLAGS["GATES_PER_HEAD"] if per_head else 0
    for kw in (dict(x_dtype=1, gate_dtype=1), dict(x_dtype=0, gate_dtype=0)):
        st, plan, nbytes = gdn.gdn_linear_plan(desc(num_heads=H, head_dim=D, max_total_tokens=T, flags=flags, **kw))
        for x in (4096, 4104, 4100):
            args = gdn.LinearArgs(**{**GOOD, "x": x, "total_tokens": T})
            for back in (False, True):
                assert gdn.gdn_linear_run_workspace(plan, args, back) <= nbytes
        gdn.gdn_linear_plan_destroy(plan)


@pytest.mark.parametrize("T", [0, 1, 2**30 - 1, 2**30, 2**31 - 65])
def test_python_plans_for_all_lengths(T):
    x = torch.empty(0, dtype=torch.bfloat16)
    plan = gdn.linear._get_plan(1, 16, x, x, 0, 0, T, 1)
    assert plan.handle and plan is gdn.linear._get_plan(1, 16, x, x, 0, 0, T, 1)


def test_states_and_pools_are_checked():
    F = gdn.LINEAR_FLAGS
    st, plan, nbytes = gdn.gdn_linear_plan(desc(flags=F["HAS_INITIAL_STATE"] | F["OUTPUT_FINAL_STATE"] | F["HAS_STATE_INDICES"]))
    pool = dict(initial_state=1 << 19, output_state=1 << 19, state_indices=128, n_pool=9)
    for kw in (dict(initial_state=None), dict(output_state=None), dict(state_indices=None), dict(n_pool=0),
               dict(state_stride=15), dict(initial_state=(1 << 19) + 2)):
        args = gdn.LinearArgs(**{**GOOD, **pool, **kw})
        assert gdn.gdn_linear_forward_run(plan, args, 1 << 22, nbytes, None) == 1
        assert gdn.gdn_linear_decode_run(plan, args, 50, None) == 1
    assert gdn.gdn_linear_backward_run(plan, gdn.LinearArgs(**{**GOOD, **pool}), 1 << 22, nbytes, None) == 2  # no pools
    assert gdn.gdn_linear_decode_run(plan, gdn.LinearArgs(**{**GOOD, **pool}), 49, None) == 1  # 2 x 49 tokens are not 100
    assert gdn.gdn_linear_decode_run(plan, gdn.LinearArgs(**{**GOOD, **pool}), 0, None) == 1
    gdn.gdn_linear_plan_destroy(plan)


def test_an_empty_batch_launches_nothing():
    st, plan, nbytes = gdn.gdn_linear_plan(desc())
    assert gdn.gdn_linear_forward_run(plan, gdn.LinearArgs(), 1 << 22, nbytes, None) == 0
    assert gdn.gdn_linear_backward_run(plan, gdn.LinearArgs(), 1 << 22, nbytes, None) == 0
    assert gdn.gdn_linear_decode_run(plan, gdn.LinearArgs(), 1, None) == 0
    gdn.gdn_linear_plan_destroy(plan)


@pytest.mark.parametrize("header", ["gdn_linear.h", "gdn_pages.h"])
def test_exports_every_declared_symbol(header):
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", header)) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = re.findall(r"\b(gdn_\w+)\s*\(", text)
    assert len(names) >= 6
    for n in names:
        assert hasattr(gdn.lib(), n), n


def test_structs_match_the_header():
    # natural alignment of include/gdn_linear.h's structs
    assert ctypes.sizeof(gdn.LinearDesc) == 40
    assert ctypes.sizeof(gdn.LinearArgs) == 224


def test_python_refuses_cpu_tensors():
    x = torch.zeros(4, 2, 8)
    with pytest.raises(ValueError, match="no CPU path"):
        gdn.gated_linear_recurrence(x, x)
    with pytest.raises(ValueError, match="no CPU path"):
        gdn.gated_linear_recurrence_decode(x, x)
    with pytest.raises(ValueError, match="no CPU path"):
        gdn.gated_linear_recurrence_backward(x, x, x)
