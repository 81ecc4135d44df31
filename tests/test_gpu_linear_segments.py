"""Narrow batches go in time segments that hand on what they do to a state: gates whose product over a segment leaves fp32's
range, while the recurrence itself stays within it.

The bounds are those of fp32 arithmetic (oracle/linear.py): the recurrence of the absolute values is finite in every case.
"""
import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from linear_testlib import check_backward, check_forward, make

pytestmark = pytest.mark.gpu

T = 6000
SHAPES = [(1, 32, "channel"), (1, 1024, "channel"), (8, 32, "head"), (8, 12, "head"), (3, 5, "channel")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.build()


def gates(kind, n):
    """[T, n]: the stretch begins 40 tokens later from one column to the next, so that it lies at every place of a segment."""
    a = torch.ones(T, n)
    for c in range(n):
        s = 300 + 40 * (c % 32)
        if kind == "shrink":  # 2^-200, and back
            a[s:s + 200, c], a[s + 200:s + 400, c] = 0.5, 2.0
        else:  # 1.25^416 = 2^134, and back
            a[s:s + 416, c], a[s + 416:s + 832, c] = 1.25, 0.8
            if kind == "zero":
                a[s + 436, c] = 0.0
    return a


def inputs(kind, H, D, per, dtype, gate_dtype, reverse):
    """Growing gates with small inputs, or a large state that shrinks and comes back; `reverse`: for the carry, from the right."""
    i = make([T], H, D, dtype, gate_dtype, gates=per, seed=40)
    a = gates(kind, H if per == "head" else H * D)
    i["a"].copy_((a.flip(0) if reverse else a).view(i["a"].shape))
    i["b"].fill_(1.0)
    big, small = ("dy", "x") if reverse else ("x", "dy")
    i[big].fill_(0.0 if kind == "shrink" else 1e-7)
    i[small].zero_()
    one, none = ("df", "h0") if reverse else ("h0", "df")
    i[one].fill_(2.0 ** 100 if kind == "shrink" else 2e-5)
    i[none].zero_()
    return i


@pytest.mark.parametrize("kind", ["grow", "zero", "shrink"])
@pytest.mark.parametrize("dtype,gate_dtype", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("H,D,per", SHAPES)
def test_forward(H, D, per, dtype, gate_dtype, kind):
    y, final, tiles = check_forward(inputs(kind, H, D, per, dtype, gate_dtype, False))
    assert torch.isfinite(y).all() and torch.isfinite(final).all() and torch.isfinite(tiles).all()


@pytest.mark.parametrize("kind", ["grow", "zero", "shrink"])
@pytest.mark.parametrize("dtype,gate_dtype", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("H,D,per", SHAPES)
def test_backward(H, D, per, dtype, gate_dtype, kind):
    i = inputs(kind, H, D, per, dtype, gate_dtype, True)
    _, _, tiles = check_forward(i)
    for got in check_backward(i, tiles):
        assert torch.isfinite(got).all()


@pytest.mark.parametrize("first", [0.0, 2.0 ** -20])
def test_a_state_of_zero_or_of_little(first):
    """A product of 2^1900 over all later segments: what is zero stays zero, and what is not grows as token by token."""
    i = make([T], 1, 32, "f32", seed=41)
    i["a"].fill_(1.25)
    i["b"].fill_(1.0)
    i["x"].zero_()
    i["h0"].fill_(first)
    y = gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], initial_state=i["h0"])
    n = 480  # 2^-20 x 1.25^480 = 2^134.5 is past the range
    if first:
        assert torch.isfinite(y[:n - 40]).all() and torch.isinf(y[n:]).all()
    else:
        assert not y.any()


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("H,D,per", [(1, 32, "channel"), (8, 32, "head"), (8, 12, "head"), (2, 17, "channel"), (16, 128, "channel"), (20, 100, "head")])
def test_what_is_not_finite_stays_in_its_sequence(H, D, per, bad):
    """Over many segments, stages and tiles: inputs, gates and states of one sequence that are not finite leave the bits of the
    others as they are, in both directions."""
    i = make([1700, 900, 1, 2100], H, D, "f32", gates=per, seed=42)
    tiles = torch.empty(-(-i["T"] // 64), H, D, device="cuda")

    def run(j):
        y, final = gdn.gated_linear_recurrence(j["x"], j["a"], j["b"], initial_state=j["h0"], cu_seqlens=j["cu"],
                                               output_final_state=True, tile_states=tiles)
        return (y, *gdn.gated_linear_recurrence_backward(j["dy"], j["x"], j["a"], j["b"], tiles, j["h0"], j["df"], j["cu"])[:3]), \
            (final, gdn.gated_linear_recurrence_backward(j["dy"], j["x"], j["a"], j["b"], tiles, j["h0"], j["df"], j["cu"])[3])

    clean = run(i)
    for where in ("x", "a", "h0", "df", "dy"):
        j = dict(i)
        j[where] = i[where].clone()
        for at in ((1, 2) if where in ("h0", "df") else (1700, 2150, 2599, 2600)):  # of the second and third sequence
            j[where][at] = bad
        got = run(j)
        for n in (0, 3):
            s, e = i["cul"][n], i["cul"][n + 1]
            assert all(torch.equal(g[s:e], w[s:e]) for g, w in zip(got[0], clean[0])), (where, n)
            assert all(torch.equal(g[n], w[n]) for g, w in zip(got[1], clean[1])), (where, n)
        assert not torch.isfinite(got[0][2 if where in ("dy", "df") else 0][1700:2600]).all()
