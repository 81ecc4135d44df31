"""The gated linear recurrence over as many channels as go in columns of 16: about 1600 to 2900 of them, all types of gates,
bounds in most stages.  Channels do not see one another, so some of them (heads, where gradients are sums over heads) are
compared with the recurrence in 64 bits."""
import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from linear_testlib import TYPES, f64, within
from oracle import linear as ref

pytestmark = pytest.mark.gpu

# over several stages of 512 tokens: long and short sequences, bounds at a stage's edge, more in a stage than a warp looks at at a time
LENS = [700, 1, 0, 1500] + [37] * 20 + [131, 512, 0, 0, 511, 1] + [0] * 40 + [3] * 100 + [64] * 8 + [1000, 0, 193]
PAIRS = [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "f32"), ("f16", "f32")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.build()


def make(lens, H, D, dtype, gate_dtype, gates, has_b, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    T, N = sum(lens), len(lens)
    gshape = (T, H, D) if gates == "channel" else (T, H)
    dt, gdt = TYPES[dtype], TYPES[gate_dtype]
    cul = [0] + torch.tensor(lens).cumsum(0).tolist()
    return dict(x=rand(T, H, D).to(dt), dy=rand(T, H, D).to(dt), h0=rand(N, H, D), df=rand(N, H, D), cul=cul,
                a=torch.exp(-torch.nn.functional.softplus(rand(*gshape)) / 16).to(gdt),
                b=torch.sigmoid(rand(*gshape)).to(gdt) if has_b else None, cu=torch.tensor(cul, dtype=torch.int32, device="cuda"))


def chosen(i, gates):
    """What is compared: a few channels (the first, the last, those at the columns' edges), or a few heads."""
    _, H, D = i["x"].shape
    if gates == "head":
        heads = sorted({0, H // 2, H - 1})
        return lambda t: None if t is None else f64(t[:, heads])
    at = sorted({0, 1, 15, 16, 31, 32, 47, H * D // 2, H * D - 17, H * D - 16, H * D - 5, H * D - 1})
    return lambda t: None if t is None else f64(t.reshape(t.shape[0], 1, -1)[:, :, at])


def check(i, gates, backward=True):
    part, T = chosen(i, gates), i["x"].shape[0]
    _, H, D = i["x"].shape
    tiles = torch.full((-(-T // 64), H, D), float("nan"), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, final = gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], initial_state=i["h0"], output_final_state=True, cu_seqlens=i["cu"],
                                           tile_states=tiles, device_status=status)
    x, a, b, h0 = (part(i[k]) for k in ("x", "a", "b", "h0"))
    want = ref.forward(x, a, b, i["cul"], h0)
    at = [min(64 * f + 63, T - 1) for f in range(tiles.shape[0])]
    within("y", torch.from_numpy(part(y)), want[0], want[3], y.dtype)
    within("final", torch.from_numpy(part(final)), want[1], want[4])
    within("tile_states", torch.from_numpy(part(tiles)), want[0][at], want[3][at])
    assert torch.isfinite(tiles).all() and torch.isfinite(y).all()
    if backward:
        dx, da, db, d0 = gdn.gated_linear_recurrence_backward(i["dy"], i["x"], i["a"], i["b"], tile_states=tiles, initial_state=i["h0"],
                                                              d_final_state=i["df"], cu_seqlens=i["cu"], device_status=status)
        val, err = ref.backward(part(i["dy"]), x, a, b, i["cul"], h0, part(i["df"]))
        for name, got in (("dx", dx), ("da", da), ("db", db), ("d0", d0)):
            if got is None:
                assert val[name] is None
                continue
            within(name, torch.from_numpy(part(got)), val[name], err[name], got.dtype)
    assert int(status) == 0
    return y, final


@pytest.mark.parametrize("has_b", [True, False])
@pytest.mark.parametrize("dtype,gate_dtype", PAIRS)
def test_gates_per_channel(dtype, gate_dtype, has_b):
    check(make(LENS, 16, 128, dtype, gate_dtype, "channel", has_b, 50), "channel")


@pytest.mark.parametrize("dtype,gate_dtype", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("C", [1600, 1608, 1624, 2800, 2904])
def test_numbers_of_channels(C, dtype, gate_dtype):
    """At the ends of the range, and where the last column is not full."""
    check(make(LENS, 1, C, dtype, gate_dtype, "channel", True, 51), "channel")


@pytest.mark.parametrize("has_b", [True, False])
@pytest.mark.parametrize("dtype,gate_dtype", PAIRS)
@pytest.mark.parametrize("H,D", [(16, 128), (20, 100), (100, 16), (203, 8)])
def test_gates_per_head(H, D, dtype, gate_dtype, has_b):
    """Heads that a column holds a part of, and heads that cross columns."""
    check(make(LENS, H, D, dtype, gate_dtype, "head", has_b, 52), "head")


@pytest.mark.parametrize("H,gate_dtype", [(12, "bf16"), (18, "bf16"), (6, "f32")])
def test_rows_of_gates_that_cannot_be_copied(H, gate_dtype):
    """Gates per head whose rows are no multiple of 16 bytes."""
    check(make(LENS, H, 128, "bf16", gate_dtype, "head", True, 53), "head")


@pytest.mark.parametrize("H,D,gates", [(16, 128, "channel"), (20, 100, "head"), (203, 8, "channel")])
def test_pool_in_place(H, D, gates):
    i = make(LENS, H, D, "bf16", "f32", gates, True, 54)
    N, P = len(LENS), len(LENS) + 9
    y, final = check(i, gates, backward=False)
    rows = torch.randperm(P, generator=torch.Generator().manual_seed(5))[:N].to(torch.int32).cuda()
    pool = torch.randn(P, H, D, device="cuda")
    pool[rows.long()] = i["h0"]
    rest = pool.clone()
    y2, out = gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], initial_state=pool, output_state=pool, state_indices=rows,
                                          output_final_state=True, cu_seqlens=i["cu"])
    assert out is pool and torch.equal(y2, y) and torch.equal(pool[rows.long()], final)
    rest[rows.long()] = final
    assert torch.equal(pool, rest)


@pytest.mark.parametrize("gates", ["channel", "head"])
def test_output_over_the_input(gates):
    i = make(LENS, 16, 128, "bf16", "bf16", gates, True, 55)
    y = gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], initial_state=i["h0"], cu_seqlens=i["cu"])
    x = i["x"].clone()
    gdn.gated_linear_recurrence(x, i["a"], i["b"], initial_state=i["h0"], cu_seqlens=i["cu"], output=x)
    assert torch.equal(x, y)


def test_repeated_runs_give_the_same_bits():
    i = make(LENS, 16, 128, "bf16", "f32", "channel", True, 56)
    tiles = torch.empty(-(-sum(LENS) // 64), 16, 128, device="cuda")
    first = None
    for _ in range(10):
        y = gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], initial_state=i["h0"], cu_seqlens=i["cu"], tile_states=tiles)
        out = [y, tiles.clone(), *gdn.gated_linear_recurrence_backward(i["dy"], i["x"], i["a"], i["b"], tiles, i["h0"], i["df"], i["cu"])]
        first = first or out
        assert all(torch.equal(p, q) for p, q in zip(out, first))
