"""The gated linear recurrence on the GPU against the token-by-token recurrence in 64 bits.

The bounds are those of fp32 arithmetic (oracle/linear.py) plus the rounding of the output's type.
"""
import numpy as np
import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from linear_testlib import check_backward, check_forward, f64, make, within
from oracle import linear as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.build()


# lengths around the tile of 64 packed tokens, empty sequences at every place, many short ones, long ones over many tiles
LENS = {
    "one": [1], "tile-1": [63], "tile": [64], "tile+1": [65], "two_tiles": [128], "ragged": [130, 0, 20, 300],
    "empty_ends": [0, 0, 5, 0, 70, 0], "ones": [1] * 150, "short": [3, 1, 7, 0, 2] * 20, "on_the_edge": [64, 64, 1, 63, 128],
    "long": [3001], "long_two": [1000, 1411], "all_empty": [0, 0, 0], "none": [0],
}
SHAPES = [(2, 128), (3, 100), (1, 1), (5, 7), (2, 64), (1, 300), (3, 8), (2, 4)]
HEADS = [(8, 16), (4, 80), (8, 48), (16, 144), (4, 32)]  # of which a column holds one, or a part


@pytest.mark.parametrize("gates", ["channel", "head"])
@pytest.mark.parametrize("lens", list(LENS))
def test_lengths(lens, gates):
    i = make(LENS[lens], 2, 40, "bf16", "f32", gates=gates, seed=1)
    _, _, tiles = check_forward(i)
    check_backward(i, tiles)


@pytest.mark.parametrize("has_b", [True, False])
@pytest.mark.parametrize("gates", ["channel", "head"])
@pytest.mark.parametrize("H,D", SHAPES)
@pytest.mark.parametrize("dtype,gate_dtype", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "f32"), ("f16", "f32")])
def test_types_and_shapes(dtype, gate_dtype, H, D, gates, has_b):
    i = make([70, 1, 0, 129], H, D, dtype, gate_dtype, gates=gates, has_b=has_b, seed=2)
    _, _, tiles = check_forward(i)
    check_backward(i, tiles)


@pytest.mark.parametrize("H,D", HEADS)
@pytest.mark.parametrize("dtype,gate_dtype", [("bf16", "bf16"), ("f32", "f32"), ("f16", "f32")])
def test_heads_in_columns(dtype, gate_dtype, H, D):
    i = make([300, 5, 0, 420], H, D, dtype, gate_dtype, gates="head", seed=30)
    _, _, tiles = check_forward(i)
    check_backward(i, tiles)


@pytest.mark.parametrize("H,D", [(2, 128), (3, 50), (1, 1)])
@pytest.mark.parametrize("states", [True, False])
def test_strided_tokens(H, D, states):
    """x, a and b as slices of one projection's output; outputs into a wider buffer."""
    i = make([100, 40], H, D, "bf16", fused=True, states=states, seed=3)
    wide = torch.full((140, H + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    _, _, tiles = check_forward(i, output=wide[:, :H])
    assert (wide[:, H] == 7).all()
    check_backward(i, tiles)


def test_misaligned_bases():
    """Tensors that start at any element."""
    i = make([90, 10], 2, 64, "bf16", "f32", seed=4)
    for k in ("x", "a", "b"):
        flat = torch.empty(i[k].numel() + 1, dtype=i[k].dtype, device="cuda")[1:]
        flat.copy_(i[k].reshape(-1))
        i[k] = flat.view(i[k].shape)
    _, _, tiles = check_forward(i)
    check_backward(i, tiles)


def test_misaligned_saved_states():
    """tile_states, and the gradients of states, that start at any float."""
    i = make([90, 30], 2, 64, "bf16", "f32", seed=25)
    want = ref.forward(f64(i["x"]), f64(i["a"]), f64(i["b"]), i["cul"], f64(i["h0"]))
    odd = lambda *shape: torch.empty(torch.Size(shape).numel() + 1, device="cuda")[1:].view(shape)  # noqa: E731
    tiles = odd(2, 2, 64)
    y, final = gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], initial_state=i["h0"], output_final_state=True,
                                           cu_seqlens=i["cu"], tile_states=tiles)
    within("tile_states", tiles, want[0][[63, 119]], want[3][[63, 119]])
    df = odd(2, 2, 64)
    df.copy_(i["df"])
    i["df"] = df
    check_backward(i, tiles)


def test_in_place():
    i = make([77, 500], 2, 128, "bf16", seed=5)
    y = gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], cu_seqlens=i["cu"])
    x = i["x"].clone()
    assert gdn.gated_linear_recurrence(x, i["a"], i["b"], cu_seqlens=i["cu"], output=x) is x
    assert torch.equal(x, y)


@pytest.mark.parametrize("H,D", [(1, 32), (2, 17)])
def test_in_place_over_many_segments(H, D):
    i = make([4000, 1500], H, D, "bf16", seed=27)
    y = gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], initial_state=i["h0"], cu_seqlens=i["cu"])
    for _ in range(5):
        x = i["x"].clone()
        gdn.gated_linear_recurrence(x, i["a"], i["b"], initial_state=i["h0"], cu_seqlens=i["cu"], output=x)
        assert torch.equal(x, y)


@pytest.mark.parametrize("lens", [[512] * 20, [1, 2, 3] * 300, [0] * 50 + [300] + [0] * 70 + [1] * 90 + [0, 2000], [255, 257] * 8])
@pytest.mark.parametrize("H,D,gates", [(1, 64, "channel"), (1, 64, "head"), (3, 6, "head")])
def test_many_sequences(lens, H, D, gates):
    """More bounds in a stage than a warp looks at at a time, and bounds at every place of a stage."""
    i = make(lens, H, D, "f32", gates=gates, seed=28)
    _, _, tiles = check_forward(i)
    check_backward(i, tiles)


def test_offsets_past_32_bits():
    """More than 2^31 elements, and the last tokens as a short sequence with the state before them gives them: gates of 1/2
    forget all but 2^-200 of what was 200 tokens ago, so the last 300 tokens alone have the same states to 2^-100."""
    T, H, D, n = 70000, 256, 128, 300
    x = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda").normal_()
    a = torch.full((T, H), 0.5, device="cuda")
    tiles = torch.empty(-(-T // 64), H, D, device="cuda")
    y = gdn.gated_linear_recurrence(x, a, tile_states=tiles)
    want = ref.forward(f64(x[-n:, :, :2]), f64(a[-n:]), None, [0, n])
    within("y", y[-50:, :, :2], want[0][-50:], want[3][-50:] + 2.0 ** -100, torch.bfloat16)
    dx = gdn.gated_linear_recurrence_backward(x, x, a, tile_states=tiles)[0]
    val, err = ref.backward(f64(x[-n:, :, :2]), f64(x[-n:, :, :2]), f64(a[-n:]), None, [0, n])
    within("dx", dx[-50:, :, :2], val["dx"][-50:], err["dx"][-50:], torch.bfloat16)


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.float8_e5m2])
def test_pool(state, index):
    """States from and to rows of a pool in place, in every storage type, over a row stride; other rows keep their bits."""
    lens, H, D, P = [70, 0, 1, 200], 2, 24, 11
    i = make(lens, H, D, "bf16", "f32", seed=6)
    rows = torch.tensor([7, 2, 10, 0], dtype=index, device="cuda")
    whole = torch.randn(P, H + 1, D, generator=torch.Generator().manual_seed(1)).to(state).cuda()
    pool, before = whole[:, :H], whole.clone()
    h0 = f64(pool[rows.long()].float())
    cu = i["cu"].to(index)
    y, out = gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], initial_state=pool, output_state=pool, state_indices=rows,
                                         output_final_state=True, cu_seqlens=cu)
    assert out is pool
    want = ref.forward(f64(i["x"]), f64(i["a"]), f64(i["b"]), i["cul"], h0)
    within("y", y, want[0], want[3], torch.bfloat16)
    within("pool", pool[rows.long()].float(), want[1], want[4], state)
    assert torch.equal(pool[2].float(), before[2, :H].float())  # an empty sequence keeps its state
    for r in range(P):
        if r not in rows.tolist():
            assert torch.equal(whole[r].float(), before[r].float())
    assert torch.equal(whole[:, H].float(), before[:, H].float())


@pytest.mark.parametrize("lens", [[5000], [1500, 3, 0, 4000, 64], [1] * 40 + [2000, 700]])
def test_pool_in_place_over_long_sequences(lens):
    """In place, where blocks far apart read and write one row: the same bits as into another pool, every time."""
    i = make(lens, 1, 32, "f32", seed=24)
    rows = torch.randperm(len(lens) + 5, generator=torch.Generator().manual_seed(2))[: len(lens)].to(torch.int32).cuda()
    pool = torch.randn(len(lens) + 5, 1, 32, device="cuda")
    call = lambda out: gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], initial_state=start, output_state=out,  # noqa: E731
                                                   state_indices=rows, output_final_state=True, cu_seqlens=i["cu"])[0]
    start = pool
    other = pool.clone()
    y = call(other)
    want = ref.forward(f64(i["x"]), f64(i["a"]), f64(i["b"]), i["cul"], f64(pool[rows.long()]))
    within("y", y, want[0], want[3])
    within("pool", other[rows.long()], want[1], want[4])
    for _ in range(30):
        start = pool.clone()
        assert torch.equal(call(start), y) and torch.equal(start, other)


def test_pool_rows_out_of_range_are_not_followed():
    i = make([10, 80, 3], 2, 16, "f32", seed=7)
    pool = torch.randn(4, 2, 16, device="cuda")
    before = pool.clone()
    for rows in ([1, 4, 2], [1, -1, 2], [1, 2 ** 31 - 1, 2]):
        p, status = pool.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
        gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], initial_state=p, output_state=p, output_final_state=True,
                                    state_indices=torch.tensor(rows, dtype=torch.int32, device="cuda"), cu_seqlens=i["cu"],
                                    device_status=status)
        assert int(status) == gdn.DEVICE_ERR["STATE_INDEX_RANGE"]
        assert torch.equal(p[[0, 3]], before[[0, 3]])


@pytest.mark.parametrize("cu", [[1, 50, 100], [0, 60, 50, 100], [0, 50, 99], [0, 50, 101], [0, 1 << 30, 100], [0, -5, 100]])
def test_malformed_cu_seqlens_are_reported(cu):
    """Reported, and nothing outside the tensors is touched."""
    i = make([100], 2, 16, "f32", states=False, seed=8)
    guard = torch.full((3, 100, 2, 16), 5.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], cu_seqlens=c, output=guard[1], device_status=status,
                                output_final_state=True)
    assert int(status) & gdn.DEVICE_ERR["CU_SEQLENS"]
    assert (guard[0] == 5).all() and (guard[2] == 5).all()
    status.zero_()
    tiles = torch.zeros(2, 2, 16, device="cuda")
    gdn.gated_linear_recurrence_backward(i["x"], i["x"], i["a"], i["b"], tile_states=tiles, cu_seqlens=c, device_status=status)
    assert int(status) & gdn.DEVICE_ERR["CU_SEQLENS"]


@pytest.mark.parametrize("bad", [float("inf"), float("nan"), float("-inf")])
def test_what_is_not_finite_stays_in_its_sequence(bad):
    lens = [50, 100, 30, 3, 200]
    i = make(lens, 2, 32, "f32", seed=9)
    clean = gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], initial_state=i["h0"], cu_seqlens=i["cu"], output_final_state=True)
    tiles = torch.empty(6, 2, 32, device="cuda")
    gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], initial_state=i["h0"], cu_seqlens=i["cu"], tile_states=tiles)
    grads = gdn.gated_linear_recurrence_backward(i["dy"], i["x"], i["a"], i["b"], tiles, i["h0"], i["df"], i["cu"])
    for where in ("x", "h0", "df"):
        j = {k: v.clone() if torch.is_tensor(v) else v for k, v in i.items()}
        if where == "x":
            j["x"][60] = bad  # in the second sequence
            j["x"][181] = bad  # in the fourth
        else:
            j[where][1] = bad
            j[where][3] = bad
        y, final = gdn.gated_linear_recurrence(j["x"], j["a"], j["b"], initial_state=j["h0"], cu_seqlens=j["cu"],
                                               output_final_state=True, tile_states=tiles)
        got = gdn.gated_linear_recurrence_backward(j["dy"], j["x"], j["a"], j["b"], tiles, j["h0"], j["df"], j["cu"])
        for n, (s, e) in enumerate(zip(j["cul"], j["cul"][1:])):
            if n in (1, 3):
                if where != "df":
                    assert not torch.isfinite(y[e - 1]).any() and not torch.isfinite(final[n]).any()
                continue
            assert torch.equal(y[s:e], clean[0][s:e]) and torch.equal(final[n], clean[1][n])
            for g, w in zip(got[:3], grads[:3]):
                assert torch.equal(g[s:e], w[s:e])
            assert torch.equal(got[3][n], grads[3][n])


@pytest.mark.parametrize("value", [0.0, 1.0, -1.0, 4.0, 1e-30])
def test_gates_of_any_value(value):
    """Zero forgets, one sums up, gates of less than four have finite products over 64 tokens (here 60 of four)."""
    n = 60 if value == 4.0 else 300
    i = make([n, 2], 2, 16, "f32", seed=10)
    i["a"].fill_(value)
    _, _, tiles = check_forward(i)
    check_backward(i, tiles)


def test_gates_above_one_without_inputs():
    """Gates whose product over a segment is infinite, and nothing for them to grow: the states stay zero until the inputs
    come, in the last tokens."""
    i = make([6000], 1, 32, "f32", states=False, seed=29)
    i["a"].fill_(1.25)
    i["x"][:5990] = 0
    y = gdn.gated_linear_recurrence(i["x"], i["a"], i["b"])
    assert not y[:5990].any()
    want = ref.forward(f64(i["x"][5990:]), f64(i["a"][5990:]), f64(i["b"][5990:]), [0, 10])
    within("y", y[5990:], want[0], want[3])


def test_growing_states_over_tiles():
    """Gates above one: states grow over many tiles, and stay finite."""
    i = make([700], 1, 40, "f32", seed=11)
    i["a"].fill_(1.1)
    _, _, tiles = check_forward(i)
    check_backward(i, tiles)


def test_without_states_and_cu_seqlens():
    i = make([333], 2, 72, "bf16", "f32", states=False, seed=12)
    y = gdn.gated_linear_recurrence(i["x"], i["a"], i["b"])
    want = ref.forward(f64(i["x"]), f64(i["a"]), f64(i["b"]), i["cul"])
    within("y", y, want[0], want[3], torch.bfloat16)
    _, final, tiles = check_forward(i)
    check_backward(i, tiles, d_final=False)


def test_repeated_runs_give_the_same_bits():
    i = make([9000, 4000], 4, 128, "bf16", "f32", seed=13)
    tiles = torch.empty(-(-13000 // 64), 4, 128, device="cuda")
    first = None
    for _ in range(20):
        y, f = gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], initial_state=i["h0"], cu_seqlens=i["cu"], tile_states=tiles,
                                           output_final_state=True)
        out = [y, f, tiles.clone(), *gdn.gated_linear_recurrence_backward(i["dy"], i["x"], i["a"], i["b"], tiles, i["h0"],
                                                                           i["df"], i["cu"])]
        first = first or out
        assert all(torch.equal(p, q) for p, q in zip(out, first))


@pytest.mark.parametrize("gates", ["channel", "head"])
def test_gradients_against_differences(gates):
    """Central differences of the loss in 64 bits at entries of every input (the loss is of degree one in each entry)."""
    i = make([90, 7], 2, 12, "f32", gates=gates, seed=14)
    leaf = {k: i[k].clone().requires_grad_() for k in ("x", "a", "b", "h0")}
    y, final = gdn.gated_linear_recurrence(leaf["x"], leaf["a"], leaf["b"], initial_state=leaf["h0"], output_final_state=True,
                                           cu_seqlens=i["cu"])
    ((y * i["dy"]).sum() + (final * i["df"]).sum()).backward()
    dy, df = f64(i["dy"]), f64(i["df"])
    _, err = ref.backward(dy, *(f64(i[k]) for k in ("x", "a", "b")), i["cul"], f64(i["h0"]), df)

    def loss(v):
        o = ref.forward(v["x"], v["a"], v["b"], i["cul"], v["h0"])
        return (o[0] * dy).sum() + (o[1] * df).sum()

    rng = np.random.default_rng(0)
    base = {k: f64(i[k]) for k in ("x", "a", "b", "h0")}
    for name, e in (("x", "dx"), ("a", "da"), ("b", "db"), ("h0", "d0")):
        grad = f64(leaf[name].grad)
        for flat in rng.integers(0, grad.size, 25):
            at = np.unravel_index(flat, grad.shape)
            hi, lo = base[name].copy(), base[name].copy()
            hi[at] += 1e-4
            lo[at] -= 1e-4
            diff = (loss({**base, name: hi}) - loss({**base, name: lo})) / 2e-4
            assert abs(diff - grad[at]) <= err[e][at] + 2.0 ** -24 * abs(diff) + 1e-7, (name, at)


def test_autograd_skips_what_needs_no_gradient():
    i = make([65, 10], 2, 16, "bf16", seed=15)
    a = i["a"].clone().requires_grad_()
    y = gdn.gated_linear_recurrence(i["x"], a, None, cu_seqlens=i["cu"])
    y.float().sum().backward()
    ones = torch.ones_like(i["x"])
    tiles = torch.empty(2, 2, 16, device="cuda")
    gdn.gated_linear_recurrence(i["x"], i["a"], cu_seqlens=i["cu"], tile_states=tiles)
    da = gdn.gated_linear_recurrence_backward(ones, i["x"], i["a"], None, tiles, cu_seqlens=i["cu"])[1]
    assert torch.equal(a.grad, da)
    with pytest.raises(ValueError, match="differentiated"):
        gdn.gated_linear_recurrence(i["x"], a, None, cu_seqlens=i["cu"], output=torch.empty_like(i["x"]))


def test_other_streams_and_graphs():
    """On a stream of the caller's, and captured once and replayed on new inputs."""
    i, j = make([500, 20], 2, 128, "bf16", seed=16), make([500, 20], 2, 128, "bf16", seed=17)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    want = [gdn.gated_linear_recurrence(k["x"], k["a"], k["b"], initial_state=k["h0"], cu_seqlens=k["cu"], output_final_state=True)
            for k in (i, j)]
    with torch.cuda.stream(s):
        got = gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], initial_state=i["h0"], cu_seqlens=i["cu"], output_final_state=True)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want[0]))
    buf = {k: i[k].clone() for k in ("x", "a", "b", "h0", "cu")}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gdn.gated_linear_recurrence(buf["x"], buf["a"], buf["b"], initial_state=buf["h0"], cu_seqlens=buf["cu"],
                                          output_final_state=True)
    for k, w in ((i, want[0]), (j, want[1]), (i, want[0])):
        for n, t in buf.items():
            t.copy_(k[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, w))


@pytest.mark.parametrize("m", [1, 2, 5])
@pytest.mark.parametrize("H,D", [(2, 128), (3, 50), (1, 1)])
@pytest.mark.parametrize("dtype,gate_dtype", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("gates", ["channel", "head"])
def test_decode(m, H, D, dtype, gate_dtype, gates):
    N, P = 19, 40
    i = make([m] * N, H, D, dtype, gate_dtype, gates=gates, seed=18)
    pool = torch.randn(P, H, D, device="cuda")
    before = pool.clone()
    rows = torch.randperm(P, device="cuda")[:N].to(torch.int32)
    y, out = gdn.gated_linear_recurrence_decode(i["x"], i["a"], i["b"], initial_state=pool, state_indices=rows, tokens_per_seq=m)
    assert out is pool
    want = ref.forward(f64(i["x"]), f64(i["a"]), f64(i["b"]), i["cul"], f64(before[rows.long()]))
    within("y", y, want[0], want[3], i["x"].dtype)
    within("pool", pool[rows.long()], want[1], want[4])
    rest = torch.ones(P, dtype=torch.bool, device="cuda")
    rest[rows.long()] = False
    assert torch.equal(pool[rest], before[rest])


@pytest.mark.parametrize("m", [1, 3, 9])
@pytest.mark.parametrize("gate_dtype,gates", [("bf16", "channel"), ("f32", "channel"), ("f32", "head")])
def test_decode_many_sequences(gate_dtype, gates, m):
    """Enough of them for loads of 16 bytes, and more tokens than are loaded at a time."""
    i = make([m] * 400, 16, 104, "bf16", gate_dtype, gates=gates, seed=26)
    y, out = gdn.gated_linear_recurrence_decode(i["x"], i["a"], i["b"], initial_state=i["h0"], tokens_per_seq=m)
    want = ref.forward(f64(i["x"]), f64(i["a"]), f64(i["b"]), i["cul"], f64(i["h0"]))
    within("y", y, want[0], want[3], torch.bfloat16)
    within("state", out, want[1], want[4])


@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.float8_e5m2])
@pytest.mark.parametrize("D", [64, 9])
def test_decode_state_types(state, D):
    i = make([1] * 6, 2, D, "bf16", has_b=False, seed=19)
    h0 = i["h0"].to(state)
    y, out = gdn.gated_linear_recurrence_decode(i["x"], i["a"], initial_state=h0)
    want = ref.forward(f64(i["x"]), f64(i["a"]), None, i["cul"], f64(h0.float()))
    within("y", y, want[0], want[3], torch.bfloat16)
    within("state", out.float(), want[1], want[4], state)
    y2 = gdn.gated_linear_recurrence_decode(i["x"], i["a"], initial_state=h0, output_final_state=False)
    assert torch.equal(y, y2)


def test_decode_follows_the_prefill():
    """A prefill, then tokens one by one, against the whole sequences at once."""
    lens, more, H, D = [130, 0, 20], 3, 2, 64
    whole = make([n + more for n in lens], H, D, "f32", seed=20)
    cul = whole["cul"]
    first = torch.cat([torch.arange(s, e - more) for s, e in zip(cul, cul[1:])]).cuda()
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    rows = torch.tensor([3, 0, 4], dtype=torch.int32, device="cuda")
    pool = torch.zeros(5, H, D, device="cuda")
    pool[rows.long()] = whole["h0"]
    part = lambda k, at: whole[k][at].contiguous()  # noqa: E731
    gdn.gated_linear_recurrence(part("x", first), part("a", first), part("b", first), initial_state=pool, output_state=pool,
                                state_indices=rows, output_final_state=True, cu_seqlens=cu)
    want = ref.forward(f64(whole["x"]), f64(whole["a"]), f64(whole["b"]), cul, f64(whole["h0"]))
    for t in range(more):
        at = torch.tensor([e - more + t for e in cul[1:]], device="cuda")
        y, _ = gdn.gated_linear_recurrence_decode(part("x", at), part("a", at), part("b", at), initial_state=pool, state_indices=rows)
        within("y", y, want[0][at.cpu().numpy()], want[3][at.cpu().numpy()])
    within("pool", pool[rows.long()], want[1], want[4])


def test_decode_skips_rows_out_of_range():
    i = make([1] * 3, 1, 16, "f32", seed=21)
    pool = torch.randn(4, 1, 16, device="cuda")
    before, status = pool.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = torch.tensor([1, 4, -1], dtype=torch.int32, device="cuda")
    gdn.gated_linear_recurrence_decode(i["x"], i["a"], i["b"], initial_state=pool, state_indices=rows, device_status=status)
    assert int(status) == gdn.DEVICE_ERR["STATE_INDEX_RANGE"]
    assert torch.equal(pool[[0, 2, 3]], before[[0, 2, 3]]) and not torch.equal(pool[1], before[1])


def test_python_refusals():
    i = make([10], 2, 8, "bf16", seed=22)
    x, a, b, cu = i["x"], i["a"], i["b"], i["cu"]
    f = gdn.gated_linear_recurrence
    bad = [lambda: f(x.view(10, 16), a), lambda: f(x.int(), a), lambda: f(x, a.half()), lambda: f(x, a[:9]),
           lambda: f(x, a, b.float()), lambda: f(x, a, b[:, 0]), lambda: f(x, a, cu_seqlens=cu.cpu()),
           lambda: f(x, a, cu_seqlens=cu.float()), lambda: f(x, a, cu_seqlens=cu[::2]) if cu.numel() > 2 else f(x, a, cu_seqlens=cu.view(1, -1)),
           lambda: f(x.transpose(1, 2), a), lambda: f(x[:1].expand(10, 2, 8), a), lambda: f(x, a, initial_state=torch.zeros(2, 2, 8, device="cuda")),
           lambda: f(x, a, initial_state=torch.zeros(1, 2, 8)), lambda: f(x, a, initial_state=torch.zeros(1, 2, 8, device="cuda").int()),
           lambda: f(x, a, initial_state=i["h0"], output_state=i["h0"].half(), output_final_state=True),
           lambda: f(x, a, state_indices=torch.zeros(1, dtype=torch.int32, device="cuda")),
           lambda: f(x, a, initial_state=i["h0"], state_indices=torch.zeros(2, dtype=torch.int32, device="cuda")),
           lambda: f(x, a, initial_state=i["h0"], state_indices=torch.zeros(1, device="cuda")),
           lambda: f(x, a, initial_state=i["h0"], output_final_state=True, state_indices=torch.zeros(1, dtype=torch.int32, device="cuda")),
           lambda: f(x, a, output=torch.empty(10, 2, 8, device="cuda")), lambda: f(x, a, tile_states=torch.empty(2, 2, 8, device="cuda")),
           lambda: f(x, a, device_status=torch.zeros(1, device="cuda")),
           lambda: gdn.gated_linear_recurrence_decode(x, a, tokens_per_seq=3),
           lambda: gdn.gated_linear_recurrence_decode(x, a, tokens_per_seq=0),
           lambda: gdn.gated_linear_recurrence_backward(x.float(), x, a),
           lambda: gdn.gated_linear_recurrence_backward(x, x, a, d_final_state=torch.zeros(2, 2, 8, device="cuda"))]
    for n, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {n} was not refused")
    j = make([70], 1, 8, "bf16", seed=23)
    with pytest.raises(ValueError, match="tile_states"):
        gdn.gated_linear_recurrence_backward(j["dy"], j["x"], j["a"])
