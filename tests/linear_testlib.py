"""Inputs and comparisons of the gated linear recurrence's tests."""
import numpy as np
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from gdn_testlib import rounding_bound
from oracle import linear as ref

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(lens, H, D, dtype="bf16", gate_dtype=None, gates="channel", has_b=True, states=True, seed=0, fused=False):
    """Inputs on the GPU, drawn on the CPU."""
    g = torch.Generator().manual_seed(seed)
    dt, gdt = TYPES[dtype], TYPES[gate_dtype or dtype]
    T, N = sum(lens), len(lens)
    gshape = (T, H, D) if gates == "channel" else (T, H)
    x = torch.randn(T, H, D, generator=g).to(dt)
    a = torch.exp(-torch.nn.functional.softplus(torch.randn(gshape, generator=g)) / 16).to(gdt)
    b = torch.sigmoid(torch.randn(gshape, generator=g)).to(gdt) if has_b else None
    h0 = torch.randn(N, H, D, generator=g) if states else None
    dy = torch.randn(T, H, D, generator=g).to(dt)
    df = torch.randn(N, H, D, generator=g) if states else None
    cu = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)
    if fused:  # slices of one projection's output
        whole = torch.empty(T, 3, H, D, dtype=dt, device="cuda")
        out = []
        for i, t in enumerate((x, a, b if b is not None else x)):
            whole[:, i] = t.cuda()
            out.append(whole[:, i])
        x, a, b = out[0], out[1], out[2] if has_b else None
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    return dict(x=dev(x), a=dev(a), b=dev(b), h0=dev(h0), dy=dev(dy), df=dev(df), cu=dev(cu), cul=cu.tolist(), T=T, N=N, H=H, D=D)


def within(name, got, want, err, dtype=torch.float32):
    """|got - want| <= the bound of fp32 arithmetic, plus the rounding to a narrower type."""
    got = f64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    lim = err + 2.0 ** -126 + 2.0 ** -23 * err
    if dtype != torch.float32:
        lim = lim + rounding_bound(np.abs(want) + err, dtype)
    else:
        lim = lim + 2.0 ** -24 * np.abs(want)
    off = np.abs(got - want)
    bad = ~(off <= lim)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.size} off, worst {np.nanmax(off - lim):.3g} at {np.argwhere(bad)[0]}"


def check_forward(i, **kw):
    """Runs the forward pass on make()'s inputs and compares outputs, final states and saved states."""
    T, H, D = i["T"], i["H"], i["D"]
    tiles = torch.full((-(-T // 64), H, D), float("nan"), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, final = gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], initial_state=i["h0"], output_final_state=True,
                                           cu_seqlens=i["cu"], tile_states=tiles, device_status=status, **kw)
    assert int(status) == 0
    want = ref.forward(f64(i["x"]), f64(i["a"]), f64(i["b"]), i["cul"], f64(i["h0"]))
    within("y", y, want[0], want[3], i["x"].dtype)
    within("final", final, want[1], want[4], final.dtype)
    at = [min(64 * f + 63, T - 1) for f in range(tiles.shape[0])]
    within("tile_states", tiles, want[0][at], want[3][at])
    return y, final, tiles


def check_backward(i, tiles, d_final=True):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    df = i["df"] if d_final else None
    dx, da, db, d0 = gdn.gated_linear_recurrence_backward(i["dy"], i["x"], i["a"], i["b"], tile_states=tiles,
                                                          initial_state=i["h0"], d_final_state=df, cu_seqlens=i["cu"],
                                                          device_status=status)
    assert int(status) == 0
    val, err = ref.backward(f64(i["dy"]), f64(i["x"]), f64(i["a"]), f64(i["b"]), i["cul"], f64(i["h0"]), f64(df))
    within("dx", dx, val["dx"], err["dx"], i["x"].dtype)
    within("da", da, val["da"], err["da"], i["a"].dtype)
    if i["b"] is not None:
        within("db", db, val["db"], err["db"], i["a"].dtype)
    else:
        assert db is None
    if i["h0"] is not None:
        within("d_initial", d0, val["d0"], err["d0"])
    else:
        assert d0 is None
    return dx, da, db, d0
