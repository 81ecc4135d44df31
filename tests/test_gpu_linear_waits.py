"""What the scans of the gated linear recurrence do when a wait for another block runs out: they end, report it, and give NaN
for whatever depends on what did not come; sequences that do not depend on it keep their values.

A scan's first place (time segment, or tile) is left out of a launch whose waits have a limit of a millisecond or so
(linear_waits.cu): its flag is one that nothing sets.
"""
import ctypes
import subprocess

import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from gated_deltanet_chunked_device_gb300 import _build
from linear_testlib import f64, within
from oracle import linear as ref

pytestmark = pytest.mark.gpu

C, CYCLES, UNTOUCHED = 128, 2_000_000, 7.0


@pytest.fixture(scope="module")
def waits(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.build()
    gdn.lib()
    out = str(tmp_path_factory.mktemp("waits") / "liblinear_waits.so")
    source = __file__.replace("test_gpu_linear_waits.py", "linear_waits.cu")
    subprocess.run([_build._nvcc(), *_build.ARCH, *_build.NVCC_FLAGS, "-I", _build.CSRC, "-shared", "-o", out, source, _build.LIB_PATH],
                   check=True, capture_output=True)
    lib = ctypes.CDLL(out)
    lib.waits_run.argtypes = [ctypes.c_int] * 2 + [ctypes.c_void_p] * 3 + [ctypes.c_int] + [ctypes.c_void_p] * 6 + [ctypes.c_int64, ctypes.c_void_p]
    return lib


def inputs(lib, column, backward, edge):
    T = lib.waits_tokens(column, backward)
    g = torch.Generator("cuda").manual_seed(60)
    x = torch.randn(T, 1, C, generator=g, device="cuda")
    a = torch.exp(-torch.nn.functional.softplus(torch.randn(T, 1, C, generator=g, device="cuda")) / 16)
    cul = [0, edge(T), T]
    return T, x, a, cul, torch.tensor(cul, dtype=torch.int32, device="cuda")


def run(lib, column, backward, x, a, cu, state, tiles):
    y, da = torch.full_like(x, UNTOUCHED), torch.full_like(x, UNTOUCHED)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(65536, dtype=torch.uint8, device="cuda")
    ptr = lambda t: t.data_ptr()  # noqa: E731
    assert lib.waits_run(column, backward, ptr(x), ptr(a), ptr(cu), C, ptr(y), ptr(da), ptr(state), ptr(tiles), ptr(status), ptr(ws),
                         CYCLES, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert int(status) == gdn.DEVICE_ERR["TIMEOUT"]
    return y, da


@pytest.mark.parametrize("column", [1, 0])
def test_forward(waits, column):
    """Of three places the first is missing; the second sequence starts in the third."""
    T, x, a, cul, cu = inputs(waits, column, 0, lambda T: 2 * T // 3 + T // 7)
    tiles, state = torch.full((-(-T // 64), 1, C), UNTOUCHED, device="cuda"), torch.full((2, 1, C), UNTOUCHED, device="cuda")
    y, _ = run(waits, column, 0, x, a, cu, state, tiles)
    start = cul[1]
    assert (y[:T // 3] == UNTOUCHED).all() and torch.isnan(y[T // 3:start]).all()
    assert torch.isnan(state[0]).all()
    want = ref.forward(f64(x[start:]), f64(a[start:]), None, [0, T - start])
    within("y", y[start:], want[0], want[3])
    within("final", state[1:], want[1], want[4])


@pytest.mark.parametrize("column", [1, 0])
def test_backward(waits, column):
    """Of three places the first from the right is missing; the first sequence ends in the third."""
    T, x, a, cul, cu = inputs(waits, column, 1, lambda T: T // 7)
    tiles = torch.empty(-(-T // 64), 1, C, device="cuda")
    h0 = torch.randn(2, 1, C, generator=torch.Generator("cuda").manual_seed(61), device="cuda")
    gdn.gated_linear_recurrence(x, a, initial_state=h0, cu_seqlens=cu, tile_states=tiles)
    state = torch.cat([torch.full_like(h0, UNTOUCHED), h0])
    dx, da = run(waits, column, 1, x, a, cu, state, tiles)
    end = cul[1]
    for got in (dx, da):
        assert (got[2 * T // 3:] == UNTOUCHED).all() and torch.isnan(got[end:2 * T // 3]).all()
    assert torch.isnan(state[1]).all()
    val, err = ref.backward(f64(x[:end]), f64(x[:end]), f64(a[:end]), None, [0, end], f64(h0[:1]))
    within("dx", dx[:end], val["dx"], err["dx"])
    within("da", da[:end], val["da"], err["da"])
    within("d_initial", state[:1], val["d0"], err["d0"])
