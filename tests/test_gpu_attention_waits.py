"""What attention over a paged cache does when a wait inside its kernel runs out: it ends, reports it, and leaves the GPU in order; every
row is NaN or right, those of units that several blocks share too.

The kernel runs with half of each tile of keys and values never fetched, so that its waits for them run out (attention_waits.cu), or
with a limit of nothing at all, so that a wait gives up as soon as it would have to go on."""
import ctypes
import subprocess

import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from gated_deltanet_chunked_device_gb300 import _build
from attention_testlib import Cache

pytestmark = pytest.mark.gpu

CYCLES = 2_000_000


@pytest.fixture(scope="module")
def waits(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.build()
    gdn.lib()
    out = str(tmp_path_factory.mktemp("waits") / "libattention_waits.so")
    source = __file__.replace("test_gpu_attention_waits.py", "attention_waits.cu")
    subprocess.run([_build._nvcc(), *_build.ARCH, *_build.NVCC_FLAGS, "-I", _build.CSRC, "-shared", "-o", out, source, _build.LIB_PATH],
                   check=True, capture_output=True)
    lib = ctypes.CDLL(out)
    lib.waits_attention.argtypes = [ctypes.c_void_p] * 4 + [ctypes.c_size_t, ctypes.c_longlong, ctypes.c_int, ctypes.c_void_p]
    return lib


def run(lib, c, cycles, missing):
    """The kernel with short waits; returns output, logarithms and status."""
    T, H, D = c.q.shape
    g, q, cu = c.gpu(), c.q.cuda(), c.cu.cuda()
    out, lse = torch.full_like(q, 7.0), torch.full((T, H), 7.0, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    S, M = g["table"].shape
    P, pt, Hk, _ = g["k_cache"].shape
    strides = [s for t in (g["k_cache"], g["v_cache"]) for s in t.stride()[:3]]
    kv = gdn.KvCache(g["k_cache"].data_ptr(), g["v_cache"].data_ptr(), *strides, Hk, D, gdn._QKV_DTYPES[c.dtype])
    batch = gdn.KvBatch(cu.data_ptr(), g["seqs"].data_ptr(), g["table"].data_ptr(), g["lengths"].data_ptr(), T, len(c.lens), 0, 0, S, M, P, pt,
                        word.data_ptr())
    args = gdn.AttentionArgs(q.data_ptr(), out.data_ptr(), lse.data_ptr(), 0, 0, H, D ** -0.5, 1, 0)
    n = gdn.lib().gdn_attention_workspace(ctypes.byref(batch), ctypes.byref(kv), ctypes.byref(args))
    ws = torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda")
    assert lib.waits_attention(ctypes.byref(batch), ctypes.byref(kv), ctypes.byref(args), ws.data_ptr(), n, cycles, missing,
                               torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    return out, lse, int(word)


SHAPES = [(64, 8, 2, [1] * 40), (128, 8, 2, [1] * 40), (256, 8, 2, [1] * 40),   # single tokens: quarters
          (64, 8, 2, [300, 1, 90]), (128, 8, 2, [300, 1, 90]),                  # two row tiles
          (256, 8, 2, [300, 1, 90]), (128, 64, 1, [1] * 40)]                    # one row tile


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,heads,kv_heads,lens", SHAPES)
@pytest.mark.parametrize("page_tokens,missing", [(64, 1), (64, 0), (20, 0)])
def test_the_kernel_ends_and_the_next_one_is_right(waits, dtype, D, heads, kv_heads, lens, page_tokens, missing):
    c = Cache(lens, [900] * len(lens), heads, kv_heads, D, page_tokens, dtype, seed=D)
    out, lse, status = run(waits, c, CYCLES if missing else -1, missing)
    assert status in ((gdn.DEVICE_ERR["TIMEOUT"],) if missing else (0, gdn.DEVICE_ERR["TIMEOUT"]))
    if missing:
        assert not bool((torch.isfinite(out) & (out != 7.0)).any())  # nothing passes for a result
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,heads,kv_heads,lens", SHAPES)
@pytest.mark.parametrize("page_tokens,missing", [(64, 1), (64, 0), (20, 0)])
def test_rows_are_nan_or_right(waits, dtype, D, heads, kv_heads, lens, page_tokens, missing):
    """Contexts long enough that most units are cut; a sequence without keys among them, whose rows are zero."""
    past = [3000 + 7 * i for i in range(len(lens))]
    past[1] = -lens[1]
    c = Cache(lens, past, heads, kv_heads, D, page_tokens, dtype, seed=D)
    want_lse = torch.empty(c.q.shape[:2], device="cuda")
    want = gdn.paged_attention(c.q.cuda(), **c.gpu(), cu_seqlens=c.cu.cuda(), lse=want_lse)
    for _ in range(1 if missing else 5):
        out, lse, status = run(waits, c, CYCLES if missing else -1, missing)
        assert bool((torch.isnan(out) | (out == want)).all()) and bool((torch.isnan(lse) | (lse == want_lse)).all())
        gone = torch.isnan(out).any(-1)
        if missing:
            keys = torch.ones(len(lens), dtype=torch.bool)
            keys[1] = False
            rows = keys.repeat_interleave(torch.tensor(lens)).cuda()
            assert bool(torch.isnan(out[rows]).all()) and bool(torch.isnan(lse[rows]).all())
        assert bool(gone.any()) == (status != 0)
