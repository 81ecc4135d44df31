"""Rotary positions, cache writes and attention without a GPU: what is refused, and the definition that the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from oracle import attention as ref

OK, INVALID, UNSUPPORTED = 0, 1, 2
F = 0x7f0000000000  # never dereferenced: every call below is refused, or has nothing to do


@pytest.fixture(scope="module")
def L():
    gdn.build()
    return gdn.lib()


def batch(**kw):
    d = dict(cu_seqlens=F, seqs=F + 0x1000, table=F + 0x2000, lengths=F + 0x3000, total_tokens=10, num_seqs=2, tokens_per_seq=0, cu_i64=0,
             max_seqs=4, max_pages=3, n_pages=20, page_tokens=16, device_status=None)
    d.update(kw)
    return gdn.KvBatch(**d)


def cache(**kw):
    d = dict(k=F + 0x10000, v=F + 0x20000, k_page_stride=16 * 128, k_token_stride=128, k_head_stride=64, v_page_stride=16 * 128,
             v_token_stride=128, v_head_stride=64, kv_heads=2, head_dim=64, dtype=gdn.DTYPE_BF16)
    d.update(kw)
    return gdn.KvCache(**d)


def rotary(**kw):
    d = dict(q=F + 0x30000, k=F + 0x40000, q_out=F + 0x50000, k_out=F + 0x60000, q_stride=0, k_stride=0, q_out_stride=0, k_out_stride=0,
             frequencies=F + 0x70000, heads=4, kv_heads=2, head_dim=64, rotary_dim=32, interleaved=0, inverse=0, magnitude=1.0,
             dtype=gdn.DTYPE_BF16)
    d.update(kw)
    return gdn.RotaryArgs(**d)


def attention(**kw):
    d = dict(q=F + 0x30000, output=F + 0x40000, lse=None, q_stride=0, output_stride=0, heads=4, scale=0.125, causal=1, window=0)
    d.update(kw)
    return gdn.AttentionArgs(**d)


def run_attention(L, b, c, a, ws=1 << 40):
    return L.gdn_attention_run(ctypes.byref(b), ctypes.byref(c), ctypes.byref(a), F + 0x100000, ws, None)


def test_structs_match_the_header():
    assert [ctypes.sizeof(t) for t in (gdn.KvBatch, gdn.KvCache, gdn.RotaryArgs, gdn.AttentionArgs)] == [80, 80, 104, 56]


BAD_BATCH = [dict(num_seqs=-1), dict(total_tokens=-1), dict(max_seqs=-1), dict(max_pages=-1), dict(n_pages=-1), dict(page_tokens=0),
             dict(lengths=None), dict(table=None), dict(lengths=F + 2), dict(table=F + 1), dict(seqs=F + 3), dict(cu_seqlens=F + 2),
             dict(cu_seqlens=F + 4, cu_i64=1), dict(device_status=F + 2), dict(cu_seqlens=None, tokens_per_seq=4),
             dict(cu_seqlens=None, tokens_per_seq=0), dict(seqs=None, num_seqs=5)]
BAD_CACHE = [dict(k=None), dict(v=None), dict(k=F + 1), dict(v=F + 1), dict(kv_heads=0), dict(head_dim=0), dict(k_head_stride=63),
             dict(k_token_stride=100), dict(v_token_stride=127), dict(v_page_stride=2000), dict(k_page_stride=0), dict(v_head_stride=-64),
             dict(k_page_stride=1 << 62)]


@pytest.mark.parametrize("kw", BAD_BATCH)
def test_batch_is_checked(L, kw):
    assert run_attention(L, batch(**kw), cache(), attention()) == INVALID
    assert L.gdn_attention_workspace(ctypes.byref(batch(**kw)), ctypes.byref(cache()), ctypes.byref(attention())) == 0
    assert L.gdn_cache_append_run(ctypes.byref(batch(**kw)), ctypes.byref(cache()), ctypes.byref(rotary()), F + 0x80000, 0, None) == INVALID


@pytest.mark.parametrize("kw", BAD_CACHE)
def test_cache_is_checked(L, kw):
    assert run_attention(L, batch(), cache(**kw), attention()) == INVALID
    assert L.gdn_cache_append_run(ctypes.byref(batch()), ctypes.byref(cache(**kw)), ctypes.byref(rotary()), F + 0x80000, 0, None) == INVALID


@pytest.mark.parametrize("b,c,a,expect", [
    ({}, {}, dict(q=None), INVALID), ({}, {}, dict(output=None), INVALID), ({}, {}, dict(q=F + 1), INVALID),
    ({}, {}, dict(lse=F + 2), INVALID), ({}, {}, dict(q_stride=255), INVALID), ({}, {}, dict(output_stride=255), INVALID),
    ({}, {}, dict(heads=0), INVALID), ({}, {}, dict(heads=5), INVALID), ({}, {}, dict(window=-1), INVALID),
    ({}, {}, dict(scale=float("nan")), INVALID), ({}, {}, dict(scale=float("inf")), INVALID), ({}, {}, dict(scale=3e38), INVALID),
    ({}, {}, dict(output=F + 0x30000), INVALID), (dict(total_tokens=0x7fff0001), {}, {}, UNSUPPORTED),
    ({}, dict(dtype=gdn.DTYPE_F8E4M3), {}, UNSUPPORTED),
    ({}, dict(head_dim=257, k_head_stride=257, k_token_stride=514, k_page_stride=16 * 514, v_head_stride=257, v_token_stride=514,
              v_page_stride=16 * 514), {}, UNSUPPORTED),
    (dict(total_tokens=1 << 31), {}, {}, UNSUPPORTED),
    (dict(total_tokens=0), {}, {}, OK), (dict(num_seqs=0), {}, {}, OK)])
def test_attention_is_checked(L, b, c, a, expect):
    assert run_attention(L, batch(**b), cache(**c), attention(**a)) == expect


# Rows of q: 10 of 4 x 64 bf16, 512 bytes each.
@pytest.mark.parametrize("kw,expect", [
    (dict(output=F + 0x30000 + 2), INVALID), (dict(output=F + 0x30000 - 2), INVALID), (dict(output=F + 0x30000 + 9 * 512), INVALID),
    (dict(output=F + 0x30000 - 10 * 512 + 2), INVALID),
    (dict(q_stride=512, output_stride=512, output=F + 0x30000 + 510), INVALID),
    (dict(q_stride=512, output_stride=512, output=F + 0x30000 + 514), INVALID),
    (dict(q_stride=512, output_stride=768, output=F + 0x30000 + 512), INVALID),
    (dict(q_stride=1 << 62, output_stride=1 << 62, output=F + 0x30000 + 2), INVALID)])
def test_output_is_apart_from_q(L, kw, expect):
    assert run_attention(L, batch(), cache(), attention(**kw)) == expect
    assert L.gdn_attention_workspace(ctypes.byref(batch()), ctypes.byref(cache()), ctypes.byref(attention(**kw))) == 0


@pytest.mark.parametrize("kw", [
    dict(output=F + 0x30000 + 10 * 512), dict(output=F + 0x30000 - 10 * 512), dict(q_stride=512, output_stride=512, output=F + 0x30000 + 512),
    dict(q_stride=512, output_stride=512, output=F + 0x30000 - 512), dict(q_stride=512, output_stride=512, output=F + 0x30000 + 1024 * 3 + 512)])
def test_output_beside_q_is_taken(L, kw):
    b, c, a = batch(), cache(), attention(**kw)  # a workspace too small is refused after the rest
    assert run_attention(L, b, c, a, ws=16) == INVALID
    assert L.gdn_attention_workspace(ctypes.byref(b), ctypes.byref(c), ctypes.byref(a)) > 0


def test_attention_needs_its_workspace(L):
    b, c, a = batch(), cache(), attention()
    assert run_attention(L, b, c, a, ws=16) == INVALID
    assert L.gdn_attention_run(ctypes.byref(b), ctypes.byref(c), ctypes.byref(a), None, 1 << 40, None) == INVALID
    assert L.gdn_attention_run(ctypes.byref(b), ctypes.byref(c), ctypes.byref(a), F + 8, 1 << 40, None) == INVALID
    assert L.gdn_attention_run(None, ctypes.byref(c), ctypes.byref(a), F, 1 << 40, None) == INVALID
    assert L.gdn_attention_run(ctypes.byref(b), ctypes.byref(c), None, F, 1 << 40, None) == INVALID


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(q_out=None), INVALID), (dict(q=F + 1), INVALID), (dict(q_stride=255), INVALID),
    (dict(k_stride=127), INVALID), (dict(rotary_dim=31), INVALID), (dict(rotary_dim=66), INVALID), (dict(rotary_dim=-2), INVALID),
    (dict(frequencies=None), INVALID), (dict(frequencies=F + 4), INVALID), (dict(heads=-1), INVALID), (dict(head_dim=0), INVALID),
    (dict(q_out=F + 0x30000, q_out_stride=300), INVALID), (dict(dtype=gdn.DTYPE_F8E5M2), UNSUPPORTED),
    (dict(head_dim=1026), UNSUPPORTED), (dict(heads=1 << 15), UNSUPPORTED)])
def test_rotary_is_checked(L, kw, expect):
    assert L.gdn_rotary_run(ctypes.byref(rotary(**kw)), None, 0, None, 0, 0, 10, None) == expect
    if "head_dim" not in kw and "dtype" not in kw:
        assert L.gdn_cache_append_run(ctypes.byref(batch()), ctypes.byref(cache()), ctypes.byref(rotary(**kw)), F + 0x80000, 0, None) == expect


def test_positions_are_checked(L):
    r = ctypes.byref(rotary())
    assert L.gdn_rotary_run(r, F + 4, 1, None, 0, 0, 10, None) == INVALID
    assert L.gdn_rotary_run(r, F + 2, 0, None, 0, 0, 10, None) == INVALID
    assert L.gdn_rotary_run(r, F, 0, F, 0, 1, 10, None) == INVALID
    assert L.gdn_rotary_run(r, None, 0, F + 4, 1, 1, 10, None) == INVALID
    assert L.gdn_rotary_run(r, None, 0, F, 0, -1, 10, None) == INVALID
    assert L.gdn_rotary_run(r, None, 0, None, 0, 0, -1, None) == INVALID
    assert L.gdn_rotary_run(r, None, 0, None, 0, 0, 0, None) == OK
    assert L.gdn_rotary_run(ctypes.byref(rotary(heads=0, kv_heads=0)), None, 0, None, 0, 0, 10, None) == OK
    assert L.gdn_rotary_run(None, None, 0, None, 0, 0, 10, None) == INVALID


@pytest.mark.parametrize("kw", [dict(kv_heads=1), dict(head_dim=32, rotary_dim=32), dict(dtype=gdn.DTYPE_F16)])
def test_append_takes_tensors_of_the_caches_kind(L, kw):
    assert L.gdn_cache_append_run(ctypes.byref(batch()), ctypes.byref(cache()), ctypes.byref(rotary(**kw)), F + 0x80000, 0, None) == INVALID


def test_append_checks_values(L):
    args = ctypes.byref(batch()), ctypes.byref(cache()), ctypes.byref(rotary())
    for v, stride in ((None, 0), (F + 1, 0), (F, 127)):
        assert L.gdn_cache_append_run(*args, v, stride, None) == INVALID


def test_python_refuses_cpu_tensors():
    x, c = torch.zeros(2, 1, 8), torch.zeros(1, 4, 1, 8)
    t, n = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    f = gdn.rotary_frequencies(8, device="cpu")
    for call in (lambda: gdn.rotary_embedding(x, x, f), lambda: gdn.rotary_embedding_backward(x, x, f),
                 lambda: gdn.cache_append(x, x, c, c, t, n), lambda: gdn.paged_attention(x, c, c, t, n)):
        with pytest.raises(ValueError, match="no CPU path"):
            call()
    for call in (lambda: gdn.rotary_embedding(None, None, f), lambda: gdn.rotary_embedding_backward(None, None, f)):
        with pytest.raises(ValueError, match="must be given"):
            call()


def test_frequencies():
    f = gdn.rotary_frequencies(8, base=100.0, device="cpu")
    assert f.dtype is torch.float64 and np.allclose(f, [1, 100 ** -0.25, 0.1, 100 ** -0.75], rtol=1e-15)
    assert torch.equal(gdn.rotary_frequencies(8, base=100.0, factor=4.0, device="cpu"), f / 4)
    # over 400 tokens these turn 63.7, 20.1, 6.4 and 2.01 times: above 32 kept, below 4 slowed, mixed in between
    g = gdn.rotary_frequencies(8, base=100.0, factor=4.0, original_length=400, slow_turns=4.0, fast_turns=32.0, device="cpu")
    turns = 400 * f / (2 * math.pi)
    assert g[0] == f[0] and g[3] == f[3] / 4
    for i in (1, 2):
        kept = float((turns[i] - 4) / 28)
        assert abs(float(g[i]) - float(f[i]) * (kept + (1 - kept) / 4)) < 1e-15
    assert gdn.rotary_frequencies(0, device="cpu").shape == (0,)
    for bad in (lambda: gdn.rotary_frequencies(3), lambda: gdn.rotary_frequencies(-2), lambda: gdn.rotary_frequencies(4, base=0.0),
                lambda: gdn.rotary_frequencies(4, factor=0.0),
                lambda: gdn.rotary_frequencies(4, original_length=10, slow_turns=2.0, fast_turns=2.0)):
        with pytest.raises(ValueError):
            bad()


def test_definition_turns_by_hand():
    """A quarter turn, an eighth, both layouts, and the way back."""
    x = np.arange(1.0, 6.0).reshape(1, 1, 5)
    y, size = ref.rotary(x, [1], [math.pi / 2, math.pi / 4])
    r = math.sqrt(0.5)
    assert np.allclose(y[0, 0], [-3, (2 - 4) * r, 1, (4 + 2) * r, 5], atol=1e-15) and size[0, 0].tolist() == [4, 6, 4, 6, 0]
    y, _ = ref.rotary(x, [1], [math.pi / 2, math.pi / 4], interleaved=True, magnitude=2.0)
    assert np.allclose(y[0, 0], [-4, 2, 2 * (3 - 4) * r, 2 * (4 + 3) * r, 5], atol=1e-14)
    back, _ = ref.rotary(y, [1], [math.pi / 2, math.pi / 4], interleaved=True, magnitude=0.5, inverse=True)
    assert np.allclose(back, x, atol=1e-14)
    # scores of turned vectors depend on the distance alone
    q, k = np.random.default_rng(0).normal(size=(2, 1, 1, 8))
    f = [1.0, 0.3, 0.01, 1e-4]
    dot = lambda a, b: float((ref.rotary(q, [a], f)[0] * ref.rotary(k, [b], f)[0]).sum())  # noqa: E731
    assert abs(dot(5, 2) - dot(1005, 1002)) < 1e-11


def test_definition_attends_by_hand():
    """Two pages of two tokens out of order, one head: the second of two new tokens sees three keys, or two of them."""
    k = np.zeros((3, 2, 1, 1))
    v = np.arange(6.0).reshape(3, 2, 1, 1)  # values 4 5 | 0 1 of pages 2, 0
    table = np.array([[-1, -1], [2, 0]])
    q = np.ones((2, 1, 1))
    out, lse, *_ = ref.attend(q, k, v, table, [0, 3], [1], [2], 1.0)
    assert np.allclose(out[:, 0, 0], [4.5, 3.0]) and np.allclose(lse[:, 0], np.log([2, 3]))
    out, lse, *_ = ref.attend(q, k, v, table, [0, 3], [1], [2], 1.0, window=2)
    assert np.allclose(out[:, 0, 0], [4.5, 2.5])
    out, lse, *_ = ref.attend(q, k, v, table, [0, 3], [1], [2], 1.0, causal=False)
    assert np.allclose(out[:, 0, 0], [3.0, 3.0])
    out, lse, *_ = ref.attend(q, k, v, table, [0, 1], [1], [2], 1.0)
    assert out[0, 0, 0] == 0 and lse[0, 0] == -np.inf and out[1, 0, 0] == 4.0
    table[1, 0] = -1
    out, *_ = ref.attend(q, k, v, table, [0, 3], [1], [2], 1.0)
    assert out[0, 0, 0] == 0 and out[1, 0, 0] == 0.0


# 10 rows of q (4 x 64 bf16, 512 bytes), and of k and v (256 bytes).  Slices of one tensor: 1024 bytes from token to token.
FUSED = dict(q=F, k=F + 512, q_stride=512, k_stride=512)


@pytest.mark.parametrize("kw", [
    dict(q_out=F + 0x30000 + 2), dict(q_out=F + 0x30000 + 128), dict(q_out=F + 0x30000 - 128), dict(q_out=F + 0x30000 + 9 * 512),
    dict(q_out=F + 0x40000), dict(q_out=F + 0x40000 - 128), dict(q_out=F + 0x40000 + 9 * 256), dict(q_out=F + 0x40000, q_out_stride=1024),
    {**FUSED, "q_out": F + 128, "q_out_stride": 512}, {**FUSED, "q_out": F + 256, "q_out_stride": 512},
    {**FUSED, "q_out": F + 640, "q_out_stride": 512}, {**FUSED, "q_out": F, "q_out_stride": 0},
    {**FUSED, "q": F + 128, "q_out": F + 128, "q_out_stride": 512}, dict(q_out=F + 0x30000 + 2, q_out_stride=1 << 62)])
def test_turned_queries_are_apart_or_in_place(L, kw):
    assert L.gdn_rotary_run(ctypes.byref(rotary(**kw)), None, 0, None, 0, 0, 10, None) == INVALID
    assert L.gdn_cache_append_run(ctypes.byref(batch()), ctypes.byref(cache()), ctypes.byref(rotary(**kw)), F + 0x80000, 0, None) == INVALID


@pytest.mark.parametrize("kw", [
    dict(k_out=F + 0x40000 + 128), dict(k_out=F + 0x30000), dict(k_out=F + 0x30000 + 9 * 512), dict(k_out=F + 0x50000),
    dict(k_out=F + 0x50000 + 4096), {**FUSED, "q_out": F, "q_out_stride": 512, "k_out": F + 256, "k_out_stride": 512},
    dict(q_out=F + 0x50000, q_out_stride=512, k_out=F + 0x50000 + 256, k_out_stride=512), dict(heads=0, q=None, q_out=None, k_out=F + 0x40000 + 2)])
def test_turned_keys_are_apart_or_in_place(L, kw):
    assert L.gdn_rotary_run(ctypes.byref(rotary(**kw)), None, 0, None, 0, 0, 10, None) == INVALID


@pytest.mark.parametrize("v,stride", [(F + 0x50000, 0), (F + 0x50000 + 9 * 512 + 510, 0), (F + 0x50000 - 9 * 256, 0), (F + 0x50000 - 4096, 512)])
def test_turned_queries_are_apart_from_the_values(L, v, stride):
    assert L.gdn_cache_append_run(ctypes.byref(batch()), ctypes.byref(cache()), ctypes.byref(rotary()), v, stride, None) == INVALID


def test_an_output_needs_its_input():
    x, f = torch.zeros(2, 1, 8), gdn.rotary_frequencies(8, device="cpu")
    for kw in (dict(q=None, k=x, q_out=x), dict(q=x, k=None, k_out=x)):
        with pytest.raises(ValueError, match="needs"):
            gdn.rotary_embedding(frequencies=f, **kw)


@pytest.mark.parametrize("lse", [F + 0x30000, F + 0x30000 + 9 * 512 + 508, F + 0x30000 - 9 * 16, F + 0x40000 + 512, F + 0x40000 - 4])
def test_logarithms_are_apart(L, lse):
    assert run_attention(L, batch(), cache(), attention(lse=lse)) == INVALID
    assert L.gdn_attention_workspace(ctypes.byref(batch()), ctypes.byref(cache()), ctypes.byref(attention(lse=lse))) == 0
    for beside in (F + 0x30000 - 160, F + 0x30000 + 10 * 512, F + 0x50000):
        assert L.gdn_attention_workspace(ctypes.byref(batch()), ctypes.byref(cache()), ctypes.byref(attention(lse=beside))) > 0
