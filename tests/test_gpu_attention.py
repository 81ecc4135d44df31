"""Attention over a paged cache on the GPU, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from attention_testlib import DEV, Cache, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.build()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [1, 6, 8, 30, 33, 64, 80, 100, 128, 130, 192, 215, 256])
def test_ragged_chunks(dtype, D):
    Cache([130, 0, 20, 1, 70], [50, 3, 0, 300, 129], 4, 2, D, 16, dtype, seed=D).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 1), (6, 2), (5, 5), (16, 1), (14, 2), (130, 1), (200, 1)])
def test_groups_of_heads(dtype, heads, kv_heads):
    Cache([17, 1, 40], [100, 260, 0], heads, kv_heads, 64, 32, dtype, seed=heads).check()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("page_tokens", [1, 3, 8, 16, 24, 48, 64, 100, 128, 200, 256])
def test_sizes_of_pages(dtype, page_tokens):
    Cache([33, 5], [250, 700], 4, 1, 64, page_tokens, dtype, seed=page_tokens).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["token", "head", "wide", "odd"])
@pytest.mark.parametrize("D,page_tokens", [(64, 16), (128, 16), (96, 5)])
def test_layouts(dtype, layout, D, page_tokens):
    Cache([60, 9], [10, 200], 8, 2, D, page_tokens, dtype, layout=layout).check(strided=True)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens", [1, 2, 5])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_single_tokens(dtype, tokens, D):
    past = [0, 1, 62, 63, 64, 127, 128, 500, 1023, 1500]
    Cache([tokens] * len(past), past, 16, 2, D, 64, dtype, seed=tokens).check(tokens=tokens)


@pytest.mark.parametrize("length", list(range(1, 12)) + [63, 64, 65, 127, 128, 129, 255, 256, 257, 1000])
def test_lengths(length):
    Cache([1, length], [length - 1, 0], 2, 1, 128, 16, "bf16", seed=length).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 2, 63, 64, 100, 128, 1000])
@pytest.mark.parametrize("causal", [True, False])
def test_windows(dtype, window, causal):
    Cache([150, 1, 40], [300, 450, 0], 4, 2, 64, 16, dtype, seed=window).check(window=window, causal=causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_key_seen(dtype):
    Cache([150, 1, 40], [300, 450, 0], 4, 2, 128, 16, dtype).check(causal=False)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_tokens_before_the_first_position_see_nothing(dtype):
    """More new tokens than the sequence has: the first ones have negative positions."""
    got = Cache([100, 7, 140], [-30, -7, -139], 4, 2, 64, 16, dtype).check()
    assert float(got[:30].abs().max()) == 0 and float(got[100:107].abs().max()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 8.0])
def test_scales(dtype, scale):
    """Up to scores of some hundreds, where one key takes all."""
    Cache([40, 3], [60, 260], 2, 1, 64, 16, dtype).check(scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_rising_scores(dtype):
    """Every tile has a larger maximum than the one before, by far: each time all sums are rescaled."""
    c = Cache([20], [900], 2, 1, 64, 16, dtype)
    for i, page in enumerate(c.table[c.seqs[0]].tolist()):
        if page >= 0:
            c.k[page] = (c.k[page].float() * 0.1 + 0.05 * i).to(c.dtype)
    c.q = c.q.abs()
    c.check(scale=0.5)
    c.check(scale=-0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("D", [64, 128, 256, 100])
def test_what_a_token_does_not_see_has_no_influence(dtype, bad, what, D):
    """A key or value in the middle of the chunk that is not finite: the tokens before it, and those that look back less far, are right."""
    lens, past = [200, 3], [100, 0]
    c = Cache(lens, past, 4, 2, D, 16, dtype)
    pos = 217
    page = int(c.table[c.seqs[0], pos // 16])
    out, lse, size, products, count = c.want(window=40)
    getattr(c, what)[page, pos % 16, 0, 5] = bad
    q = c.q.cuda()
    got = f64(gdn.paged_attention(q, **c.gpu(), cu_seqlens=c.cu.cuda(), window=40))
    from attention_testlib import attention_bound
    lim = attention_bound(out, size, products, count, D, c.dtype)
    sees = np.zeros((203, 4), dtype=bool)
    at = np.arange(100, 300)
    sees[:200, :2] = ((at >= pos) & (at < pos + 40))[:, None]
    assert (np.abs(got - out) <= lim)[~sees].all()
    if what == "v" or bad != bad:
        assert not np.isfinite(got[sees]).all(-1).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page_tokens", [16, 64, 7])
@pytest.mark.parametrize("heads", [4, 64])
def test_bad_pages_are_left_out_and_reported(dtype, page_tokens, heads):
    c = Cache([30, 2, 5], [200, 100, 0], heads, 1, 64, page_tokens, dtype)
    s = c.seqs.tolist()
    c.table[s[0], 1] = -1
    c.table[s[0], 3] = c.k.shape[0]
    c.table[s[1], 0] = -2 ** 31
    c.check(status=DEV["PAGE"])


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements, pages at both of its ends."""
    c = Cache([20, 1], [300, 100], 4, 2, 128, 64, "bf16", fill=0.0)
    g = c.gpu()
    pages, old = 140000, c.k.shape[0]
    whole = [torch.empty(pages, *c.k.shape[1:], dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for t, small in zip(whole, (g["k_cache"], g["v_cache"])):
        t[pages - old:] = small
    want = gdn.paged_attention(c.q.cuda(), **g, cu_seqlens=c.cu.cuda())
    g["table"] = torch.where(g["table"] >= 0, g["table"] + (pages - old), -1)
    got = gdn.paged_attention(c.q.cuda(), **{**g, "k_cache": whole[0], "v_cache": whole[1]}, cu_seqlens=c.cu.cuda())
    assert torch.equal(got, want)
    f = gdn.rotary_frequencies(128)
    k, v = torch.randn(21, 2, 128, device="cuda").bfloat16(), torch.randn(21, 2, 128, device="cuda").bfloat16()
    gdn.cache_append(k, v, whole[0], whole[1], g["table"], g["lengths"], seqs=g["seqs"], cu_seqlens=c.cu.cuda(), frequencies=f)
    small = c.gpu()
    gdn.cache_append(k, v, small["k_cache"], small["v_cache"], small["table"], g["lengths"], seqs=g["seqs"], cu_seqlens=c.cu.cuda(), frequencies=f)
    assert torch.equal(whole[0][pages - old:], small["k_cache"]) and torch.equal(whole[1][pages - old:], small["v_cache"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_sequences_and_lengths(dtype):
    c = Cache([3, 2, 5, 4], [20, 10, 0, 30], 2, 1, 64, 16, dtype)
    c.seqs[0], c.seqs[2] = -1, 10 ** 6
    c.check(status=DEV["SEQ"])
    c = Cache([3, 2, 5], [20, 10, 0], 2, 1, 64, 16, dtype)
    c.lengths[c.seqs[1]] = -4
    c.check(status=DEV["PAGE"])
    c = Cache([3, 2, 5], [20, 10, 0], 2, 1, 64, 16, dtype)
    c.lengths[c.seqs[0]] = 1000  # past the table
    c.check(status=DEV["PAGE"])
    c.check(status=DEV["PAGE"], causal=False)
    c.check(status=DEV["PAGE"], window=980)


def test_bad_bounds_are_reported_and_followed_nowhere():
    c = Cache([30, 20, 10], [0, 5, 9], 2, 1, 64, 16, "bf16")
    for cu in ([0, 40, 20, 60], [0, 30, 50, 70], [5, 30, 50, 60], [0, -3, 50, 60], [0, 2 ** 31 - 1, -2 ** 31, 60]):
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        gdn.paged_attention(c.q.cuda(), **c.gpu(), cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), device_status=word)
        assert int(word) & DEV["CU_SEQLENS"]
        gdn.cache_append(c.k.cuda().flatten(0, 1)[:60], c.v.cuda().flatten(0, 1)[:60], **c.gpu(),
                         cu_seqlens=torch.tensor(cu, dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()


def test_padding_is_left_alone():
    for dtype in ("bf16", "f32"):
        c = Cache([30, 0, 7], [0, 5, 100], 2, 1, 64, 16, dtype)
        q = torch.cat([c.q, torch.full_like(c.q[:20], float("nan"))]).cuda()
        out = torch.full_like(q, 3.0)
        lse = torch.full(q.shape[:2], 3.0, device="cuda")
        gdn.paged_attention(q, **c.gpu(), cu_seqlens=c.cu.cuda(), output=out, lse=lse)
        assert bool((out[37:] == 3.0).all()) and bool((lse[37:] == 3.0).all()) and bool(torch.isfinite(out[:37]).all())


def test_no_tokens_and_no_pages():
    c = Cache([0, 0], [5, 0], 2, 1, 64, 16, "bf16")
    assert gdn.paged_attention(c.q.cuda(), **c.gpu(), cu_seqlens=c.cu.cuda()).shape == (0, 2, 64)
    for dtype in (torch.bfloat16, torch.float32):  # an empty cache, an empty table
        q = torch.ones(3, 2, 64, dtype=dtype, device="cuda")
        cache = torch.empty(0, 16, 1, 64, dtype=dtype, device="cuda")
        z = dict(dtype=torch.int32, device="cuda")
        for table in (torch.full((3, 2), -1, **z), torch.empty(3, 0, **z)):
            got = gdn.paged_attention(q, cache, cache.clone(), table, torch.zeros(3, **z), tokens_per_seq=1)
            assert float(got.abs().max()) == 0


def test_many_sequences():
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 4, (1700,), generator=g).tolist()
    past = torch.randint(0, 90, (1700,), generator=g).tolist()
    for dtype in ("bf16", "f32"):
        Cache(lens, past, 2, 1, 64, 16, dtype).check()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D,tokens,page_tokens", [(64, 1, 16), (128, 1, 16), (128, 2, 64), (256, 1, 32), (128, 1, 12), (99, 1, 64), (250, 1, 10)])
def test_many_units_a_block(dtype, D, tokens, page_tokens):
    """Each block goes through several sequences with several tiles and a partly filled last one."""
    g = torch.Generator().manual_seed(D + tokens)
    past = torch.randint(0, 1300, (320,), generator=g).tolist()
    Cache([tokens] * 320, past, 4, 2, D, page_tokens, dtype, seed=D).check(tokens=tokens)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page_tokens", [(64, 16), (128, 64), (256, 64), (128, 10), (100, 64), (47, 7), (200, 20)])
def test_many_units_of_many_rows_a_block(dtype, D, page_tokens):
    """The same for chunks of tokens: units of several hundred rows, whole ones and cut ones."""
    g = torch.Generator().manual_seed(D)
    lens = torch.randint(0, 60, (60,), generator=g).tolist()
    past = torch.randint(0, 1000, (60,), generator=g).tolist()
    Cache(lens, past, 32, 2, D, page_tokens, dtype, seed=D).check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads,kv_heads", [(4, 1), (16, 2)])
def test_long_context_of_one_sequence(dtype, D, heads, kv_heads):
    """Few rows, many keys: every block has a piece of the same unit."""
    Cache([1], [9000], heads, kv_heads, D, 64, dtype, seed=1).check(tokens=1)


def same_bits(a, b):
    t = torch.int16 if a.element_size() == 2 else torch.int32
    return torch.equal(a.view(t), b.view(t))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_same_inputs_give_the_same_bits(dtype):
    c = Cache([300, 1, 1, 40], [700, 2000, 3, 0], 8, 2, 128, 16, dtype)
    g, q, cu = c.gpu(), c.q.cuda(), c.cu.cuda()
    first = gdn.paged_attention(q, **g, cu_seqlens=cu)
    for _ in range(5):
        assert torch.equal(first, gdn.paged_attention(q, **g, cu_seqlens=cu))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_graphs_that_share_a_pool_and_replay_with_other_lengths(dtype):
    c = Cache([1] * 6, [300, 10, 0, 77, 500, 64], 8, 2, 128, 16, dtype)
    d = Cache([1] * 6, [30, 10, 340, 7, 100, 50], 8, 2, 128, 16, dtype, seed=9)
    g, q = c.gpu(), c.q.cuda()
    out = torch.empty_like(q), torch.empty_like(q)
    call = lambda o: gdn.paged_attention(q, **g, tokens_per_seq=1, output=o)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(out[0])
    s.synchronize()
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        call(out[0])
    with torch.cuda.graph(two, pool=one.pool()):
        call(out[1])
    one.replay()
    two.replay()
    want = call(None)
    assert same_bits(out[0], want) and same_bits(out[1], want)
    pages = min(c.k.shape[0], d.k.shape[0])
    if int(d.table.max()) < pages and d.table.shape[1] <= c.table.shape[1]:
        g["k_cache"][:pages] = d.k[:pages].cuda()
        g["v_cache"][:pages] = d.v[:pages].cuda()
    g["lengths"].copy_((c.lengths.clamp_max(40)).cuda())
    one.replay()
    two.replay()
    want = call(None)
    assert same_bits(out[0], want) and same_bits(out[1], want)  # some of what is seen now is NaN


def test_on_another_stream():
    c = Cache([60, 1], [100, 700], 8, 2, 128, 16, "bf16")
    g, q, cu = c.gpu(), c.q.cuda(), c.cu.cuda()
    want = gdn.paged_attention(q, **g, cu_seqlens=cu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [gdn.paged_attention(q, **g, cu_seqlens=cu) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(x, want) for x in got)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page_tokens", [(60, 64), (62, 64), (63, 64), (64, 46), (100, 64), (101, 64), (102, 64), (104, 46), (250, 16), (252, 16)])
def test_rows_that_tiled_copies_cannot_fetch(dtype, D, page_tokens):
    """Few rows and many, in pieces of 16, 8, 4 and 2 bytes."""
    Cache([1] * 5, [0, 45, 130, 700, 1000], 16, 2, D, page_tokens, dtype, seed=D).check(tokens=1)
    Cache([300, 1], [100, 700], 16, 2, D, page_tokens, dtype, seed=D + 1).check()


def test_output_and_queries_as_slices_of_one_tensor():
    c = Cache([130, 20], [50, 300], 4, 2, 64, 16, "bf16")
    g, cu, q = c.gpu(), c.cu.cuda(), c.q.cuda()
    want = gdn.paged_attention(q, **g, cu_seqlens=cu)
    both = torch.cat([q, torch.zeros_like(q)], 1)
    gdn.paged_attention(both[:, :4], **g, cu_seqlens=cu, output=both[:, 4:])
    assert torch.equal(both[:, :4], q) and torch.equal(both[:, 4:], want)
    with pytest.raises(gdn.GdnError):
        gdn.paged_attention(both[:, :4], **g, cu_seqlens=cu, output=both[:, 1:5])


def test_refusals():
    c = Cache([4], [10], 4, 2, 64, 16, "bf16")
    g, q = c.gpu(), c.q.cuda()
    call = lambda q=q, **kw: gdn.paged_attention(q, **{**g, **kw})  # noqa: E731
    bad = [dict(cu_seqlens=c.cu.cuda(), tokens_per_seq=1), dict(tokens_per_seq=3), dict(tokens_per_seq=0), dict(seqs=g["seqs"].long()),
           dict(table=g["table"].long()), dict(lengths=g["lengths"][:1]), dict(lengths=g["lengths"].cpu()), dict(window=-1),
           dict(k_cache=g["k_cache"].float()), dict(k_cache=g["k_cache"][:, :, :, :32]), dict(v_cache=g["v_cache"][:, :8]),
           dict(k_cache=g["k_cache"].transpose(2, 3).contiguous().transpose(2, 3)), dict(output=torch.empty(4, 4, 32, device="cuda").bfloat16()),
           dict(output=q), dict(lse=torch.empty(4, 2, device="cuda")), dict(lse=torch.empty(4, 4, device="cuda").half()),
           dict(q=q[:, :3]), dict(q=q.double()), dict(q=q[0]), dict(device_status=torch.zeros(1, device="cuda")), dict(cu_seqlens=c.cu.cuda().float()),
           dict(seqs=None, tokens_per_seq=1, table=g["table"][:2], lengths=g["lengths"][:2])]
    for kw in bad:
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(gdn.GdnError):
        call(scale=float("nan"))
    with pytest.raises(gdn.GdnError):
        call(k_cache=g["k_cache"][:1].expand(g["k_cache"].shape))  # pages that overlap
