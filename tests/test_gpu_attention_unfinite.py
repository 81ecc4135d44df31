"""Attention over a paged cache with values that are infinite or NaN: rows that do not see them are what they are without them, rows
that do have the definition's infinity or NaN in those channels and their values in the others, and no wait runs out on the way."""
import numpy as np
import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from attention_testlib import Cache, attention_bound, f64

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.build()


def put(c, seq, pos, head, channel, value):
    page = int(c.table[c.seqs[seq], pos // c.k.shape[1]])
    c.v[page, pos % c.k.shape[1], head, channel] = value


def check(c, exact_kind=True, **how):
    """Against the definition: infinities and NaN where it has them (its weights are all above zero here), and the values beside them."""
    with np.errstate(invalid="ignore"):
        out, lse, size, products, count = c.want(**how)
        lim = attention_bound(out, size, products, count, c.D, c.dtype)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = f64(gdn.paged_attention(c.q.cuda(), **c.gpu(), cu_seqlens=c.cu.cuda(), device_status=word, **how))
    assert int(word) == 0
    fine = np.isfinite(out)
    assert not np.isfinite(got[~fine]).any()
    assert (np.abs(got[fine] - out[fine]) <= lim[fine]).all()
    if exact_kind:
        assert ((got == out) | (np.isnan(got) & np.isnan(out)))[~fine].all()
    return fine


# (heads, key heads, head size, page tokens): quarters, one and two row tiles, tiled and plain copies
SHAPES = [(4, 2, 64, 16), (8, 2, 128, 64), (16, 2, 256, 64), (4, 4, 128, 16), (32, 2, 64, 16), (4, 2, 100, 16), (8, 2, 128, 20), (4, 2, 250, 12)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,kv_heads,D,page_tokens", SHAPES)
@pytest.mark.parametrize("tokens,past,window", [(1, 700, 0), (4, 700, 0), (4, 700, 300), (1, 3000, 0), (200, 300, 0), (200, 300, 150), (300, 0, 40)])
def test_a_value_at_every_kind_of_place(dtype, heads, kv_heads, D, page_tokens, tokens, past, window):
    """At the first position, within, before and at the window's start, at the chunk's start and at its last token; in one sequence of three."""
    lens, pasts = [tokens, tokens, 1], [past, past, 90]
    for i, pos in enumerate([0, 131, past - 1, past, past + tokens // 2, past + tokens - 1, past + tokens - 1 - window]):
        if not 0 <= pos < past + tokens:
            continue
        c = Cache(lens, pasts, heads, kv_heads, D, page_tokens, dtype, seed=i)
        put(c, 1, pos, kv_heads - 1, (7 * i) % D, (INF, -INF, NAN)[i % 3])
        # where rows see it whole tiles ahead, fp16 weights below 2^-32 of the largest give NaN for an infinity
        check(c, exact_kind=dtype == "bf16" or tokens * heads // kv_heads <= 32, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("tokens", [1, 4])
def test_several_values_of_one_channel(dtype, D, tokens):
    """In one quarter of a tile, in several, in several tiles; of one sign, of both, and NaN: few rows."""
    for places, values in (([3, 5], [INF, INF]), ([3, 40, 100], [INF, INF, INF]), ([3, 70], [INF, -INF]), ([10, 300, 590], [-INF] * 3),
                           ([10, 300, 590], [-INF, NAN, -INF]), ([599], [-INF]), (range(600), [INF] * 600)):
        c = Cache([tokens] * 3, [600 - tokens] * 3, 8, 2, D, 64, dtype, seed=D)
        for pos, value in zip(places, values):
            put(c, 2, pos, 0, 9, value)
        check(c)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,kv_heads,D,page_tokens", SHAPES)
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 100), (False, 100), (False, 0)])
def test_many_values(dtype, heads, kv_heads, D, page_tokens, causal, window):
    """Every token from the middle of a chunk on, in all channels of one head: the rows before them are right."""
    c = Cache([150, 40], [200, 260], heads, kv_heads, D, page_tokens, dtype, seed=4)
    for pos in range(275, 350):
        put(c, 0, pos, 0, slice(None), NAN if pos % 2 else INF)
    fine = check(c, exact_kind=False, causal=causal, window=window)
    assert fine[150:].all() and fine[:75, :heads // kv_heads].all() == causal


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,kv_heads,D,page_tokens", [(16, 4, 128, 64), (4, 1, 256, 64), (4, 2, 128, 20)])
def test_a_long_context(dtype, heads, kv_heads, D, page_tokens):
    """A chunk of 2048 tokens over 129024 whose last token has an infinite value: all other rows, and another sequence's, have the bits that
    they have without it.  The same for a value that all rows see, at position 0, and with few rows."""
    T, past = (2048, 129024) if page_tokens == 64 else (300, 131072 - 300)
    g = torch.Generator("cuda").manual_seed(1)
    pages = -(-(past + T) // page_tokens)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float16)  # noqa: E731
    k, v = r(pages + 40, page_tokens, kv_heads, D), r(pages + 40, page_tokens, kv_heads, D)
    table = torch.full((2, pages), -1, dtype=torch.int32, device="cuda")
    table[0] = torch.randperm(pages, generator=g, device="cuda").int()
    table[1, :40] = torch.arange(pages, pages + 40, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    for n in (T, 4):
        q = r(n + 5, heads, D)
        lengths = torch.tensor([past + n, 300], dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, n, n + 5], dtype=torch.int32, device="cuda")
        call = lambda: gdn.paged_attention(q, k, v, table, lengths, cu_seqlens=cu, device_status=word)  # noqa: E731
        want = call()
        assert bool(torch.isfinite(want).all())
        for pos, first in ((past + n - 1, n - 1), (0, 0)):
            at = int(table[0, pos // page_tokens]), pos % page_tokens, 0, 5
            kept = v[at].clone()
            v[at] = INF
            got = call()
            v[at] = kept
            sees = torch.zeros_like(want, dtype=torch.bool)
            sees[first:n, :heads // kv_heads, 5] = True
            assert torch.equal(got[~sees], want[~sees]) and not bool(torch.isfinite(got[sees]).any()), (n, pos)
    assert int(word) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page_tokens", [(64, 64), (128, 64), (256, 64), (128, 20)])
@pytest.mark.parametrize("tokens", [1, 4, 500])
def test_a_channel_that_is_infinite_throughout(dtype, D, page_tokens, tokens):
    """As where a projection overflows: over 131072 tokens one channel of one head is infinite, another one of both signs, a third NaN."""
    past, heads, kv_heads = 131072 - tokens, 4, 2
    g = torch.Generator("cuda").manual_seed(1)
    pages = -(-(past + tokens) // page_tokens)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float16)  # noqa: E731
    q, k, v = r(tokens, heads, D), r(pages, page_tokens, kv_heads, D), r(pages, page_tokens, kv_heads, D)
    table = torch.randperm(pages, generator=g, device="cuda").int()[None]
    lengths = torch.tensor([past + tokens], dtype=torch.int32, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda: gdn.paged_attention(q, k, v, table, lengths, device_status=word)  # noqa: E731
    want = call()
    v[:, :, 1, 3] = -INF
    v[:, :, 1, 10] = INF
    v[0, :, 1, 10] = -INF
    v[:, :, 1, 63] = NAN
    got = call()
    same = torch.ones_like(want, dtype=torch.bool)
    same[:, 2:, [3, 10, 63]] = False
    assert int(word) == 0 and torch.equal(got[same], want[same])
    if tokens < 500 or dtype == "bf16":  # fp16 weights below 2^-32 of the largest make NaN of an infinity in the products
        assert bool((got[:, 2:, 3] == -INF).all())
    assert not bool(torch.isfinite(got[:, 2:, 3]).any()) and bool(torch.isnan(got[:, 2:, [10, 63]]).all())
