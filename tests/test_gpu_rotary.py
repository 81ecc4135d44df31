"""Rotary positions and writes into a paged cache on the GPU, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from attention_testlib import DEV, TYPES, Cache, close_rotary, f64
from oracle import attention as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.build()


def tensors(T, Hq, Hk, D, dtype, seed=0, fused=False):
    g = torch.Generator().manual_seed(seed)
    whole = torch.randn(T, Hq + 2 * Hk, D, generator=g).to(TYPES[dtype]).cuda()
    q, k, v = whole.split([Hq, Hk, Hk], dim=1)
    return (q, k, v) if fused else tuple(t.contiguous() for t in (q, k, v))


def compare(name, got, x, pos, f, dtype, **kw):
    want, size = ref.rotary(f64(x), pos, f64(f), **kw)
    close_rotary(name, got, want, size, TYPES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(128, 128), (128, 64), (256, 64), (100, 50), (80, 80), (7, 2), (64, 0), (72, 24), (1000, 12)])
def test_turn(dtype, interleaved, D, R):
    lens = [130, 0, 20, 1, 3]
    T = sum(lens)
    q, k, _ = tensors(T, 3, 2, D, dtype)
    f = gdn.rotary_frequencies(R)
    cu = torch.tensor([0] + lens).cumsum(0).cuda()
    a, b = gdn.rotary_embedding(q, k, f, cu_seqlens=cu, interleaved=interleaved, magnitude=1.25)
    pos = ref.positions(lens)
    compare("q", a, q, pos, f, dtype, interleaved=interleaved, magnitude=1.25)
    compare("k", b, k, pos, f, dtype, interleaved=interleaved, magnitude=1.25)
    a, b = gdn.rotary_embedding_backward(q, k, f, cu_seqlens=cu.int(), interleaved=interleaved, magnitude=1.25)
    compare("dq", a, q, pos, f, dtype, interleaved=interleaved, magnitude=1.25, inverse=True)
    compare("dk", b, k, pos, f, dtype, interleaved=interleaved, magnitude=1.25, inverse=True)


@pytest.mark.parametrize("T", [1, 2, 700, 20000])
def test_many_and_few_tokens(T):
    q, k, _ = tensors(T, 5, 1, 64, "bf16", fused=True)
    f = gdn.rotary_frequencies(64)
    a, b = gdn.rotary_embedding(q, k, f)
    compare("q", a, q, np.arange(T), f, "bf16")
    compare("k", b, k, np.arange(T), f, "bf16")


def test_far_and_negative_positions():
    pos = [0, 1, -1, 12345678, -7, 2 ** 20 + 1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1]
    q, _, _ = tensors(len(pos), 2, 1, 128, "f32")
    f = gdn.rotary_frequencies(128)
    for dt in (torch.int32, torch.int64):
        a, none = gdn.rotary_embedding(q, None, f, positions=torch.tensor(pos, dtype=dt, device="cuda"))
        assert none is None
        compare("q", a, q, pos, f, "f32")


def test_many_sequences_and_rows_past_them():
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 3, (2500,), generator=g).tolist()
    T = sum(lens) + 5
    _, k, _ = tensors(T, 1, 2, 16, "f32")
    f = gdn.rotary_frequencies(16)
    last = max(i for i, n in enumerate(lens) if n)
    cu = torch.tensor([0] + lens).cumsum(0).int().cuda()
    _, b = gdn.rotary_embedding(None, k, f, cu_seqlens=cu)
    pos = list(ref.positions(lens))
    tail = [T - 5 + j - int(cu[-2]) for j in range(5)]
    assert last <= len(lens) - 1
    compare("k", b, k, pos + tail, f, "f32")


def test_in_place_and_into_wider_rows():
    q, k, _ = tensors(50, 4, 2, 96, "bf16", fused=True)
    q0, k0 = q.clone(), k.clone()
    f = gdn.rotary_frequencies(32)
    a, b = gdn.rotary_embedding(q, k, f, q_out=q, k_out=k)
    assert a is q and b is k
    compare("q", q, q0, np.arange(50), f, "bf16")
    compare("k", k, k0, np.arange(50), f, "bf16")


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients(interleaved):
    f = gdn.rotary_frequencies(6, base=100.0)
    cu = torch.tensor([0, 5, 5, 9], device="cuda")
    q, k, _ = (t.requires_grad_() for t in tensors(9, 2, 1, 10, "f32"))
    a, b = gdn.rotary_embedding(q, k, f, cu_seqlens=cu, interleaved=interleaved, magnitude=0.75)
    wa, wb = torch.randn_like(a), torch.randn_like(b)
    ((a * wa).sum() + (b * wb).sum()).backward()
    pos = ref.positions([5, 0, 4])
    compare("dq", q.grad, wa, pos, f, "f32", interleaved=interleaved, magnitude=0.75, inverse=True)
    compare("dk", k.grad, wb, pos, f, "f32", interleaved=interleaved, magnitude=0.75, inverse=True)
    # against differences of the definition: it is linear, so that one difference is exact but for rounding
    e = np.zeros(q.shape)
    e[6, 1, 3] = 1.0
    d = (ref.rotary(e, pos, f64(f), interleaved, 0.75)[0] * f64(wa)).sum()
    assert abs(float(q.grad[6, 1, 3]) - d) < 1e-5


def test_gradient_of_one_of_two():
    f = gdn.rotary_frequencies(8)
    q, k, _ = tensors(4, 1, 1, 8, "f32")
    k.requires_grad_()
    a, b = gdn.rotary_embedding(q, k, f)
    b.sum().backward()
    compare("dk", k.grad, torch.ones_like(b), np.arange(4), f, "f32", inverse=True)
    assert q.grad is None and not a.grad_fn is None
    q.requires_grad_()
    a, b = gdn.rotary_embedding(q, k, f)
    k.grad = None
    a.sum().backward()
    assert k.grad is None and q.grad is not None


def test_changes_in_place_are_seen_by_autograd():
    f = gdn.rotary_frequencies(8)
    x, _, _ = tensors(4, 1, 1, 8, "f32")
    w = torch.randn(4, 1, 8, device="cuda", requires_grad=True)
    y = w * x
    gdn.rotary_embedding(x, None, f, q_out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.sum().backward()
    y, _ = gdn.rotary_embedding(w, None, f)
    f.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.sum().backward()


# ------------------------------------------------------------------------------------------------ into the cache

def check_append(lens, past, Hq, Hk, D, R, pt, dtype, tokens=None, layout="token", interleaved=False, with_q=True, fused=True, seed=0):
    c = Cache(lens, past, Hq, Hk, D, pt, dtype, seed=seed, layout=layout, fill=7.0)
    T = sum(lens)
    q, k, v = tensors(T, Hq, Hk, D, dtype, seed=seed + 1, fused=fused)
    g = c.gpu()
    f = gdn.rotary_frequencies(R) if R else None
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    how = dict(tokens_per_seq=tokens) if tokens else dict(cu_seqlens=c.cu.cuda())
    out = gdn.cache_append(k, v, **g, **how, q=q if with_q else None, frequencies=f, interleaved=interleaved, magnitude=1.5 if R else 1.0,
                           device_status=word)
    assert int(word) == 0
    pos = ref.positions(lens, c.lengths.tolist(), c.seqs.tolist())
    fr = f64(f) if R else np.zeros(0)
    kw = dict(interleaved=interleaved, magnitude=1.5 if R else 1.0)
    if with_q:
        compare("q", out, q, pos, f if R else torch.zeros(0), dtype, **kw)
    else:
        assert out is None
    want_k, size = ref.rotary(f64(k), pos, fr, **kw)
    wk, sk, wv = f64(c.k), np.zeros(c.k.shape), f64(c.v)
    row = [s for n, s in zip(lens, c.seqs.tolist()) for _ in range(n)]
    for t in range(T):
        if pos[t] < 0:
            continue
        page = int(c.table[row[t], pos[t] // pt])
        wk[page, pos[t] % pt], sk[page, pos[t] % pt], wv[page, pos[t] % pt] = want_k[t], size[t], f64(v[t])
    close_rotary("k_cache", g["k_cache"], wk, sk, TYPES[dtype])
    assert np.array_equal(f64(g["v_cache"]), wv)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("layout", ["token", "head", "wide"])
@pytest.mark.parametrize("D,R,pt", [(128, 128, 16), (64, 32, 1), (100, 50, 7), (33, 0, 64)])
def test_append_ragged(dtype, layout, D, R, pt):
    check_append([13, 0, 20, 1, 64], [5, 3, 0, 100, 63], 4, 2, D, R, pt, dtype, layout=layout)


def test_append_single_tokens():
    check_append([1] * 5, [0, 15, 16, 17, 300], 8, 1, 128, 128, 16, "bf16", tokens=1)
    check_append([3] * 4, [0, 15, 16, 300], 8, 1, 128, 64, 16, "f16", tokens=3, interleaved=True)


def test_append_without_queries_and_from_dense_tensors():
    check_append([40, 2], [0, 9], 4, 4, 64, 64, 16, "bf16", with_q=False, fused=False)


def test_append_reports_what_has_no_page():
    c = Cache([4, 2, 3], [30, 0, 1], 1, 1, 8, 16, "f32", fill=7.0)
    k, v = (torch.randn(9, 1, 8, device="cuda") for _ in range(2))
    for change, bit in (("page", "PAGE"), ("far", "PAGE"), ("seq", "SEQ"), ("length", "PAGE"), ("table", "PAGE")):
        g = c.gpu()
        before = g["k_cache"].clone(), g["v_cache"].clone()
        s = c.seqs.tolist()
        if change == "page":
            g["table"][s[0]] = -1
        elif change == "far":
            g["table"][s[0]] = g["k_cache"].shape[0]
        elif change == "seq":
            g["seqs"][0] = 99
        elif change == "length":
            g["lengths"][s[0]] = -5
        else:
            g["lengths"][s[0]] = 1000
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        gdn.cache_append(k, v, **g, cu_seqlens=c.cu.cuda(), device_status=word)
        assert int(word) & DEV[bit], change
        changed = ((g["k_cache"] != before[0]).any(-1).any(-1).sum(), (g["v_cache"] != before[1]).any(-1).any(-1).sum())
        assert [int(x) for x in changed] == [5, 5], change  # the other two sequences' tokens


def test_append_leaves_padding_alone():
    c = Cache([2, 3], [0, 4], 2, 1, 16, 8, "f32", fill=7.0)
    q, k, v = tensors(9, 2, 1, 16, "f32")
    out = torch.full_like(q, 3.0)
    g = c.gpu()
    gdn.cache_append(k, v, **g, cu_seqlens=c.cu.cuda(), q=q, frequencies=gdn.rotary_frequencies(16), output=out)
    assert bool((out[5:] == 3.0).all()) and not bool((out[:5] == 3.0).any())
    assert int((g["v_cache"] != c.v.cuda()).any(-1).any(-1).sum()) == 5


def test_graph_replay_and_other_streams():
    c = Cache([1] * 4, [3, 40, 0, 17], 4, 2, 64, 16, "bf16", fill=0.0)
    q, k, v = tensors(4, 4, 2, 64, "bf16")
    f = gdn.rotary_frequencies(64)
    g = c.gpu()
    out = torch.empty_like(q)
    call = lambda d: gdn.cache_append(k, v, **d, tokens_per_seq=1, q=q, frequencies=f, output=out)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(g)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(g)
    g["lengths"].copy_((c.lengths + (c.lengths > 0) * 5).clamp_max(g["table"].shape[1] * 16).cuda())
    g["table"].copy_(torch.where(c.table < 0, torch.tensor(0, dtype=torch.int32), c.table).cuda())
    g["k_cache"].zero_()
    graph.replay()
    again = {n: t.clone() for n, t in g.items()}
    again["k_cache"].zero_()
    replayed = out.clone()
    call(again)
    torch.cuda.synchronize()
    assert torch.equal(out, replayed) and torch.equal(again["k_cache"], g["k_cache"])


def test_offsets_past_32_bits():
    """Tokens 20001 elements apart, 120000 of them."""
    T = 120000
    whole = torch.zeros(T, 20001, dtype=torch.bfloat16, device="cuda")
    x = whole[:, :16].view(T, 1, 16)
    rows = [0, 1, 107000, 107375, T - 1]
    x[rows] = torch.randn(len(rows), 1, 16, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    f = gdn.rotary_frequencies(16)
    y, _ = gdn.rotary_embedding(x, None, f)
    compare("q", y[rows], x[rows], rows, f, "bf16")


def test_refusals():
    q, k, v = tensors(6, 2, 1, 16, "bf16")
    f, p = gdn.rotary_frequencies(16), torch.arange(6, device="cuda")
    bad = [dict(positions=p, cu_seqlens=p), dict(positions=p[:5]), dict(positions=p.float()), dict(positions=p.cpu()), dict(frequencies=f.float()),
           dict(frequencies=gdn.rotary_frequencies(18)), dict(frequencies=f.cpu()), dict(frequencies=f[None]), dict(cu_seqlens=p.float()),
           dict(q_out=q[:3]), dict(k_out=k.float()), dict(q=q.double()), dict(k=k[:, :, :8]), dict(k=k[:5]), dict(q=q[0]), dict(q=None, k=None)]
    for kw in bad:
        with pytest.raises(ValueError):
            gdn.rotary_embedding(**{**dict(q=q, k=k, frequencies=f), **kw})
    with pytest.raises(ValueError, match="differentiated"):
        gdn.rotary_embedding(q.requires_grad_(), k, f, k_out=torch.empty_like(k))
    q.requires_grad_(False)
    c = Cache([6], [0], 2, 1, 16, 8, "bf16")
    g = c.gpu()
    for kw in (dict(output=q), dict(v=v[:5]), dict(k=k[:, :, :8]), dict(q=q.float()), dict(cu_seqlens=c.cu.cuda(), tokens_per_seq=6),
               dict(k_cache=g["k_cache"].float()), dict(frequencies=gdn.rotary_frequencies(18))):
        with pytest.raises(ValueError):
            gdn.cache_append(**{**dict(k=k, v=v), **g, **kw})
