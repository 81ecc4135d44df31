"""Cases of rotary positions (forward and backward), of writing rotated keys and values into a paged cache, and of attention
over that cache (chunks of new tokens, single tokens).

`run` computes an operator in its plain form (elementary torch operations in 32 bits, angles in 64) or, where `own` is
true, with the framework's own calls.  Sizes follow the framework's workloads: the ragged batch 130/0/20/300, batches of
2 x 2048 tokens and of 8 sequences of up to 8192, one sequence of 32768, decode steps of 512 sequences, heads of 128 channels,
key/value pages of 64 tokens and 2 heads.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EIGHT = "5419,1,8192,777,6044,2380,7001,3906"


def _rotary(name, kind, lens, heads, kv_heads, dim, rot, dtype, **kw):
    c = dict(name=name, kind=kind, lens=lens, heads=heads, kv_heads=kv_heads, dim=dim, rot=rot, dtype=dtype, interleaved=False,
             fused=False, first=0, factor=1.0, magnitude=1.0)
    c.update(kw)
    return c


def _attend(name, lens, past, heads, kv_heads, dim, page_tokens, dtype, **kw):
    c = dict(name=name, kind="attend", lens=lens, past=past, tokens=0, heads=heads, kv_heads=kv_heads, dim=dim,
             page_tokens=page_tokens, window=0, dtype=dtype)
    c.update(kw)
    return c


def listed():
    return [
        # the ragged batch with an empty sequence, fp32, half of a head of 100 channels: no power of two; small, latency counts
        _rotary("rotary_ragged_f32", "rotary", "130,0,20,300", 16, 2, 100, 50, "f32"),
        # training: a micro batch of 2 x 2048 tokens, q and k as slices of one projection's output
        _rotary("rotary_2x2048_bf16", "rotary", "2048,2048", 32, 16, 128, 128, "bf16", fused=True),
        # training on one long document far from its start, pairs side by side, half of the head, frequencies of an extended context
        _rotary("rotary_backward_32768_bf16", "rotary_backward", "32768", 32, 16, 128, 64, "bf16", interleaved=True, first=1 << 20,
                factor=16.0, magnitude=1.2772588722239782),
        # decode of a few sequences: pure latency
        _rotary("append_4seq_bf16", "append", "1,1,1,1", 16, 2, 128, 128, "bf16", past="1000,17,0,4095", page_tokens=64),
        # prefill of 8 prompts into pages, slices of one projection's output, a quarter of a head of 256 channels rotated
        _rotary("append_8seq_bf16", "append", EIGHT, 16, 2, 256, 64, "bf16", past="0,0,0,0,0,0,0,0", page_tokens=64, fused=True,
                factor=4.0),
        # the ragged batch as a second chunk, heads of 100 channels, fp32, pages of 16: a small call away from the fast sizes
        _attend("attend_ragged_f32", "130,0,20,300", "500,40,7,0", 16, 2, 100, 16, "f32"),
        # prefill of 8 whole prompts, bf16, 4 query heads a key head
        _attend("attend_8seq_bf16", EIGHT, "0,0,0,0,0,0,0,0", 32, 8, 128, 64, "bf16"),
        # a chunk of one long prompt over what is cached already, fp16, as many key heads as the long workload has
        _attend("attend_2048_of_32768_f16", "2048", "30720", 32, 16, 128, 64, "f16"),
        # a step of a server that mixes one prompt's chunk with decoding sequences, heads of 256
        _attend("attend_mixed_bf16", "1000," + ",".join(["1"] * 63), "2500," + ",".join(str(61 * i) for i in range(63)), 16, 2, 256,
                64, "bf16"),
        # decode of a few sequences: latency
        _attend("decode_4seq_bf16", "", "1000,17,0,4095", 16, 2, 128, 64, "bf16", tokens=1),
        # decode of a full batch, contexts from none to 8128 tokens
        _attend("decode_512seq_bf16", "", ",".join(str((i * 2731) % 512 * 8192 // 516) for i in range(512)), 16, 2, 128, 64, "bf16",
                tokens=1),
        # four speculated tokens of 64 sequences, each layer looks back 1024 tokens only, small pages, heads of 64
        _attend("decode_64seq_x4_window_f16", "", ",".join(str(500 + 117 * i) for i in range(64)), 32, 8, 64, 16, "f16", tokens=4,
                window=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _split(rng, total, most):
    n = min(_log(rng, 1, most), total)
    ends = [0] + sorted(rng.randrange(0, total + 1) for _ in range(n - 1)) + [total]
    return [q - p for p, q in zip(ends, ends[1:])]


def draw(rng):
    kind = rng.choice(["rotary", "rotary_backward", "append", "attend", "attend", "decode", "decode"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    dim = rng.choice([128, 128, 64, 256, 96, 80, rng.randrange(2, 200)])
    kv_heads = rng.choice([1, 2, 2, 4, 8, 16])
    heads = kv_heads * rng.choice([g for g in (1, 2, 3, 4, 6, 8, 16) if g * kv_heads <= 64])
    page_tokens = rng.choice([16, 64, 64, 128, 256, 48, rng.randrange(1, 100)])
    c = dict(heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype)
    if kind in ("rotary", "rotary_backward", "append"):
        rot = max(2, rng.choice([dim, dim, dim // 2, dim // 4]) // 2 * 2)
        one = 2 * (heads + 2 * kv_heads) * dim * BYTES[dtype]
        lens = _split(rng, _log(rng, 1, min(32768, 800_000_000 // one)), 64)
        c.update(kind=kind, lens=",".join(map(str, lens)), rot=rot, interleaved=rng.random() < 0.5,
                 fused=kind != "rotary_backward" and rng.random() < 0.5, first=0, factor=rng.choice([1.0, 1.0, 4.0, 32.0]),
                 magnitude=rng.choice([1.0, 1.0, 1.1386294361119891]))
        if kind == "append":
            c.update(past=",".join(str(rng.choice([0, _log(rng, 1, 8192)])) for _ in lens), page_tokens=page_tokens)
        else:
            c["first"] = rng.choice([0, 0, _log(rng, 1, 1 << 20)])
        return c
    c.update(kind="attend", tokens=0, lens="", page_tokens=page_tokens, window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]))
    bound = 2.0e11 if dtype == "f32" else 1.2e12  # operations of one pass
    if kind == "decode":
        c["tokens"] = rng.choice([1, 1, 1, 2, 4, 5])
        n = _log(rng, 1, 512)
        longest = _log(rng, 16, 131072)
        row = 2 * kv_heads * dim * BYTES[dtype]
        longest = max(16, min(longest, 2_000_000_000 // (row * n), int(bound / (4 * heads * dim * n * c["tokens"]))))
        c["past"] = ",".join(str(rng.randrange(0, longest)) for _ in range(n))
        return c
    lens = _split(rng, _log(rng, 1, 16384), 64)
    deep = _log(rng, 1, 32768)
    past = [rng.choice([0, rng.randrange(0, deep + 1)]) for _ in lens]
    while 4 * dim * heads * sum(n * (p + n) for n, p in zip(lens, past)) > bound:
        lens, past = [n // 2 for n in lens], [p // 2 for p in past]
    c.update(lens=",".join(map(str, lens)), past=",".join(map(str, past)))
    return c


# ------------------------------------------------------------------------------------------------ inputs

def _ints(text):
    return [int(v) for v in text.split(",")] if text else []


def _lens(case):
    """(new tokens, tokens before them) of each sequence."""
    past = _ints(case["past"]) if "past" in case else None
    lens = [case["tokens"]] * len(past) if case.get("tokens") else _ints(case["lens"])
    return lens, past


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _frequencies(rot, factor):
    """Radians a token, in 64 bits: 10000^(-2i/rot); with a factor, a context of 4096 tokens stretched: what turns less than once
    over it is slowed by the factor, what turns 32 times and more is kept, in between there is a ramp."""
    f = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    if factor != 1.0:
        keep = ((4096 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
    return f.cuda()


def _cache(case, g, lengths):
    """Pages in random order, a table of them, and the pools; a third of the pages belongs to nobody here."""
    pt, dt = case["page_tokens"], DTYPES[case["dtype"]]
    need = [-(-n // pt) for n in lengths]
    width, pages = max(1, max(need)), sum(need) + sum(need) // 2 + 1
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    row = torch.tensor(need, device="cuda")
    col = torch.arange(width, device="cuda")[None]
    start = (row.cumsum(0) - row)[:, None]
    table = torch.where(col < row[:, None], order[(start + col).clamp_max(pages - 1)], -1)
    seqs = torch.randperm(len(need) + 3, generator=g, device="cuda")[: len(need)]
    whole = torch.full((len(need) + 3, width), -1, dtype=torch.int32, device="cuda")
    whole[seqs] = table
    length = torch.zeros(len(need) + 3, dtype=torch.int32, device="cuda")
    length[seqs] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    shape = (pages, pt, case["kv_heads"], case["dim"])
    return dict(table=whole, lengths=length, seqs=seqs.to(torch.int32), k_cache=_randn(g, shape, dt), v_cache=_randn(g, shape, dt))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, D, Hq, Hk = DTYPES[case["dtype"]], case["dim"], case["heads"], case["kv_heads"]
    lens, past = _lens(case)
    T = sum(lens)
    s = dict(case=case, lens=lens, past=past)
    s["cu"] = None if case.get("tokens") else torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
    if past is not None:
        s.update(_cache(case, g, [p + n for p, n in zip(past, lens)]))
    if case["kind"] == "attend":
        s["q"] = _randn(g, (T, Hq, D), torch.float32).mul_(1.5).to(dt)
        return s
    if case["fused"]:
        s["q"], s["k"], s["v"] = _randn(g, (T, Hq + 2 * Hk, D), dt).split([Hq, Hk, Hk], dim=1)
    else:
        s["q"], s["k"], s["v"] = (_randn(g, (T, h, D), dt) for h in (Hq, Hk, Hk))
    s["frequencies"] = _frequencies(case["rot"], case["factor"])
    if case["first"]:  # positions of a document's later part, as a loader gives them
        s["positions"] = torch.cat([torch.arange(n) for n in lens]).cuda() + case["first"]
    return s


# ------------------------------------------------------------------------------------------------ one pass

def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["kind"]](state)


def _own_rotary(s):
    import gated_deltanet_chunked_device_gb300 as gdn

    c = s["case"]
    call = gdn.rotary_embedding if c["kind"] == "rotary" else gdn.rotary_embedding_backward
    where = dict(positions=s["positions"]) if "positions" in s else dict(cu_seqlens=s["cu"])
    return call(s["q"], s["k"], s["frequencies"], interleaved=c["interleaved"], magnitude=c["magnitude"], **where)


def _own_append(s):
    import gated_deltanet_chunked_device_gb300 as gdn

    c = s["case"]
    q = gdn.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], seqs=s["seqs"], cu_seqlens=s["cu"],
                         q=s["q"], frequencies=s["frequencies"], interleaved=c["interleaved"], magnitude=c["magnitude"])
    return q, s["k_cache"], s["v_cache"]


def _own_attend(s):
    import gated_deltanet_chunked_device_gb300 as gdn

    c = s["case"]
    how = dict(tokens_per_seq=c["tokens"]) if c["tokens"] else dict(cu_seqlens=s["cu"])
    return gdn.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], seqs=s["seqs"], window=c["window"], **how)


_OWN = dict(rotary=_own_rotary, rotary_backward=_own_rotary, append=_own_append, attend=_own_attend)


def _token_positions(s):
    """Each packed token's position, on the device."""
    if "positions" in s:
        return s["positions"]
    cu = s["cu"].long()
    t = torch.arange(s["q"].shape[0], device="cuda")
    i = torch.searchsorted(cu[1:], t, right=True)
    pos = t - cu[i]
    if s["past"] is not None:
        pos = pos + s["lengths"].long()[s["seqs"].long()[i]] - (cu[i + 1] - cu[i])
    return pos


def _rotate(x, cos, sin, interleaved):
    half, rot = cos.shape[1], 2 * cos.shape[1]
    w = x.float()
    cos, sin = cos[:, None], sin[:, None]
    a, b = (w[..., 0:rot:2], w[..., 1:rot:2]) if interleaved else (w[..., :half], w[..., half:rot])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([turned, w[..., rot:]], -1).to(x.dtype)


def _angles(s):
    a = _token_positions(s).double()[:, None] * s["frequencies"]
    m = s["case"]["magnitude"]
    return (a.cos() * m).float(), (a.sin() * m).float()


def _plain_rotary(s):
    cos, sin = _angles(s)
    if s["case"]["kind"] == "rotary_backward":
        sin = -sin
    return tuple(_rotate(s[n], cos, sin, s["case"]["interleaved"]) for n in ("q", "k"))


def _plain_append(s):
    cos, sin = _angles(s)
    inter, pt = s["case"]["interleaved"], s["case"]["page_tokens"]
    pos = _token_positions(s)
    i = torch.searchsorted(s["cu"].long()[1:], torch.arange(pos.numel(), device="cuda"), right=True)
    page = s["table"][s["seqs"].long()[i], pos // pt].long()
    s["k_cache"][page, pos % pt] = _rotate(s["k"], cos, sin, inter)
    s["v_cache"][page, pos % pt] = s["v"]
    return _rotate(s["q"], cos, sin, inter), s["k_cache"], s["v_cache"]


def _plain_softmax_values(scores, seen, v):
    """Softmax over the last axis where `seen`, times v; rows that see nothing are zero."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)


def _seen(at, keys, window):
    ok = keys <= at[..., None]
    return ok & (keys > at[..., None] - window) if window else ok


def _plain_attend(s):
    c, q = s["case"], s["q"]
    Hq, Hk, D, pt, window = c["heads"], c["kv_heads"], c["dim"], c["page_tokens"], c["window"]
    G, scale = Hq // Hk, 1.0 / math.sqrt(D)
    out = torch.empty_like(q)
    if c["tokens"]:  # equal numbers of tokens: sequences side by side, in groups that share a padded length
        m, N = c["tokens"], len(s["lens"])
        rows = s["table"][s["seqs"].long()]
        length = s["lengths"][s["seqs"].long()].long()
        qs, outs = q.view(N, m, Hk, G, D), out.view(N, m, Hk, G, D)
        step = max(1, 1_000_000_000 // (4 * Hk * D * max(p + m for p in s["past"])))
        for i in range(0, N, step):
            e = min(N, i + step)
            L = max(p + m for p in s["past"][i:e])
            pages = rows[i:e, : -(-L // pt)].clamp_min(0).long()
            k, v = (t[pages].flatten(1, 2)[:, :L].float().permute(0, 2, 1, 3) for t in (s["k_cache"], s["v_cache"]))
            w = qs[i:e].float().permute(0, 2, 1, 3, 4).flatten(2, 3)
            at = length[i:e, None] - m + torch.arange(m, device="cuda")
            seen = _seen(at, torch.arange(L, device="cuda"), window)[:, None, :, None].expand(-1, 1, -1, G, -1).flatten(2, 3)
            o = _plain_softmax_values(torch.matmul(w, k.transpose(-1, -2)) * scale, seen, v)
            outs[i:e] = o.view(e - i, Hk, m, G, D).permute(0, 2, 1, 3, 4).to(q.dtype)
        return out
    first = 0
    for i, (n, p) in enumerate(zip(s["lens"], s["past"])):
        L = n + p
        if n:
            pages = s["table"][s["seqs"][i].long(), : -(-L // pt)].long()
            k, v = (t[pages].flatten(0, 1)[:L].float().transpose(0, 1) for t in (s["k_cache"], s["v_cache"]))
        for b in range(0, n, 512):
            e = min(n, b + 512)
            lo, hi = max(0, p + b - window + 1) if window else 0, p + e
            w = q[first + b: first + e].float().view(e - b, Hk, G, D).permute(1, 0, 2, 3).flatten(1, 2)
            seen = _seen(torch.arange(p + b, p + e, device="cuda"), torch.arange(lo, hi, device="cuda"), window)
            seen = seen[:, None].expand(-1, G, -1).flatten(0, 1)
            o = _plain_softmax_values(torch.matmul(w, k[:, lo:hi].transpose(-1, -2)) * scale, seen, v[:, lo:hi])
            out[first + b: first + e] = o.view(Hk, e - b, G, D).permute(1, 0, 2, 3).flatten(1, 2).to(q.dtype)
        first += n
    return out


_PLAIN = dict(rotary=_plain_rotary, rotary_backward=_plain_rotary, append=_plain_append, attend=_plain_attend)


# ------------------------------------------------------------------------------------------------ accounting and values

def _pairs(n, p, window):
    """(query, key) pairs that see each other, and keys that some query sees."""
    if not n:
        return 0, 0
    if not window:
        return n * p + n * (n + 1) // 2, p + n
    full = max(0, min(n, p + n - window + 1))  # queries that see `window` keys: the last ones
    short = n - full
    return full * window + short * p + short * (short + 1) // 2, p + n - max(0, p + 1 - window)


def work(case):
    Hq, Hk, D, e = case["heads"], case["kv_heads"], case["dim"], BYTES[case["dtype"]]
    lens, past = _lens(case)
    T = sum(lens)
    if case["kind"] == "attend":
        seen = [_pairs(n, p, case["window"]) for n, p in zip(lens, past)]
        return dict(bytes=2 * T * Hq * D * e + 2 * sum(k for _, k in seen) * Hk * D * e, flops=4 * D * Hq * sum(n for n, _ in seen))
    heads = Hq + Hk * (2 if case["kind"] == "append" else 1)
    return dict(bytes=2 * T * heads * D * e + 8 * (T if case["first"] else len(lens)), flops=3 * T * (Hq + Hk) * case["rot"])


def exact(case, seed):
    """Rotations as complex products, attention key by key through the table, in 64 bits."""
    s = prepare(case, seed)
    lens, past = s["lens"], s["past"]
    if case["kind"] == "attend":
        return None if work(case)["flops"] > 3e12 else _exact_attend(s)
    start = [0] * len(lens) if past is None else past
    pos = torch.tensor([p + j for n, p in zip(lens, start) for j in range(n)], dtype=torch.float64, device="cuda") + case["first"]
    turn = torch.polar(torch.full_like(pos, case["magnitude"])[:, None].expand(-1, case["rot"] // 2).contiguous(),
                       pos[:, None] * s["frequencies"])[:, None]
    if case["kind"] == "rotary_backward":
        turn = turn.conj()

    def rotated(x):
        w = x.double()
        r = w[..., : case["rot"]]
        pairs = r.unflatten(-1, (-1, 2)) if case["interleaved"] else r.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, w[..., case["rot"]:]], -1)

    if case["kind"] != "append":
        return rotated(s["q"]), rotated(s["k"])
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    k, v, at = rotated(s["k"]), s["v"].double(), 0
    for i, (n, p) in enumerate(zip(lens, past)):
        token = torch.arange(p, p + n, device="cuda")
        page = s["table"][s["seqs"][i].long(), token // case["page_tokens"]].long()
        k_cache[page, token % case["page_tokens"]] = k[at: at + n]
        v_cache[page, token % case["page_tokens"]] = v[at: at + n]
        at += n
    return rotated(s["q"]), k_cache, v_cache


def _exact_attend(s):
    c = s["case"]
    G, pt = c["heads"] // c["kv_heads"], c["page_tokens"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for i, (n, p) in enumerate(zip(s["lens"], s["past"])):
        token = torch.arange(p + n, device="cuda")
        page = s["table"][s["seqs"][i].long()].long()[token // pt]
        k, v = s["k_cache"][page, token % pt], s["v_cache"][page, token % pt]
        for b in range(0, n, 1024):
            e = min(n, b + 1024)
            far = (token[None, : p + e] - torch.arange(p + b, p + e, device="cuda")[:, None])  # key's position less the query's
            hidden = (far > 0) | (far <= -c["window"] if c["window"] else False)
            for h in range(c["heads"]):
                z = torch.einsum("td,sd->ts", s["q"][at + b: at + e, h].double(), k[: p + e, h // G].double()) / c["dim"] ** 0.5
                out[at + b: at + e, h] = torch.softmax(z.masked_fill(hidden, -math.inf), 1) @ v[: p + e, h // G].double()
        at += n
    return out
