"""Cases of the gated linear recurrence (forward, backward, decode step) and of the cache's page operators.

`run` computes an operator in its plain form (elementary torch operations in 32 bits) or, where `own` is true, with
the framework's own calls.  Sizes follow the framework's workloads: 16 or 32 heads of 128 channels, the ragged batch
130/0/20/300, the batches of 2 x 2048 tokens and of 8 sequences of up to 8192, one sequence of 32768, decode steps of 512
sequences on a pool of 1024 rows, states of 128 x 128 a head.
"""
import math

import torch

own = False

TILE = 64  # packed tokens between two saved states of the recurrence's forward pass
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # the ragged batch with an empty sequence, fp32, gates per head as the delta rule has them, states from a pool:
        # a small prompt batch, where latency counts; 100 channels a head: no power of two
        dict(name="forward_ragged_f32", kind="forward", lens="130,0,20,300", heads=16, dim=100, dtype="f32", gate_dtype="f32",
             gates="head", has_b=True, fused=False, n_pool=64),
        # 8 prompts of random length, gates per channel, x, a and b as slices of one projection's output: a prefill step
        dict(name="forward_8seq_bf16", kind="forward", lens="5419,1,8192,777,6044,2380,7001,3906", heads=32, dim=128, dtype="bf16",
             gate_dtype="bf16", gates="channel", has_b=True, fused=True, n_pool=0),
        # training: a micro batch of 2 x 2048 tokens, gates per channel in fp32 (decays near one), bf16 activations
        dict(name="backward_2x2048_bf16", kind="backward", lens="2048,2048", heads=16, dim=128, dtype="bf16", gate_dtype="f32",
             gates="channel", has_b=True, fused=False, n_pool=0),
        # training on one long document, gates per head
        dict(name="backward_32768_bf16", kind="backward", lens="32768", heads=32, dim=128, dtype="bf16", gate_dtype="f32",
             gates="head", has_b=True, fused=False, n_pool=0),
        # decode of a few sequences, one token each: pure latency
        dict(name="decode_4seq_bf16", kind="decode", seqs=4, tokens=1, heads=16, dim=128, dtype="bf16", gate_dtype="bf16",
             gates="channel", has_b=True, n_pool=64),
        # decode of a full batch with four tokens each (speculated), on the pool of 1024 rows
        dict(name="decode_512seq_x4_bf16", kind="decode", seqs=512, tokens=4, heads=32, dim=128, dtype="bf16", gate_dtype="bf16",
             gates="channel", has_b=True, n_pool=1024),
        # a scheduler's step on a small pool of recurrence states: admit 2, fork 4, drop them all: latency
        dict(name="turn_states_small", kind="turn", pages=64, buffers=1, page_elems=16 * 128, dtype="f32", seqs=64, max_pages=1,
             page_tokens=0, live=24, admit=2, fork=4),
        # the same on the delta rule's states (32 heads of 128 x 128, fp32, 2 MiB a row): 64 answers forked from 8 prompts
        dict(name="turn_states_gdn", kind="turn", pages=1024, buffers=1, page_elems=32 * 128 * 128, dtype="f32", seqs=1024,
             max_pages=1, page_tokens=0, live=512, admit=32, fork=64),
        # closing the holes of a key/value cache: 8 buffers (K and V of 4 layers) of 64-token pages, half of them live
        dict(name="compact_kv_bf16", kind="compact", pages=8191, buffers=8, page_elems=64 * 2 * 128, dtype="bf16", seqs=129, max_pages=64,
             live=4095, moves=1999),
        # a small pool of states after some sequences ended
        dict(name="compact_states_small", kind="compact", pages=64, buffers=2, page_elems=16 * 128, dtype="f32", seqs=64, max_pages=1,
             live=29, moves=7),
        # restoring checkpoints into the rows of a state pool: 384 rows of the delta rule's states
        dict(name="copy_checkpoints_bf16", kind="copy", pages=1024, src_pages=512, buffers=1, page_elems=32 * 128 * 128, dtype="bf16",
             pairs=384),
        # a few rows of an odd size (7 heads of 43 fp16 channels: 602 bytes), two buffers
        dict(name="copy_odd_small_f16", kind="copy", pages=100, src_pages=37, buffers=2, page_elems=7 * 43, dtype="f16", pairs=11),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["forward", "backward", "decode", "turn", "compact", "copy"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if kind in ("forward", "backward", "decode"):
        dim = rng.choice([128, 128, 64, 256, 96, rng.randrange(1, 200)])
        heads = max(1, min(64, _log(rng, 128, 4096) // dim))
        c = dict(kind=kind, heads=heads, dim=dim, dtype=dtype, gate_dtype=rng.choice([dtype, "f32"]),
                 gates=rng.choice(["channel", "head"]), has_b=rng.random() < 0.8)
        if kind == "decode":
            seqs = _log(rng, 1, 512)
            c.update(seqs=seqs, tokens=rng.choice([1, 1, 2, 4, 5]), n_pool=seqs + _log(rng, 1, 512))
            return c
        one = work(dict(c, kind=kind, lens="1000"))["bytes"] // 1000  # bytes a token, about
        total = _log(rng, 1, min(32768, 900_000_000 // one))
        n = min(_log(rng, 1, 64), total)
        cuts = sorted(rng.randrange(0, total + 1) for _ in range(n - 1))
        ends = [0] + cuts + [total]
        c["lens"] = ",".join(str(q - p) for p, q in zip(ends, ends[1:]))
        c["fused"] = kind == "forward" and c["gates"] == "channel" and c["gate_dtype"] == dtype and rng.random() < 0.5
        c["n_pool"] = n + _log(rng, 1, 64) if kind == "forward" and rng.random() < 0.5 else 0
        return c
    elems = _log(rng, 100, 32 * 128 * 128)
    if rng.random() < 0.7:
        elems = (elems + 127) // 128 * 128
    buffers = rng.choice([1, 1, 2, 4, 8])
    per_page = buffers * elems * BYTES[dtype]
    pages = max(8, min(8192, _log(rng, 8, 8192), (1 << 30) // per_page))
    if kind == "copy":
        src = max(1, _log(rng, 1, pages))
        return dict(kind=kind, pages=pages, src_pages=src, buffers=buffers, page_elems=elems, dtype=dtype,
                    pairs=_log(rng, 1, pages // 2))
    if kind == "compact":
        live = rng.randrange(1, pages)
        seqs = _log(rng, 1, 512)
        return dict(kind=kind, pages=pages, buffers=buffers, page_elems=elems, dtype=dtype, seqs=seqs,
                    max_pages=-(-pages // seqs), live=live, moves=rng.randrange(0, min(live, pages - live) + 1))
    page_tokens = rng.choice([0, 16, 64])
    max_pages = rng.choice([1, 2]) if page_tokens == 0 else _log(rng, 1, 32)
    live = max(1, min(pages // (4 * max_pages), 256))
    fork, admit = _log(rng, 1, live), _log(rng, 1, live)
    return dict(kind=kind, pages=max(pages, 4 * max_pages), buffers=buffers, page_elems=elems, dtype=dtype, seqs=live + fork + admit,
                max_pages=max_pages, page_tokens=page_tokens, live=live, admit=admit, fork=fork)


# ------------------------------------------------------------------------------------------------ inputs

def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _gate(g, shape, kind):
    r = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    # decays: exp(-softplus / 16), most of them near one; input gates: a sigmoid
    return torch.exp(-torch.nn.functional.softplus(r) / 16.0) if kind == "a" else torch.sigmoid(r)


def _pool_ids(g, n, count):
    return torch.randperm(n, generator=g, device="cuda")[:count].to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = case["kind"]
    if kind in ("forward", "backward", "decode"):
        return _prepare_recurrence(case, g)
    dt = DTYPES[case["dtype"]]
    pools = [_randn(g, (case["pages"], case["page_elems"]), dt) for _ in range(case["buffers"])]
    if kind == "copy":
        src = [_randn(g, (case["src_pages"], case["page_elems"]), dt) for _ in range(case["buffers"])]
        return dict(case=case, src_pools=src, pools=pools, dst=_pool_ids(g, case["pages"], case["pairs"]),
                    src=torch.randint(0, case["src_pages"], (case["pairs"],), generator=g, device="cuda", dtype=torch.int32))
    if kind == "compact":
        return dict(case=case, pools=pools, **_prepare_compact(case, g))
    return dict(case=case, pools=pools, **_prepare_turn(case, g))


def _prepare_recurrence(case, g):
    H, D, dt, gdt = case["heads"], case["dim"], DTYPES[case["dtype"]], DTYPES[case["gate_dtype"]]
    if case["kind"] == "decode":
        lens = [case["tokens"]] * case["seqs"]
    else:
        lens = [int(v) for v in case["lens"].split(",")]
    T, N = sum(lens), len(lens)
    gshape = (T, H, D) if case["gates"] == "channel" else (T, H)
    if case.get("fused"):
        x, a, b = torch.empty(T, 3, H, D, device="cuda", dtype=dt).unbind(1)
    else:
        x, a, b = (torch.empty(s, device="cuda", dtype=t) for s, t in (((T, H, D), dt), (gshape, gdt), (gshape, gdt)))
    x.copy_(_randn(g, (T, H, D), dt))
    a.copy_(_gate(g, gshape, "a"))
    b.copy_(_gate(g, gshape, "b"))
    s = dict(case=case, lens=lens, x=x, a=a, b=b if case["has_b"] else None, state_indices=None)
    ends = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32)
    s["cu"] = ends.cuda()
    if case["n_pool"]:
        s["pool"] = 0.5 * _randn(g, (case["n_pool"], H, D), torch.float32)
        s["pool_out"] = s["pool"].clone()
        s["state_indices"] = _pool_ids(g, case["n_pool"], N)
    else:
        s["pool"] = 0.5 * _randn(g, (N, H, D), torch.float32)
    if case["kind"] == "backward":
        s["dy"] = _randn(g, (T, H, D), dt)
        s["d_final"] = _randn(g, (N, H, D), torch.float32)
        # what the forward pass has left: the state after every 64th packed token
        h = _plain_states(s)
        rows = torch.arange(TILE - 1, TILE * (-(-T // TILE)), TILE, device="cuda").clamp_max(max(T - 1, 0))
        s["tile_states"] = h[rows].contiguous() if T else h
    return s


def _prepare_turn(case, g):
    P, S, M, live = case["pages"], case["seqs"], case["max_pages"], case["live"]
    pt = case["page_tokens"]
    ids = torch.arange(live, device="cuda")
    if pt:  # a partly filled last page each: it is what a fork copies
        used = torch.randint(1, M + 1, (live,), generator=g, device="cuda")
        left = torch.randint(1, pt, (live,), generator=g, device="cuda")
        lengths = (used - 1) * pt + left
    else:
        used, lengths = torch.full((live,), M, device="cuda"), torch.randint(1, 9999, (live,), generator=g, device="cuda")
    seq_ids = torch.randperm(S, generator=g, device="cuda")
    pages = torch.randperm(P, generator=g, device="cuda")[: live * M].view(live, M)
    rows = torch.where(torch.arange(M, device="cuda")[None] < used[:, None], pages, -1)
    table = torch.full((S, M), -1, device="cuda", dtype=torch.int32)
    table[seq_ids[:live]] = rows.to(torch.int32)
    refs = torch.zeros(P + 1, device="cuda", dtype=torch.int32)
    refs[torch.where(rows >= 0, rows, P).view(-1)] = 1
    length = torch.zeros(S, device="cuda", dtype=torch.int32)
    length[seq_ids[:live]] = lengths.to(torch.int32)
    parents = seq_ids[torch.randint(0, max(1, -(-live // 8)), (case["fork"],), generator=g, device="cuda") % live]
    return dict(table=table, refcounts=refs[:P].contiguous(), lengths=length, parents=parents.to(torch.int32),
                children=seq_ids[live: live + case["fork"]].to(torch.int32),
                new=seq_ids[live + case["fork"]: live + case["fork"] + case["admit"]].to(torch.int32),
                counts=torch.randint(1, M + 1, (case["admit"],), generator=g, device="cuda", dtype=torch.int32),
                drop=seq_ids[live: live + case["fork"] + case["admit"]].to(torch.int32))


def _prepare_compact(case, g):
    P, S, M, live, moves = case["pages"], case["seqs"], case["max_pages"], case["live"], case["moves"]
    low = torch.randperm(live, generator=g, device="cuda")[: live - moves]  # the others below `live` are the holes
    high = live + torch.randperm(P - live, generator=g, device="cuda")[:moves]
    pages = torch.cat([low, high])[torch.randperm(live, generator=g, device="cuda")]
    table = torch.full((S * M,), -1, device="cuda", dtype=torch.int32)
    table[torch.randperm(S * M, generator=g, device="cuda")[:live]] = pages[: S * M].to(torch.int32)
    refs = torch.zeros(P, device="cuda", dtype=torch.int32)
    refs[pages] = torch.randint(1, 4, (live,), generator=g, device="cuda", dtype=torch.int32)
    return dict(table=table.view(S, M), refcounts=refs, table_out=torch.empty(S, M, device="cuda", dtype=torch.int32),
                refcounts_out=torch.empty_like(refs))


# ------------------------------------------------------------------------------------------------ one pass

def run(state):
    kind = state["case"]["kind"]
    if own:
        return _OWN[kind](state)
    return _PLAIN[kind](state)


def _own_forward(s):
    import gated_deltanet_chunked_device_gb300 as gdn

    if s["state_indices"] is not None:
        return gdn.gated_linear_recurrence(s["x"], s["a"], s["b"], initial_state=s["pool"], state_indices=s["state_indices"],
                                           output_state=s["pool_out"], output_final_state=True, cu_seqlens=s["cu"])
    return gdn.gated_linear_recurrence(s["x"], s["a"], s["b"], initial_state=s["pool"], output_final_state=True,
                                       cu_seqlens=s["cu"])


def _own_backward(s):
    import gated_deltanet_chunked_device_gb300 as gdn

    return gdn.gated_linear_recurrence_backward(s["dy"], s["x"], s["a"], s["b"], tile_states=s["tile_states"],
                                                initial_state=s["pool"], d_final_state=s["d_final"], cu_seqlens=s["cu"])


def _own_decode(s):
    import gated_deltanet_chunked_device_gb300 as gdn

    return gdn.gated_linear_recurrence_decode(s["x"], s["a"], s["b"], initial_state=s["pool"], output_state=s["pool_out"],
                                              state_indices=s["state_indices"], tokens_per_seq=s["case"]["tokens"])


def _own_turn(s):
    import gated_deltanet_chunked_device_gb300 as gdn

    book = s["table"], s["refcounts"]
    admitted = gdn.cache_reserve(*book, s["new"], s["counts"])
    forked = gdn.cache_fork(s["pools"], *book, s["parents"], s["children"], page_tokens=s["case"]["page_tokens"], lengths=s["lengths"])
    gdn.cache_free(*book, s["drop"], lengths=s["lengths"])
    return admitted, forked, s["pools"], s["table"], s["refcounts"], s["lengths"]


def _own_compact(s):
    import gated_deltanet_chunked_device_gb300 as gdn

    remap, n_live = gdn.cache_compact(s["pools"], s["table"], s["refcounts"], table_out=s["table_out"],
                                      refcounts_out=s["refcounts_out"])
    return remap, n_live, s["table_out"], s["refcounts_out"], s["pools"]


def _own_copy(s):
    import gated_deltanet_chunked_device_gb300 as gdn

    gdn.cache_copy(s["src_pools"], s["pools"], s["src"], s["dst"])
    return s["pools"]


_OWN = dict(forward=_own_forward, backward=_own_backward, decode=_own_decode, turn=_own_turn, compact=_own_compact, copy=_own_copy)


def _wide(gate, D):
    return gate.float() if gate.dim() == 3 else gate.float()[:, :, None].expand(-1, -1, D)


def _scan(a, u, reverse=False):
    """h_t = a_t h_{t-1} + u_t along dim 0 (from the end with `reverse`), by doubling: log2(T) steps of whole tensors."""
    T, k = u.shape[0], 1
    a, u = a.contiguous(), u.contiguous()
    while k < T:
        if reverse:
            u = torch.cat([torch.addcmul(u[:-k], a[:-k], u[k:]), u[-k:]])
            a = torch.cat([a[:-k] * a[k:], a[-k:]])
        else:
            u = torch.cat([u[:k], torch.addcmul(u[k:], a[k:], u[:-k])])
            a = torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    return u


def _bounds(s):
    """Per packed token: whether it is the first, and the last, of its sequence; per sequence: whether it is empty, its last token."""
    cu, T = s["cu"].long(), s["x"].shape[0]
    full = cu[1:] > cu[:-1]
    first = torch.zeros(T + 1, device="cuda", dtype=torch.bool)
    last = torch.zeros(T + 1, device="cuda", dtype=torch.bool)
    first[torch.where(full, cu[:-1], T)] = True
    last[torch.where(full, cu[1:] - 1, T)] = True
    return first[:T], last[:T], full, torch.where(full, cu[1:] - 1, 0)


def _spread(rows, cu, full, T, at_end):
    """[T, H, D] with each non-empty sequence's row at its first (or last) token, zeros elsewhere."""
    where = torch.where(full, cu[1:].long() - 1 if at_end else cu[:-1].long(), T)
    out = torch.zeros(T + 1, *rows.shape[1:], device="cuda", dtype=torch.float32)
    out[where] = rows.float()
    return out[:T]


def _start(s):
    return s["pool"] if s["state_indices"] is None else s["pool"][s["state_indices"].long()]


def _plain_states(s):
    x = s["x"].float()
    T, H, D = x.shape
    a = _wide(s["a"], D)
    u = x if s["b"] is None else x * _wide(s["b"], D)
    first, _, full, _ = _bounds(s)
    u = u + a * _spread(_start(s), s["cu"], full, T, False)
    return _scan(torch.where(first[:, None, None], torch.zeros_like(a), a), u)


def _plain_forward(s):
    h = _plain_states(s)
    _, _, full, at = _bounds(s)
    start = _start(s)
    final = torch.where(full[:, None, None], h[at], start) if h.shape[0] else start
    if s["state_indices"] is not None:
        s["pool_out"][s["state_indices"].long()] = final
        final = s["pool_out"]
    return h.to(s["x"].dtype), final


def _plain_backward(s):
    x, dy = s["x"].float(), s["dy"].float()
    T, H, D = x.shape
    h = _plain_states(s)
    a = _wide(s["a"], D)
    b = None if s["b"] is None else _wide(s["b"], D)
    first, last, full, _ = _bounds(s)
    fm = first[:, None, None]
    before = torch.where(fm, _spread(s["pool"], s["cu"], full, T, False), torch.cat([h[:1], h[:-1]]))
    # g_t = dy_t + a_{t+1} g_{t+1} inside a sequence, from its final state's gradient at the last token
    a_next = torch.where(last[:, None, None], torch.zeros_like(a), torch.cat([a[1:], a[:1]]))
    gr = _scan(a_next, dy + _spread(s["d_final"], s["cu"], full, T, True), reverse=True)
    da, dx = gr * before, gr if b is None else gr * b
    db = None if b is None else gr * x
    if s["a"].dim() == 2:
        da, db = da.sum(2), None if db is None else db.sum(2)
    starts = torch.where(full, s["cu"][:-1].long(), 0)
    d0 = torch.where(full[:, None, None], (a * gr)[starts], s["d_final"]) if T else s["d_final"]
    gt = s["a"].dtype
    return dx.to(s["x"].dtype), da.to(gt), None if db is None else db.to(gt), d0


def _plain_decode(s):
    m, D = s["case"]["tokens"], s["x"].shape[2]
    x, a = s["x"].float(), _wide(s["a"], D)
    u = x if s["b"] is None else x * _wide(s["b"], D)
    a, u = (t.reshape(-1, m, *t.shape[1:]) for t in (a, u))
    rows = s["state_indices"].long()
    h, y = s["pool"][rows], torch.empty_like(u)
    for j in range(m):
        h = torch.addcmul(u[:, j], a[:, j], h)
        y[:, j] = h
    s["pool_out"][rows] = h
    return y.reshape(x.shape).to(s["x"].dtype), s["pool_out"]


def _free_pages(refcounts):
    return torch.sort((refcounts != 0).to(torch.int32), stable=True).indices, (refcounts == 0).sum()


def _plain_turn(s):
    table, refs, lengths, pt = s["table"], s["refcounts"], s["lengths"], s["case"]["page_tokens"]
    M, col = table.shape[1], torch.arange(table.shape[1], device="cuda")[None]

    def take(need):
        order, free = _free_pages(refs)
        served = need.sum(1).cumsum(0) <= free  # in order, up to the first that does not fit
        need = need & served[:, None]
        rank = need.view(-1).to(torch.int32).cumsum(0) - 1
        pages = order[rank.clamp(0, order.numel() - 1)].view(need.shape)
        refs.index_add_(0, pages.view(-1), need.view(-1).to(torch.int32))
        return need, pages.to(torch.int32), served

    # admit
    rows = table[s["new"].long()]
    need, pages, _ = take((rows < 0) & (col < s["counts"][:, None]))
    admitted = torch.where(need, pages, rows)
    table[s["new"].long()] = admitted
    # fork
    rows, length = table[s["parents"].long()], lengths[s["parents"].long()]
    if pt:
        n = (length + pt - 1) // pt
        copied = (col == n[:, None] - 1) & (length % pt != 0)[:, None]
        shared = (col < n[:, None]) & ~copied
    else:
        copied, shared = rows >= 0, torch.zeros_like(rows, dtype=torch.bool)
    got, pages, served = take(copied)
    shared = shared & served[:, None]
    forked = torch.where(shared, rows, torch.where(got, pages, -1))
    table[s["children"].long()] = forked
    refs.index_add_(0, rows.clamp_min(0).view(-1).long(), shared.view(-1).to(torch.int32))
    lengths[s["children"].long()] = torch.where(served, length, 0)
    at = (n.long() - 1).clamp_min(0)[:, None] if pt else col.expand(rows.shape[0], M)
    src = rows.gather(1, at).view(-1).long().clamp_min(0)
    dst = torch.where(got, pages, rows).gather(1, at).view(-1).long().clamp_min(0)
    for p in s["pools"]:
        p[dst] = p[src]
    # drop
    gone = table[s["drop"].long()]
    refs.index_add_(0, gone.clamp_min(0).view(-1).long(), -(gone >= 0).view(-1).to(torch.int32))
    table[s["drop"].long()] = -1
    lengths[s["drop"].long()] = 0
    return admitted, forked, s["pools"], table, refs, lengths


def _plain_compact(s):
    table, refs = s["table"], s["refcounts"]
    live = refs > 0
    idx = torch.arange(refs.numel(), device="cuda")
    n_live = live.sum()
    holes, movers = (~live & (idx < n_live)).nonzero().view(-1), (live & (idx >= n_live)).nonzero().view(-1)
    remap = torch.where(live, idx, -1).to(torch.int32)
    remap[movers] = holes.to(torch.int32)
    s["table_out"].copy_(torch.where(table >= 0, remap[table.clamp_min(0).long()], -1))
    out = torch.where(idx < n_live, refs, 0)
    out[holes] = refs[movers]
    s["refcounts_out"].copy_(out)
    for p in s["pools"]:
        p[holes] = p[movers]
    return remap, n_live.to(torch.int32).view(1), s["table_out"], s["refcounts_out"], s["pools"]


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for p, q in zip(s["pools"], s["src_pools"]):
        p[dst] = q[src]
    return s["pools"]


_PLAIN = dict(forward=_plain_forward, backward=_plain_backward, decode=_plain_decode, turn=_plain_turn, compact=_plain_compact,
              copy=_plain_copy)


# ------------------------------------------------------------------------------------------------ accounting and values

def work(case):
    kind = case["kind"]
    if kind in ("forward", "backward", "decode"):
        H, D, e, ge = case["heads"], case["dim"], BYTES[case["dtype"]], BYTES[case["gate_dtype"]]
        lens = [case["tokens"]] * case["seqs"] if kind == "decode" else [int(v) for v in case["lens"].split(",")]
        T, N = sum(lens), len(lens)
        tok, gate = T * H * D * e, T * H * (D if case["gates"] == "channel" else 1) * ge * (2 if case["has_b"] else 1)
        state = N * H * D * 4
        if kind == "backward":  # x, dy, dx; the gates and their gradients; initial and final states' gradients, the saved states
            return dict(bytes=3 * tok + 2 * gate + 3 * state + (T // TILE) * H * D * 4, flops=9 * T * H * D)
        return dict(bytes=2 * tok + gate + 2 * state + 4 * (N + 1), flops=3 * T * H * D)
    page = case["buffers"] * case["page_elems"] * BYTES[case["dtype"]]
    if kind == "copy":  # a source page is read once however often it is copied
        return dict(bytes=(min(case["pairs"], case["src_pages"]) + case["pairs"]) * page + 8 * case["pairs"], flops=0)
    table = 4 * case["max_pages"]
    if kind == "compact":
        return dict(bytes=2 * case["moves"] * page + 2 * case["seqs"] * table + 12 * case["pages"], flops=0)
    copied = case["fork"] * (1 if case["page_tokens"] else case["max_pages"])
    sources = min(copied, (-(-case["live"] // 8)) * (1 if case["page_tokens"] else case["max_pages"]))
    return dict(bytes=(copied + sources) * page + 4 * case["pages"] + 3 * (case["fork"] + case["admit"]) * table, flops=0)


def exact(case, seed):
    """The recurrence token by token in 64 bits, all sequences side by side.  Pages are moved, not computed: no values."""
    if case["kind"] not in ("forward", "backward", "decode"):
        return None
    s = prepare(case, seed)
    D = case["dim"]
    lens, N = s["lens"], len(s["lens"])
    x = s["x"].double()
    T, H, _ = x.shape
    L = max(lens)
    at = torch.zeros(N, L, dtype=torch.int64, device="cuda")
    for i, n in enumerate(lens):
        at[i, :n] = torch.arange(n, device="cuda") + sum(lens[:i])
    on = torch.arange(L, device="cuda")[None] < torch.tensor(lens, device="cuda")[:, None]

    def gate(t):
        return None if t is None else (t.double() if t.dim() == 3 else t.double()[:, :, None].expand(-1, -1, D))

    a, b = gate(s["a"]), gate(s["b"])
    h = (s["pool"] if s["state_indices"] is None else s["pool"][s["state_indices"].long()]).double()
    ys = torch.zeros(T + 1, H, D, dtype=torch.float64, device="cuda")
    prev = torch.zeros(T + 1, H, D, dtype=torch.float64, device="cuda")
    slot = torch.where(on, at, T)
    for t in range(L):
        i = at[:, t]
        m = on[:, t, None, None]
        prev[slot[:, t]] = h
        h = torch.where(m, a[i] * h + (x[i] if b is None else b[i] * x[i]), h)
        ys[slot[:, t]] = h
    if case["kind"] != "backward":
        if s["state_indices"] is None:
            return ys[:T], h
        pool = s["pool"].double()
        pool[s["state_indices"].long()] = h
        return ys[:T], pool
    dy = s["dy"].double()
    gs = torch.zeros(T + 1, H, D, dtype=torch.float64, device="cuda")
    c = s["d_final"].double()
    for t in range(L - 1, -1, -1):
        i = at[:, t]
        gt = dy[i] + c
        gs[slot[:, t]] = gt
        c = torch.where(on[:, t, None, None], a[i] * gt, c)
    gs, prev = gs[:T], prev[:T]
    da, db = gs * prev, None if b is None else gs * x
    if s["a"].dim() == 2:
        da, db = da.sum(2), None if db is None else db.sum(2)
    return gs if b is None else gs * b, da, db, c
