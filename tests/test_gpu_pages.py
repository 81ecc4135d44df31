"""The page operators on the GPU against the one-entry-after-the-other model: every table, count and byte is equal."""
import numpy as np
import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from pages_testlib import ERR, Book

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.build()


def i32(v):
    return torch.as_tensor(np.asarray(v), dtype=torch.int32).cuda()


class Pair:
    """The same bookkeeping on the GPU and in the model."""

    def __init__(self, table, refs, lengths, pools):
        self.m = Book(table, refs, lengths, [p.view(torch.uint8).cpu().numpy() if p.dtype != torch.uint8 else p.cpu().numpy()
                                             for p in pools])
        self.table, self.refs = i32(table).view(len(table), -1), i32(refs)
        self.lengths = None if lengths is None else i32(lengths)
        self.pools, self.status = pools, torch.zeros(1, dtype=torch.int32, device="cuda")

    def reserve(self, seqs, counts):
        rows = gdn.cache_reserve(self.table, self.refs, i32(seqs), i32(counts), device_status=self.status)
        assert np.array_equal(rows.cpu(), self.m.reserve(seqs, counts))
        self.check()

    def fork(self, parents, children, page_tokens):
        rows = gdn.cache_fork(self.pools, self.table, self.refs, i32(parents), i32(children), page_tokens=page_tokens,
                              lengths=self.lengths, device_status=self.status)
        assert np.array_equal(rows.cpu(), self.m.fork(parents, children, page_tokens))
        self.check()

    def free(self, seqs):
        gdn.cache_free(self.table, self.refs, i32(seqs), lengths=self.lengths, device_status=self.status)
        self.m.free(seqs)
        self.check()

    def compact(self):
        remap, n = gdn.cache_compact(self.pools, self.table, self.refs, device_status=self.status)
        want, L = self.m.compact()
        assert np.array_equal(remap.cpu(), want) and n.tolist() == [L]
        self.check()

    def check(self):
        assert np.array_equal(self.table.cpu(), self.m.table) and np.array_equal(self.refs.cpu(), self.m.refs)
        if self.lengths is not None:
            assert np.array_equal(self.lengths.cpu(), self.m.lengths)
        for p, q in zip(self.pools, self.m.pools):
            assert np.array_equal(p.view(torch.uint8).cpu().numpy() if p.dtype != torch.uint8 else p.cpu().numpy(), q)
        assert int(self.status) == self.m.status


def pools_of(P, kind, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randint(0, 255, s, generator=g, dtype=torch.uint8).cuda()  # noqa: E731
    return {"one": lambda: [r(P, 64)], "odd": lambda: [r(P, 7), r(P, 602), r(P, 33)], "none": lambda: [],
            "empty_rows": lambda: [r(P, 0), r(P, 16)], "large": lambda: [r(P, 40000), r(P, 16384), r(P, 16400)],
            "pieces": lambda: [r(P, 3 * 16384 + 1), r(P, 5)]}[kind]()


def random_pair(rng, P, S, M, live, page_tokens=0, kind="one"):
    table, refs, lengths = np.full((S, M), -1), np.zeros(P, dtype=int), np.zeros(S, dtype=int)
    pages = rng.permutation(P)
    at = 0
    for s in rng.permutation(S)[:live]:
        n = int(rng.integers(0, M + 1))
        n = min(n, P - at)
        table[s, :n] = pages[at:at + n]
        refs[table[s, :n]] = 1
        at += n
        lengths[s] = 0 if n == 0 else rng.integers((n - 1) * page_tokens + 1, n * page_tokens + 1) if page_tokens else rng.integers(1, 99)
    return Pair(table, refs, lengths, pools_of(P, kind))


@pytest.mark.parametrize("kind", ["one", "odd", "none", "empty_rows", "large", "pieces"])
@pytest.mark.parametrize("page_tokens", [0, 1, 16])
@pytest.mark.parametrize("seed", [0, 1])
def test_random_turns(seed, page_tokens, kind):
    """Admit, fork, free and compact in turn, with lists of every length, until pages run out now and then."""
    rng = np.random.default_rng(seed)
    S, M, P = 24, 5, 61
    p = random_pair(rng, P, S, M, 8, page_tokens, kind)
    for _ in range(12):
        n = int(rng.integers(1, 6))
        what = rng.integers(0, 4)
        if what == 0:
            p.reserve(rng.permutation(S)[:n].tolist(), rng.integers(0, M + 1, n).tolist())
        elif what == 1:
            p.fork(rng.integers(0, S, n).tolist(), rng.permutation(S)[:n].tolist(), page_tokens)
        elif what == 2:
            p.free(rng.permutation(S)[:n].tolist())
        else:
            p.compact()


@pytest.mark.parametrize("P,S,M", [(1, 1, 1), (32, 7, 1), (1025, 300, 2), (40000, 2000, 3), (5000, 3, 1500)])
def test_sizes(P, S, M):
    rng = np.random.default_rng(5)
    p = random_pair(rng, P, S, M, S // 2, 4, "one")
    empty = np.flatnonzero((p.m.table < 0).all(1) & (p.m.lengths == 0))
    live = np.flatnonzero((p.m.table >= 0).any(1))
    if len(live):
        p.fork(rng.choice(live, len(empty[::2])).tolist(), empty[::2].tolist(), 4)
    p.reserve(empty[1::2].tolist(), rng.integers(0, M + 1, len(empty[1::2])).tolist())
    p.free(rng.permutation(S)[: S // 3].tolist())
    p.compact()
    p.compact()  # nothing left to move
    p.free(list(range(S)))
    assert not p.m.refs.any()
    p.compact()
    p.reserve([0], [M])


def test_pages_run_out_in_order():
    """Whoever does not fit, and all after them, get nothing, even where a later one would fit."""
    p = Pair(np.full((5, 3), -1), np.array([1, 0, 0, 1, 0]), np.zeros(5), pools_of(5, "one"))
    p.reserve([4, 2, 0], [2, 2, 1])
    assert p.m.status == ERR["NO_PAGES"] and p.m.table[4].tolist() == [1, 2, -1] and (p.m.table[[0, 2]] == -1).all()
    p.fork([4, 4], [0, 1], 0)
    assert (p.m.table[[0, 1]] == -1).all()


@pytest.mark.parametrize("page_tokens", [0, 8])
def test_entries_at_fault_are_skipped(page_tokens):
    """Sequences out of range, twice or their own parents, children with pages, pages out of range: reported, the others served."""
    table = np.array([[0, 1], [2, -1], [-1, -1], [-1, -1], [9, 3], [-1, -1], [-1, -1]])
    p = Pair(table, np.array([1, 1, 1, 1, 0, 0, 0, 0, 0]), np.array([12, 5, 0, 0, 16, 0, 0]), pools_of(9, "odd"))
    p.fork([0, -1, 7, 1, 2, 0, 4, 1, 2], [2, 3, 3, 3, 2, 1, 5, 6, 3], page_tokens)
    p.reserve([-1, 7, 3, 3, 5, 5], [1, 1, 3, 1, -1, 1])
    p.free([-1, 7, 2, 2, 4])
    p.compact()


def test_freeing_twice_and_what_is_free():
    p = Pair([[0, 1], [1, 1]], [1, 2, 0], [3, 3], pools_of(3, "one"))
    p.free([0, 0, 1])  # page 1 is named three times and counted twice
    assert p.m.status == ERR["PAGE"] and p.m.refs.tolist() == [0, 0, 0]


def test_parents_are_taken_as_they_were():
    """A sequence that another entry of the list makes is still empty as a parent."""
    p = Pair([[0], [-1], [-1], [-1]], [1, 0, 0, 0, 0], [5, 0, 0, 0], pools_of(5, "one"))
    p.fork([1, 0, 1], [2, 1, 3], 0)
    assert p.m.table.tolist() == [[0], [1], [-1], [-1]]


def test_compact_beside_the_running_tables():
    """Into other tables: the old bookkeeping and the pages that it names stay as they are."""
    rng = np.random.default_rng(3)
    p = random_pair(rng, 200, 30, 4, 20, 4, "odd")
    p.free(np.flatnonzero(p.m.table[:, 0] >= 0)[::2].tolist())
    table, refs, before = p.table.clone(), p.refs.clone(), [q.clone() for q in p.pools]
    t2, r2 = torch.empty_like(table), torch.empty_like(refs)
    remap, n = gdn.cache_compact(p.pools, p.table, p.refs, table_out=t2, refcounts_out=r2)
    assert torch.equal(p.table, table) and torch.equal(p.refs, refs)
    for q, b in zip(p.pools, before):
        assert torch.equal(q[refs > 0], b[refs > 0])
    want, L = p.m.compact()
    assert np.array_equal(t2.cpu(), p.m.table) and np.array_equal(r2.cpu(), p.m.refs) and n.tolist() == [L]
    assert np.array_equal(remap.cpu(), want)
    for q, b in zip(p.pools, p.m.pools):
        assert np.array_equal(q.cpu().numpy(), b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.uint8])
@pytest.mark.parametrize("row", [(1,), (3,), (8,), (7, 43), (16, 128), (2, 100, 100)])
def test_copy(row, dtype):
    g = torch.Generator().manual_seed(1)
    src = torch.randn(9, *row, generator=g).to(dtype).cuda()
    dst = torch.randn(14, *row, generator=g).to(dtype).cuda()
    want = dst.clone()
    s, d = [3, 3, -1, 8, 0], [13, 0, 4, -1, 7]
    for i, j in zip(s, d):
        if i >= 0 and j >= 0:
            want[j] = src[i]
    gdn.cache_copy([src], [dst], i32(s), i32(d))
    assert torch.equal(dst.view(torch.uint8), want.view(torch.uint8))


def test_copy_between_strided_pools():
    """Rows of a wider buffer, at any alignment; what lies between the rows stays."""
    for shift in (0, 1, 4, 8):
        wide_s, wide_d = torch.randn(6, 50, device="cuda"), torch.randn(8, 61, device="cuda")
        want = wide_d.clone()
        src, dst = wide_s[:, shift: shift + 24], wide_d[:, 1: 25]
        want[[5, 0], 1:25] = wide_s[[2, 4], shift: shift + 24]
        gdn.cache_copy(src, dst, i32([2, 4]), i32([5, 0]))
        assert torch.equal(wide_d, want)


def test_copy_within_a_pool_and_out_of_range():
    pool = torch.randn(6, 40, device="cuda")
    want, status = pool.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    want[4] = pool[1]
    gdn.cache_copy(pool, pool, i32([1, 6, 2, 2 ** 31 - 1]), i32([4, 0, 6, 2]), device_status=status)
    assert torch.equal(pool, want) and int(status) == ERR["PAGE"]


def test_copy_many_rows_many_buffers():
    g = torch.Generator(device="cuda").manual_seed(2)
    src = [torch.randn(700, 130 + 8 * i, generator=g, device="cuda") for i in range(40)]
    dst = [torch.zeros(900, 130 + 8 * i, device="cuda") for i in range(40)]
    d = torch.randperm(900, generator=g, device="cuda")[:800].to(torch.int32)
    s = torch.randint(0, 700, (800,), generator=g, device="cuda", dtype=torch.int32)
    gdn.cache_copy(src, dst, s, d)
    for p, q in zip(src, dst):
        want = torch.zeros_like(q)
        want[d.long()] = p[s.long()]
        assert torch.equal(q, want)


def test_offsets_past_32_bits():
    """Rows that start more than 2^32 bytes into a buffer."""
    pool = torch.zeros(5, 1 << 30, dtype=torch.uint8, device="cuda")
    pool[0, -5:] = 7
    pool[0, :5] = 9
    gdn.cache_copy(pool, pool, i32([0]), i32([4]))
    assert torch.equal(pool[4], pool[0]) and not pool[1:4].any()


def test_graph_capture():
    """A scheduler's step captured once and replayed."""
    rng = np.random.default_rng(4)
    p, q = random_pair(rng, 64, 20, 1, 6, 0, "one"), None
    live, empty = np.flatnonzero(p.m.table[:, 0] >= 0), np.flatnonzero(p.m.table[:, 0] < 0)
    par, kids = i32(live[:2]), i32(empty[:2])
    gdn.cache_fork(p.pools, p.table, p.refs, par, kids, lengths=p.lengths)  # loads the library before the capture
    gdn.cache_free(p.table, p.refs, kids, lengths=p.lengths)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rows = gdn.cache_fork(p.pools, p.table, p.refs, par, kids, lengths=p.lengths, device_status=p.status)
    for _ in range(3):
        graph.replay()
        want = p.m.fork(live[:2].tolist(), empty[:2].tolist(), 0)
        torch.cuda.synchronize()
        assert np.array_equal(rows.cpu(), want)
        p.check()
        p.free(empty[:2].tolist())


def test_states_of_a_recurrence_are_forked():
    """Prefill, fork, decode: the children go on from their parent's state, and apart from it."""
    H, D, P = 2, 64, 12
    g = torch.Generator(device="cuda").manual_seed(6)
    pool = torch.zeros(P, H, D, device="cuda")
    table, refs = torch.full((8, 1), -1, dtype=torch.int32, device="cuda"), torch.zeros(P, dtype=torch.int32, device="cuda")
    rows = gdn.cache_reserve(table, refs, i32([0]), i32([1]))
    x, a = torch.randn(90, H, D, generator=g, device="cuda"), torch.rand(90, H, D, generator=g, device="cuda")
    gdn.gated_linear_recurrence(x, a, initial_state=pool, output_state=pool, state_indices=rows.view(-1), output_final_state=True)
    kids = gdn.cache_fork(pool, table, refs, i32([0, 0]), i32([5, 6]))
    assert kids.view(-1).tolist() == [1, 2] and torch.equal(pool[1], pool[0]) and torch.equal(pool[2], pool[0])
    x1, a1 = torch.randn(2, H, D, generator=g, device="cuda"), torch.rand(2, H, D, generator=g, device="cuda")
    y, _ = gdn.gated_linear_recurrence_decode(x1, a1, initial_state=pool, state_indices=kids.view(-1))
    assert torch.equal(pool[1], y[0]) and torch.equal(pool[2], y[1]) and not torch.equal(pool[1], pool[0])
    torch.testing.assert_close(y, a1 * pool[0] + x1, rtol=2 ** -22, atol=2 ** -22)  # one product and one sum, fused or not


def test_python_refusals():
    t, r, le = i32(np.full((3, 2), -1)), i32(np.zeros(5)), i32(np.zeros(3))
    pool, s = torch.zeros(5, 4, device="cuda"), i32([0])
    bad = [lambda: gdn.cache_reserve(t.long(), r, s, s), lambda: gdn.cache_reserve(t[:, :1], r, s, s),
           lambda: gdn.cache_reserve(t, r.view(5, 1), s, s), lambda: gdn.cache_reserve(t, r, s, i32([0, 1])),
           lambda: gdn.cache_reserve(t, r, s.cpu(), s), lambda: gdn.cache_fork([pool[:4]], t, r, s, s),
           lambda: gdn.cache_fork([pool.cpu()], t, r, s, s), lambda: gdn.cache_fork([torch.zeros(4, 5, device="cuda").t()], t, r, s, s),
           lambda: gdn.cache_fork([pool[:1].expand(5, 4)], t, r, s, s), lambda: gdn.cache_fork([pool], t, r, s, s, page_tokens=16),
           lambda: gdn.cache_fork([pool] * 129, t, r, s, s), lambda: gdn.cache_fork([pool], t, r, s, s, lengths=le[:2]),
           lambda: gdn.cache_free(t, r, s.long()), lambda: gdn.cache_compact([pool], t, r, table_out=t[:2]),
           lambda: gdn.cache_compact([pool], t, r, refcounts_out=r[:4]), lambda: gdn.cache_copy([pool], [pool, pool], s, s),
           lambda: gdn.cache_copy([pool], [pool.half()], s, s), lambda: gdn.cache_copy([pool], [torch.zeros(5, 3, device="cuda")], s, s),
           lambda: gdn.cache_copy([pool], [pool], s, i32([0, 1]))]
    for n, call in enumerate(bad):
        with pytest.raises((ValueError, gdn.GdnError)):
            call()
            pytest.fail(f"call {n} was not refused")
    with pytest.raises(gdn.GdnError):  # host-checked by the library
        gdn.cache_fork([pool], t, r, s, s, page_tokens=-1, lengths=le)
