"""The page operators around the sizes up to which their lists lie in shared memory: 1024 entries of a list, 4096 sequences,
2048 pages given at a time; against the one-entry-after-the-other model."""
import numpy as np
import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from pages_testlib import ERR
from test_gpu_pages import Pair, pools_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.build()


def empty_pair(S, M, P, kind="one"):
    return Pair(np.full((S, M), -1), np.zeros(P, dtype=int), np.zeros(S, dtype=int), pools_of(P, kind))


def lengths(p, seqs, n):
    for s in seqs:
        p.m.lengths[s] = p.lengths[int(s)] = n


@pytest.mark.parametrize("n", [1023, 1024, 1025, 2500])
@pytest.mark.parametrize("page_tokens", [0, 4])
def test_long_lists(n, page_tokens):
    """Every second entry asks for a page; every sequence is forked from one of a few."""
    S, rng = 2 * n + 8, np.random.default_rng(n)
    p = empty_pair(S, 2, 4 * n + 20)
    seqs = rng.permutation(S)
    p.reserve(seqs[:n].tolist(), (np.arange(n) % 3).tolist())
    full = [int(s) for s in seqs[:n] if (p.m.table[s] >= 0).all()][:4]
    lengths(p, full, 7)
    p.fork([full[k % 4] for k in range(n)], seqs[n:2 * n].tolist(), page_tokens)
    assert p.m.status == 0
    p.free(seqs[: 2 * n].tolist())
    assert not p.m.refs.any()


@pytest.mark.parametrize("S", [4095, 4096, 4097, 9000])
def test_many_sequences(S):
    rng = np.random.default_rng(S)
    p = empty_pair(S, 1, 700)
    seqs = rng.permutation(S)
    seqs[:2] = S - 1, 0
    p.reserve(seqs[:300].tolist() + [S - 1, 0, S, -1], [1] * 304)  # the last ones are named before, or outside
    assert p.m.status == ERR["SEQ"]
    empty = np.flatnonzero(p.m.table[:, 0] < 0)[-300:]
    p.fork(seqs[:300].tolist(), empty.tolist(), 0)
    p.free(rng.permutation(S)[:2000].tolist())
    p.compact()


@pytest.mark.parametrize("wanted", [2047, 2048, 2049, 6000])
@pytest.mark.parametrize("short", [0, 5])
def test_many_pages_at_a_time(wanted, short):
    """All of the wanted pages are there, or a few too few."""
    n = 40
    counts = [wanted // n + (k < wanted % n) for k in range(n)]
    p = empty_pair(2 * n, max(counts), wanted - short)
    p.reserve(list(range(n)), counts)
    assert p.m.status == (ERR["NO_PAGES"] if short else 0)
    p.free(list(range(n)))
    q = empty_pair(2 * n, max(counts), 2 * wanted - short)
    q.reserve(list(range(n)), counts)
    q.fork(list(range(n)), list(range(n, 2 * n)), 0)
    assert q.m.status == (ERR["NO_PAGES"] if short else 0)


@pytest.mark.parametrize("page_tokens", [0, 4])
def test_past_all_limits_at_once(page_tokens):
    """Long lists over many sequences that want many pages, with entries twice, out of range and at fault, until pages run out."""
    S, M, P, n = 5001, 3, 4500, 1800
    rng = np.random.default_rng(7)
    p = empty_pair(S, M, P)
    seqs = rng.integers(-3, S + 3, n)
    p.reserve(seqs.tolist(), rng.integers(0, M + 2, n).tolist())
    assert p.m.status == ERR["SEQ"] | ERR["PAGE"]
    live = np.flatnonzero((p.m.table >= 0).any(1))
    for s in live[:200]:
        lengths(p, [s], int((p.m.table[s] >= 0).sum()) * 4 - int(s) % 3)
    children = rng.integers(-3, S + 3, n)
    children[::2] = rng.permutation(np.flatnonzero((p.m.table < 0).all(1)))[: n // 2]
    p.fork(rng.choice(live, n).tolist(), children.tolist(), page_tokens)
    p.reserve(rng.permutation(S)[:2500].tolist(), [M] * 2500)
    assert p.m.status & ERR["NO_PAGES"]
    p.free(rng.integers(0, S, 3000).tolist())
    p.compact()


def test_page_tokens_past_32_bits_are_refused():
    """Not taken modulo 2^32, by which 2^32 + 4 tokens a page would be 4."""
    p = empty_pair(3, 2, 6)
    p.reserve([0], [2])
    lengths(p, [0], 7)
    for n in (1 << 31, (1 << 32) + 4, 1 << 70):
        with pytest.raises(ValueError, match="page_tokens"):
            p.fork([0], [1], n)
    p.fork([0], [1], 0x7fffffff)  # one page, partly filled
    assert p.m.table[1].tolist() == [2, -1]
