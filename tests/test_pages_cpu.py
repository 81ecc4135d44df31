"""The page operators without a GPU: what the entry points refuse, and the model that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from pages_testlib import ERR, Book


@pytest.fixture(scope="module")
def L():
    gdn.build()
    return gdn.lib()


def book(**kw):
    d = dict(table=4096, refcounts=8192, lengths=12288, max_seqs=4, max_pages=3, n_pages=20)
    d.update(kw)
    return ctypes.byref(gdn.PagesBook(**d))


def bufs(*rows):
    return (gdn.PagesBuffer * max(1, len(rows)))(*rows)


WS = 1 << 20


@pytest.mark.parametrize("kw", [dict(table=None), dict(refcounts=None), dict(table=4098), dict(refcounts=8193), dict(lengths=2),
                                dict(max_seqs=-1), dict(max_pages=-1), dict(n_pages=-1)])
def test_book_is_checked(L, kw):
    b, n = book(**kw), 1 << 20
    assert L.gdn_pages_reserve_run(b, 64, 128, 2, None, None, WS, n, None) == 1
    assert L.gdn_pages_fork_run(b, bufs(), 0, 64, 128, 2, 0, None, None, WS, n, None) == 1
    assert L.gdn_pages_free_run(b, 64, 2, None, None) == 1
    assert L.gdn_pages_compact_run(b, bufs(), 0, 64, 128, 256, 512, None, WS, n, None) == 1


def test_lists_and_workspaces_are_checked(L):
    b, n = book(), L.gdn_pages_workspace_bytes(4, 3, 20, 2)
    assert n > 0 and L.gdn_pages_workspace_bytes(-1, 3, 20, 2) == 0
    for args in ((None, 128, 2), (64, None, 2), (64, 128, -1), (65, 128, 2)):
        assert L.gdn_pages_reserve_run(b, *args, None, None, WS, n, None) == 1
        assert L.gdn_pages_fork_run(b, bufs(), 0, *args, 0, None, None, WS, n, None) == 1
    assert L.gdn_pages_free_run(b, None, 2, None, None) == 1
    for ws, size in ((None, n), (WS, n - 1), (WS + 4, n)):
        assert L.gdn_pages_reserve_run(b, 64, 128, 2, None, None, ws, size, None) == 1
        assert L.gdn_pages_fork_run(b, bufs(), 0, 64, 128, 2, 0, None, None, ws, size, None) == 1
    assert L.gdn_pages_reserve_run(book(max_pages=1 << 20), 64, 128, 4096, None, None, WS, 1 << 40, None) == 2  # 2^32 pages
    assert L.gdn_pages_fork_run(b, bufs(), 0, 64, 128, 2, -1, None, None, WS, n, None) == 1
    assert L.gdn_pages_fork_run(book(lengths=None), bufs(), 0, 64, 128, 2, 16, None, None, WS, n, None) == 1
    for out in ((None, 128, 256, 512), (64, None, 256, 512), (64, 128, None, 512), (64, 128, 256, None), (66, 128, 256, 512)):
        assert L.gdn_pages_compact_run(b, bufs(), 0, *out, None, WS, n, None) == 1


@pytest.mark.parametrize("row", [(None, 16, 16), (4096, 8, 16), (4096, 16, -1)])
def test_buffers_are_checked(L, row):
    n = 1 << 20
    assert L.gdn_pages_fork_run(book(), bufs(row), 1, 64, 128, 2, 0, None, None, WS, n, None) == 1
    assert L.gdn_pages_compact_run(book(), bufs(row), 1, 64, 128, 256, 512, None, WS, n, None) == 1
    good = bufs((4096, 16, 16))
    assert L.gdn_pages_copy_run(bufs(row), 4, good, 4, 1, 64, 128, 2, None, None) == 1
    assert L.gdn_pages_copy_run(good, 4, bufs(row), 4, 1, 64, 128, 2, None, None) == 1


def test_copy_is_checked(L):
    good, other = bufs((4096, 16, 16)), bufs((8192, 32, 32))
    assert L.gdn_pages_copy_run(good, 4, other, 4, 1, 64, 128, 2, None, None) == 1  # rows of two sizes
    for args in ((-1, 4, 1, 64, 128, 2), (4, -1, 1, 64, 128, 2), (4, 4, -1, 64, 128, 2), (4, 4, 129, 64, 128, 2),
                 (4, 4, 1, None, 128, 2), (4, 4, 1, 64, None, 2), (4, 4, 1, 64, 128, -1)):
        assert L.gdn_pages_copy_run(good, args[0], good, *args[1:], None, None) == 1
    assert L.gdn_pages_copy_run(good, 4, good, 4, 1, None, None, 0, None, None) == 0  # nothing to do, nothing launched
    assert L.gdn_pages_copy_run(good, 4, good, 4, 0, 64, 128, 2, None, None) == 0


def test_empty_lists_launch_nothing(L):
    n = 1 << 20
    assert L.gdn_pages_reserve_run(book(), None, None, 0, None, None, WS, n, None) == 0
    assert L.gdn_pages_fork_run(book(), bufs(), 0, None, None, 0, 0, None, None, WS, n, None) == 0
    assert L.gdn_pages_free_run(book(), None, 0, None, None) == 0


def test_structs_match_the_header():
    assert ctypes.sizeof(gdn.PagesBook) == 40 and ctypes.sizeof(gdn.PagesBuffer) == 24


def test_python_refuses_cpu_tensors():
    t, r, s = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    p = torch.zeros(4, 8)
    for call in (lambda: gdn.cache_reserve(t, r, s, s), lambda: gdn.cache_fork([p], t, r, s, s), lambda: gdn.cache_free(t, r, s),
                 lambda: gdn.cache_compact([p], t, r), lambda: gdn.cache_copy([p], [p], s, s)):
        with pytest.raises(ValueError, match="no CPU path"):
            call()


def test_model_forks_shares_and_copies():
    """A hand-made case: two full pages shared, the partly filled third copied into the lowest free page."""
    b = Book([[4, 1, 3], [-1, -1, -1]], [0, 1, 0, 1, 1], [40, 0], [np.arange(5.0)])
    assert b.fork([0], [1], 16).tolist() == [[4, 1, 0]]
    assert b.refs.tolist() == [1, 2, 0, 1, 2] and b.lengths.tolist() == [40, 40] and b.pools[0].tolist() == [3, 1, 2, 3, 4]
    b.free([0])
    assert b.refs.tolist() == [1, 1, 0, 0, 1]
    remap, n = b.compact()
    assert n == 3 and remap.tolist() == [0, 1, -1, -1, 2] and b.table.tolist() == [[-1, -1, -1], [2, 1, 0]]
    assert b.pools[0].tolist() == [3, 1, 4, 3, 4] and b.status == 0
    b.reserve([0, 1], [3, 3])
    assert b.status == ERR["NO_PAGES"] and (b.table[0] == -1).all()
