"""The page operators' changes in place, as autograd sees them."""
import numpy as np
import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.build()


def i32(v):
    return torch.as_tensor(np.asarray(v), dtype=torch.int32).cuda()


CHANGES = {
    "reserve": (("table", "refs"), lambda s: gdn.cache_reserve(s["table"], s["refs"], i32([2]), i32([1]))),
    "fork": (("table", "refs", "lengths", "pool"),
             lambda s: gdn.cache_fork([s["pool"]], s["table"], s["refs"], i32([0]), i32([2]), lengths=s["lengths"])),
    "free": (("table", "refs", "lengths"), lambda s: gdn.cache_free(s["table"], s["refs"], i32([0]), lengths=s["lengths"])),
    "compact": (("table", "refs", "pool"), lambda s: gdn.cache_compact(s["pool"], s["table"], s["refs"])),
    "compact_beside": (("table2", "refs2", "pool"), lambda s: gdn.cache_compact(
        s["pool"], s["table"], s["refs"], table_out=s["table2"], refcounts_out=s["refs2"])),
    "copy": (("pool",), lambda s: gdn.cache_copy([s["other"]], [s["pool"]], i32([0]), i32([3]))),
}


@pytest.mark.parametrize("what", list(CHANGES))
def test_changes_in_place_are_counted(what):
    """What an operator writes counts as changed in place, what it reads does not: a backward pass that saved a pool's rows
    refuses to go on with other values."""
    written, call = CHANGES[what]
    s = {"table": i32([[0], [4], [-1]]), "refs": i32([1, 0, 0, 0, 1, 0]), "lengths": i32([3, 2, 0]),
         "pool": torch.randn(6, 8, device="cuda"), "other": torch.randn(6, 8, device="cuda")}
    s["table2"], s["refs2"] = s["table"].clone(), s["refs"].clone()
    w = torch.ones(6, 8, device="cuda", requires_grad=True)
    loss = (w * s["pool"]).sum()
    before = {k: t._version for k, t in s.items()}
    call(s)
    assert {k for k, t in s.items() if t._version != before[k]} == set(written)
    if "pool" in written:
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()
    else:
        loss.backward()


def test_inference_mode():
    with torch.inference_mode():
        table, refs, pool = i32([[0], [-1]]), i32([1, 0, 0]), torch.randn(3, 8, device="cuda")
        assert gdn.cache_fork(pool, table, refs, i32([0]), i32([1])).tolist() == [[1]]
        assert torch.equal(pool[1], pool[0])
        gdn.cache_copy(pool, pool, i32([0]), i32([2]))
        assert torch.equal(pool[2], pool[0])
        gdn.cache_free(table, refs, i32([0]))
        gdn.cache_compact(pool, table, refs)
        assert table.tolist() == [[-1], [0]] and refs.tolist() == [1, 0, 0]
