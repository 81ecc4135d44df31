"""State indices of empty sequences: looked at like any others, although no token reads or writes their rows."""
import pytest
import torch

import gated_deltanet_chunked_device_gb300 as gdn
from linear_testlib import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.build()


@pytest.mark.parametrize("lens", [[70, 0, 200], [0, 30, 0], [0, 0], [5000, 0, 900]])
@pytest.mark.parametrize("H,D", [(2, 16), (1, 17), (16, 128)])
@pytest.mark.parametrize("states", ["in_place", "apart", "only_read"])
def test_an_empty_sequences_index_is_checked(lens, H, D, states):
    i = make(lens, H, D, "f32", seed=70)
    at = lens.index(0)
    pool = torch.randn(9, H, D, device="cuda")
    for bad in (None, -1, 9):
        rows = torch.tensor([6, 2, 4][: len(lens)], dtype=torch.int32, device="cuda")
        if bad is not None:
            rows[at] = bad
        start, status = pool.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
        out = {"in_place": start, "apart": torch.full_like(pool, 7.0), "only_read": None}[states]
        gdn.gated_linear_recurrence(i["x"], i["a"], i["b"], initial_state=start, output_state=out, state_indices=rows,
                                    output_final_state=out is not None, cu_seqlens=i["cu"], device_status=status)
        assert int(status) == (gdn.DEVICE_ERR["STATE_INDEX_RANGE"] if bad is not None else 0)
        used = rows.tolist()
        if out is not None:
            rest = [r for r in range(9) if r not in used]
            assert torch.equal(out[rest], pool[rest] if states == "in_place" else torch.full_like(out[rest], 7.0))
            if bad is None:
                assert torch.equal(out[used[at]], pool[used[at]])
