"""Problems of the batch maps' inputs where some of the outputs are left out."""
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from hybrid_linear_attention_gdn_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("held", [-1, -7])
def test_negative_held_entry_of_a_completed_block(cuda, held, rows):
    """A request of 60 tokens whose held block has no id completes it: no
    checkpoint, and an error whether the row maps are asked for or not."""
    d = lambda v, t=torch.int32: torch.tensor(v, dtype=t, device="cuda")
    table, cu, ck, nf, err = d([[held, -1], [5, -1]]), d([9, 9, 9]), d([[9], [9]]), d([4]), d([0])
    maps = dict(seq_ids=d([9] * 12), slot_map=d([9] * 12, torch.int64)) if rows else {}
    gdn.batch_maps(d([6, 4]), d([60, 60], torch.int64), 64, table, d([10, 11, 12, 13]), nf, cu, ck, dev_err=err, **maps)
    assert err.tolist() == [binding.DEV_ERR_SLOT_OOB]
    assert cu.tolist() == [0, 6, 10] and ck.tolist() == [[-1], [5]] and nf.tolist() == [3]
    assert table.tolist() == [[held, 13], [5, -1]]
    if rows:
        assert maps["slot_map"].tolist() == [-1] * 4 + [13 * 64, 13 * 64 + 1] + [5 * 64 + 60 + i for i in range(4)] + [-1] * 2
