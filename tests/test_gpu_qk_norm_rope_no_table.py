"""A rotation table of no positions: every row's outputs are zeros, nothing goes
to the cache, the table is not read."""
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from hybrid_linear_attention_gdn_gb300 import binding
from test_gpu_qk_norm_rope import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot", [(64, 32), (20, 4), (128, 0)])
def test_through_the_binding(cuda, d, rot, act):
    c = Case(d, 5, 3, 1, d, rot, act)
    c.cs = torch.ones((0, rot))
    c.x.fill_(2.0)
    kc = torch.full((2, 4, 1, d), 9.0, dtype=c.act, device="cuda")
    vc, qo, ko = kc.clone(), torch.full_like(c.q, 3.0), torch.full_like(c.k, 3.0)
    c.call(q_out=qo, k_out=ko, v=c.v, k_cache=kc, v_cache=vc, slot_map=torch.arange(5, device="cuda"))
    assert not bool(qo.any()) and not bool(ko.any())
    assert bool((kc == 9).all()) and bool((vc == 9).all()) and bool((c.x == 2).all())
    assert int(c.err) == binding.DEV_ERR_SEQLENS


@pytest.mark.parametrize("d,rot", [(64, 32), (20, 4)])
def test_a_table_of_rows_that_do_not_count(cuda, d, rot):
    """max_pos 0 with a table behind the pointer, NaN where it must not be read."""
    c = Case(d + 1, 7, 2, 2, d, rot, "bf16")
    table = torch.full((4, rot), float("nan"), device="cuda")
    c.pos.zero_()
    pos, w, row = c.pos.cuda(), c.qw.cuda(), c.x.stride(0)
    qo, ko = torch.full((7, 2, d), 3.0, dtype=c.act, device="cuda"), torch.full((7, 2, d), 3.0, dtype=c.act, device="cuda")
    rows, none = binding.CRows, binding.CPages(None, 0, 0, 0)
    st = gdn.load().gdn_qk_norm_rope(
        1, 2, 2, d, 0, 0, 7, rows(c.q.data_ptr(), row, d), rows(c.k.data_ptr(), row, d), rows(None, 0, 0), w.data_ptr(),
        w.data_ptr(), 1e-6, table.data_ptr(), 0, rot, 0, pos.data_ptr(), rows(qo.data_ptr(), 2 * d, d),
        rows(ko.data_ptr(), 2 * d, d), none, none, 0, 1, None, c.err.data_ptr(),
        torch.cuda.current_stream().cuda_stream)
    assert st == binding.OK
    assert not bool(qo.any()) and not bool(ko.any()) and int(c.err) == binding.DEV_ERR_SEQLENS
