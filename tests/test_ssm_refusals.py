"""Refusals of the state space, norm and map calls beyond their first ones, on
the CPU by their messages and next to a GPU by what they leave alone."""
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from hybrid_linear_attention_gdn_gb300 import binding
from ssm_helpers import SsmSetup, shape

TABLES = {"flat": lambda t: t[0], "deep": lambda t: t[None], "rows": lambda t: t.repeat(2, 1),
          "no_rows": lambda t: t[:0], "scalar": lambda t: t[0, 0]}


def _prefill_with(st, table, device):
    sh, n = st.shape, 70
    qkv, a = (t.to(device) for t in st.tokens(n))
    out = torch.zeros((n, sh.hv, sh.dv), dtype=sh.act_dtype, device=device)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=device)
    ck, _ = st.ckpt_pool(2, device)
    gdn.ssm_prefill(st.dims, st.pool, ck, st.params, i32([1]), i32([0, n]), torch.tensor([0], device=device), n,
                    table(i32([[0, 1]])), 64, qkv, a, out, None)
    return ck


@pytest.mark.parametrize("table", list(TABLES))
def test_checkpoint_table_of_another_shape(table):
    """[n_seq][max_ckpt] or nothing: a table of any other shape wrote no
    checkpoint and said nothing."""
    with pytest.raises(gdn.GdnError, match="ckpt_ids") as e:
        _prefill_with(SsmSetup(shape("tiny"), 1, device="cpu"), TABLES[table], "cpu")
    assert e.value.status == binding.ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("table", list(TABLES))
def test_checkpoint_table_of_another_shape_next_to_a_gpu(cuda, table):
    st = SsmSetup(shape("tiny"), 1)
    before, n0 = st.pool.ssm.clone(), binding.launch_counts()
    with pytest.raises(gdn.GdnError, match="ckpt_ids"):
        _prefill_with(st, TABLES[table], "cuda")
    assert binding.launch_counts() == n0 and torch.equal(st.pool.ssm, before)


@pytest.mark.gpu
def test_checkpoint_table_of_its_shape(cuda):
    st = SsmSetup(shape("tiny"), 1)
    ck = _prefill_with(st, lambda t: t, "cuda")
    assert (ck.ssm[0] != -5).all() and (ck.ssm[1] == -5).all()
    _prefill_with(st, lambda t: t[:, :0], "cuda")  # room for none


@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("device", ["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def test_norm_of_rows_of_nothing(device, group):
    """Rows of no values have no norm; with an 8-bit output the scales' shape
    divided by zero."""
    if device == "cuda" and not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    e = lambda *s, dt=torch.float32: torch.zeros(s, device=device).to(dt)
    for kw in ({}, dict(q8=e(3, 0, dt=torch.float8_e4m3fn), group=group)):
        with pytest.raises(gdn.GdnError, match="no values") as err:
            gdn.add_rmsnorm(e(3, 0), None, e(0), **kw)
        assert err.value.status == binding.ERR_INVALID_ARG
