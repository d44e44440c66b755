"""Positions at the end of the 64-bit range: the next block boundary may lie beyond it."""
import numpy as np
import pytest
import torch

from hybrid_linear_attention_gdn_gb300 import binding
from lin_helpers import LinSetup, assert_out_close, f64
from oracle import linear
from test_gpu_lin import _state_close, run_prefill
from test_gpu_lin_paths import _call, _i32, _i64

pytestmark = pytest.mark.gpu
LAST = 2 ** 63 - 1


@pytest.mark.parametrize("name", ["square", "narrow", "tiny"])
@pytest.mark.parametrize("lens,starts,block", [
    ([100, 7], [LAST - 64 - 100, LAST - 64 - 7], 64),
    ([100, 7], [LAST - 64 - 100, LAST - 64 - 7], 2 ** 31 - 64),
    ([300], [2 ** 63 - 2 ** 30 - 150], 2 ** 30),                     # a boundary inside, the next beyond
    ([2100], [LAST - 64 - 2100], 1024),                              # cut
    ([2100], [2 ** 63 - 2 ** 20 - 1000], 2 ** 20),
])
def test_far_positions(cuda, name, lens, starts, block):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    run_prefill(LinSetup(name, 51), lens, starts, block=block, gaps=(2, 3), err=err)
    assert int(err) == 0


@pytest.mark.parametrize("name", ["square", "narrow", "tiny"])
def test_the_last_64_positions_are_refused(cuda, name):
    """The second sequence would end at 2^63 - 64: it is left out, the first one runs."""
    st, err = LinSetup(name, 51), torch.zeros(1, dtype=torch.int32, device="cuda")
    x, out, before = st.tokens(364), st.out(364), st.pool.ssm.clone()
    starts = [2 ** 63 - 2 ** 30 - 150, 2 ** 63 - 128]
    _call(st, st.pool, _i32([1, 2]), _i32([0, 300, 364]), _i64(starts), x.cuda(), out, err=err)
    ref = linear.prefill(st.od, st.opool, None, st.old, st.scale, [1], [0, 300], starts[:1], np.zeros((1, 0), int), 64,
                         f64(x))
    assert_out_close(out[:300], ref[:300], st.dims.dv)
    _state_close(st.pool, st.opool)
    assert bool((out[300:] == 7).all()) and torch.equal(st.pool.ssm[2], before[2])
    assert int(err) == binding.DEV_ERR_SEQLENS
