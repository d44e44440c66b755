"""The state space prefill's workspace: what it may hold, and that its places
suffice for batches of many short sequences."""
import ctypes

import numpy as np
import pytest

import hybrid_linear_attention_gdn_gb300 as gdn
from hybrid_linear_attention_gdn_gb300 import _build, binding
from ssm_helpers import SsmSetup, shape

RECORD = 57 * 1024  # bytes of a chunk's operands, per group


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gdn.load()


def _size(lib, n_seq, total, hk=8, hv=64, dv=64):
    d = binding.CDims(hk=hk, hv=hv, dk=128, dv=dv, conv_width=4, act_dtype=1, conv_dtype=1)
    return lib.gdn_ssm_prefill_workspace_size(ctypes.byref(d), n_seq, total)


@pytest.mark.parametrize("n_seq,total", [(1, 1), (512, 512), (512, 700), (4096, 4100), (512, 40000)])
def test_no_more_records_than_tokens(lib, n_seq, total):
    """A record belongs to a chunk that holds a token, so that many sequences
    of a token or two need a record per token at most."""
    history = 3 * n_seq * 64 * 64 * 2
    records = min(total, total // 64 + 2 * n_seq) * 8 * RECORD
    # whole sequences: with 512 of them no call is cut; one token is one chunk
    assert records + history <= _size(lib, n_seq, total) <= records + history + 256 + 1024


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[1] * 40, [1, 0, 0, 2, 1, 65, 0, 1, 1, 1, 130, 2], [0, 0, 1], [2, 64, 1, 66, 1]])
@pytest.mark.parametrize("seed", range(3))
def test_short_sequences(cuda, lens, seed):
    """Starts at any place of a chunk, empty sequences between, rows around."""
    from test_gpu_ssm import _prefill
    rng = np.random.default_rng(seed)
    starts = rng.choice([0, 1, 62, 63, 64, 127, 200], len(lens)).tolist()
    st = SsmSetup(shape("one_group", num_slots=len(lens)), seed=91)
    _prefill(st, rng.permutation(len(lens)).tolist(), lens, starts, 64, lead=seed, extra=7 * seed)
