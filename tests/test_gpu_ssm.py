"""The selective state space step on the GPU against its float64 recurrence."""
import numpy as np
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from hybrid_linear_attention_gdn_gb300 import binding
from oracle import state_space
from helpers import assert_out_close, conv_bits_equal, max_rel_l2, out_tol
from ssm_helpers import SHAPES, STATE_TOL, SsmSetup, f64, shape

pytestmark = pytest.mark.gpu


def _check_states(st, pool, opool):
    n = st.shape.dv * st.shape.dk
    assert max_rel_l2(f64(pool.ssm), opool.ssm, n) <= STATE_TOL
    assert conv_bits_equal(pool.conv, opool.conv)


def _decode(st, ids, out=None):
    qkv, a = st.tokens(len(ids))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if out is None:
        out = torch.full((len(ids), st.shape.hv, st.shape.dv), 7.0, dtype=st.shape.act_dtype, device="cuda")
    gdn.ssm_decode_step(st.dims, st.pool, st.params, torch.tensor(ids, dtype=torch.int32, device="cuda"),
                        qkv.cuda(), a.cuda(), out, err)
    ref, bad = state_space.decode_step(st.od, st.opool, st.oparams, ids, f64(qkv), f64(a))
    torch.cuda.synchronize()
    assert int(err.item()) == (binding.DEV_ERR_SLOT_OOB if bad else 0)
    return out, ref


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("ids", [[3], [5, 0, 7, 2, 1], [4, -1, 0, -1, 6]])
def test_decode(cuda, name, ids):
    sh = shape(name)
    st = SsmSetup(sh, seed=1 + len(ids))
    n0 = binding.launch_count(binding.K_SSM_DECODE)
    out, ref = _decode(st, ids)
    assert binding.launch_count(binding.K_SSM_DECODE) == n0 + 1
    assert_out_close(out, ref, sh.dv, out_tol(sh))
    _check_states(st, st.pool, st.opool)


def test_decode_chain_and_out_of_range_id(cuda):
    """Several steps in a row on moving slots; an id outside the pool is
    skipped, zeroed and reported."""
    sh = shape("wide")
    st = SsmSetup(sh, seed=9)
    for ids in ([1, 2, 3], [3, 8, 1], [-2, 1, 5], [5, 3, 1]):
        out, ref = _decode(st, ids)
        assert_out_close(out, ref, sh.dv, out_tol(sh))
    _check_states(st, st.pool, st.opool)


def test_decode_without_bias_and_skip_many_requests(cuda):
    """More requests than SMs: the rows of a group are no longer split."""
    sh = shape("wide", num_slots=400)
    st = SsmSetup(sh, seed=10, bias=False, skip=False)
    ids = torch.randperm(400, generator=st.gen)[:333].tolist()
    out, ref = _decode(st, ids)
    assert_out_close(out, ref, sh.dv, out_tol(sh))
    _check_states(st, st.pool, st.opool)


def test_decode_zero_decay_and_nan_gate(cuda):
    """dt large enough for an exact zero decay replaces the state; a NaN gate
    poisons its own head only."""
    sh = shape("tiny")
    st = SsmSetup(sh, seed=11)
    qkv, a = st.tokens(2)
    a[0, 1] = 500.0
    a[1, 2] = float("nan")
    out = torch.empty((2, sh.hv, sh.dv), device="cuda")
    gdn.ssm_decode_step(st.dims, st.pool, st.params, torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                        qkv.cuda(), a.cuda(), out)
    ref, _ = state_space.decode_step(st.od, st.opool, st.oparams, [0, 1], f64(qkv), f64(a))
    got = f64(out)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    assert np.linalg.norm(got[ok] - ref[ok]) <= 1e-4 * np.linalg.norm(ref[ok])
    assert np.isnan(f64(st.pool.ssm)[1, 2]).all() and not np.isnan(f64(st.pool.ssm)[1, [0, 1, 3]]).any()


def _prefill(st, ids, lens, starts, block, max_ckpt=None, extra=0, lead=0):
    """Runs the call and the recurrence; `lead` and `extra` rows before and
    behind the sequences stay as they were."""
    sh = st.shape
    cu = np.concatenate([[0], np.cumsum(lens)]) + lead
    total = int(cu[-1]) + extra
    counts = [(s + l) // block - s // block for s, l in zip(starts, lens)]
    mc = max(counts) if max_ckpt is None else max_ckpt
    n_ck = sum(counts) + 1
    table = np.full((len(lens), max(mc, 1)), -1, np.int32)
    perm = torch.randperm(n_ck, generator=st.gen).tolist()
    for r, c in enumerate(counts):
        for k in range(min(c, mc)):
            table[r, k] = perm.pop()
    ck, ock = st.ckpt_pool(n_ck)
    qkv, a = st.tokens(total)
    out = torch.full((total, sh.hv, sh.dv), 7.0, dtype=sh.act_dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    size = gdn.ssm_prefill_workspace_size(st.dims, len(lens), total)
    ws = torch.full((size,), 0xff, dtype=torch.uint8, device="cuda") if size else None
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    gdn.ssm_prefill(st.dims, st.pool, ck, st.params, i32(ids), i32(cu), torch.tensor(starts, device="cuda"), total,
                    i32(table), block, qkv.cuda(), a.cuda(), out, ws, err)
    ref = state_space.prefill(st.od, st.opool, ock, st.oparams, ids, cu, starts, table, block, f64(qkv), f64(a))
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert (out[:lead] == 7).all() and (out[total - extra:] == 7).all()
    lo, hi = lead, total - extra
    if hi > lo:
        assert_out_close(out[lo:hi], ref[lo:hi], sh.dv, out_tol(sh), row_floor_rms=True)
    _check_states(st, st.pool, st.opool)
    _check_states(st, ck, ock)


CASES = {
    "one_token": ([2], [1], [0], 64),
    "one_chunk": ([2], [64], [0], 64),
    "short": ([2], [37], [320], 256),
    "unaligned": ([1, 5, 0], [130, 65, 200], [7, 63, 1001], 64),
    "empty_between": ([1, 5, 0, 3], [70, 0, 1, 0], [64, 10, 127, 0], 64),
    "long": ([6, 2], [700, 515], [0, 300], 128),
}


@pytest.mark.parametrize("case", list(CASES))
@pytest.mark.parametrize("name", list(SHAPES))
def test_prefill(cuda, name, case):
    ids, lens, starts, block = CASES[case]
    if case == "long" and name not in ("wide", "square", "tiny"):
        lens = [v // 4 for v in lens]
    n0 = binding.launch_count(binding.K_SSM_PREFILL)
    _prefill(SsmSetup(shape(name), seed=21), ids, lens, starts, block)
    assert binding.launch_count(binding.K_SSM_PREFILL) == n0 + 1


@pytest.mark.parametrize("name", ["wide", "square", "tiny"])
def test_prefill_leaves_other_rows(cuda, name):
    _prefill(SsmSetup(shape(name), seed=22), [4, 1], [90, 40], [5, 0], 64, lead=3, extra=70)


@pytest.mark.parametrize("name", ["wide", "tiny"])
def test_prefill_fewer_checkpoints_than_boundaries(cuda, name):
    _prefill(SsmSetup(shape(name), seed=23, bias=False, skip=False), [4, 1], [300, 150], [5, 0], 64, max_ckpt=2)


@pytest.mark.parametrize("decay", [(1.0, 4.0), (1e-5, 1e-4)])
@pytest.mark.parametrize("name", ["wide", "square"])
def test_prefill_strong_and_weak_decay(cuda, name, decay):
    """Decays that forget within a token (chunk sums of log decays in the
    thousands) and that hardly forget at all."""
    _prefill(SsmSetup(shape(name), seed=24, decay=decay), [4, 1], [200, 130], [33, 64], 64)


@pytest.mark.parametrize("scale", [1e-6, 1e6])
@pytest.mark.parametrize("name", ["wide", "square"])
def test_prefill_small_and_large_inputs(cuda, name, scale):
    """Features far from 1: SiLU(y) ~ y / 2 for the small ones, y or a tiny
    negative for the large ones; the split operands are scaled per chunk."""
    st = SsmSetup(shape(name), seed=25, bias=False)
    plain = st.tokens

    def tokens(n):
        qkv, a = plain(n)
        return (qkv.float() * scale).to(qkv.dtype), a

    st.tokens = tokens
    st.pool.conv *= scale
    st.pool.ssm *= scale * scale
    st.opool.conv[:], st.opool.ssm[:] = f64(st.pool.conv), f64(st.pool.ssm)  # the rounded products
    _prefill(st, [4, 1], [100, 130], [33, 64], 64)


def test_prefill_padding_and_bad_sequences(cuda):
    sh = shape("wide")
    st = SsmSetup(sh, seed=26)
    before = st.pool.ssm.clone()
    qkv, a = st.tokens(100)
    out = torch.full((100, sh.hv, sh.dv), 7.0, dtype=sh.act_dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    size = gdn.ssm_prefill_workspace_size(st.dims, 4, 100)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None

    def call(ids, cu, sp):
        err.zero_()
        gdn.ssm_prefill(st.dims, st.pool, None, st.params, i32(ids), i32(cu), torch.tensor(sp, device="cuda"), 100,
                        None, 64, qkv.cuda(), a.cuda(), out, ws, err)
        torch.cuda.synchronize()
        return int(err.item())

    # a padded sequence's rows are zeros, an id outside the pool too
    assert call([-1, 99], [0, 40, 60], [0, 0]) == binding.DEV_ERR_SLOT_OOB
    assert (out[:60] == 0).all() and (out[60:] == 7).all()
    # decreasing offsets, rows past the end, a negative start: skipped, reported
    out.fill_(7.0)
    assert call([1, 2, 3, 4], [0, 50, 30, 30, 30], [0, 0, -5, 0]) == binding.DEV_ERR_SEQLENS
    assert (out[50:] == 7).all() and torch.equal(st.pool.ssm[2:], before[2:])
    assert call([5], [60, 140], [0]) == binding.DEV_ERR_SEQLENS
    assert torch.equal(st.pool.ssm[5], before[5])


@pytest.mark.parametrize("name", ["wide", "one_group", "square", "tiny"])
def test_prefill_then_decode_equals_one_prefill(cuda, name):
    """A prompt's prefill followed by decode steps, and a prefill resumed from
    a checkpoint: the states of one long recurrence."""
    sh = shape(name)
    st = SsmSetup(sh, seed=27)
    _prefill(st, [3], [77], [0], 64)
    for _ in range(3):
        out, ref = _decode(st, [3])
        assert_out_close(out, ref, sh.dv, out_tol(sh))
    _prefill(st, [3], [60], [80], 64)


def test_captured_and_replayed(cuda):
    """Decode and prefill in one captured graph, replayed on new inputs, while
    another stream's call is in flight; workspaces of their own."""
    sh = shape("wide")
    st, st2 = SsmSetup(sh, seed=28), SsmSetup(sh, seed=29)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    ids, cu, sp = i32([1, 4]), i32([0, 100, 170]), torch.tensor([0, 30], device="cuda")
    qkv, a = (t.cuda() for t in st.tokens(170))
    dq, da = (t.cuda() for t in st.tokens(2))
    out = torch.zeros((170, sh.hv, sh.dv), dtype=sh.act_dtype, device="cuda")
    dout = torch.zeros((2, sh.hv, sh.dv), dtype=sh.act_dtype, device="cuda")
    size = max(16, gdn.ssm_prefill_workspace_size(st.dims, 2, 170))
    ws, ws2 = (torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2))

    def step(s, w, o, do):
        gdn.ssm_prefill(s.dims, s.pool, None, s.params, ids, cu, sp, 170, None, 64, qkv, a, o, w)
        gdn.ssm_decode_step(s.dims, s.pool, s.params, ids, dq, da, do)

    step(st2, ws2, out, dout)  # loads the kernels
    start = st.pool.ssm.clone(), st.pool.conv.clone()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(st, ws, out, dout)
    out2, dout2 = torch.empty_like(out), torch.empty_like(dout)
    for _ in range(2):
        qkv.copy_(torch.randn(qkv.shape, device="cuda"))
        st.pool.ssm.copy_(start[0]), st.pool.conv.copy_(start[1])
        other = SsmSetup(sh, seed=28)
        torch.cuda.synchronize()
        g.replay()
        with torch.cuda.stream(side):
            step(other, ws2, out2, dout2)
        torch.cuda.synchronize()
        assert torch.equal(out, out2) and torch.equal(dout, dout2)
        assert torch.equal(st.pool.ssm, other.pool.ssm) and torch.equal(st.pool.conv, other.pool.conv)
