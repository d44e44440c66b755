"""The state space prefill on both sides of the rule that cuts sequences into
segments, each call first asserted to be cut or whole: the segments' states
are what makes the workspace larger than the records.  (On the 152 SMs of this
GPU a segment of the calls below is 8 chunks of 64 tokens.)

States after n chunks: 13 n roundings of 2^-24 as in the tests of the paths,
and 2 for each join of a segment: 25 chunks and three joins stay below 1.98e-5,
within the 2e-5 of the others.
"""
import numpy as np
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from hybrid_linear_attention_gdn_gb300 import StatePool
from helpers import assert_out_close, conv_bits_equal, max_rel_l2, out_tol
from oracle import state_space
from ssm_helpers import SsmSetup, f64, shape
from test_gpu_ssm import _prefill

pytestmark = pytest.mark.gpu

RECORD = 57 * 1024  # bytes of a chunk's operands, per group


def _cut(sh, n_seq, total):
    """Whether a call of these sizes is cut: with segments the workspace holds
    at least one state more per sequence."""
    st = SsmSetup(sh, seed=0, device="cpu")
    records = (total // 64 + 2 * n_seq) * sh.hk * RECORD
    history = 3 * n_seq * sh.hv * sh.dv * 2 + 256
    size = gdn.ssm_prefill_workspace_size(st.dims, n_seq, total)
    return size > records + history + 1024


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("name", ["wide", "one_group", "square"])
@pytest.mark.parametrize("total,starts,cut", [(1024, [0], False), (1025, [0], True), (1536, [0, 63], False),
                                              (1537, [0, 63], True)])
def test_both_sides_of_the_rule(cuda, name, total, starts, cut):
    """16 and 17 chunks of one sequence, 24 and 25 of two."""
    sh = shape(name)
    lens = [total] if len(starts) == 1 else [1000, total - 1000]
    assert _cut(sh, len(lens), total) == cut
    _prefill(SsmSetup(sh, seed=81), [5, 2][:len(lens)], lens, starts, 128)


@pytest.mark.parametrize("lens,starts", [([1536], [0]), ([1537], [0]), ([1535], [0]), ([1535], [1]), ([1530], [63]),
                                         ([1088], [0]), ([1089], [63]), ([1100, 0, 512], [0, 5, 0]),
                                         ([1, 1535, 64], [511, 1, 448])])
def test_edges_of_segments(cuda, lens, starts):
    """Sequences that end at, before and behind a segment's last token, and
    neighbours that are one chunk, one token or none."""
    sh = shape("square")
    assert _cut(sh, len(lens), sum(lens))
    _prefill(SsmSetup(sh, seed=82), list(range(len(lens))), lens, starts, 64)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38])
def test_neighbours_of_cut_sequences(cuda, value):
    """Cut sequences, padded ones and unused rows that are not finite leave
    the others' results as they are, bit for bit."""
    sh, lens = shape("wide"), [700, 600, 560]
    one, two = SsmSetup(sh, seed=83), SsmSetup(sh, seed=83)
    cu = np.concatenate([[0], np.cumsum(lens)]) + 2
    total = int(cu[-1]) + 50
    assert _cut(sh, 3, total)
    qkv, a = (t.cuda() for t in one.tokens(total))
    bad_q, bad_a = qkv.clone(), a.clone()
    for lo, hi in ((0, cu[0]), (cu[1], cu[2]), (cu[3], total)):
        bad_q[lo:hi], bad_a[lo:hi] = value, value
    # NaN everywhere: no state or record is read that the call did not write
    ws = torch.full((gdn.ssm_prefill_workspace_size(one.dims, 3, total),), 0xff, dtype=torch.uint8, device="cuda")
    table = _i32([list(range(11)), [-1] * 11, list(range(11, 22))])
    for mid in (3, -1):  # the middle sequence first with a slot of its own, then padded
        outs, cks = [], []
        for s, q, g in ((one, qkv, a), (two, bad_q, bad_a)):
            ck, _ = s.ckpt_pool(22)
            out = torch.full((total, sh.hv, sh.dv), 7.0, dtype=sh.act_dtype, device="cuda")
            gdn.ssm_prefill(s.dims, s.pool, ck, s.params, _i32([1, mid, 6]), _i32(cu.tolist()),
                            torch.tensor([5, 0, 64], device="cuda"), total, table, 64, q, g, out, ws)
            outs.append(out), cks.append(ck)
        for lo, hi in ((0, cu[1]), (cu[2], total)):
            assert torch.equal(outs[0][lo:hi], outs[1][lo:hi]) and torch.isfinite(outs[1][lo:hi]).all()
        assert torch.equal(cks[0].ssm, cks[1].ssm) and torch.equal(cks[0].conv, cks[1].conv)
        if mid == -1:
            assert (outs[1][cu[1]:cu[2]] == 0).all()
    keep = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(one.pool.ssm[keep], two.pool.ssm[keep]) and torch.equal(one.pool.conv[keep], two.pool.conv[keep])


@pytest.mark.parametrize("token", [70, 700, 1499])
@pytest.mark.parametrize("part", ["q", "k", "v", "a"])
def test_a_nan_in_a_segment(cuda, part, token):
    """Nothing before its block of 64 positions in any segment; from its token
    on, in every later segment too, what the recurrence gives it."""
    sh, T = shape("wide"), 1500
    assert _cut(sh, 1, T)
    one, two = SsmSetup(sh, seed=84), SsmSetup(sh, seed=84)
    qkv, a = (t.cuda() for t in one.tokens(T))
    bad_q, bad_a = qkv.clone(), a.clone()
    h, ch = 3, 1  # of the first group
    if part == "a":
        bad_a[token, h] = float("nan")
    else:
        bad_q[token, {"q": 5, "k": sh.hk * sh.dk + 5, "v": 2 * sh.hk * sh.dk + h * sh.dv + ch}[part]] = float("nan")
    ws = torch.full((gdn.ssm_prefill_workspace_size(one.dims, 1, T),), 0xff, dtype=torch.uint8, device="cuda")
    outs, cks = [], []
    for s, q, g in ((one, qkv, a), (two, bad_q, bad_a)):
        ck, _ = s.ckpt_pool(24)
        out = torch.empty((T, sh.hv, sh.dv), dtype=sh.act_dtype, device="cuda")
        gdn.ssm_prefill(s.dims, s.pool, ck, s.params, _i32([1]), _i32([0, T]), torch.tensor([0], device="cuda"), T,
                        _i32([list(range(24))]), 64, q, g, out, ws)
        outs.append(out), cks.append(ck)
    first = token // 64 * 64
    assert torch.equal(outs[0][:first], outs[1][:first])
    assert torch.equal(cks[0].ssm[:first // 64], cks[1].ssm[:first // 64])
    G = sh.hv // sh.hk
    touched = [h] if part in "av" else list(range(G))
    rest = [i for i in range(sh.hv) if i not in touched]
    assert torch.equal(outs[0][:, rest], outs[1][:, rest])
    assert torch.equal(one.pool.ssm[1, rest], two.pool.ssm[1, rest])
    got, state = outs[1][:, touched], two.pool.ssm[1, touched]
    if part == "q":  # four tokens' queries, no state
        assert torch.isnan(got[token:token + 4]).all()
    elif part == "k":  # a column of the state: every output from then on
        assert torch.isnan(got[token:]).all() and torch.isnan(state[:, :, 5]).all()
    elif part == "v":  # a row of the state
        assert torch.isnan(got[token:, 0, ch]).all() and torch.isnan(state[0, ch]).all()
    else:
        assert torch.isnan(got[token:]).all() and torch.isnan(state).all()


@pytest.mark.parametrize("name", ["wide", "square"])
def test_prompt_in_pieces_equals_whole(cuda, name):
    """A cut prompt resumed from its own checkpoint, cut again: the states and
    outputs of the one recurrence."""
    sh, T, at = shape(name), 2700, 1216
    st = SsmSetup(sh, seed=85)
    qkv, a = st.tokens(T)
    out = torch.empty((T, sh.hv, sh.dv), dtype=sh.act_dtype, device="cuda")
    ref = state_space.prefill(st.od, st.opool, None, st.oparams, [6], [0, T], [0], None, 64, f64(qkv), f64(a))
    ck = StatePool.empty(st.dims, 19, "cuda")
    for lo, hi in ((0, at), (at, T)):
        n = hi - lo
        assert _cut(sh, 1, n)
        ws = torch.full((gdn.ssm_prefill_workspace_size(st.dims, 1, n),), 0xff, dtype=torch.uint8, device="cuda")
        gdn.ssm_prefill(st.dims, st.pool, ck if lo == 0 else None, st.params, _i32([6]), _i32([0, n]),
                        torch.tensor([lo], device="cuda"), n, _i32([list(range(19))]) if lo == 0 else None, 64,
                        qkv[lo:hi].cuda(), a[lo:hi].cuda(), out[lo:hi], ws)
        if lo == 0:  # on from the last checkpoint, at the piece's end
            assert torch.equal(ck.ssm[18], st.pool.ssm[6]) and torch.equal(ck.conv[18], st.pool.conv[6])
            st.pool.ssm[6], st.pool.conv[6] = ck.ssm[18], ck.conv[18]
    assert_out_close(out, ref, sh.dv, out_tol(sh), row_floor_rms=True)
    # 43 chunks and five joins: 569 roundings of 2^-24
    assert max_rel_l2(f64(st.pool.ssm), st.opool.ssm, sh.dv * sh.dk) <= 569 * 2.0 ** -24
    assert conv_bits_equal(st.pool.conv, st.opool.conv)


def test_cut_call_captured_and_replayed(cuda):
    """A cut prefill, its checkpoints in free slots of the working pool, and a
    decode step behind it in one graph, replayed on new inputs: the eager
    calls' results, with a workspace that holds what the last replay left."""
    sh, lens = shape("wide", num_slots=24), [1100, 600]
    T = sum(lens)
    assert _cut(sh, 2, T)
    st, ref = SsmSetup(sh, seed=86), SsmSetup(sh, seed=86)
    start = st.pool.ssm.clone(), st.pool.conv.clone()
    ids, cu, sp = _i32([1, 4]), _i32([0, lens[0], T]), torch.tensor([0, 30], device="cuda")
    table = _i32([[5, 6, 7, 8, 9, 10, 11, 12], [13, 14, 15, 16, -1, -1, -1, -1]])
    qkv, a = (t.cuda() for t in st.tokens(T))

    def step(s, ws, out, tok):
        gdn.ssm_prefill(s.dims, s.pool, s.pool, s.params, ids, cu, sp, T, table, 128, qkv, a, out, ws)
        gdn.ssm_decode_step(s.dims, s.pool, s.params, ids, qkv[:2], a[:2], tok)

    size = gdn.ssm_prefill_workspace_size(st.dims, 2, T)
    ws = [torch.full((size,), 0xff, dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = [torch.zeros((T, sh.hv, sh.dv), dtype=sh.act_dtype, device="cuda") for _ in range(2)]
    tok = [torch.zeros((2, sh.hv, sh.dv), dtype=sh.act_dtype, device="cuda") for _ in range(2)]
    step(ref, ws[1], out[1], tok[1])  # loads the kernels
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(st, ws[0], out[0], tok[0])
    for seed in range(3):
        gen = torch.Generator().manual_seed(seed)
        qkv.copy_(torch.randn(qkv.shape, generator=gen))
        for s in (st, ref):
            s.pool.ssm.copy_(start[0]), s.pool.conv.copy_(start[1])
        g.replay()
        step(ref, ws[1], out[1], tok[1])
        torch.cuda.synchronize()
        assert torch.equal(out[0], out[1]) and torch.equal(tok[0], tok[1])
        assert torch.equal(st.pool.ssm, ref.pool.ssm) and torch.equal(st.pool.conv, ref.pool.conv)
        assert torch.equal(st.pool.ssm[[0, 2, 3, 17]], start[0][[0, 2, 3, 17]])  # no other slot
