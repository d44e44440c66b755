"""The state space prefill's ways of working, each against the recurrence:
segments, the token recurrence on shapes of the chunked form, tensors beyond
32-bit offsets, inputs that are not finite next to it, other streams.

States after 24 chunks: a chunk adds at most 13 roundings of 2^-24 to a state
(split operands 2^-22 each, scales, the carried state's product and sum), so
24 chunks stay below 24 * 13 * 2^-24 = 1.9e-5, within the 2e-5 of the others.
"""
import numpy as np
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from hybrid_linear_attention_gdn_gb300 import SsmParams, StatePool, binding
from ssm_helpers import SsmSetup, f64, shape
from test_gpu_ssm import _decode, _prefill
from helpers import assert_out_close, out_tol

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("name", ["wide", "one_group", "square"])
def test_few_long_sequences(cuda, name):
    """Few chains: the long sequence is cut into segments, checkpoints fall
    into every one of them, the short ones stay whole."""
    _prefill(SsmSetup(shape(name), seed=31), [3, 1, 6], [1450, 300, 2], [37, 64, 0], 128)


@pytest.mark.parametrize("lens,starts", [([512], [0]), ([513], [0]), ([511], [1]), ([1024, 1024], [0, 64]),
                                         ([1025, 0, 700], [63, 0, 1])])
def test_segment_edges(cuda, lens, starts):
    """Lengths at and beside whole segments of 8 chunks."""
    _prefill(SsmSetup(shape("square"), seed=32), list(range(len(lens))), lens, starts, 64)


@pytest.mark.parametrize("decay", [(1.0, 4.0), (1e-5, 1e-4)])
def test_segments_strong_and_weak_decay(cuda, decay):
    _prefill(SsmSetup(shape("wide"), seed=33, decay=decay), [4], [1400], [33], 256)


def test_segments_zero_decay(cuda):
    """A decay of exactly 0 forgets everything before the token."""
    st = SsmSetup(shape("wide"), seed=34)
    st.params.A_log[::3] = 30.0
    st.oparams.A_log[::3] = 30.0
    _prefill(st, [4], [1200], [0], 128)


@pytest.mark.parametrize("name", ["wide", "square"])
@pytest.mark.parametrize("lens,starts", [([130, 65, 0, 200], [7, 63, 0, 1001]), ([300], [0])])
def test_recurrence_on_chunked_shapes(cuda, name, lens, starts, monkeypatch):
    monkeypatch.setenv("GDN_SSM_PREFILL_PATH", "recurrent")
    _prefill(SsmSetup(shape(name), seed=35), [5, 1, 0, 2][:len(lens)], lens, starts, 64, lead=1, extra=3)


def test_unaligned_rows_take_the_recurrence(cuda):
    """Rows that do not start on a 16-byte boundary: no copy engine."""
    sh = shape("wide")
    st, st2 = SsmSetup(sh, seed=36), SsmSetup(sh, seed=36)
    qkv, a = (t.cuda() for t in st.tokens(150))
    odd = torch.empty(qkv.numel() + 1, dtype=qkv.dtype, device="cuda")[1:].view_as(qkv).copy_(qkv)
    ws = torch.empty(gdn.ssm_prefill_workspace_size(st.dims, 1, 150), dtype=torch.uint8, device="cuda")
    outs = [torch.empty((150, sh.hv, sh.dv), dtype=sh.act_dtype, device="cuda") for _ in range(2)]
    for s, x, o in ((st, qkv, outs[0]), (st2, odd, outs[1])):
        gdn.ssm_prefill(s.dims, s.pool, None, s.params, _i32([2]), _i32([0, 150]), torch.tensor([0], device="cuda"),
                        150, None, 64, x, a, o, ws)
    # two bf16 roundings of values within out_tol of the exact ones: a row's
    # elements differ by at most 2 * 2^-8 relative for the roundings, and
    # 2 out_tol for what was rounded
    assert_out_close(outs[1], f64(outs[0]), sh.dv, 2 * 2.0 ** -8 + 2 * out_tol(sh), row_floor_rms=True)
    assert torch.equal(st.pool.conv, st2.pool.conv)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("lens", [[70, 41, 65], [600, 100, 37]])
def test_neighbours_that_are_not_finite(cuda, value, lens):
    """Sequences, padded sequences and unused rows that are not finite leave
    the others' results as they are, bit for bit."""
    sh = shape("wide")
    one, two = SsmSetup(sh, seed=37), SsmSetup(sh, seed=37)
    cu = np.concatenate([[0], np.cumsum(lens)]) + 2
    total = int(cu[-1]) + 50
    qkv, a = (t.cuda() for t in one.tokens(total))
    bad_q, bad_a = qkv.clone(), a.clone()
    for lo, hi in ((0, cu[0]), (cu[1], cu[2]), (cu[3], total)):
        bad_q[lo:hi], bad_a[lo:hi] = value, value
    ws = torch.full((gdn.ssm_prefill_workspace_size(one.dims, 3, total),), 0xff, dtype=torch.uint8, device="cuda")
    outs, cks = [], []
    # the middle sequence first with a slot of its own, then padded
    for mid in (3, -1):
        for s, q, g in ((one, qkv, a), (two, bad_q, bad_a)):
            ck, _ = s.ckpt_pool(24)
            table = _i32([[0, 1, 2, 3, 4, 5, 6, 7, 8, 9], [-1] * 10, list(range(10, 20))])
            out = torch.full((total, sh.hv, sh.dv), 7.0, dtype=sh.act_dtype, device="cuda")
            gdn.ssm_prefill(s.dims, s.pool, ck, s.params, _i32([1, mid, 6]), _i32(cu.tolist()),
                            torch.tensor([5, 0, 64], device="cuda"), total, table, 64, q, g, out, ws)
            outs.append(out), cks.append(ck)
    for k in (0, 2):
        for lo, hi in ((0, cu[1]), (cu[2], total)):
            assert torch.equal(outs[k][lo:hi], outs[k + 1][lo:hi])
        assert torch.equal(cks[k].ssm, cks[k + 1].ssm) and torch.equal(cks[k].conv, cks[k + 1].conv)
        assert torch.isfinite(outs[k + 1][cu[0]:cu[1]]).all() and torch.isfinite(outs[k + 1][cu[2]:cu[3]]).all()
    assert (outs[3][cu[1]:cu[2]] == 0).all()
    keep = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(one.pool.ssm[keep], two.pool.ssm[keep]) and torch.equal(one.pool.conv[keep], two.pool.conv[keep])


@pytest.mark.parametrize("part", ["q", "v", "a"])
def test_a_nan_reaches_nothing_before_its_chunk(cuda, part):
    sh = shape("wide")
    one, two = SsmSetup(sh, seed=38), SsmSetup(sh, seed=38)
    qkv, a = (t.cuda() for t in one.tokens(200))
    bad_q, bad_a = qkv.clone(), a.clone()
    if part == "a":
        bad_a[140, 3] = float("nan")
    else:
        bad_q[140, 5 if part == "q" else 2 * sh.hk * sh.dk + 3 * sh.dv + 1] = float("nan")
    ws = torch.empty(gdn.ssm_prefill_workspace_size(one.dims, 1, 200), dtype=torch.uint8, device="cuda")
    outs, cks = [], []
    for s, q, g in ((one, qkv, a), (two, bad_q, bad_a)):
        ck, _ = s.ckpt_pool(4)
        out = torch.empty((200, sh.hv, sh.dv), dtype=sh.act_dtype, device="cuda")
        gdn.ssm_prefill(s.dims, s.pool, ck, s.params, _i32([1]), _i32([0, 200]), torch.tensor([0], device="cuda"),
                        200, _i32([[0, 1, 2]]), 64, q, g, out, ws)
        outs.append(out), cks.append(ck)
    assert torch.equal(outs[0][:128], outs[1][:128]) and torch.isnan(outs[1][140]).any()
    assert torch.equal(cks[0].ssm[:2], cks[1].ssm[:2])
    heads = [h for h in range(sh.hv) if h != 3] if part != "q" else list(range(sh.hv // sh.hk, sh.hv))
    if part == "v":  # the two heads of a tile's products share no row
        assert torch.isnan(outs[1][140, 3]).any()
    assert torch.equal(outs[0][:, heads], outs[1][:, heads])


def test_slots_and_rows_beyond_32_bits(cuda):
    """A pool of more than 2^31 state elements and packed rows of more than
    2^31 elements: the same results as at the front."""
    sh = shape("wide")
    st = SsmSetup(sh, seed=39)
    slots = 2 ** 31 // (sh.hv * sh.dv * sh.dk) + 60
    rows = 2 ** 31 // sh.channels + 100
    far = StatePool.empty(st.dims, slots, "cuda")
    qkv, a = (t.cuda() for t in st.tokens(90))
    big_q = torch.zeros((rows, sh.channels), dtype=sh.act_dtype, device="cuda")
    big_a = torch.zeros((rows, sh.hv), dtype=sh.act_dtype, device="cuda")
    big_o = torch.zeros((rows, sh.hv, sh.dv), dtype=sh.act_dtype, device="cuda")
    big_q[-90:], big_a[-90:] = qkv, a
    for s in (slots - 1, slots - 2):
        far.ssm[s], far.conv[s] = st.pool.ssm[slots - s], st.pool.conv[slots - s]
    sp = torch.tensor([60, 0], device="cuda")

    def run(pool, ids, lo, total, q, g, out):
        ws = torch.empty(gdn.ssm_prefill_workspace_size(st.dims, 2, total), dtype=torch.uint8, device="cuda")
        ck, _ = st.ckpt_pool(4)
        gdn.ssm_prefill(st.dims, pool, ck, st.params, _i32(ids), _i32([lo, lo + 50, lo + 90]), sp, total,
                        _i32([[1], [2]]), 64, q, g, out, ws)
        o = out[-90:].clone()
        d = torch.empty((2, sh.hv, sh.dv), dtype=sh.act_dtype, device="cuda")
        gdn.ssm_decode_step(st.dims, pool, st.params, _i32(ids), q[-2:], g[-2:], d)
        return o, d, ck, pool.ssm[ids], pool.conv[ids]

    out = torch.zeros((90, sh.hv, sh.dv), dtype=sh.act_dtype, device="cuda")
    got = run(far, [slots - 1, slots - 2], rows - 90, rows, big_q, big_a, big_o)
    ref = run(st.pool, [1, 2], 0, 90, qkv, a, out)
    assert torch.equal(got[2].ssm, ref[2].ssm) and torch.equal(got[2].conv, ref[2].conv)
    for k in (0, 1, 3, 4):
        assert torch.equal(got[k], ref[k])
    assert (big_o[:-90] == 0).all() if big_o[:-90].numel() < 2 ** 31 else True


def test_many_sequences(cuda):
    """More sequences than a lookup pass, most of one token, some empty."""
    rng = np.random.default_rng(40)
    lens = np.where(rng.random(700) < 0.8, 1, rng.integers(0, 70, 700)).tolist()
    st = SsmSetup(shape("one_group", num_slots=701), seed=40)
    _prefill(st, rng.permutation(701)[:700].tolist(), lens, rng.integers(0, 130, 700).tolist(), 64)


@pytest.mark.parametrize("name", ["wide", "tiny"])
def test_other_streams_and_order(cuda, name):
    """Prefill and decode on a stream that waits for the current one, passed
    explicitly and as the current stream; the calls of a stream stay in order."""
    sh = shape(name)
    one, two = SsmSetup(sh, seed=41), SsmSetup(sh, seed=41)
    qkv, a = (t.cuda() for t in one.tokens(130))
    res = []
    for s, given in ((one, True), (two, False)):
        stream = torch.cuda.Stream()
        size = gdn.ssm_prefill_workspace_size(s.dims, 1, 130)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
        out = torch.zeros((130, sh.hv, sh.dv), dtype=sh.act_dtype, device="cuda")
        d = torch.zeros((1, sh.hv, sh.dv), dtype=sh.act_dtype, device="cuda")
        ids, cu, sp = _i32([2]), _i32([0, 130]), torch.tensor([0], device="cuda")
        stream.wait_stream(torch.cuda.current_stream())
        kw = dict(stream=stream) if given else {}
        with torch.cuda.stream(torch.cuda.current_stream() if given else stream):
            for _ in range(3):
                gdn.ssm_prefill(s.dims, s.pool, None, s.params, ids, cu, sp, 130, None, 64, qkv, a, out, ws, **kw)
                gdn.ssm_decode_step(s.dims, s.pool, s.params, ids, qkv[:1], a[:1], d, **kw)
        torch.cuda.current_stream().wait_stream(stream)
        res.append((out, d, s.pool.ssm, s.pool.conv))
    torch.cuda.synchronize()
    for x, y in zip(*res):
        assert torch.equal(x, y)


def test_no_tokens(cuda):
    """No sequences, or sequences of no tokens: nothing changes."""
    sh = shape("wide")
    st = SsmSetup(sh, seed=42)
    before = st.pool.ssm.clone(), st.pool.conv.clone()
    e = lambda *s, dt=sh.act_dtype: torch.empty(s, dtype=dt, device="cuda")
    for n in (0, 2):
        gdn.ssm_prefill(st.dims, st.pool, None, st.params, _i32(list(range(n))), _i32([0] * (n + 1)),
                        e(n, dt=torch.int64).zero_(), 0, None, 64, e(0, sh.channels), e(0, sh.hv), e(0, sh.hv, sh.dv),
                        None)
    gdn.ssm_decode_step(st.dims, st.pool, st.params, _i32([]), e(0, sh.channels), e(0, sh.hv), e(0, sh.hv, sh.dv))
    torch.cuda.synchronize()
    assert torch.equal(st.pool.ssm, before[0]) and torch.equal(st.pool.conv, before[1])


def test_refusals_next_to_a_gpu(cuda):
    """Host tensors, short or missing workspaces and wrong error words are
    refused before anything is launched."""
    sh = shape("wide")
    st = SsmSetup(sh, seed=43)
    qkv, a = (t.cuda() for t in st.tokens(100))
    out = torch.empty((100, sh.hv, sh.dv), dtype=sh.act_dtype, device="cuda")
    size = gdn.ssm_prefill_workspace_size(st.dims, 1, 100)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    sp = torch.tensor([0], device="cuda")
    good = dict(ids=_i32([1]), cu=_i32([0, 100]), sp=sp, ck=None, ck_ids=None, block=64, qkv=qkv, a=a, out=out, ws=ws,
                err=_i32([0]))
    before, n0 = st.pool.ssm.clone(), binding.launch_counts()
    for bad in (dict(ids=torch.tensor([1], dtype=torch.int32)), dict(cu=_i32([0, 100]).cpu()), dict(sp=sp.cpu()),
                dict(sp=sp.int()), dict(ws=None), dict(ws=ws[:-1]), dict(ws=ws[1:]), dict(ws=ws.cpu()), dict(block=0),
                dict(block=96), dict(err=torch.zeros(1, dtype=torch.int32)), dict(err=sp), dict(qkv=qkv.cpu()),
                dict(out=out.transpose(1, 2)), dict(a=a[:99]), dict(ck_ids=_i32([[0]]))):
        k = {**good, **bad}
        with pytest.raises(gdn.GdnError) as e:
            gdn.ssm_prefill(st.dims, st.pool, k["ck"], st.params, k["ids"], k["cu"], k["sp"], 100, k["ck_ids"],
                            k["block"], k["qkv"], k["a"], k["out"], k["ws"], k["err"])
        assert e.value.status == binding.ERR_INVALID_ARG, bad
    with pytest.raises(gdn.GdnError):
        gdn.ssm_decode_step(st.dims, st.pool, st.params, _i32([1]), qkv[:1], a[:1], out[:1], good["err"].cpu())
    with pytest.raises(gdn.GdnError):
        gdn.ssm_decode_step(st.dims, st.pool, SsmParams(*(getattr(st.params, k).cpu() for k in
                                                          ("conv_w", "conv_bias", "A_log", "dt_bias", "D"))),
                            _i32([1]), qkv[:1], a[:1], out[:1])
    assert binding.launch_counts() == n0 and torch.equal(st.pool.ssm, before)
