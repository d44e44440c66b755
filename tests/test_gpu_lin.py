"""Linear attention with a fixed decay against the float64 recurrence: decode
and prefill at every kind of shape, padding, bad ids, odd lengths and starts,
checkpoints, rows outside the sequences, decays at both ends."""
import math

import numpy as np
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from hybrid_linear_attention_gdn_gb300 import binding
from oracle import linear
from helpers import max_rel_l2
from lin_helpers import SHAPES, STATE_TOL, LinSetup, assert_out_close, ckpt_table, f64

pytestmark = pytest.mark.gpu


def _state_close(pool, ref, tol=STATE_TOL):
    d = pool.ssm.shape
    assert max_rel_l2(f64(pool.ssm), ref, d[2] * d[3]) <= tol


def _word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("name", sorted(SHAPES))
@pytest.mark.parametrize("B", [1, 5, 70])
def test_decode(cuda, name, B):
    st = LinSetup(name, 10 + B, num_slots=B + 3)
    ids = torch.randperm(B + 3, generator=st.gen)[:B].to(torch.int32)
    if B > 1:
        ids[B // 2] = -1
    if B > 10:
        ids[3], ids[4] = B + 3, -7  # outside the pool
    err = _word()
    for step in range(2):
        x, out = st.tokens(B), st.out(B)
        n0 = gdn.launch_count(binding.K_LIN_DECODE)
        gdn.lin_decode_step(st.dims, st.pool, st.ld, ids.cuda(), x.cuda(), out, scale=st.scale, dev_err=err)
        assert gdn.launch_count(binding.K_LIN_DECODE) == n0 + 1
        ref = linear.decode_step(st.od, st.opool, st.old, st.scale, ids.tolist(), f64(x))
        assert_out_close(out, ref, st.dims.dv)
    _state_close(st.pool, st.opool)
    assert int(err) == (binding.DEV_ERR_SLOT_OOB if B > 10 else 0)


def test_decode_without_requests_and_strides_of_rows(cuda):
    st = LinSetup("odd_dv", 3)
    before = st.pool.ssm.clone()
    gdn.lin_decode_step(st.dims, st.pool, st.ld, torch.zeros(0, dtype=torch.int32, device="cuda"),
                        st.tokens(0).cuda(), st.out(0))
    assert torch.equal(before, st.pool.ssm)


def test_decode_of_rows_at_odd_addresses(cuda):
    """qkv that starts 2 bytes into its allocation."""
    st = LinSetup("square", 4)
    x, out = st.tokens(3), st.out(3)
    buf = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")
    odd = buf[1:].view(x.shape)
    odd.copy_(x)
    ids = torch.tensor([2, 0, 5], dtype=torch.int32)
    gdn.lin_decode_step(st.dims, st.pool, st.ld, ids.cuda(), odd, out, scale=st.scale)
    ref = linear.decode_step(st.od, st.opool, st.old, st.scale, ids.tolist(), f64(x))
    assert_out_close(out, ref, st.dims.dv)
    _state_close(st.pool, st.opool)


def run_prefill(st, lens, starts, block=64, slots=None, gaps=(0, 0), ckpt=True, max_ckpt=None, err=None):
    """Both sides; `gaps` rows before and behind the sequences must stay."""
    n, total = len(lens), sum(lens) + sum(gaps)
    cu = [gaps[0]]
    for v in lens:
        cu.append(cu[-1] + v)
    ids = torch.randperm(st.opool.shape[0], generator=st.gen)[:n].to(torch.int32) if slots is None \
        else torch.tensor(slots, dtype=torch.int32)
    table, n_ck = ckpt_table(lens, starts, block, st.gen)
    if max_ckpt is not None:
        table = np.ascontiguousarray(table[:, :max_ckpt])
    ck, ock = st.ckpt(n_ck)
    x, out = st.tokens(total), st.out(total)
    oout = np.full(out.shape, 7.0)
    size = gdn.lin_prefill_workspace_size(st.dims, n, total)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda") if size else None
    gdn.lin_prefill(st.dims, st.pool, ck if ckpt else None, st.ld, ids.cuda(),
                    torch.tensor(cu, dtype=torch.int32, device="cuda"),
                    torch.tensor(starts, dtype=torch.int64, device="cuda"), total,
                    torch.from_numpy(table).cuda() if ckpt else None, block, x.cuda(), out, ws, scale=st.scale,
                    dev_err=err)
    linear.prefill(st.od, st.opool, ock if ckpt else None, st.old, st.scale, ids.tolist(), cu, starts, table, block,
                   f64(x), oout)
    assert_out_close(out, oout, st.dims.dv)
    if gaps[0]:
        assert (out[:gaps[0]] == 7).all()
    if gaps[1]:
        assert (out[-gaps[1]:] == 7).all()
    _state_close(st.pool, st.opool)
    _state_close(ck, ock)
    return out, ck


@pytest.mark.parametrize("name", sorted(SHAPES))
@pytest.mark.parametrize("lens,starts", [
    ([1], [0]), ([37], [320]), ([64], [0]), ([65], [63]), ([200, 33], [0, 10]),
    ([129, 0, 1, 64, 70], [77, 5, 63, 64, 4095]),
])
def test_prefill(cuda, name, lens, starts):
    st = LinSetup(name, sum(lens) + sum(starts))
    n0 = gdn.launch_count(binding.K_LIN_PREFILL)
    run_prefill(st, lens, starts)
    assert gdn.launch_count(binding.K_LIN_PREFILL) == n0 + 1


@pytest.mark.parametrize("name", ["square", "narrow", "tiny"])
def test_prefill_around_the_sequences(cuda, name):
    """Padded and out-of-range slots, rows around the sequences, checkpoint
    blocks of 128, a table with fewer columns than boundaries."""
    st, err = LinSetup(name, 5), _word()
    run_prefill(st, [70, 3, 150, 66], [0, 9, 100, 64], block=128, slots=[3, -1, 0, 99], gaps=(5, 9), err=err)
    assert int(err) == binding.DEV_ERR_SLOT_OOB
    run_prefill(LinSetup(name, 6), [300, 20], [0, 50], max_ckpt=2)
    run_prefill(LinSetup(name, 7), [300, 20], [0, 50], ckpt=False)


@pytest.mark.parametrize("name", ["square", "tiny"])
@pytest.mark.parametrize("log_decay", [0.0, -1e-7, -3.0, -40.0, -1e4, -math.inf])
def test_extreme_decays(cuda, name, log_decay):
    st = LinSetup(name, 8)
    st.log_decay.fill_(log_decay)
    st.ld, st.old = st.log_decay.cuda(), f64(st.log_decay)
    run_prefill(st, [60, 7], [0, 30])
    x, out = st.tokens(2), st.out(2)
    ids = torch.tensor([1, 6], dtype=torch.int32)
    gdn.lin_decode_step(st.dims, st.pool, st.ld, ids.cuda(), x.cuda(), out, scale=st.scale)
    ref = linear.decode_step(st.od, st.opool, st.old, st.scale, ids.tolist(), f64(x))
    assert_out_close(out, ref, st.dims.dv)
    _state_close(st.pool, st.opool)


@pytest.mark.parametrize("name", ["square", "tiny"])
def test_inconsistent_sequences(cuda, name):
    """Rows outside the batch or a negative position: that sequence is skipped, the others run."""
    st, err = LinSetup(name, 9), _word()
    x, out = st.tokens(50), st.out(50)
    before = st.pool.ssm.clone()
    cu = torch.tensor([0, 20, 30, 60], dtype=torch.int32, device="cuda")
    sp = torch.tensor([0, -1, 0], dtype=torch.int64, device="cuda")
    ids = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    size = gdn.lin_prefill_workspace_size(st.dims, 3, 50)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    gdn.lin_prefill(st.dims, st.pool, None, st.ld, ids, cu, sp, 50, None, 64, x.cuda(), out, ws, scale=st.scale,
                    dev_err=err)
    ref = linear.prefill(st.od, st.opool, None, st.old, st.scale, [0], [0, 20], [0], np.zeros((1, 0), int), 64, f64(x))
    assert int(err) == binding.DEV_ERR_SEQLENS
    assert_out_close(out[:20], ref[:20], st.dims.dv)
    assert (out[20:] == 7).all() and torch.equal(st.pool.ssm[1:], before[1:])
    _state_close(st.pool, st.opool)


def test_bad_checkpoint_ids_are_reported(cuda):
    st, err = LinSetup("square", 11), _word()
    ck, _ = st.ckpt(2)
    x, out = st.tokens(200), st.out(200)
    size = gdn.lin_prefill_workspace_size(st.dims, 1, 200)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    gdn.lin_prefill(st.dims, st.pool, ck, st.ld, i32([0]), i32([0, 200]), torch.zeros(1, dtype=torch.int64, device="cuda"),
                    200, i32([[-1, 7, 1]]), 64, x.cuda(), out, ws, scale=st.scale, dev_err=err)
    assert int(err) == binding.DEV_ERR_SLOT_OOB
    assert (ck.ssm[0] == -5).all()
    o = st.opool[:1].copy()
    linear.prefill(st.od, o, None, st.old, st.scale, [0], [0, 192], [0], np.zeros((1, 0), int), 64, f64(x))
    assert max_rel_l2(f64(ck.ssm[1:]), o, 128 * 128) <= STATE_TOL


def test_states_move_between_slots(cuda):
    """Copies, zeroing and records of slots without a conv history."""
    st = LinSetup("square", 12)
    pool, dims = st.pool, st.dims
    before = pool.ssm.clone()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    gdn.slot_copy(dims, pool, pool, i32([1]), i32([4]))
    gdn.slot_zero(dims, pool, i32([2]))
    rec = torch.empty(2 * gdn.state_record_bytes(dims), dtype=torch.uint8, device="cuda")
    gdn.state_pack(dims, pool, i32([0, 3]), rec)
    gdn.state_unpack(dims, rec, pool, i32([6, 5]))
    want = before.clone()
    want[4], want[2], want[6], want[5] = before[1], 0, before[0], before[3]
    assert torch.equal(pool.ssm, want)


def test_workspace_refusals(cuda):
    """A long prompt is cut and needs its workspace."""
    st = LinSetup("square", 13)
    n = 8192
    size = gdn.lin_prefill_workspace_size(st.dims, 1, n)
    assert size > 0
    x, out = st.tokens(n).cuda(), st.out(n)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    ws = torch.empty(size + 256, dtype=torch.uint8, device="cuda")
    before = st.pool.ssm.clone()
    for bad in (None, ws[:size - 1], ws[16:size + 16]):
        with pytest.raises(gdn.GdnError, match="INVALID_ARG"):
            gdn.lin_prefill(st.dims, st.pool, None, st.ld, i32([0]), i32([0, n]),
                            torch.zeros(1, dtype=torch.int64, device="cuda"), n, None, 64, x, out, bad)
    assert torch.equal(before, st.pool.ssm) and (out == 7).all()


@pytest.mark.parametrize("name", ["square", "tiny", "dk64"])
@pytest.mark.parametrize("lens,starts", [([1500], [0]), ([1300, 700], [77, 5000]), ([40, 2100, 3], [1, 63, 64])])
def test_segments(cuda, name, lens, starts):
    """Sequences that are cut: states, outputs and checkpoints across the cuts."""
    st = LinSetup(name, 14)
    assert gdn.lin_prefill_workspace_size(st.dims, len(lens), sum(lens)) > 0
    run_prefill(st, lens, starts, block=128)


def test_segments_of_padded_sequences(cuda):
    st, err = LinSetup("square", 15), torch.zeros(1, dtype=torch.int32, device="cuda")
    run_prefill(st, [1300, 900], [5, 0], slots=[-1, 3], gaps=(3, 70), err=err)
    assert int(err) == 0


@pytest.mark.parametrize("name", ["square", "tiny"])
def test_long_memory(cuda, name):
    """Decays that remember some 2,000 tokens: a rounded lambda would be off by
    2000 * 2^-25 = 6e-5.  A token's roundings (at most 2^-23 of the state) are
    independent: some sqrt(2000) 2^-24 = 3e-6 at the state."""
    st = LinSetup(name, 16, rates=(1 / 1500, 1 / 2500))
    run_prefill(st, [3000], [10], block=1024)
    ids = torch.tensor([2], dtype=torch.int32)
    st.opool = f64(st.pool.ssm).copy()
    x, out = st.tokens(2500), st.out(1)
    xd, idd = x.cuda(), ids.cuda()
    for i in range(2500):
        gdn.lin_decode_step(st.dims, st.pool, st.ld, idd, xd[i:i + 1], out, scale=st.scale)
        ref = linear.decode_step(st.od, st.opool, st.old, st.scale, [2], f64(x[i:i + 1]))
    assert_out_close(out, ref, st.dims.dv)
    _state_close(st.pool, st.opool)
