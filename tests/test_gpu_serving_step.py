"""The step of a serving loop as its calls run together: maps of the batch,
residual norm, projection, state space prefill or decode with the maps'
offsets and checkpoint ids, gated norm, residual norm with 8-bit output; a
prompt resumed from a checkpoint; a decode step captured once and replayed.

The recurrence runs in float64 on the projected rows the device used, the
norms on their own inputs; tolerances as in the files of the single calls.
"""
import numpy as np
import pytest
import torch

import oracle
import hybrid_linear_attention_gdn_gb300 as gdn
from hybrid_linear_attention_gdn_gb300 import binding
from oracle import state_space
from helpers import assert_out_close, conv_bits_equal, max_rel_l2, out_tol
from ssm_helpers import STATE_TOL, SsmSetup, f64, shape

pytestmark = pytest.mark.gpu

BLOCK, MAX_BLOCKS, D = 64, 8, 256


class Loop:
    """One state space layer behind a residual norm; states, KV block tables
    and the float64 twin of the states."""

    def __init__(self, name, n_seq, rows, seed):
        self.sh = sh = shape(name, num_slots=n_seq + 2)
        self.st = st = SsmSetup(sh, seed)
        g = torch.Generator().manual_seed(seed)
        self.n, self.rows = n_seq, rows
        dev = lambda t: t.cuda()
        self.w_norm = dev(1 + 0.1 * torch.randn(D, generator=g))
        self.w_gate = dev(1 + 0.1 * torch.randn(sh.dv, generator=g))
        cols = sh.channels + sh.hv + sh.hv * sh.dv
        self.proj = dev((torch.randn((D, cols), generator=g) / D ** 0.5).to(sh.act_dtype))
        self.back = dev((torch.randn((sh.hv * sh.dv, D), generator=g) / (sh.hv * sh.dv) ** 0.5).to(sh.act_dtype))
        n_ids = n_seq * MAX_BLOCKS
        self.ck, self.ock = st.ckpt_pool(n_ids)
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
        self.lens, self.starts = i32(n_seq), torch.zeros(n_seq, dtype=torch.int64, device="cuda")
        self.table, self.free = i32(n_seq, MAX_BLOCKS) - 1, torch.randperm(n_ids, generator=g).to(torch.int32).cuda()
        self.n_free = i32(1) + n_ids
        self.cu, self.ckpt = i32(n_seq + 1), i32(n_seq, MAX_BLOCKS)
        self.seq, self.pos = i32(rows), torch.zeros(rows, dtype=torch.int64, device="cuda")
        self.slot = torch.zeros(rows, dtype=torch.int64, device="cuda")
        self.err = i32(1)
        self.ids = torch.arange(n_seq, dtype=torch.int32, device="cuda") + 1
        size = gdn.ssm_prefill_workspace_size(st.dims, n_seq, rows)
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
        act = lambda *s: torch.zeros(s, dtype=sh.act_dtype, device="cuda")
        self.x, self.y, self.out = act(rows, D), act(rows, D), act(rows, sh.hv, sh.dv)
        self.h = torch.zeros((rows, D), device="cuda")
        self.q8 = torch.zeros((rows, D), dtype=torch.float8_e4m3fn, device="cuda")
        self.sc = torch.zeros((rows, D // 32), dtype=torch.uint8, device="cuda")

    def step(self, decode):
        """Everything on the device; nothing is read back."""
        sh, st = self.sh, self.st
        gdn.batch_maps(self.lens, self.starts, BLOCK, self.table, self.free, self.n_free, self.cu, self.ckpt, self.seq,
                       self.pos, self.slot, dev_err=self.err)
        gdn.add_rmsnorm(self.x, self.h, self.w_norm, y=self.y)
        p = self.y @ self.proj
        self.qkv, self.a, z = (t.contiguous() for t in p.split([sh.channels, sh.hv, sh.hv * sh.dv], dim=1))
        if decode:
            gdn.ssm_decode_step(st.dims, st.pool, st.params, self.ids, self.qkv[:self.n], self.a[:self.n],
                                self.out[:self.n], self.err)
        else:
            gdn.ssm_prefill(st.dims, st.pool, self.ck, st.params, self.ids, self.cu, self.starts, self.rows, self.ckpt,
                            BLOCK, self.qkv, self.a, self.out, self.ws, self.err)
        self.gated = gdn.gated_rmsnorm(st.dims, self.out.clone(), z.view(-1, sh.hv, sh.dv), self.w_gate)
        self.x.copy_(self.gated.view(self.rows, -1) @ self.back)
        gdn.add_rmsnorm(self.x, self.h, self.w_norm, q8=self.q8, scales=self.sc, group=32)
        self.starts += self.lens

    def check(self, decode, lens, starts):
        """The states, checkpoints and outputs of the step that ran."""
        sh, st = self.sh, self.st
        torch.cuda.synchronize()
        assert int(self.err.item()) == 0
        ids, cu = self.ids.tolist(), np.concatenate([[0], np.cumsum(lens)])
        assert self.cu.tolist() == cu.tolist()
        if decode:
            ref, _ = state_space.decode_step(st.od, st.opool, st.oparams, ids, f64(self.qkv)[:self.n],
                                             f64(self.a)[:self.n])
        else:
            ref = state_space.prefill(st.od, st.opool, self.ock, st.oparams, ids, cu, starts, self.ckpt.cpu().numpy(),
                                      BLOCK, f64(self.qkv), f64(self.a))
            assert max_rel_l2(f64(self.ck.ssm), self.ock.ssm, sh.dv * sh.dk) <= STATE_TOL
            assert conv_bits_equal(self.ck.conv, self.ock.conv)
        n = int(cu[-1])
        assert_out_close(self.out[:n], ref[:n], sh.dv, out_tol(sh), row_floor_rms=not decode)
        assert max_rel_l2(f64(st.pool.ssm), st.opool.ssm, sh.dv * sh.dk) <= STATE_TOL
        assert conv_bits_equal(st.pool.conv, st.opool.conv)
        # the blocks a request completed hold the states at their ends
        for r in range(self.n):
            full = range(starts[r] // BLOCK, (starts[r] + lens[r]) // BLOCK)
            want = [int(self.table[r, i]) for i in full]
            assert self.ckpt[r].tolist() == want + [-1] * (MAX_BLOCKS - len(want))
        # the residual's norm in 8 bits: half an e4m3 step of y / scale
        h = self.h.double()
        y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * self.w_norm.double()
        z = y / torch.exp2(self.sc.double() - 127).repeat_interleave(32, 1)
        step = torch.maximum(z.abs() * 2.0 ** -4, torch.full_like(z, 2.0 ** -10))
        assert ((self.q8.double() - z).abs() <= step + 1e-4 * z.abs()).all()


@pytest.mark.parametrize("name", ["wide", "square", "tiny"])
def test_prompts_then_decode_then_more_prompt(cuda, name):
    n, lens = 3, [150, 70, 9]
    L = Loop(name, n, 260, seed=51)
    starts = [0, 0, 0]
    for lens in ([150, 70, 9], [1, 1, 1], [1, 1, 1], [40, 0, 200], [1, 1, 1]):
        decode = lens == [1, 1, 1]
        L.lens.copy_(torch.tensor(lens))
        L.x.copy_(torch.randn((L.rows, D), generator=L.st.gen))
        L.step(decode)
        L.check(decode, lens, starts)
        starts = [s + l for s, l in zip(starts, lens)]
    assert L.starts.tolist() == starts


@pytest.mark.parametrize("name", ["wide", "tiny"])
def test_prefix_resumed_from_its_checkpoint(cuda, name):
    """A prompt whose first two blocks another request computed: the state at
    their end is copied from the checkpoint, and the rest of the prompt gives
    what the whole prompt gives."""
    L = Loop(name, 1, 190, seed=52)
    st, sh = L.st, L.sh
    L.lens.fill_(190)
    L.x.copy_(torch.randn((190, D), generator=st.gen))
    L.step(False)
    qkv, a, whole = L.qkv, L.a, L.out.clone()
    gdn.slot_copy(st.dims, L.ck, st.pool, L.table[0, 1:2].contiguous(),
                  torch.tensor([2], dtype=torch.int32, device="cuda"))
    out = torch.empty((62, sh.hv, sh.dv), dtype=sh.act_dtype, device="cuda")
    size = gdn.ssm_prefill_workspace_size(st.dims, 1, 62)
    gdn.ssm_prefill(st.dims, st.pool, None, st.params, torch.tensor([2], dtype=torch.int32, device="cuda"),
                    torch.tensor([0, 62], dtype=torch.int32, device="cuda"), torch.tensor([128], device="cuda"), 62,
                    None, BLOCK, qkv[128:], a[128:], out,
                    torch.empty(size, dtype=torch.uint8, device="cuda") if size else None)
    torch.cuda.synchronize()
    # the chunks' boundaries are the positions' in both: the same arithmetic
    # (were it not, two roundings of at most 2^-8 and 2 out_tol would part them)
    assert_out_close(out, f64(whole[128:]), sh.dv, 2 * 2.0 ** -8 + 2 * out_tol(sh), row_floor_rms=True)
    assert max_rel_l2(f64(st.pool.ssm[2]), f64(st.pool.ssm[1]), sh.dv * sh.dk) <= 2 * STATE_TOL
    assert torch.equal(st.pool.conv[2], st.pool.conv[1])


@pytest.mark.parametrize("name", ["wide", "tiny"])
def test_captured_decode_loop(cuda, name):
    """The whole decode step in one graph: lengths, block tables and states
    move on by themselves from replay to replay, as in eager steps."""
    n = 5
    one, two = Loop(name, n, n, seed=53), Loop(name, n, n, seed=53)
    x = torch.randn((6, n, D), generator=one.st.gen)
    for L in (one, two):
        L.lens.fill_(1)
        L.starts += torch.arange(n, device="cuda") + 60
        L.table[:, 0] = L.free[-n:]
        L.n_free -= n
    warm = Loop(name, n, n, seed=53)  # loads the kernels
    warm.lens.fill_(1)
    warm.step(True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    counts = binding.launch_counts()
    with torch.cuda.graph(graph):
        one.step(True)
    assert binding.launch_counts()[binding.K_SSM_DECODE] == counts[binding.K_SSM_DECODE] + 1
    for t in range(6):
        one.x.copy_(x[t]), two.x.copy_(x[t])
        graph.replay()
        two.step(True)
        torch.cuda.synchronize()
        for k in ("out", "h", "q8", "sc", "cu", "table", "n_free", "starts", "slot", "pos", "ckpt", "err"):
            assert torch.equal(getattr(one, k).view(torch.uint8), getattr(two, k).view(torch.uint8)), (t, k)
        assert torch.equal(one.st.pool.ssm, two.st.pool.ssm)
    assert int(one.err.item()) == 0 and (one.table[:, 1] >= 0).all()
    assert int(one.n_free.item()) == n * MAX_BLOCKS - 2 * n
