"""The calls of a hybrid model's step together, as a server makes them: maps,
norm, a linear-attention layer with rotated heads and a gated norm, an
attention layer's keys and values into pages; then branches of a request, their
tokens, their end, and a compaction of the pages.  Values against float64, the
blocks against plain lists, a captured step against eager calls bit for bit.

Tolerances: those of the single calls.  Their inputs are taken as the calls
before them left them, so that no error is counted twice.
"""
import numpy as np
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
import oracle
from hybrid_linear_attention_gdn_gb300 import Dims, StatePool
from helpers import max_rel_l2
from lin_helpers import STATE_TOL, assert_out_close, f64
from oracle import linear
from test_gpu_qk_norm_rope import TOL, close, reference, table

pytestmark = pytest.mark.gpu
BLOCK, ROWS, MB, NB = 64, 5, 8, 32
HQ, HK, D, MODEL = 4, 2, 64, 256


class Server:
    def __init__(self, seed):
        self.g = g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g)
        self.dims = d = Dims(2, 4, 128, 128, 1, torch.bfloat16, torch.bfloat16)
        self.pool = StatePool(torch.zeros((ROWS, d.hv, d.dv, d.dk), device="cuda"))
        self.ck = StatePool(torch.zeros((NB, d.hv, d.dv, d.dk), device="cuda"))
        self.ld = -(0.02 + 0.1 * torch.rand(d.hv, generator=g)).cuda()
        w = lambda n: (rnd(MODEL, n) * MODEL ** -0.5).to(torch.bfloat16).cuda()
        self.w_lin, self.w_z, self.w_att = w(d.channels), w(d.hv * d.dv), w((HQ + 2 * HK) * D)
        self.norm, self.qn, self.kn, self.aq, self.ak, self.on = (
            (1 + 0.2 * rnd(n)).cuda() for n in (MODEL, 128, 128, D, D, d.dv))
        self.cs, self.cs2 = table(BLOCK * MB, 128).cuda(), table(BLOCK * MB, 32).cuda()
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        self.free = i32(torch.randperm(NB, generator=g).tolist())
        self.nf, self.refs = i32([NB]), i32([0] * NB)
        self.table = torch.full((ROWS, MB), -1, dtype=torch.int32, device="cuda")
        self.k, self.v = (torch.zeros((NB, BLOCK, HK, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.planes = gdn.PagePlanes([self.k, self.v])
        self.err, self.slots = i32([0]), torch.arange(ROWS, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
        self.cs_src, self.cs_dst = i32([-1] * 2), i32([-1] * 2)
        self.mv_src, self.mv_dst, self.n_mv = i32([-1] * NB), i32([-1] * NB), i32([0])
        self.cws = torch.empty(gdn.block_compact_workspace_size(NB), dtype=torch.uint8, device="cuda")

    def tensors(self):
        return [self.pool.ssm, self.ck.ssm, self.free, self.nf, self.refs, self.table, self.k, self.v]

    def step(self, x, residual, new, start, decode_rows=None):
        """One model step of new[r] tokens per row of the table (x: their
        capacity of rows); decode_rows: all have one token, of these slots."""
        d, n = self.dims, x.shape[0]
        e = lambda *s, t=torch.int32: torch.empty(s, dtype=t, device="cuda")
        self.cu, seq, pos, slot = e(ROWS + 1), e(n), e(n, t=torch.int64), e(n, t=torch.int64)
        ids = e(ROWS, 2 * MB)
        gdn.batch_maps(new, start, BLOCK, self.table, self.free, self.nf, self.cu, ids, seq, pos, slot, dev_err=self.err)
        y = gdn.add_rmsnorm(x, residual, self.norm)[0]
        # the linear layer: heads rotated in place in its projection
        qkv = y @ self.w_lin
        kd = d.hk * d.dk
        raw = qkv.clone()
        gdn.qk_norm_rope(qkv[:, :kd].unflatten(1, (d.hk, d.dk)), qkv[:, kd:2 * kd].unflatten(1, (d.hk, d.dk)), self.qn,
                         self.kn, self.cs, pos, dev_err=self.err)
        o = torch.zeros((n, d.hv, d.dv), dtype=torch.bfloat16, device="cuda")
        if decode_rows is None:
            gdn.lin_prefill(d, self.pool, self.ck, self.ld, self.slots, self.cu, start, n, ids, BLOCK, qkv, o, self.ws,
                            scale=128 ** -0.5, dev_err=self.err)
        else:
            gdn.lin_decode_step(d, self.pool, self.ld, decode_rows, qkv, o, scale=128 ** -0.5, dev_err=self.err)
        lin = o.clone()
        z = (y @ self.w_z).view_as(o)
        gdn.gated_rmsnorm(d, o, z, self.on)
        # the attention layer: a new q, keys and values to their pages
        att = y @ self.w_att
        q, k, v = (t.unflatten(1, (-1, D)) for t in att.split([HQ * D, HK * D, HK * D], 1))
        qo = torch.zeros_like(q)
        gdn.qk_norm_rope(q, k, self.aq, self.ak, self.cs2, pos, q_out=qo, v=v, k_cache=self.k, v_cache=self.v,
                         slot_map=slot, dev_err=self.err)
        return dict(y=y, raw=raw, qkv=qkv, lin=lin, z=z, o=o, att=att, qo=qo, pos=pos, seq=seq, slot=slot)

    def fork(self, src, dst, lens):
        gdn.block_fork(src, dst, lens, BLOCK, self.table, self.refs, self.free, self.nf, self.cs_src, self.cs_dst,
                       dev_err=self.err)
        gdn.page_copy(self.planes, self.cs_src, self.cs_dst, dev_err=self.err)
        gdn.slot_copy(self.dims, self.pool, self.pool, src, dst, dev_err=self.err)

    def end(self, rows, old, new):
        gdn.block_release(rows, old, new, BLOCK, self.table, self.refs, self.free, self.nf, dev_err=self.err)
        gdn.block_compact(self.table, self.refs, self.free, self.nf, self.mv_src, self.mv_dst, self.n_mv, self.cws,
                          dev_err=self.err)
        gdn.page_copy(self.planes, self.mv_src, self.mv_dst, dev_err=self.err)
        gdn.slot_copy(self.dims, self.ck, self.ck, self.mv_src, self.mv_dst, dev_err=self.err)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _i64(v):
    return torch.tensor(v, dtype=torch.int64, device="cuda")


def _tokens(sv, n):
    return (torch.randn((n, MODEL), generator=sv.g).to(torch.bfloat16).cuda(),
            torch.randn((n, MODEL), generator=sv.g).cuda())


def _check_step(sv, r, n, hist, refs):
    """Values of a step's n rows; keys and values go to hist, refs: the states."""
    d, kd = sv.dims, sv.dims.hk * sv.dims.dk
    pos, seq = r["pos"].cpu()[:n], r["seq"].cpu()[:n].tolist()
    raw, qkv = f64t(r["raw"][:n]), r["qkv"][:n]
    for part, w in ((slice(0, kd), sv.qn), (slice(kd, 2 * kd), sv.kn)):
        close(qkv[:, part].unflatten(1, (d.hk, d.dk)),
              reference(raw[:, part].unflatten(1, (d.hk, d.dk)), w.cpu(), sv.cs.cpu(), pos, 1e-6, False))
    assert torch.equal(qkv[:, 2 * kd:], r["raw"][:n, 2 * kd:])
    od, want, done = oracle.Dims(d.hk, d.hv, d.dk, d.dv, 1), np.zeros((n, d.hv, d.dv)), 0
    while done < n:  # one sequence after the other
        s = seq[done]
        m = next((i for i in range(done, n) if seq[i] != s), n)
        want[done:m] = linear.prefill(od, refs, None, f64(sv.ld), 128 ** -0.5, [s], [0, m - done], [int(pos[done])],
                                      np.zeros((1, 0), int), BLOCK, f64(qkv[done:m]))
        done = m
    assert_out_close(r["lin"][:n], want, d.dv)
    gated = oracle.gated_rmsnorm(od, f64(r["lin"][:n]), f64(r["z"][:n]), f64(sv.on), eps=1e-6)
    assert_out_close(r["o"][:n], gated, d.dv)
    q, k, v = (t.unflatten(1, (-1, D)) for t in r["att"][:n].split([HQ * D, HK * D, HK * D], 1))
    close(r["qo"][:n], reference(f64t(q), sv.aq.cpu(), sv.cs2.cpu(), pos, 1e-6, False))
    kw = reference(f64t(k), sv.ak.cpu(), sv.cs2.cpu(), pos, 1e-6, False)
    for i, s in enumerate(seq):
        hist[s] = hist[s][:int(pos[i])] + [(kw[i], v[i].cpu())]


def f64t(t):
    return t.detach().cpu().double()


def _check_pages(sv, hist):
    table, free, nf = sv.table.tolist(), sv.free.tolist(), int(sv.nf)
    held = {}
    for row, h in hist.items():
        blocks = table[row][:-(-len(h) // BLOCK)]
        assert table[row][len(blocks):] == [-1] * (MB - len(blocks))
        for b in blocks:
            held[b] = held.get(b, 0) + 1
        if h:
            k, v = (t[blocks].flatten(0, 1)[:len(h)] for t in (sv.k, sv.v))
            close(k, torch.stack([x for x, _ in h]))
            assert torch.equal(v.cpu(), torch.stack([x for _, x in h]))
    assert sorted(free[:nf] + list(held)) == list(range(NB))
    refs = sv.refs.tolist()
    assert all(refs[b] == c - 1 for b, c in held.items()) and all(refs[b] == 0 for b in free[:nf])
    return held


def test_a_servers_life(cuda):
    sv = Server(1)
    hist = {r: [] for r in range(ROWS)}
    refs = np.zeros((ROWS, 4, 128, 128))
    x, res = _tokens(sv, 360)
    r = sv.step(x, res, _i32([310, 0, 37, 0, 0]), _i64([0] * 5))
    assert int(sv.cu[-1]) == 347 and r["seq"][347:].tolist() == [-1] * 13
    _check_step(sv, r, 347, hist, refs)
    assert not bool(r["lin"][347:].any())
    _check_pages(sv, hist)
    ck = {b: sv.ck.ssm[b].clone() for b in sv.table[0].tolist()[:4]}
    # two branches of row 0; they and row 0 each get a token of their own
    sv.fork(_i32([0, 0]), _i32([1, 3]), _i64([310, 310]))
    for c in (1, 3):
        hist[c], refs[c] = list(hist[0]), refs[0]
    _check_pages(sv, hist)
    lens = [310, 310, 37, 310, 0]
    for _ in range(12):  # past the end of a block
        x, res = _tokens(sv, 4)
        r = sv.step(x, res, _i32([1, 1, 1, 1, 0]), _i64(lens), decode_rows=_i32([0, 1, 2, 3]))
        _check_step(sv, r, 4, hist, refs)
        lens = [n + 1 for n in lens[:4]] + [0]
    assert max_rel_l2(f64(sv.pool.ssm), refs, 128 * 128) <= STATE_TOL
    held = _check_pages(sv, hist)
    assert max(held.values()) == 3
    # the parent ends, a branch goes back by 32 tokens; the rest moves together
    before = {row: list(h) for row, h in hist.items()}
    old_table = sv.table.clone()
    sv.end(_i32([0, 3]), _i64([322, 322]), _i64([0, 290]))
    hist[0], hist[3] = [], before[3][:290]
    held = _check_pages(sv, hist)
    assert max(held) == len(held) - 1 and int(sv.n_mv) > 0
    for j in range(4):  # the shared blocks' checkpoints went with them
        assert torch.equal(sv.ck.ssm[int(sv.table[1, j])], ck[int(old_table[1, j])])
    # a prompt in the freed row, and the branch goes on from a block's checkpoint
    sv.end(_i32([3]), _i64([290]), _i64([256]))
    hist[3] = hist[3][:256]
    gdn.slot_copy(sv.dims, sv.ck, sv.pool, sv.table[3, 3:4].clone(), _i32([3]), dev_err=sv.err)
    gdn.slot_zero(sv.dims, sv.pool, _i32([0]), dev_err=sv.err)
    refs[0], refs[3] = 0, f64(sv.pool.ssm[3])
    x, res = _tokens(sv, 90)
    r = sv.step(x, res, _i32([50, 0, 1, 39, 0]), _i64([0, 322, 49, 256, 0]))
    _check_step(sv, r, 90, hist, refs)
    _check_pages(sv, hist)
    assert max_rel_l2(f64(sv.pool.ssm), refs, 128 * 128) <= STATE_TOL
    assert int(sv.err) == 0


def test_a_captured_step_with_a_branch(cuda):
    """Prefill, fork, a token each, the branch's end and compaction in one graph,
    replayed twice on other inputs, against eager calls bit for bit."""
    sv = Server(2)
    x, res = _tokens(sv, 220)
    start, zero = _i64([0] * 5), _i32([70, 0, 150, 0, 0])
    one, at, rows = _i32([1, 1, 1, 0, 0]), _i64([70, 70, 150, 0, 0]), _i32([0, 1, 2])
    src, dst, lens = _i32([0, -1]), _i32([1, 4]), _i64([70, 3])
    end, old, new = _i32([1, 2]), _i64([71, 151]), _i64([0, 70])

    def step():
        a = sv.step(x, res, zero, start)
        sv.fork(src, dst, lens)
        b = sv.step(x[:3], res[:3], one, at, decode_rows=rows)
        sv.end(end, old, new)
        return [r[k] for r in (a, b) for k in ("o", "qo", "pos", "seq", "slot")]

    first = [t.clone() for t in sv.tensors()]

    def reset():
        for t, f in zip(sv.tensors(), first):
            t.copy_(f)

    step()
    torch.cuda.synchronize()
    reset()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for _ in range(2):
        nx, nr = _tokens(sv, 220)
        reset()
        x.copy_(nx), res.copy_(nr)
        g.replay()
        got = [t.clone() for t in outs + sv.tensors()]
        reset()
        res.copy_(nr)
        want = step() + sv.tensors()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert int(sv.err) == 0 and int(sv.nf) == NB - 2 - 2
