"""Query and key norms with rotation against float64: head sizes, rotated
parts, both pairings, views of a projection, caches by rows and by heads,
padding, positions and slots out of range.

Tolerances: everything is computed in fp32 from inputs that are exact: the sum
of squares (d / 2 roundings at most of half a step each in a sum of positive
terms, through a square root: d 2^-26), four further products and one sum of
two rotated terms.  With d <= 1024 that is below (16 + 6) 2^-24 relative to
|a| + |b| of a pair, 2e-6 of the row's L2 norm; bf16 outputs add their own
rounding, 2^-8 / 2 of each value.  Bounds: L2 per head 1e-5 (fp32) and, beyond
the rounding, 1e-5 (bf16).
"""
import numpy as np
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from hybrid_linear_attention_gdn_gb300 import binding

pytestmark = pytest.mark.gpu
TOL = 1e-5


def f64(t):
    return t.detach().cpu().double()


def table(max_pos, rot, base=1e4):
    f = base ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / max(rot, 1))
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * f
    return torch.cat([torch.cos(ang), torch.sin(ang)], 1).float()


def reference(x, w, cs, pos, eps, interleaved):
    """x [rows][heads][d] in float64."""
    y = x if w is None else x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    rot = cs.shape[1]
    c, s = cs.double()[pos][:, None, :rot // 2], cs.double()[pos][:, None, rot // 2:]
    out = y.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def close(got, want):
    """L2 per head: beyond the rounding of the exact values to the output's type."""
    g, w = f64(got), want
    rnd = w.to(got.dtype).double()
    err, own = (g - w).norm(dim=-1), (rnd - w).norm(dim=-1)
    assert bool((err - own <= TOL * w.norm(dim=-1)).all()), float(((err - own) / w.norm(dim=-1)).max())


class Case:
    def __init__(self, seed, rows, hq, hk, d, rot, act, max_pos=300, hv=None, dv=None):
        g = self.g = torch.Generator().manual_seed(seed)
        self.rows, self.hq, self.hk, self.d = rows, hq, hk, d
        self.hv, self.dv = hk if hv is None else hv, d if dv is None else dv
        self.act = torch.bfloat16 if act == "bf16" else torch.float32
        x = torch.randn((rows, (hq + hk) * d + self.hv * self.dv), generator=g).to(self.act)
        self.x = x.cuda()
        self.q = self.x[:, :hq * d].unflatten(1, (hq, d))
        self.k = self.x[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        self.v = self.x[:, (hq + hk) * d:].unflatten(1, (self.hv, self.dv))
        self.qw, self.kw = (1 + 0.3 * torch.randn(d, generator=g) for _ in range(2))
        self.cs = table(max_pos, rot)
        self.pos = torch.randint(0, max_pos, (rows,), generator=g)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def want(self, interleaved, eps=1e-6):
        return (reference(f64(self.q), self.qw, self.cs, self.pos, eps, interleaved),
                reference(f64(self.k), self.kw, self.cs, self.pos, eps, interleaved))

    def call(self, **kw):
        return gdn.qk_norm_rope(self.q, self.k, self.qw.cuda(), self.kw.cuda(), self.cs.cuda(), self.pos.cuda(),
                                dev_err=self.err, **kw)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (128, 64), (256, 64), (128, 32), (256, 256), (64, 16),
                                   (128, 0), (128, 6), (96, 96), (80, 20), (8, 8), (7, 4), (1, 0), (1024, 512)])
def test_new_tensors(cuda, d, rot, interleaved, act):
    c = Case(d + rot, 37, 6, 2, d, rot, act)
    q, k = c.want(interleaved)
    qo, ko = torch.empty((37, 6, d), dtype=c.act, device="cuda"), torch.empty((37, 2, d), dtype=c.act, device="cuda")
    before = c.x.clone()
    n0 = gdn.launch_count(binding.K_QK_NORM_ROPE)
    r = c.call(interleaved=interleaved, q_out=qo, k_out=ko)
    assert r[0] is qo and r[1] is ko and gdn.launch_count(binding.K_QK_NORM_ROPE) == n0 + 1
    close(qo, q)
    close(ko, k)
    assert torch.equal(c.x, before) and int(c.err) == 0


@pytest.mark.parametrize("rows", [1, 3, 64, 1000])
@pytest.mark.parametrize("hq,hk,d", [(1, 1, 64), (32, 4, 128), (5, 3, 128), (16, 2, 256), (3, 1, 96)])
def test_in_place(cuda, rows, hq, hk, d):
    """The projection's q and k replaced, its v left alone."""
    c = Case(rows + d, rows, hq, hk, d, d, "bf16")
    (q, k), v = c.want(False), c.v.clone()
    c.call()
    close(c.q, q)
    close(c.k, k)
    assert torch.equal(c.v, v)


@pytest.mark.parametrize("by_heads", [False, True])
@pytest.mark.parametrize("act,d,dv,hv,block", [("bf16", 128, 128, 4, 64), ("bf16", 128, 64, 2, 16), ("f32", 64, 64, 4, 1),
                                               ("bf16", 96, 40, 3, 32), ("bf16", 256, 256, 4, 128)])
def test_cache(cuda, act, d, dv, hv, block, by_heads):
    rows, hk, pages = 75, 4, 200 // block + 3
    c = Case(d + dv, rows, 8, hk, d, d, act, hv=hv, dv=dv)
    q, k = c.want(False)
    n = pages * block
    slot = torch.randperm(n, generator=c.g)[:rows]
    slot[5], slot[40] = -1, -1
    kc, vc = (torch.full((pages, h, block, w) if by_heads else (pages, block, h, w), 9.0, dtype=c.act, device="cuda")
              for h, w in ((hk, d), (hv, dv)))
    view = (lambda t: t.transpose(1, 2)) if by_heads else (lambda t: t)
    before = c.x.clone()
    qo = torch.empty((rows, 8, d), dtype=c.act, device="cuda")
    r = c.call(q_out=qo, v=c.v, k_cache=view(kc), v_cache=view(vc), slot_map=slot.cuda())
    assert r[1] is None and torch.equal(c.x, before) and int(c.err) == 0
    close(qo, q)
    flat = lambda t: view(t).reshape(n, *view(t).shape[2:])
    live = slot >= 0
    close(flat(kc)[slot[live].cuda()], k[live])
    assert torch.equal(flat(vc)[slot[live].cuda()], c.v[live.cuda()])
    rest = torch.ones(n, dtype=torch.bool)
    rest[slot[live]] = False
    assert bool((flat(kc)[rest.cuda()] == 9).all()) and bool((flat(vc)[rest.cuda()] == 9).all())


def test_positions_and_slots_out_of_range(cuda):
    c = Case(1, 9, 4, 2, 64, 64, "bf16", max_pos=50)
    q, k = c.want(False)
    c.pos[2], c.pos[7] = 50, -1
    slot = torch.arange(9)
    slot[4], slot[5] = 16, -2
    kc = torch.full((1, 16, 2, 64), 9.0, dtype=c.act, device="cuda")
    vc = kc.clone()
    qo, ko = torch.empty_like(c.q.contiguous()), torch.empty_like(c.k.contiguous())
    c.call(q_out=qo, k_out=ko, v=c.v, k_cache=kc, v_cache=vc, slot_map=slot.cuda())
    assert int(c.err) == binding.DEV_ERR_SEQLENS | binding.DEV_ERR_SLOT_OOB
    ok = torch.tensor([0, 1, 3, 4, 5, 6, 8])
    close(qo[ok.cuda()], q[ok])
    close(ko[ok.cuda()], k[ok])
    assert not qo[[2, 7]].any() and not ko[[2, 7]].any()
    written = torch.tensor([0, 1, 3, 6, 8])
    close(kc[0][written.cuda()], k[written])
    rest = [r for r in range(16) if r not in written.tolist()]
    assert bool((kc[0, rest] == 9).all()) and bool((vc[0, rest] == 9).all())


def test_parts_alone(cuda):
    """Only queries, only keys, no norm, keys without values in the cache, no rows."""
    c = Case(2, 10, 4, 2, 64, 32, "f32")
    q, k = c.want(False)
    cs, pos = c.cs.cuda(), c.pos.cuda()
    qo = torch.empty((10, 4, 64), device="cuda")
    r = gdn.qk_norm_rope(c.q, None, c.qw.cuda(), None, cs, pos, q_out=qo)
    close(qo, q)
    assert r[1] is None
    ko = torch.empty((10, 2, 64), device="cuda")
    gdn.qk_norm_rope(None, c.k, None, c.kw.cuda(), cs, pos, k_out=ko)
    close(ko, k)
    gdn.qk_norm_rope(c.q, c.k, None, None, cs, pos, q_out=qo, k_out=ko)
    close(qo, reference(f64(c.q), None, c.cs, c.pos, 0, False))
    close(ko, reference(f64(c.k), None, c.cs, c.pos, 0, False))
    kc = torch.zeros((1, 16, 2, 64), device="cuda")
    gdn.qk_norm_rope(c.q, c.k, c.qw.cuda(), c.kw.cuda(), cs, pos, q_out=qo, k_cache=kc,
                     slot_map=torch.arange(10, device="cuda"))
    close(kc[0, :10], k)
    none = torch.zeros((0, 4, 64), device="cuda")
    gdn.qk_norm_rope(none, none, None, None, cs, pos[:0])


def test_zero_and_non_finite_heads(cuda):
    """A head of zeros stays zeros; a NaN stays in its head; the values of a padded row reach no other."""
    c = Case(3, 6, 4, 2, 128, 128, "bf16")
    c.x[1] = 0
    c.q[2, 1, 5] = float("nan")
    c.q[3, 0, 100] = float("inf")
    q, k = c.want(False)
    c.call()
    assert not c.q[1].any() and not c.k[1].any()
    assert bool(c.q[2, 1].isnan().all())
    ok = torch.ones((6, 4), dtype=torch.bool)
    ok[1], ok[2, 1], ok[3, 0] = False, False, False
    close(c.q[ok.cuda()], q[ok])


def test_far_positions(cuda):
    c = Case(4, 16, 2, 1, 64, 64, "f32", max_pos=1 << 20)
    c.pos[0] = (1 << 20) - 1
    q, k = c.want(False)
    c.call()
    close(c.q, q)
    close(c.k, k)


def test_refusals(cuda):
    c = Case(5, 4, 2, 1, 64, 64, "bf16")
    cs, pos, w = c.cs.cuda(), c.pos.cuda(), c.qw.cuda()
    kc = torch.zeros((1, 16, 1, 64), dtype=c.act, device="cuda")
    slot = torch.arange(4, device="cuda")
    bad = [
        lambda: gdn.qk_norm_rope(c.q.half(), None, w, None, cs, pos),
        lambda: gdn.qk_norm_rope(c.q, c.k.float(), w, w, cs, pos),
        lambda: gdn.qk_norm_rope(c.q.transpose(1, 2), None, w, None, cs, pos),
        lambda: gdn.qk_norm_rope(c.q, c.k, w[:32], w, cs, pos),
        lambda: gdn.qk_norm_rope(c.q, c.k, w, w, cs.cpu(), pos),
        lambda: gdn.qk_norm_rope(c.q, c.k, w, w, cs, pos.int()),
        lambda: gdn.qk_norm_rope(c.q, c.k, w, w, torch.cat([cs, cs], 1), pos),             # rot > d
        lambda: gdn.qk_norm_rope(c.q, c.k, w, w, cs[:, :3].contiguous(), pos),              # odd rot
        lambda: gdn.qk_norm_rope(c.q, c.k, w, w, cs, pos, eps=-1.0),
        lambda: gdn.qk_norm_rope(c.q, c.k, w, w, cs, pos, eps=float("nan")),
        lambda: gdn.qk_norm_rope(c.q, c.k, w, w, cs, pos, slot_map=slot),                   # no cache
        lambda: gdn.qk_norm_rope(c.q, c.k, w, w, cs, pos, k_cache=kc),                      # no slots
        lambda: gdn.qk_norm_rope(c.q, c.k, w, w, cs, pos, k_cache=kc, v=c.v, slot_map=slot),
        lambda: gdn.qk_norm_rope(c.q, c.k, w, w, cs, pos, k_cache=kc[:, :12], slot_map=slot),  # 12 rows a page
        lambda: gdn.qk_norm_rope(c.q, c.k, w, w, cs, pos, k_cache=kc.float(), slot_map=slot),
        lambda: gdn.qk_norm_rope(c.q, c.k, w, w, cs, pos, q_out=c.q[:1].expand(4, -1, -1)),
        lambda: gdn.qk_norm_rope(None, None, w, w, cs, pos),
    ]
    before = c.x.clone()
    for i, f in enumerate(bad):
        with pytest.raises(gdn.GdnError):
            f()
            pytest.fail(f"case {i} was accepted")
    assert torch.equal(before, c.x)


@pytest.mark.parametrize("d", [64, 20])
def test_a_table_of_no_positions(cuda, d):
    """Every position lies outside: zeros, and the table is not read."""
    c = Case(40, 5, 3, 1, d, 4 if d == 20 else 32, "bf16")
    c.cs = torch.ones((3, c.cs.shape[1]))
    tab = c.cs.cuda()[:0]
    q, k = gdn.qk_norm_rope(c.q, c.k, c.qw.cuda(), c.kw.cuda(), tab, c.pos.cuda(), dev_err=c.err) \
        if tab.data_ptr() else (c.q.zero_(), c.k.zero_())
    assert not bool(q.any()) and not bool(k.any())
    assert not tab.data_ptr() or int(c.err) == binding.DEV_ERR_SEQLENS
