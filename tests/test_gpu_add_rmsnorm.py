"""The residual RMS norm with its 8-bit output against float64.

Tolerances.  h is one fp32 addition: 2^-24 relative to it, so the stored
residual is the fp32 sum's rounding, exactly.  y: the sum of squares of d
terms in a tree of depth <= 40 and a square root, division and two products:
relative error at most 64 2^-24 = 4e-6 on fp32 (plus the sum's cancellation,
relative to |x| + |residual|), and half a step more in bf16 (2^-8 with the
4e-6).  Scales: the same 4e-6.  q8: y / scale lies within 448 (4e-6 + 2 2^-24)
of the exact quotient, so q8 is one of the two e4m3 neighbours of it, and the
nearest except within that distance of a midpoint: the error is at most half
an e4m3 step (2^-4 of the value, or 2^-10 below the smallest normal 2^-6)
plus 1e-5 of the value.
"""
import numpy as np
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from hybrid_linear_attention_gdn_gb300 import binding

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _case(rows, d, act, res, seed, std=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, d), generator=g).to(act)
    r = (torch.randn((rows, d), generator=g) * std).to(res) if res is not None else None
    w = 1 + 0.2 * torch.randn(d, generator=g)
    return x, r, w


def _ref(x, r, w, eps):
    h = x.double() + (r.double() if r is not None else 0)
    return h, h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w.double()


def _check_q8(q, scale, y, group):
    """Half an e4m3 step of y / scale, with the scale that was stored."""
    z = y / scale.double().repeat_interleave(group, dim=1)
    got = q.float().double()
    step = torch.maximum(z.abs() * 2.0 ** -4, torch.full_like(z, 2.0 ** -10))
    assert ((got - z.clamp(-448, 448)).abs() <= step * (1 + 1e-5) + 1e-5 * z.abs()).all()


@pytest.mark.parametrize("rows,d", [(1, 32), (5, 256), (3, 288), (7, 1024), (2, 1056), (9, 2048), (4, 4096),
                                    (3, 5120), (2, 8192), (2, 16384), (1, 32768)])
@pytest.mark.parametrize("act,res", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
def test_norm_and_q8(cuda, rows, d, act, res):
    x, r, w = _case(rows, d, act, res, 3 + rows)
    h, y = _ref(x, r, w, 1e-6)
    for group in (0, 32, 128 if d % 128 == 0 else 32):
        rd = r.cuda()
        q = torch.empty((rows, d), dtype=torch.float8_e4m3fn, device="cuda")
        n0 = binding.launch_count(binding.K_ADD_RMSNORM)
        yd, q, s = gdn.add_rmsnorm(x.cuda(), rd, w.cuda(), 1e-6, y=torch.empty_like(x, device="cuda"), q8=q,
                                   group=group)
        assert binding.launch_count(binding.K_ADD_RMSNORM) == n0 + 1
        assert torch.equal(rd.cpu(), (x.float() + r.float()).to(res))
        mag = (x.double().abs() + r.double().abs()) / h.abs().clamp(min=1e-30)
        half = torch.finfo(act).eps / 2
        assert ((yd.cpu().double() - y).abs() <= y.abs() * (half + 4e-6 + mag * 2.0 ** -24) + 1e-12).all()
        gs = group or d
        top = y.reshape(rows, -1, gs).abs().amax(-1)
        assert s.shape == top.shape and ((s.cpu().double() - top / 448).abs() <= 5e-6 * top / 448).all()
        _check_q8(q.cpu(), s.cpu(), y, gs)


@pytest.mark.parametrize("rows,d", [(6, 96), (3, 4096)])
def test_power_of_two_scales(cuda, rows, d):
    x, r, w = _case(rows, d, BF16, F32, 4)
    x[0, :32] = 0.0
    r[0, :32] = 0.0
    _, y = _ref(x, r, w, 1e-6)
    for dt in (torch.uint8, torch.float8_e8m0fnu):
        q = torch.empty((rows, d), dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty((rows, d // 32), dtype=dt, device="cuda")
        gdn.add_rmsnorm(x.cuda(), r.cuda(), w.cuda(), 1e-6, q8=q, scales=s, group=32)
        b = s.view(torch.uint8).cpu().double()
        top = y.reshape(rows, -1, 32).abs().amax(-1)
        exact = torch.where(top > 0, torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)) + 127, 127.0)
        near = (torch.log2(top.clamp(min=1e-300) / 448).frac().abs().sub(0.5).abs() > 0.49999) & (top > 0)
        assert ((b == exact) | near).all()
        assert b[0, 0] == 127 and (q.cpu().float()[0, :32] == 0).all()
        _check_q8(q.cpu(), torch.exp2(b - 127), y, 32)


@pytest.mark.parametrize("d", [1, 7, 33, 1000, 4099])
@pytest.mark.parametrize("act", [BF16, F32])
def test_odd_sizes_and_unaligned(cuda, act, d):
    """Any d with a scale per row, and tensors that start at an odd element."""
    x, r, w = _case(5, d, act, act, 5)
    h, y = _ref(x, r, w, 1e-5)

    def off(t):
        big = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        big[1:] = t.reshape(-1).cuda()
        return big[1:].view(t.shape)

    q = off(torch.zeros((5, d), dtype=torch.uint8)).view(torch.float8_e4m3fn)
    rd = off(r)
    yd, q, s = gdn.add_rmsnorm(off(x), rd, off(w), 1e-5, y=off(x), q8=q)
    assert torch.equal(rd.cpu(), (x.float() + r.float()).to(act))
    mag = (x.double().abs() + r.double().abs()) / h.abs().clamp(min=1e-30)
    half = torch.finfo(act).eps / 2
    assert ((yd.cpu().double() - y).abs() <= y.abs() * (half + 4e-6 + mag * 2.0 ** -24) + 1e-12).all()
    _check_q8(q.cpu(), s.cpu(), y, d)


def test_without_residual_in_place_and_extremes(cuda):
    x, _, w = _case(6, 512, F32, None, 6)
    x[1] = 0.0                       # an empty row: y 0, scale 1
    x[2] *= 1e-18                    # squares below the smallest float
    x[3] *= 1e15                     # squares near 1e30
    x[4, 3] = float("nan")
    x[5, 7] = float("inf")
    xd = x.cuda()
    q = torch.empty((6, 512), dtype=torch.float8_e4m3fn, device="cuda")
    yd, q, s = gdn.add_rmsnorm(xd, None, w.cuda(), 0.0 + 1e-12, y=xd, q8=q, group=256)
    _, y = _ref(x, None, w, 1e-12)
    got = yd.cpu().double()
    for row in (0, 1, 2, 3):
        assert ((got[row] - y[row]).abs() <= 8e-6 * y[row].abs() + 1e-30).all(), row
    assert (s.cpu()[1] == 1).all() and (q.cpu().float()[1] == 0).all()
    # the NaN's row is NaN throughout; an infinity leaves NaN in its own place and zeros elsewhere
    assert torch.isnan(got[4]).all() and torch.isnan(s.cpu()[4]).all() and torch.isnan(q.cpu().float()[4]).all()
    assert torch.isnan(got[5, 7]) and (got[5, :7] == 0).all() and (got[5, 8:] == 0).all()
    assert torch.isnan(s.cpu()[5, 0]) and s.cpu()[5, 1] == 1


def test_rows_of_higher_rank_and_none(cuda):
    x, r, w = _case(6, 64, BF16, BF16, 7)
    y, q8, s = gdn.add_rmsnorm(x.view(2, 3, 64).cuda(), r.view(2, 3, 64).cuda(), w.cuda())
    assert y.shape == (2, 3, 64) and q8 is None and s is None
    e = gdn.add_rmsnorm(x[:0].cuda(), r[:0].cuda(), w.cuda())[0]
    assert e.shape == (0, 64)


def _e4m3(z):
    """float64 to the nearest e4m3 value, ties to even, at most 448."""
    m = z.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(m.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(z) * (torch.round(m / step) * step).clamp(max=448.0)


@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("act,res", [(BF16, BF16), (BF16, F32), (F32, F32), (BF16, None)])
def test_q8_is_the_nearest_to_the_exact_quotient(cuda, act, res, group):
    """The only rounding between y / scale and q8 is q8's: the kernel's
    quotient is within 2^-40 of the exact one, so that of 2 million values in
    float64 not one is expected on the other side of a midpoint."""
    for rows, d in ((512, 4096), (64, 256), (40, 16384)) + (((9, 1001),) if group == 0 else ()):
        x, r, w = _case(rows, d, act, res, 12 + d)
        x[1] = x[0]  # equal rows, and in one of them equal largest values
        x[2, ::2] = x[2, 0]
        h = x.cuda().double() + (r.cuda().double() if r is not None else 0)
        p = h * w.cuda().double()
        gs = group or d
        top = p.reshape(rows, -1, gs).abs().amax(-1, keepdim=True)
        z = (448 * p.reshape(rows, -1, gs) / top).reshape(rows, d)
        q = torch.empty((rows, d), dtype=torch.float8_e4m3fn, device="cuda")
        gdn.add_rmsnorm(x.cuda(), r.cuda() if r is not None else None, w.cuda(), 1e-6, q8=q, group=group)
        assert torch.equal(q.double(), _e4m3(z))


def test_q8_at_midpoints(cuda):
    """Quotients that are midpoints go to the even neighbour, in normal and
    subnormal range; a step of the input's last bit decides beside them."""
    top = 448.0
    mid = torch.tensor([17 / 16, 19 / 16, 208.0 + 8, 224 + 16, 2.0 ** -7 * 1.25, 2.0 ** -10, 3 * 2.0 ** -10,
                        5 * 2.0 ** -10])
    vals = torch.cat([mid, mid * (1 + 2.0 ** -23), mid * (1 - 2.0 ** -24), -mid])
    x = torch.zeros(2, 64)
    x[0, :32], x[1, :32] = vals, vals.flip(0)
    x[:, 40] = top
    q = torch.empty((2, 64), dtype=torch.float8_e4m3fn, device="cuda")
    for group in (0, 64):
        gdn.add_rmsnorm(x.cuda(), None, torch.ones(64).cuda(), 1e-6, q8=q, group=group)
        assert torch.equal(q.cpu().double(), _e4m3(x.double()))
