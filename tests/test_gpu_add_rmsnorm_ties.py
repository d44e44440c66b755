"""q8 at quotients that are exactly half way between two e4m3 values, for
largest values whose reciprocal is not exact: to the even neighbour."""
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from test_gpu_add_rmsnorm import _e4m3

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
MIDS = [21.0 / 16 * 2.0 ** k for k in range(-6, 8)] + [7 * 2.0 ** -10, 21 / 16 * 2.0 ** 8]  # multiples of 7


def _rows(d, group):
    """Row T - 1: T the largest value of every group, the others 448-ths of
    it that make halves of e4m3 steps, with one fp32 step less and more."""
    t = torch.arange(1, 86, dtype=torch.float64)[:, None]
    mid = torch.tensor(MIDS, dtype=torch.float64)
    x = (t * mid[torch.arange(d) % len(MIDS)] / 448)
    x[:, 1::2] *= -1
    x[:, 3::group or d] = t  # the largest
    return x


@pytest.mark.parametrize("act,res", [(BF16, None), (BF16, BF16), (BF16, F32), (F32, None), (F32, F32)])
@pytest.mark.parametrize("d,group", [(64, 0), (1000, 0), (4096, 0), (64, 32), (4096, 128), (8192, 256)])
def test_halves_go_to_the_even_value(cuda, act, res, d, group):
    h = _rows(d, group)
    x, r = h.to(act), None
    if res is not None:  # the same sums from two parts, exact in both types
        r = (h / 2).to(res)
        x = (h / 2).to(act)
    assert torch.equal(x.double() + (r.double() if r is not None else 0), h)
    for w in (torch.ones(d), torch.full((d,), 1.5), torch.full((d,), -0.7109375)):
        q = torch.empty((85, d), dtype=torch.float8_e4m3fn, device="cuda")
        gdn.add_rmsnorm(x.cuda(), r.cuda() if r is not None else None, w.cuda(), 1e-6, q8=q, group=group)
        p = h * w.double()
        z = 448 * p / p.abs().amax(-1, keepdim=True)
        assert torch.equal(q.cpu().double(), _e4m3(z))


@pytest.mark.parametrize("d,group", [(1000, 0), (4096, 0), (4096, 32)])
def test_a_step_beside_a_half_decides(cuda, d, group):
    """fp32 values one step below and above those: to their own side."""
    h = _rows(d, group).float()
    rest = (h.abs() < h.abs().amax(-1, keepdim=True))
    for to in (0.0, float("inf")):
        x = torch.where(rest, torch.nextafter(h.abs(), torch.full_like(h, to)).copysign(h), h)
        q = torch.empty((85, d), dtype=torch.float8_e4m3fn, device="cuda")
        gdn.add_rmsnorm(x.cuda(), None, torch.ones(d).cuda(), 1e-6, q8=q, group=group)
        xd = x.double()
        assert torch.equal(q.cpu().double(), _e4m3(448 * xd / xd.abs().amax(-1, keepdim=True)))
