"""Outputs of the rotation kept by heads, padded, or beyond 32 bits: any
strides that keep the elements apart.  Bounds as in test_gpu_qk_norm_rope."""
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from test_gpu_qk_norm_rope import Case, close

pytestmark = pytest.mark.gpu


def by_heads(t):
    """t [rows][heads][d] as a view of [heads][rows][d]."""
    return t.transpose(0, 1).contiguous().transpose(0, 1)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("rows,hq,hk,d,rot", [(37, 6, 2, 128, 64), (1, 4, 4, 64, 64), (5, 3, 1, 96, 96), (300, 1, 1, 20, 4),
                                              (2, 5, 5, 256, 256)])
@pytest.mark.parametrize("in_place", [False, True])
def test_outputs_by_heads(cuda, rows, hq, hk, d, rot, act, in_place):
    c = Case(rows + d, rows, hq, hk, d, rot, act)
    q, k = c.want(False)
    c.q, c.k = by_heads(c.q), by_heads(c.k)
    if in_place:
        qo, ko = c.call()
        assert qo is c.q and ko is c.k
    else:
        before = c.q.clone(), c.k.clone()
        qo, ko = c.call(q_out=torch.zeros_like(c.q), k_out=by_heads(torch.zeros_like(c.k)))
        assert torch.equal(before[0], c.q) and torch.equal(before[1], c.k)
    close(qo, q)
    close(ko, k)
    assert int(c.err) == 0


@pytest.mark.parametrize("d", [64, 20])
def test_outputs_with_room_between(cuda, d):
    """Heads within rows and rows within heads, with unused elements between them that stay."""
    for rows_first in (True, False):
        c = Case(d, 9, 3, 2, d, 4 * (d // 8), "bf16")
        q, k = c.want(True)
        size = (9, 4, d + 12) if rows_first else (4, 11, d + 12)
        buf = torch.full(size, 5.0, dtype=c.act, device="cuda")
        view = (buf if rows_first else buf.transpose(0, 1))[:9, :3, 4:4 + d]
        c.call(q_out=view, k_out=by_heads(c.k), interleaved=True)
        close(view, q)
        kept = buf.clone()
        (kept if rows_first else kept.transpose(0, 1))[:9, :3, 4:4 + d] = 5.0
        assert bool((kept == 5).all())


def test_outputs_that_overlap_are_refused(cuda):
    c = Case(3, 6, 4, 2, 64, 64, "bf16")
    flat = torch.zeros(6 * 4 * 64 * 2, dtype=c.act, device="cuda")
    before = c.x.clone()
    for strides in ((64, 64, 1), (0, 64, 1), (256, 0, 1), (256, 32, 1), (32, 256, 1), (65, 64, 1), (64, 320, 1)):
        with pytest.raises(gdn.GdnError, match="separate"):
            c.call(q_out=flat.as_strided((6, 4, 64), strides), k_out=torch.empty_like(c.k))
    with pytest.raises(gdn.GdnError, match="consecutive"):
        c.call(q_out=flat.as_strided((6, 4, 64), (512, 128, 2)), k_out=torch.empty_like(c.k))
    assert not bool(flat.any()) and torch.equal(before, c.x)


@pytest.mark.parametrize("d", [128, 96])
@pytest.mark.parametrize("heads_far", [False, True])
def test_elements_beyond_32_bits(cuda, d, heads_far):
    """Rows or heads 2^30 and more elements apart, the last ones beyond 2^31."""
    c = Case(d, 4, 4, 2, d, d, "bf16")
    q, k = c.want(False)
    far = 2 ** 30 - 2 ** 20
    s = (1024, far, 1) if heads_far else (far, 1024, 1)
    buf = torch.empty(3 * far + 20000, dtype=c.act, device="cuda")
    qo, ko = buf.as_strided((4, 4, d), s), buf[8192:].as_strided((4, 2, d), s)
    qo.copy_(c.q)
    ko.copy_(c.k)
    kc = buf[16384:].as_strided((4, 1, 2, d), (far, 256, 128, 1))
    kc.zero_()
    c.q, c.k = qo, ko
    c.call(k_out=ko, k_cache=kc, slot_map=torch.tensor([3, -1, 0, 1], device="cuda"))
    close(qo, q)
    close(ko, k)
    close(kc[:, 0][[3, 0, 1]], k[[0, 2, 3]])
    assert not bool(kc[2].any()) and int(c.err) == 0
