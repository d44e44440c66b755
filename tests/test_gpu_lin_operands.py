"""The outputs of the chunk form where their terms cancel, so that the operands'
own roundings show: at most 2^-17 of a term.

An operand is two bf16 parts.  For |x| in [2^e, 2^(e + 1)) the first one, rounded
to nearest, leaves at most 2^(e - 8), the second one of that at most 2^(e - 17):
2^-17 of |x|.  (A first part by truncation leaves up to 2^(e - 7), whose rounding
is off by up to 2^(e - 16).)  Everything else is fp32: products of bf16 parts are
exact, at most eight accumulations and three factors follow, 2^-20 of the terms in
all; and the output's own half step, 2^-8 of it.
"""
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from hybrid_linear_attention_gdn_gb300 import StatePool

pytestmark = pytest.mark.gpu
D = 128
BOUND = 2 ** -17 + 2 ** -20


def call(hk, hv, ssm, ld, x, lens, scale):
    n, total = len(lens), sum(lens)
    dims = gdn.Dims(hk, hv, D, D, 1, torch.bfloat16, torch.bfloat16)
    cu = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
    out = torch.empty((total, hv, D), dtype=torch.bfloat16, device="cuda")
    size = gdn.lin_prefill_workspace_size(dims, n, total)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    gdn.lin_prefill(dims, StatePool(ssm), None, ld, torch.arange(n, dtype=torch.int32, device="cuda"), cu,
                    torch.zeros(n, dtype=torch.int64, device="cuda"), total, None, 64, x, out, ws, scale=scale)
    return out.double()


def check(got, want, terms):
    off = (got - want).abs() - 2 ** -8 * want.abs()
    worst = float((off / terms).max())
    assert worst <= BOUND, f"off by 2^{torch.tensor(worst).log2():.2f} of the terms"


def test_states_that_cancel(cuda):
    """o = S[:, 0] - S[:, 1] of one token without a key, S[:, 1] within 2^-11 of S[:, 0]."""
    g = torch.Generator(device="cuda").manual_seed(61)
    hv, n = 4, 30
    rand = lambda *shape: torch.rand(shape, generator=g, device="cuda")
    ssm = torch.zeros((n, hv, D, D), device="cuda")
    ssm[..., 0] = (1 + rand(n, hv, D)) * 2.0 ** torch.randint(-9, 9, (n, hv, D), generator=g, device="cuda")
    ssm[..., 1] = ssm[..., 0] * (1 + (rand(n, hv, D) - 0.5) * 2 ** -10)
    a, b = ssm[..., 0].double(), ssm[..., 1].double()
    x = torch.zeros((n, 2 * hv * D + hv * D), dtype=torch.bfloat16, device="cuda")
    q = x[:, :hv * D].view(n, hv, D)
    q[..., 0], q[..., 1] = 1, -1
    check(call(hv, hv, ssm, torch.zeros(hv, device="cuda"), x, [1] * n, 1.0), a - b, a + b)


def test_tokens_that_cancel(cuda):
    """Two tokens with opposite values and the same key, nearly without decay."""
    g = torch.Generator(device="cuda").manual_seed(62)
    hv, n = 8, 120
    x = torch.zeros((2 * n, 3 * hv * D), dtype=torch.bfloat16, device="cuda")
    q, k, v = x[:, :hv * D].view(2 * n, hv, D), x[:, hv * D:2 * hv * D].view(2 * n, hv, D), x[:, 2 * hv * D:].view(2 * n, hv, D)
    c = torch.rand((n, hv), generator=g, device="cuda").add(1).bfloat16()
    q[..., 0], k[0::2, :, 0], k[1::2, :, 0] = 1, c, c
    v[0::2], v[1::2] = 1, -1
    ld = -torch.rand(hv, generator=g, device="cuda") * 2 ** -11
    scale = 0.7310585975646973
    p = c.double() * scale
    old = p * torch.exp(ld.double())
    got = call(hv, hv, torch.zeros((n, hv, D, D), device="cuda"), ld, x, [2] * n, scale)
    want, terms = torch.empty_like(got), torch.empty_like(got)
    want[0::2], want[1::2] = p[..., None].expand(-1, -1, D), (old - p)[..., None].expand(-1, -1, D)
    terms[0::2], terms[1::2] = p[..., None].expand(-1, -1, D), (old + p)[..., None].expand(-1, -1, D)
    check(got, want, terms)
