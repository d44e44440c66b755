"""Decays that remember some 65,000 to 1,000,000 tokens, over prompts of as
many: the state of every form of the prefill against its closed form in 64 bits.

Tolerance.  A state that is multiplied by one rounded factor per 64 tokens is
off by the factor's error (up to 2^-25, the same every time) times the
multiplications that it remembers: 2^14 * 2^-25 = 5e-4 at 2^20 tokens, which is
what these tests are for, with decays whose lambda^64 lies as far from a float
as it can.  What may remain: the part of a factor below 1, 64 / M for a memory
of M tokens, off by 2^-23 of itself, so that M / 64 of them put the state off
by 2^-23; and two roundings of an update, 2^-24 of the state each at most and
independent.  The chunk form updates once per 64 tokens, 2^14 times here:
sqrt(2^15) 2^-24 = 1.1e-5.  The recurrence updates once per token, 2^17 times
here, by two roundings of which one is relative to the addend (2^-8 of the state
and less): sqrt(2^17) 2^-24 = 2.2e-5 if every one were at its bound of half a
step and the state had its last size all along; errors spread over that step
evenly are 1 / sqrt(3) of it, 1.3e-5.  Both are below the 2e-5 of the other tests.
"""
import math

import numpy as np
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from hybrid_linear_attention_gdn_gb300 import StatePool
from lin_helpers import STATE_TOL

pytestmark = pytest.mark.gpu
MEMORIES = (65536, 131072, 262144, 1048576)


def worst_decay(memory, tokens):
    """A log decay of some 1 / memory whose lambda^tokens, rounded to a float, is off by most."""
    cand = np.float32(-1 / memory) * (1 + np.arange(400, dtype=np.float32) / 1000)
    exact = np.exp(cand.astype(np.float64) * tokens)
    return float(cand[np.abs(exact.astype(np.float32).astype(np.float64) / exact - 1).argmax()])


def rel(got, want):
    return ((got.double() - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)).tolist()


@pytest.mark.parametrize("form,tokens,calls", [
    ("cut", 65536, 16),         # 16 segments a call
    ("whole", 65536, 16),       # one of 33 sequences
    ("cut", 2048, 64),          # several segments of 8 blocks and more a call
    ("recurrent", 2048, 64),    # segments of one block
])
def test_long_memory(cuda, monkeypatch, form, tokens, calls):
    if form == "recurrent":
        monkeypatch.setenv("GDN_LIN_PREFILL_PATH", "recurrent")
    dims = gdn.Dims(1, len(MEMORIES), 128, 128, 1, torch.bfloat16, torch.bfloat16)
    ld = torch.tensor([worst_decay(m, 64) for m in MEMORIES])
    n = 33 if form == "whole" else 1
    g = torch.Generator(device="cuda").manual_seed(tokens + n)
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    pool = StatePool(normal(2, dims.hv, dims.dv, dims.dk))
    S = pool.ssm[1].double()
    ids = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    ids[0] = 1
    cu = torch.full((n + 1,), tokens, dtype=torch.int32, device="cuda")
    cu[0] = 0
    size = gdn.lin_prefill_workspace_size(dims, n, tokens)
    assert (size > 0) == (form != "whole")
    ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    ldd, out = ld.cuda(), torch.empty((tokens, dims.hv, dims.dv), dtype=torch.bfloat16, device="cuda")
    ages = torch.arange(tokens - 1, -1, -1, device="cuda", dtype=torch.float64)
    w, keep = torch.exp(ages[:, None] * ldd.double()), torch.exp(tokens * ldd.double())
    for c in range(calls):
        x = normal(tokens, dims.channels).bfloat16()
        start = torch.zeros(n, dtype=torch.int64, device="cuda")
        start[0] = c * tokens
        gdn.lin_prefill(dims, pool, None, ldd, ids, cu, start, tokens, None, 64, x, out, ws, scale=1 / math.sqrt(128))
        k, v = x[:, 128:256].double(), x[:, 256:].double().view(tokens, dims.hv, dims.dv)
        S = keep[:, None, None] * S + torch.stack([(v[:, h] * w[:, h:h + 1]).T @ k for h in range(dims.hv)])
    off = rel(pool.ssm[1], S)
    assert max(off) <= STATE_TOL, f"states of memories {MEMORIES} are off by {off}"
    # the last outputs are those of that state: bf16's half step, and 16-bit operands
    q = x[-1, :128].double()
    want = torch.einsum("hvk,k->hv", S, q) / math.sqrt(128)
    bound = 2 ** -8 * want.abs() + 2 ** -15 * (S.abs() @ q.abs()) / math.sqrt(128)
    assert bool(((out[-1].double() - want).abs() <= bound).all())
