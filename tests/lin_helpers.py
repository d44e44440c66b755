"""Set-ups of the tests of linear attention with a fixed decay.

Tolerances.  States and checkpoints are fp32 (relative L2 per (slot, head)
matrix).  A token multiplies what is kept by lambda (its own error at most
2^-23, the product's 2^-24) and adds v k^T (2^-24): at most 2^-22 of what a
state remembers, and a state remembers at most some 80 tokens' worth here
(rates from 1/8 to 1/80 a token, or at most 60 tokens without decay), in the
worst case 80 * 2^-22 = 1.9e-5 <= 2e-5.  The chunk form takes the products of v
and lambda^n exactly as their fp32 value (24 bits in three parts) and adds a
chunk's terms in twelve products, each off by at most 2^-23 of the terms'
magnitudes in sum, which for 64 independent terms are up to 8 times their sum:
12 * 8 * 2^-23 = 1.1e-5; a state takes two roundings per chunk, with a decay of two
floats, fewer than the recurrence's.  Together below the same bound.
Outputs: 2e-3 (bf16) and 1e-4 (fp32), the bounds of the other steps, beyond the
error of the exact values' own rounding: where a strong decay leaves
o = (q.k) v, one factor times bf16 values, a row's rounding errors are not
independent and reach any part of their bound of half a step, 2^-8 in bf16,
which is above 2e-3 without any error of a kernel.
"""
import math

import numpy as np
import torch

import oracle
from hybrid_linear_attention_gdn_gb300 import Dims, StatePool

STATE_TOL = 2e-5

# (hk, hv, dk, dv, type)
SHAPES = {
    "square": (2, 4, 128, 128, "bf16"),
    "own_keys": (3, 3, 128, 128, "bf16"),
    "narrow": (2, 4, 64, 64, "bf16"),
    "half_dv": (2, 2, 128, 64, "bf16"),
    "odd_dv": (1, 2, 128, 7, "bf16"),
    "dk64": (2, 4, 64, 96, "bf16"),
    "one_dv": (1, 1, 64, 1, "f32"),
    "tiny": (2, 4, 16, 16, "f32"),
    "ragged_dv": (1, 2, 16, 33, "f32"),
    "wide_dv": (1, 2, 64, 200, "f32"),
    "square_f32": (2, 2, 128, 128, "f32"),
}


def f64(t):
    return t.detach().cpu().double().numpy()


class LinSetup:
    def __init__(self, name, seed, num_slots=8, device="cuda", rates=(1 / 8, 1 / 80)):
        hk, hv, dk, dv, act = SHAPES[name]
        self.gen = g = torch.Generator().manual_seed(seed)
        self.act = torch.bfloat16 if act == "bf16" else torch.float32
        self.dims = Dims(hk, hv, dk, dv, 1, self.act, self.act)
        lo, hi = math.log(rates[0]), math.log(rates[1])
        self.log_decay = -torch.exp(torch.rand(hv, generator=g) * (hi - lo) + lo)
        self.scale = dk ** -0.5
        ssm = torch.randn((num_slots, hv, dv, dk), generator=g)
        self.pool, self.opool = StatePool(ssm.to(device)), f64(ssm).copy()
        self.ld = self.log_decay.to(device)
        self.od, self.old = oracle.Dims(hk, hv, dk, dv, 1), f64(self.log_decay)
        self.device = device

    def tokens(self, n):
        return torch.randn((n, self.dims.channels), generator=self.gen).to(self.act)

    def ckpt(self, n):
        d = self.dims
        p = torch.full((n, d.hv, d.dv, d.dk), -5.0)
        return StatePool(p.to(self.device)), f64(p).copy()

    def out(self, n, fill=7.0):
        return torch.full((n, self.dims.hv, self.dims.dv), fill, dtype=self.act, device=self.device)


def assert_out_close(out, ref, row):
    """Rows and tensor within the bound beyond their own rounding; a row counts
    as at least the tensor's RMS row (the chunk form's errors are absolute)."""
    tol = 2e-3 if out.dtype == torch.bfloat16 else 1e-4
    x, ref = f64(out).reshape(-1, row), np.asarray(ref).reshape(-1, row)
    rnd = torch.from_numpy(ref).to(out.dtype).double().numpy()
    err, own, nrm = (np.linalg.norm(t, axis=1) for t in (x - ref, rnd - ref, ref))
    floor = np.sqrt(np.mean(nrm ** 2))
    assert np.isfinite(x).all() and np.linalg.norm(err) - np.linalg.norm(own) <= tol * np.linalg.norm(nrm)
    worst = ((err - own) - tol * np.maximum(nrm, floor)).max()
    assert worst <= 0, f"a row is off by {worst:.3e} more than its bound"


def ckpt_table(lens, starts, block, gen):
    """Distinct checkpoint ids for every boundary: (table [n][max], ids in all)."""
    counts = [(p + v) // block - p // block for v, p in zip(lens, starts)]
    table = np.full((len(lens), max(1, max(counts))), -1, np.int32)
    ids = torch.randperm(sum(counts) + 1, generator=gen).numpy()
    at = 0
    for r, c in enumerate(counts):
        table[r, :c] = ids[at:at + c]
        at += c
    return table, sum(counts) + 1
