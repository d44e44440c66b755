"""Set-ups of the selective state space tests: both sides from one seed.

Tolerances.  States and checkpoints are fp32 (relative L2 per (slot, head)
matrix): a token adds two roundings of at most 2^-24 to what it keeps, and its
own term carries the conv's and SiLU's few; with the rounding errors of n
remembered tokens adding in the worst case, n 2^-24 + 16 2^-24 <= 2e-5 for
the at most 320 tokens that a decay of these tests' distributions lets a state
remember (a decay of exp(-1e-3 .. -1.6) per token).  The chunked form's split
operands (22 bits) and chunk sums stay below the same bound.  Outputs: bf16
2e-3 beyond the row's own rounding; fp32 1e-4, the bounds of the other steps.
"""
import math

import numpy as np
import torch

import oracle
from oracle import state_space
from hybrid_linear_attention_gdn_gb300 import Dims, SsmParams, StatePool, synth

STATE_TOL = 2e-5

# (hk, hv, dk, dv, W, activations, conv history)
SHAPES = {
    "wide": (2, 16, 128, 64, 4, "bf16", "bf16"),
    "one_group": (1, 6, 128, 64, 4, "bf16", "bf16"),
    "square": (2, 4, 128, 128, 4, "bf16", "bf16"),
    "odd_heads": (3, 3, 128, 64, 4, "bf16", "bf16"),
    "dk64": (2, 4, 64, 96, 4, "bf16", "f32"),
    "tiny": (2, 4, 16, 16, 4, "f32", "f32"),
    "ragged_dv": (1, 2, 16, 33, 3, "f32", "f32"),
    "wide_conv": (1, 2, 64, 200, 8, "f32", "f32"),
    "short_conv": (2, 2, 128, 7, 2, "bf16", "bf16"),
}


def shape(name, num_slots=8):
    hk, hv, dk, dv, w, act, conv = SHAPES[name]
    return synth.LayerShape(name, hk, hv, dk, dv, w, num_slots, act, conv)


class SsmSetup:
    """One layer: parameters, a device pool and its float64 twin."""

    def __init__(self, sh, seed, device="cuda", bias=True, skip=True, decay=(1e-3, 1e-1)):
        g = self.gen = synth.generator(seed)
        self.shape, self.dims = sh, Dims.of(sh)
        conv_w = synth.normal((sh.channels, sh.w), 0.5, g)
        conv_b = synth.normal((sh.channels,), 0.2, g) if bias else None
        A_log = torch.log(1 + 15 * torch.rand((sh.hv,), generator=g))
        lo, hi = math.log(decay[0]), math.log(decay[1])
        dt = torch.exp(torch.rand((sh.hv,), generator=g) * (hi - lo) + lo)
        dt_bias = dt + torch.log(-torch.expm1(-dt))
        D = 1 + synth.normal((sh.hv,), 0.2, g) if skip else None
        ssm, conv = synth.pool(sh, g)
        dev = lambda t: None if t is None else t.to(device)
        f64 = lambda t: None if t is None else t.double().numpy().copy()
        self.params = SsmParams(dev(conv_w), dev(conv_b), dev(A_log), dev(dt_bias), dev(D))
        self.oparams = state_space.SsmParams(f64(conv_w), f64(conv_b), f64(A_log), f64(dt_bias), f64(D))
        self.pool = StatePool(ssm.to(device), conv.to(device))
        self.opool = oracle.Pool(f64(ssm), f64(conv))
        self.od = oracle.Dims(sh.hk, sh.hv, sh.dk, sh.dv, sh.w)

    def tokens(self, n):
        sh = self.shape
        qkv = synth.normal((n, sh.channels), 1.0, self.gen, sh.act_dtype)
        a = synth.normal((n, sh.hv), 1.0, self.gen, sh.act_dtype)
        return qkv, a

    def ckpt_pool(self, n, device="cuda"):
        p = StatePool.empty(self.dims, n, device)
        p.ssm.fill_(-5.0)
        p.conv.fill_(9.0)
        return p, oracle.Pool(np.full(p.ssm.shape, -5.0), np.full(p.conv.shape, 9.0))


def f64(t):
    return t.detach().cpu().double().numpy()
