"""Double-precision selective state space step, token by token (TEST
INFRASTRUCTURE ONLY, like the rest of this package; no code shared with the
CUDA sources).

The published recurrence (Gu & Dao, "Mamba", 2023; Dao & Gu, "Transformers
are SSMs", ICML 2024) over the slot pool's layouts: head h reads q and k of
group h // (hv // hk), the conv history holds the last W - 1 raw inputs,
oldest first, the state is St[hv][dv][dk].
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

from . import Dims, Pool


@dataclass
class SsmParams:
    conv_w: np.ndarray            # [C][W]
    conv_bias: np.ndarray | None  # [C]
    A_log: np.ndarray             # [hv]
    dt_bias: np.ndarray           # [hv]
    D: np.ndarray | None          # [hv]


def token(d: Dims, p: SsmParams, ssm, conv, x, a):
    """One token on one slot's state [hv][dv][dk] and history [W-1][C], both
    updated in place; returns o [hv][dv]."""
    G = d.hv // d.hk
    win = np.concatenate([conv, x[None]])
    y = (win * p.conv_w.T).sum(0) + (0.0 if p.conv_bias is None else p.conv_bias)
    y = y / (1.0 + np.exp(-y))
    q = y[:d.hk * d.dk].reshape(d.hk, d.dk).repeat(G, 0)
    k = y[d.hk * d.dk:2 * d.hk * d.dk].reshape(d.hk, d.dk).repeat(G, 0)
    v = y[2 * d.hk * d.dk:].reshape(d.hv, d.dv)
    dt = np.logaddexp(0.0, a + p.dt_bias)
    ssm *= np.exp(-np.exp(p.A_log) * dt)[:, None, None]
    ssm += (dt[:, None] * v)[:, :, None] * k[:, None, :]
    conv[:] = win[1:]
    o = np.einsum("hvk,hk->hv", ssm, q)
    return o if p.D is None else o + p.D[:, None] * v


def _usable(slot, n):
    return 0 <= slot < n


def decode_step(d: Dims, pool: Pool, p: SsmParams, slot_ids, qkv, a):
    """One token per request, in place on ``pool``.  Returns (out, an id was out of range)."""
    out = np.zeros((len(slot_ids), d.hv, d.dv))
    n = pool.ssm.shape[0]
    for r, s in enumerate(slot_ids):
        if _usable(s, n):
            out[r] = token(d, p, pool.ssm[s], pool.conv[s], qkv[r], a[r])
    return out, any(s != -1 and not _usable(s, n) for s in slot_ids)


def prefill(d: Dims, pool: Pool, ckpt: Pool | None, p: SsmParams, slot_ids, cu, start_pos, ckpt_ids, block, qkv, a):
    """Packed sequences, in place on ``pool``; state and history copied into
    ``ckpt`` at the block boundaries.  Returns out (zeros for unusable slots)."""
    out = np.zeros((qkv.shape[0], d.hv, d.dv))
    for n, s in enumerate(slot_ids):
        if not _usable(s, pool.ssm.shape[0]):
            continue
        for i in range(cu[n], cu[n + 1]):
            out[i] = token(d, p, pool.ssm[s], pool.conv[s], qkv[i], a[i])
            P = int(start_pos[n]) + i - int(cu[n]) + 1
            if P % block or ckpt is None:
                continue
            idx = P // block - int(start_pos[n]) // block - 1
            if idx < ckpt_ids.shape[1] and _usable(ckpt_ids[n][idx], ckpt.ssm.shape[0]):
                ckpt.ssm[ckpt_ids[n][idx]] = pool.ssm[s]
                ckpt.conv[ckpt_ids[n][idx]] = pool.conv[s]
    return out
