"""Double-precision linear attention with a fixed decay per head, token by
token (TEST INFRASTRUCTURE ONLY, like the rest of this package; no code shared
with the CUDA sources).

The published recurrence (Sun et al., "Retentive Network", 2023) over the slot
pool's layouts: head h reads q and k of group h // (hv // hk), the state is
St[hv][dv][dk]:  St <- lambda St + v k^T,  o = scale St q.
"""
from __future__ import annotations

import numpy as np


def token(d, log_decay, scale, ssm, x):
    """One token on one slot's state [hv][dv][dk], updated in place; o [hv][dv]."""
    G = d.hv // d.hk
    q = x[:d.hk * d.dk].reshape(d.hk, d.dk).repeat(G, 0)
    k = x[d.hk * d.dk:2 * d.hk * d.dk].reshape(d.hk, d.dk).repeat(G, 0)
    v = x[2 * d.hk * d.dk:].reshape(d.hv, d.dv)
    ssm *= np.exp(log_decay)[:, None, None]
    ssm += v[:, :, None] * k[:, None, :]
    return scale * np.einsum("hvk,hk->hv", ssm, q)


def decode_step(d, pool, log_decay, scale, slot_ids, qkv):
    """One token per request, in place on ``pool`` [slots][hv][dv][dk]."""
    out = np.zeros((len(slot_ids), d.hv, d.dv))
    for r, s in enumerate(slot_ids):
        if 0 <= s < pool.shape[0]:
            out[r] = token(d, log_decay, scale, pool[s], qkv[r])
    return out


def prefill(d, pool, ckpt, log_decay, scale, slot_ids, cu, start_pos, ckpt_ids, block, qkv, out=None):
    """Packed sequences, in place on ``pool`` and, at the block boundaries, on
    ``ckpt`` (None: no checkpoints).  Rows outside the sequences stay as in
    ``out``; those of unusable slots are zeros."""
    out = np.zeros((qkv.shape[0], d.hv, d.dv)) if out is None else out
    for n, s in enumerate(slot_ids):
        for i in range(cu[n], cu[n + 1]):
            if not 0 <= s < pool.shape[0]:
                out[i] = 0
                continue
            out[i] = token(d, log_decay, scale, pool[s], qkv[i])
            P = int(start_pos[n]) + i - int(cu[n]) + 1
            if P % block or ckpt is None:
                continue
            idx = P // block - int(start_pos[n]) // block - 1
            if idx < ckpt_ids.shape[1] and 0 <= ckpt_ids[n][idx] < ckpt.shape[0]:
                ckpt[ckpt_ids[n][idx]] = pool[s]
    return out
