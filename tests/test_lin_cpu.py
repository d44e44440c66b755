"""Refusals of the linear-attention calls without a GPU, slot calls without a
conv history, and the float64 recurrence against its definition."""
import ctypes

import numpy as np
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
import oracle
from hybrid_linear_attention_gdn_gb300 import _build, binding
from oracle import linear


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gdn.load()


def _dims(**kw):
    d = dict(hk=2, hv=4, dk=128, dv=128, conv_width=1, act_dtype=1, conv_dtype=1)
    d.update(kw)
    return binding.CDims(**d)


POOL = binding.CPool(0x10000, None, 4)


def _decode(lib, d=None, pool=POOL, ld=0x80, ids=0x100, B=1, qkv=0x200, out=0x400):
    return lib.gdn_lin_decode_step(ctypes.byref(d or _dims()), pool, ld, 1.0, ids, B, qkv, out, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=_dims(dk=32)), binding.ERR_UNSUPPORTED),
    (dict(d=_dims(dv=257)), binding.ERR_UNSUPPORTED),
    (dict(d=_dims(conv_width=4)), binding.ERR_UNSUPPORTED),
    (dict(d=_dims(conv_width=0)), binding.ERR_INVALID_ARG),
    (dict(d=_dims(hk=1, hv=65536)), binding.ERR_UNSUPPORTED),
    (dict(d=_dims(hv=3)), binding.ERR_INVALID_ARG),
    (dict(d=_dims(act_dtype=2)), binding.ERR_INVALID_ARG),
    (dict(B=-1), binding.ERR_INVALID_ARG),
    (dict(B=65536), binding.ERR_UNSUPPORTED),
    (dict(ld=None), binding.ERR_INVALID_ARG),
    (dict(ids=None), binding.ERR_INVALID_ARG),
    (dict(qkv=None), binding.ERR_INVALID_ARG),
    (dict(out=None), binding.ERR_INVALID_ARG),
    (dict(pool=binding.CPool(None, None, 4)), binding.ERR_INVALID_ARG),
    (dict(pool=binding.CPool(0x10004, None, 4)), binding.ERR_INVALID_ARG),
    (dict(B=0, ld=None, ids=None), binding.OK),
])
def test_decode_refusals(lib, kw, status):
    n0 = lib.gdn_launch_count(binding.K_LIN_DECODE)
    assert _decode(lib, **kw) == status
    assert lib.gdn_launch_count(binding.K_LIN_DECODE) == n0


def _prefill(lib, d=None, pool=POOL, ck=POOL, ld=0x80, ids=0x100, cu=0x180, sp=0x200, n=2, total=100, ck_ids=0x280,
             mc=2, block=64, qkv=0x300, out=0x400, ws=0x10000, ws_bytes=1 << 30):
    return lib.gdn_lin_prefill(ctypes.byref(d or _dims()), pool, ck, ld, 1.0, ids, cu, sp, n, total, ck_ids, mc, block,
                               qkv, out, ws, ws_bytes, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=_dims(conv_width=4)), binding.ERR_UNSUPPORTED),
    (dict(d=_dims(dk=48)), binding.ERR_UNSUPPORTED),
    (dict(n=-1), binding.ERR_INVALID_ARG),
    (dict(total=-1), binding.ERR_INVALID_ARG),
    (dict(mc=-1), binding.ERR_INVALID_ARG),
    (dict(block=0), binding.ERR_INVALID_ARG),
    (dict(block=100), binding.ERR_INVALID_ARG),
    (dict(n=16385), binding.ERR_UNSUPPORTED),
    (dict(total=1 << 31), binding.ERR_UNSUPPORTED),
    (dict(ld=None), binding.ERR_INVALID_ARG),
    (dict(ids=None), binding.ERR_INVALID_ARG),
    (dict(cu=None), binding.ERR_INVALID_ARG),
    (dict(sp=None), binding.ERR_INVALID_ARG),
    (dict(ck_ids=None), binding.ERR_INVALID_ARG),
    (dict(qkv=None), binding.ERR_INVALID_ARG),
    (dict(out=None), binding.ERR_INVALID_ARG),
    (dict(pool=binding.CPool(None, None, 1)), binding.ERR_INVALID_ARG),
    (dict(ck=binding.CPool(0x10001, None, 1)), binding.ERR_INVALID_ARG),
    (dict(n=0, ld=None), binding.OK),
])
def test_prefill_refusals(lib, kw, status):
    n0 = lib.gdn_launch_count(binding.K_LIN_PREFILL)
    assert _prefill(lib, **kw) == status
    assert lib.gdn_launch_count(binding.K_LIN_PREFILL) == n0


def test_workspace_size_is_host_only(lib):
    size = lambda d, n, t: lib.gdn_lin_prefill_workspace_size(ctypes.byref(d), n, t)
    assert size(_dims(conv_width=4), 1, 1 << 20) == 0
    assert size(_dims(), 0, 100) == 0 and size(_dims(), 1, 0) == 0


def test_slot_calls_without_a_conv_history(lib):
    d = _dims()
    assert lib.gdn_state_record_bytes(ctypes.byref(d)) == 4 * 128 * 128 * 4
    assert lib.gdn_slot_zero(ctypes.byref(d), POOL, None, 0, None, None) == binding.OK
    # the steps that have a conv still refuse such layers
    assert lib.gdn_decode_step(ctypes.byref(d), POOL, None, None, 1, None, None, None, None, None,
                               None) == binding.ERR_UNSUPPORTED
    assert lib.gdn_ssm_decode_step(ctypes.byref(d), POOL, None, None, 1, None, None, None, None,
                                   None) == binding.ERR_UNSUPPORTED
    # and a conv history is still required where there is one
    assert lib.gdn_slot_zero(ctypes.byref(_dims(conv_width=2)), POOL, 0x100, 1, None, None) == binding.ERR_INVALID_ARG


def test_pools_of_the_binding():
    dims = gdn.Dims(2, 4, 16, 16, 1, torch.float32, torch.float32)
    p = gdn.StatePool.empty(dims, 3, "cpu")
    assert p.conv is None and p.c().conv is None and p.c().num_slots == 3
    with pytest.raises(gdn.GdnError, match="not on the current CUDA device"):
        gdn.lin_decode_step(dims, p, torch.zeros(4), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 128),
                            torch.zeros(1, 4, 16))
    w4 = gdn.Dims(2, 4, 16, 16, 4, torch.float32, torch.float32)
    with pytest.raises(gdn.GdnError):
        gdn.lin_decode_step(w4, p, torch.zeros(4), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 128),
                            torch.zeros(1, 4, 16))


def test_recurrence_against_the_sum():
    """St = lambda^n S0 + sum_j lambda^(n - 1 - j) v_j k_j^T, o_i = scale St_i q_i."""
    rng = np.random.default_rng(1)
    d = oracle.Dims(2, 4, 16, 8, 1)
    n = 23
    x = rng.standard_normal((n, 2 * 2 * 16 + 4 * 8))
    ld = -rng.random(4)
    S0 = rng.standard_normal((1, 4, 8, 16))
    S = S0.copy()
    out = linear.prefill(d, S, None, ld, 0.25, [0], [0, n], [0], np.zeros((1, 0), int), 64, x)
    q = x[:, :32].reshape(n, 2, 16).repeat(2, 1)
    k = x[:, 32:64].reshape(n, 2, 16).repeat(2, 1)
    v = x[:, 64:].reshape(n, 4, 8)
    for i in (0, 7, n - 1):
        w = np.exp(ld[None] * (i - np.arange(i + 1))[:, None])
        St = np.exp(ld * (i + 1))[:, None, None] * S0[0] + np.einsum("jh,jhv,jhk->hvk", w, v[:i + 1], k[:i + 1])
        np.testing.assert_allclose(out[i], 0.25 * np.einsum("hvk,hk->hv", St, q[i]), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(S[0], St, rtol=1e-12, atol=1e-12)
