"""Refusals of the state space, norm and batch-map calls, without a GPU, and
the float64 recurrence against its definition."""
import ctypes

import numpy as np
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from hybrid_linear_attention_gdn_gb300 import _build, binding
import oracle
from oracle import state_space
from ssm_helpers import SsmSetup, f64, shape


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gdn.load()


def _dims(**kw):
    d = dict(hk=2, hv=16, dk=128, dv=64, conv_width=4, act_dtype=1, conv_dtype=1)
    d.update(kw)
    return binding.CDims(**d)


POOL = binding.CPool(0x10000, 0x20000, 4)
PARAMS = binding.CSsmParams(0x1000, None, 0x2000, 0x3000, None)


def _decode(lib, d=None, pool=POOL, p=PARAMS, ids=0x100, B=1, qkv=0x200, a=0x300, out=0x400):
    return lib.gdn_ssm_decode_step(ctypes.byref(d or _dims()), pool, ctypes.byref(p) if p else None, ids, B, qkv, a,
                                   out, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=_dims(dk=32)), binding.ERR_UNSUPPORTED),
    (dict(d=_dims(hv=15)), binding.ERR_INVALID_ARG),
    (dict(d=_dims(hk=1, hv=256)), binding.ERR_UNSUPPORTED),   # 16384 rows in one group
    (dict(B=-1), binding.ERR_INVALID_ARG),
    (dict(B=65536), binding.ERR_UNSUPPORTED),
    (dict(p=None), binding.ERR_INVALID_ARG),
    (dict(p=binding.CSsmParams(None, None, 0x2000, 0x3000, None)), binding.ERR_INVALID_ARG),
    (dict(p=binding.CSsmParams(0x1000, None, 0x2000, None, None)), binding.ERR_INVALID_ARG),
    (dict(ids=None), binding.ERR_INVALID_ARG),
    (dict(qkv=None), binding.ERR_INVALID_ARG),
    (dict(a=None), binding.ERR_INVALID_ARG),
    (dict(out=None), binding.ERR_INVALID_ARG),
    (dict(pool=binding.CPool(None, None, 4)), binding.ERR_INVALID_ARG),
    (dict(pool=binding.CPool(0x10004, 0x20000, 4)), binding.ERR_INVALID_ARG),
    (dict(B=0, p=None), binding.OK),
])
def test_decode_refusals(lib, kw, status):
    n0 = lib.gdn_launch_count(binding.K_SSM_DECODE)
    assert _decode(lib, **kw) == status
    assert lib.gdn_launch_count(binding.K_SSM_DECODE) == n0


def _prefill(lib, d=None, pool=POOL, ck=POOL, p=PARAMS, ids=0x100, cu=0x180, sp=0x200, n=2, total=100, ck_ids=0x280,
             mc=1, block=64, qkv=0x300, a=0x400, out=0x500, ws=0x600, nbytes=None):
    d = d or _dims()
    if nbytes is None:
        nbytes = 1 << 40
    return lib.gdn_ssm_prefill(ctypes.byref(d), pool, ck, ctypes.byref(p) if p else None, ids, cu, sp, n, total,
                               ck_ids, mc, block, qkv, a, out, ws, nbytes, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=_dims(dk=32)), binding.ERR_UNSUPPORTED),
    (dict(n=-1), binding.ERR_INVALID_ARG),
    (dict(total=-1), binding.ERR_INVALID_ARG),
    (dict(mc=-1), binding.ERR_INVALID_ARG),
    (dict(block=0), binding.ERR_INVALID_ARG),
    (dict(block=100), binding.ERR_INVALID_ARG),
    (dict(n=65536), binding.ERR_UNSUPPORTED),
    (dict(total=1 << 31), binding.ERR_UNSUPPORTED),
    (dict(mc=4 * 65536), binding.ERR_UNSUPPORTED),
    (dict(p=None), binding.ERR_INVALID_ARG),
    (dict(ids=None), binding.ERR_INVALID_ARG),
    (dict(cu=None), binding.ERR_INVALID_ARG),
    (dict(sp=None), binding.ERR_INVALID_ARG),
    (dict(ck_ids=None), binding.ERR_INVALID_ARG),
    (dict(ck=binding.CPool(None, None, 4)), binding.ERR_INVALID_ARG),
    (dict(qkv=None), binding.ERR_INVALID_ARG),
    (dict(a=None), binding.ERR_INVALID_ARG),
    (dict(out=None), binding.ERR_INVALID_ARG),
    (dict(n=0, p=None), binding.OK),
])
def test_prefill_refusals(lib, kw, status):
    n0 = lib.gdn_launch_count(binding.K_SSM_PREFILL)
    assert _prefill(lib, **kw) == status
    assert lib.gdn_launch_count(binding.K_SSM_PREFILL) == n0


def test_prefill_workspace(lib):
    d = _dims()
    size = lib.gdn_ssm_prefill_workspace_size(ctypes.byref(d), 2, 100)
    assert lib.gdn_ssm_prefill_workspace_size(ctypes.byref(d), 0, 100) == 0
    assert lib.gdn_ssm_prefill_workspace_size(ctypes.byref(d), 2, 0) == 0
    assert lib.gdn_ssm_prefill_workspace_size(ctypes.byref(_dims(dk=32)), 2, 100) == 0
    if size:  # missing, short, misaligned
        assert _prefill(lib, ws=None) == binding.ERR_INVALID_ARG
        assert _prefill(lib, nbytes=size - 1) == binding.ERR_INVALID_ARG
        assert _prefill(lib, ws=0x610) == binding.ERR_INVALID_ARG


def _norm(lib, act=1, res=1, x=0x100, r=0x200, w=0x300, eps=1e-6, n=4, d=256, y=0x400, q=0x500, s=0x600, g=32, st=0):
    return lib.gdn_add_rmsnorm(act, res, x, r, w, eps, n, d, y, q, s, g, st, None)


@pytest.mark.parametrize("kw,status", [
    (dict(act=2), binding.ERR_INVALID_ARG),
    (dict(res=-1), binding.ERR_INVALID_ARG),
    (dict(x=None), binding.ERR_INVALID_ARG),
    (dict(w=None), binding.ERR_INVALID_ARG),
    (dict(y=None, q=None), binding.ERR_INVALID_ARG),
    (dict(s=None), binding.ERR_INVALID_ARG),
    (dict(eps=-1.0), binding.ERR_INVALID_ARG),
    (dict(eps=float("nan")), binding.ERR_INVALID_ARG),
    (dict(n=-1), binding.ERR_INVALID_ARG),
    (dict(d=0), binding.ERR_INVALID_ARG),
    (dict(g=48), binding.ERR_INVALID_ARG),
    (dict(g=-32), binding.ERR_INVALID_ARG),
    (dict(d=240), binding.ERR_INVALID_ARG),               # 32 does not divide it
    (dict(st=2), binding.ERR_INVALID_ARG),
    (dict(x=0x101), binding.ERR_INVALID_ARG),
    (dict(s=0x602), binding.ERR_INVALID_ARG),
    (dict(d=32769, g=0), binding.ERR_UNSUPPORTED),
    (dict(n=0, x=None), binding.OK),
])
def test_norm_refusals(lib, kw, status):
    n0 = lib.gdn_launch_count(binding.K_ADD_RMSNORM)
    assert _norm(lib, **kw) == status
    assert lib.gdn_launch_count(binding.K_ADD_RMSNORM) == n0


def _maps(lib, lens=0x100, sp=0x200, n=4, block=64, table=0x300, mb=8, free=0x400, cap=16, nf=0x500, nfo=0x500,
          cu=0x600, ck=0x700, mc=2, seq=None, pos=None, slot=None, rows=100):
    return lib.gdn_batch_maps(lens, sp, n, block, table, mb, free, cap, nf, nfo, cu, ck, mc, seq, pos, slot, rows,
                              None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), binding.ERR_INVALID_ARG),
    (dict(block=0), binding.ERR_INVALID_ARG),
    (dict(block=96), binding.ERR_INVALID_ARG),            # not a power of two
    (dict(mb=-1), binding.ERR_INVALID_ARG),
    (dict(cap=-1), binding.ERR_INVALID_ARG),
    (dict(mc=-1), binding.ERR_INVALID_ARG),
    (dict(rows=-1), binding.ERR_INVALID_ARG),
    (dict(lens=None), binding.ERR_INVALID_ARG),
    (dict(sp=None), binding.ERR_INVALID_ARG),
    (dict(table=None), binding.ERR_INVALID_ARG),
    (dict(free=None), binding.ERR_INVALID_ARG),
    (dict(nf=None), binding.ERR_INVALID_ARG),
    (dict(nfo=None), binding.ERR_INVALID_ARG),
    (dict(cu=None), binding.ERR_INVALID_ARG),
    (dict(ck=None), binding.ERR_INVALID_ARG),
    (dict(n=8193), binding.ERR_UNSUPPORTED),
    (dict(rows=1 << 31), binding.ERR_UNSUPPORTED),
])
def test_maps_refusals(lib, kw, status):
    n0 = lib.gdn_launch_count(binding.K_BATCH_MAPS)
    assert _maps(lib, **kw) == status
    assert lib.gdn_launch_count(binding.K_BATCH_MAPS) == n0


def test_binding_refuses_wrong_tensors():
    """Types, shapes, strides and devices are checked before the call."""
    sh = shape("tiny")
    st = SsmSetup(sh, 1, device="cpu")
    qkv, a = st.tokens(2)
    ids, out = torch.tensor([0, 1], dtype=torch.int32), torch.zeros(2, sh.hv, sh.dv)
    for bad in (dict(qkv=qkv.double()), dict(qkv=qkv[:1]), dict(a=a.t().contiguous().t()), dict(out=out[:, :, 1:]),
                dict(ids=ids.long()), {}):  # the last: right, but not on a GPU
        kw = dict(ids=ids, qkv=qkv, a=a, out=out)
        kw.update(bad)
        with pytest.raises(gdn.GdnError) as e:
            gdn.ssm_decode_step(st.dims, st.pool, st.params, kw["ids"], kw["qkv"], kw["a"], kw["out"])
        assert e.value.status == binding.ERR_INVALID_ARG
    x = torch.zeros(3, 64)
    for kw in (dict(x=x.half()), dict(weight=torch.ones(63)), dict(q8=torch.zeros(3, 64)), dict(x=x[:, ::2]),
               dict(q8=torch.zeros(3, 64).to(torch.float8_e4m3fn), group=48)):
        args = dict(x=x, residual=None, weight=torch.ones(64))
        args.update(kw)
        with pytest.raises(gdn.GdnError):
            gdn.add_rmsnorm(**args)


def test_recurrence_by_hand():
    """One head of one channel: the recurrence written out for three tokens."""
    d = oracle.Dims(1, 1, 1, 1, 2)
    p = state_space.SsmParams(np.array([[0.5, 1.0], [0.0, 2.0], [-1.0, 1.0]]), np.array([0.1, 0.0, 0.2]),
                              np.array([0.3]), np.array([-0.4]), np.array([0.7]))
    ssm, conv = np.array([[[0.25]]]), np.array([[0.1, -0.2, 0.3]])
    xs, as_ = np.array([[1.0, 0.5, -1.0], [0.2, -0.3, 2.0], [0.0, 1.0, 1.0]]), np.array([[0.1], [-2.0], [1.5]])
    S, prev = 0.25, [0.1, -0.2, 0.3]
    silu = lambda v: v / (1 + np.exp(-v))
    for x, a in zip(xs, as_):
        q, k, v = (silu(p.conv_w[c, 0] * prev[c] + p.conv_w[c, 1] * x[c] + p.conv_bias[c]) for c in range(3))
        dt = np.log(1 + np.exp(a[0] - 0.4))
        S = np.exp(-np.exp(0.3) * dt) * S + dt * v * k
        prev = list(x)
        assert np.allclose(state_space.token(d, p, ssm, conv, x, a), S * q + 0.7 * v, rtol=1e-13)
        assert np.allclose(ssm, S, rtol=1e-13) and np.array_equal(conv[0], x)
