"""The state space prefill over the range of its inputs: saturated SiLU,
queries or keys that are zero, values at the top of fp32, heads of very
different sizes.  Each head is compared at its own size; tolerances as in the
other state space tests unless derived here.
"""
import numpy as np
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
import oracle
from hybrid_linear_attention_gdn_gb300 import synth
from oracle import state_space
from helpers import assert_out_close, out_tol
from ssm_helpers import SsmSetup, f64, shape
from test_gpu_ssm import _check_states

pytestmark = pytest.mark.gpu

IDS, LENS, STARTS = [4, 1], [100, 130], [33, 64]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _call(st, qkv, a, ids=IDS, lens=LENS, starts=STARTS):
    """One prefill and its recurrence: both outputs."""
    sh, total = st.shape, sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    out = torch.full((total, sh.hv, sh.dv), 7.0, dtype=sh.act_dtype, device="cuda")
    size = gdn.ssm_prefill_workspace_size(st.dims, len(lens), total)
    ws = torch.full((size,), 0xff, dtype=torch.uint8, device="cuda") if size else None
    gdn.ssm_prefill(st.dims, st.pool, None, st.params, _i32(ids), _i32(cu), torch.tensor(starts, device="cuda"), total,
                    None, 64, qkv.cuda(), a.cuda(), out, ws)
    ref = state_space.prefill(st.od, st.opool, None, st.oparams, ids, cu, starts, None, 64, f64(qkv), f64(a))
    return out, ref


def _check_heads(st, out, ref):
    for h in range(st.shape.hv):
        assert_out_close(out[:, h], ref[:, h], st.shape.dv, out_tol(st.shape), row_floor_rms=True)
    _check_states(st, st.pool, st.opool)


def _silu(x, qk=0.0):
    """SiLU as the token recurrence takes it: a layer whose output is D v (and
    S q with queries and keys of SiLU(qk))."""
    hv = 64
    sh = synth.LayerShape("silu", 1, hv, 16, 16, 2, 1, "f32", "f32")
    st = SsmSetup(sh, seed=70, bias=False)
    st.params.conv_w[:] = torch.tensor([0.0, 1.0], device="cuda")
    st.params.D[:] = 1.0
    st.pool.conv.zero_(), st.pool.ssm.zero_()
    T = x.numel() // (hv * 16)
    qkv = torch.cat([torch.full((T, 2 * 16), qk), x.reshape(T, hv * 16)], 1).cuda()
    out = torch.empty((T, hv, 16), device="cuda")
    gdn.ssm_prefill(st.dims, st.pool, None, st.params, _i32([0]), _i32([0, T]), torch.tensor([0], device="cuda"), T, None,
                    64, qkv, torch.zeros((T, hv), device="cuda"), out, None)
    return out.cpu().reshape(-1)


def test_silu_of_the_recurrence(cuda):
    """From -3e38 to 3e38.  For x >= -87 the exponential's 2 units in the last
    place and half a one for each of its correction, the sum, the product and
    the quotient's 2: 5.5 <= 6 units of at most 2^-23; below, where the
    exponential leaves the normal range, what is lost is at most 90 2^-126."""
    big = torch.logspace(2, 38.4, 4096, dtype=torch.float64)
    x = torch.cat([torch.linspace(-110, 110, 57344, dtype=torch.float64), -big, big]).float()
    got = _silu(x).double()
    xd = x.double()
    ref = xd / (1 + torch.exp(-xd))
    assert torch.isfinite(got).all()
    assert ((got - ref).abs() <= 6 * 2.0 ** -23 * ref.abs() + 90 * 2.0 ** -126).all()


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_silu_of_the_recurrence_not_finite(cuda, value):
    """As in the decode step: infinity, NaN, NaN.  With keys of 0 the state
    takes infinity times 0, so that every output is NaN."""
    x = torch.full((1024,), value)
    assert torch.isnan(_silu(x)).all()
    got = _silu(x, qk=1.0)
    assert (got == float("inf")).all() if value > 0 else torch.isnan(got).all()


@pytest.mark.parametrize("name", ["tiny", "dk64", "wide_conv", "ragged_dv"])
@pytest.mark.parametrize("value", [-1e30, -1e37])
def test_saturated_channels(cuda, name, value):
    """Channels whose conv sums are far below zero: features of 0."""
    st = SsmSetup(shape(name), seed=71)
    st.params.conv_w.abs_()
    st.oparams.conv_w[:] = f64(st.params.conv_w)
    qkv, a = st.tokens(sum(LENS))
    qkv[:, ::3] = value
    _check_heads(st, *_call(st, qkv, a))


@pytest.mark.parametrize("scale", [1e-6, 1e6])
@pytest.mark.parametrize("name", ["tiny", "dk64", "wide_conv"])
def test_recurrence_small_and_large_inputs(cuda, name, scale):
    st = SsmSetup(shape(name), seed=72, bias=False)
    qkv, a = st.tokens(sum(LENS))
    st.pool.conv *= scale
    st.pool.ssm *= scale * scale
    st.opool.conv[:], st.opool.ssm[:] = f64(st.pool.conv), f64(st.pool.ssm)  # the rounded products
    _check_heads(st, *_call(st, (qkv.float() * scale).to(qkv.dtype), a))


@pytest.mark.parametrize("zero", ["q", "k", "qk"])
@pytest.mark.parametrize("name", ["wide", "square"])
def test_zero_queries_and_keys(cuda, name, zero):
    """Where q.k is zero throughout, D v is all that P holds: it keeps its
    bits at any dt and for skips from 0.01 to 5."""
    st = SsmSetup(shape(name), seed=73, decay=(0.1, 3.0))
    n = st.shape.hk * st.shape.dk
    cols = slice(0 if "q" in zero else n, 2 * n if "k" in zero else n)
    for p in (st.params, st.oparams):
        p.conv_bias[cols] = 0.0
        p.A_log[:] = -7.0  # a state that fp32 still holds at the end
    for p in (st.pool, st.opool):
        p.conv[:, :, cols] = 0.0
    st.params.D[:] = torch.tensor([0.1, 0.5, 0.01, 5.0] * (st.shape.hv // 4))
    st.oparams.D[:] = f64(st.params.D)
    qkv, a = st.tokens(sum(LENS))
    qkv[:, cols] = 0.0
    _check_heads(st, *_call(st, qkv, a))


@pytest.mark.parametrize("name", ["wide", "square"])
def test_zero_everything(cuda, name):
    """No inputs, no bias, no skip term: the state decays, every output is 0."""
    st = SsmSetup(shape(name), seed=74, bias=False, skip=False)
    st.params.A_log[:] = -7.0
    st.oparams.A_log[:] = -7.0
    st.pool.conv.zero_()
    st.opool.conv[:] = 0.0
    qkv, a = st.tokens(sum(LENS))
    out, ref = _call(st, torch.zeros_like(qkv), a)
    assert (out == 0).all() and (ref == 0).all()
    _check_states(st, st.pool, st.opool)


@pytest.mark.parametrize("big,small", [(1.0, 1e-12), (1e6, 1e-6), (1e20, 1.0), (1.0, 0.0)])
def test_heads_of_different_sizes(cuda, big, small):
    """Neighbouring heads that share a tile's products: each keeps its bits,
    whatever the other's size."""
    st = SsmSetup(shape("wide"), seed=76, bias=False)
    sh = st.shape
    c = 2 * sh.hk * sh.dk
    qkv, a = st.tokens(sum(LENS))
    for h in range(sh.hv):
        f = big if h % 2 else small
        cols = slice(c + h * sh.dv, c + (h + 1) * sh.dv)
        qkv[:, cols] = (qkv[:, cols].float() * f).to(qkv.dtype)
        st.pool.conv[:, :, cols] *= f
        st.pool.ssm[:, h] *= f
    st.opool.conv[:], st.opool.ssm[:] = f64(st.pool.conv), f64(st.pool.ssm)
    _check_heads(st, *_call(st, qkv, a))


def _sum_of_terms(st, opool, qkv, a, h, ch):
    """The readouts of head h's channel ch with every term's magnitude."""
    p, sh, n, rows, out = st.oparams, st.shape, st.shape.hk * st.shape.dk, f64(qkv), []
    hq, vc = h // (sh.hv // sh.hk), 2 * n + h * sh.dv + ch
    cols = [hq * sh.dk + np.arange(sh.dk), n + hq * sh.dk + np.arange(sh.dk), np.array([vc])]
    dt = np.logaddexp(0.0, f64(a)[:, h] + p.dt_bias[h])
    for slot, lo, hi in zip(IDS, [0, LENS[0]], [LENS[0], sum(LENS)]):
        x = np.concatenate([opool.conv[slot], rows[lo:hi]])
        y = [sum(p.conv_w[c, j] * x[j:len(x) - sh.w + 1 + j, c] for j in range(sh.w)) + p.conv_bias[c] for c in cols]
        q, k, v = (np.abs(f / (1 + np.exp(-f))) for f in y)
        s = np.abs(opool.ssm[slot, h, ch])
        for t in range(hi - lo):
            s = np.exp(-np.exp(p.A_log[h]) * dt[lo + t]) * s + dt[lo + t] * v[t] * k[t]
            out.append(s @ q[t] + (0.0 if p.D is None else abs(p.D[h]) * v[t, 0]))
    return np.array(out)


@pytest.mark.parametrize("wide_bound", [False, True])
@pytest.mark.parametrize("scale", [1e30, 1e34, 1e36])
@pytest.mark.parametrize("name", ["wide", "square"])
def test_values_at_the_top_of_the_range(cuda, name, scale, wide_bound):
    """A channel of head 0 with raw values up to some 1e36: bounds of |V| and
    |S| pass the largest fp32 value, V, the state and the outputs do not.
    wide_bound: another channel's taps are large, so that the bound of |V|
    (largest tap sum times largest input) overflows by itself.

    Head 0's rows are that one channel, not the dv of which a row's bound
    takes the norm.  Its elements: q, k, G, P, V (or q and S) are rounded to
    11 bits, 2^-11 of every term each, and the sum to bf16, 2^-8."""
    st = SsmSetup(shape(name), seed=75, skip=not wide_bound)
    c, ch = 2 * st.shape.hk * st.shape.dk, 5
    if wide_bound:
        st.params.conv_w[c + 2] = 60.0
        st.oparams.conv_w[c + 2] = 60.0
    qkv, a = st.tokens(sum(LENS))
    qkv[:, c + ch] = (qkv[:, c + ch].float() * scale).to(qkv.dtype)
    before = oracle.Pool(st.opool.ssm.copy(), st.opool.conv.copy())
    with np.errstate(over="ignore"):
        out, ref = _call(st, qkv, a)
        terms = _sum_of_terms(st, before, qkv, a, 0, ch)
    assert torch.isfinite(out).all()
    got, want = f64(out[:, 0, ch]), ref[:, 0, ch]
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 5.1 * 2.0 ** -11 * terms).all()
    for h in range(1, st.shape.hv):
        assert_out_close(out[:, h], ref[:, h], st.shape.dv, out_tol(st.shape), row_floor_rms=True)
    _check_states(st, st.pool, st.opool)


@pytest.mark.parametrize("name", ["wide", "square"])
def test_rows_before_an_infinite_step(cuda, name):
    """An infinite dt: the rows before it, in its own block of 64 too, keep
    their values; from it on its head is not finite."""
    st = SsmSetup(shape(name), seed=77, decay=(0.1, 1.0))
    qkv, a = st.tokens(100)
    a[50, 2] = float("inf")
    with np.errstate(all="ignore"):
        out, ref = _call(st, qkv, a, [3], [100], [0])
    heads = [h for h in range(st.shape.hv) if h != 2]
    for h, end in [(2, 50)] + [(h, 100) for h in heads]:
        assert_out_close(out[:end, h], ref[:end, h], st.shape.dv, out_tol(st.shape), row_floor_rms=True)
    assert not torch.isfinite(out[50:, 2]).any()
    assert not torch.isfinite(st.pool.ssm[3, 2]).any() and torch.isfinite(st.pool.ssm[3, heads]).all()


@pytest.mark.parametrize("name", ["wide", "square"])
@pytest.mark.parametrize("T", [64, 150])
def test_small_steps_after_a_strong_decay(cuda, name, T):
    """Heads that forget within a token, with time steps between 1e-5 and 60
    in a block: the state is what the last, small steps gave."""
    st = SsmSetup(shape(name), seed=78)
    for p in (st.params, st.oparams):
        p.A_log[::2] = 30.0
        p.dt_bias[:] = 0.0
    qkv, a = st.tokens(T)
    a[:] = torch.where(torch.rand(a.shape, generator=st.gen) < 0.2, 60.0, -2.0 + a.float()).to(a.dtype)
    a[-6:] = -11.0
    out, ref = _call(st, qkv, a, [3], [T], [0])
    # (the few rows of large steps hold a head's norm, where bf16's rounding
    # alone may reach 2^-8: the whole tensor, not head by head)
    assert_out_close(out, ref, st.shape.dv, out_tol(st.shape), row_floor_rms=True)
    _check_states(st, st.pool, st.opool)
