"""The state space decode's two forms (a CTA or cluster per group; persistent
CTAs with a copy engine ahead) against the float64 recurrence, forced and by
the number of groups; tolerances as in the other state space tests."""
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from hybrid_linear_attention_gdn_gb300 import synth
from hybrid_linear_attention_gdn_gb300 import binding
from oracle import state_space
from helpers import assert_out_close, conv_bits_equal, max_rel_l2, out_tol
from ssm_helpers import STATE_TOL, SsmSetup, f64, shape

pytestmark = pytest.mark.gpu

# groups of 32 to 512 rows: what the persistent form takes
EXTRA = {
    "row32_f32": (3, 3, 128, 32, 4, "f32", "f32"),
    "rows288_f32conv": (2, 6, 128, 96, 4, "bf16", "f32"),
    "rows512": (2, 8, 128, 128, 4, "bf16", "bf16"),
    "rows96": (5, 5, 128, 96, 4, "bf16", "bf16"),
}


def _shape(name, slots):
    return synth.LayerShape(name, *EXTRA[name][:5], slots, *EXTRA[name][5:]) if name in EXTRA else shape(name, slots)


def _steps(st, calls):
    sh = st.shape
    for ids in calls:
        qkv, a = st.tokens(len(ids))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((len(ids), sh.hv, sh.dv), 7.0, dtype=sh.act_dtype, device="cuda")
        gdn.ssm_decode_step(st.dims, st.pool, st.params, torch.tensor(ids, dtype=torch.int32, device="cuda"),
                            qkv.cuda(), a.cuda(), out, err)
        ref, bad = state_space.decode_step(st.od, st.opool, st.oparams, ids, f64(qkv), f64(a))
        torch.cuda.synchronize()
        assert int(err.item()) == (binding.DEV_ERR_SLOT_OOB if bad else 0)
        assert_out_close(out, ref, sh.dv, out_tol(sh))
    assert max_rel_l2(f64(st.pool.ssm), st.opool.ssm, sh.dv * sh.dk) <= STATE_TOL
    assert conv_bits_equal(st.pool.conv, st.opool.conv)


@pytest.mark.parametrize("path", ["ring", "split"])
@pytest.mark.parametrize("name", ["wide", "square", "odd_heads", *EXTRA])
def test_forced(cuda, name, path, monkeypatch):
    monkeypatch.setenv("GDN_SSM_DECODE_PATH", path)
    st = SsmSetup(_shape(name, 8), seed=61, bias=name != "square", skip=name != "wide")
    _steps(st, [[3], [5, -1, 0, 7, 2, 99, 1], [-1], [1, 3]])


@pytest.mark.parametrize("path", ["ring", "split", ""])
@pytest.mark.parametrize("n", [47, 76, 130, 301, 512, 530])
def test_many_requests(cuda, n, path, monkeypatch):
    """Around one and several rounds of a group per SM, padded rows among them."""
    monkeypatch.setenv("GDN_SSM_DECODE_PATH", path)
    st = SsmSetup(shape("wide", n + 9), seed=62)
    ids = torch.randperm(n + 9, generator=st.gen)[:n].tolist()
    ids[5:n:17] = [-1] * len(ids[5:n:17])
    _steps(st, [ids, ids[::-1]])


@pytest.mark.parametrize("n", [60, 600])
def test_all_padded(cuda, n, monkeypatch):
    monkeypatch.setenv("GDN_SSM_DECODE_PATH", "ring")
    _steps(SsmSetup(shape("square", 8), seed=65), [[-1] * n, [-1] * (n - 1) + [8], [-1] * (n // 2) + [3, -1]])


@pytest.mark.parametrize("what", ["qkv", "conv_w", "conv_bias"])
def test_unaligned_inputs_take_the_split_form(cuda, what, monkeypatch):
    """Tensors that the copy engine cannot start at, with the persistent form asked for."""
    monkeypatch.setenv("GDN_SSM_DECODE_PATH", "ring")
    st, st2 = SsmSetup(shape("wide"), seed=63), SsmSetup(shape("wide"), seed=63)
    qkv, a = (t.cuda() for t in st.tokens(3))

    def off(t):
        return torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view_as(t).copy_(t)

    q2, p2 = qkv, st2.params
    if what == "qkv":
        q2 = off(qkv)
    else:
        p2 = gdn.SsmParams(**{k: off(getattr(p2, k)) if k == what else getattr(p2, k)
                              for k in ("conv_w", "conv_bias", "A_log", "dt_bias", "D")})
    ids = torch.tensor([4, 1, 6], dtype=torch.int32, device="cuda")
    outs = [torch.empty((3, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    gdn.ssm_decode_step(st.dims, st.pool, st.params, ids, qkv, a, outs[0])
    gdn.ssm_decode_step(st2.dims, st2.pool, p2, ids, q2, a, outs[1])
    ref, _ = state_space.decode_step(st.od, st.opool, st.oparams, ids.tolist(), f64(qkv), f64(a))
    for o in outs:
        assert_out_close(o, ref, 64, out_tol(st.shape))
    for p in (st.pool, st2.pool):
        assert max_rel_l2(f64(p.ssm), st.opool.ssm, 64 * 128) <= STATE_TOL and conv_bits_equal(p.conv, st.opool.conv)


def test_back_to_back_launches_and_replays(cuda, monkeypatch):
    """Dependent launches of both forms in one graph on the same slots: each
    sees the state and history of the one before."""
    st, two = SsmSetup(shape("wide", 90), seed=64), SsmSetup(shape("wide", 90), seed=64)
    ids = torch.randperm(90, generator=st.gen).to(torch.int32).cuda()
    qkv, a = (t.cuda() for t in st.tokens(90))
    out = torch.empty((90, 16, 64), dtype=torch.bfloat16, device="cuda")

    def four(s, sync):
        for path in ("ring", "split", "ring", "ring"):
            monkeypatch.setenv("GDN_SSM_DECODE_PATH", path)
            gdn.ssm_decode_step(s.dims, s.pool, s.params, ids, qkv, a, out)
            if sync:
                torch.cuda.synchronize()

    four(two, True)
    start = st.pool.ssm.clone(), st.pool.conv.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        four(st, False)
    for _ in range(3):
        st.pool.ssm.copy_(start[0]), st.pool.conv.copy_(start[1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(st.pool.ssm, two.pool.ssm) and torch.equal(st.pool.conv, two.pool.conv)
