"""Linear attention with a fixed decay: both forms of the prefill on the same
calls, values of any size, neighbours that are not finite, prompts in parts,
captured and repeated calls, several streams and threads, many short
sequences, tensors beyond 32 bits."""
import threading

import numpy as np
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from hybrid_linear_attention_gdn_gb300 import StatePool
from oracle import linear
from helpers import max_rel_l2
from lin_helpers import STATE_TOL, LinSetup, assert_out_close, ckpt_table, f64
from test_gpu_lin import _state_close, run_prefill

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _i64(v):
    return torch.tensor(v, dtype=torch.int64, device="cuda")


def _ws(st, n, total):
    size = gdn.lin_prefill_workspace_size(st.dims, n, total)
    return torch.empty(size, dtype=torch.uint8, device="cuda") if size else None


def _call(st, pool, ids, cu, sp, x, out, ck=None, table=None, block=64, ws=None, err=None):
    n, total = len(ids), x.shape[0]
    gdn.lin_prefill(st.dims, pool, ck, st.ld, ids, cu, sp, total, table, block, x, out,
                    _ws(st, n, total) if ws is None else ws, scale=st.scale, dev_err=err)


@pytest.mark.parametrize("lens,starts", [([64], [0]), ([200, 33], [7, 64]), ([1300, 5, 700], [3, 63, 0])])
def test_recurrence_on_the_chunk_forms_shape(cuda, monkeypatch, lens, starts):
    monkeypatch.setenv("GDN_LIN_PREFILL_PATH", "recurrent")
    run_prefill(LinSetup("square", 21), lens, starts, block=128)


def test_rows_off_their_alignment(cuda):
    """qkv 2 bytes into its allocation, out 2 bytes into its: no chunk form."""
    st = LinSetup("square", 22)
    x = st.tokens(200)
    buf = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")
    xo = buf[1:].view(x.shape)
    xo.copy_(x)
    ob = torch.empty(200 * 4 * 128 + 1, dtype=x.dtype, device="cuda")
    out = ob[1:].view(200, 4, 128)
    _call(st, st.pool, _i32([3, 1]), _i32([0, 130, 200]), _i64([5, 0]), xo, out)
    ref = linear.prefill(st.od, st.opool, None, st.old, st.scale, [3, 1], [0, 130, 200], [5, 0], np.zeros((2, 0), int),
                         64, f64(x))
    assert_out_close(out, ref, 128)
    _state_close(st.pool, st.opool)


@pytest.mark.parametrize("name", ["square", "own_keys", "dk64", "tiny"])
@pytest.mark.parametrize("q,k,v,s", [(1e-15, 1e-12, 1e12, 1.0), (1e10, 1e8, 1e9, 1e17), (1.0, 1e-18, 1e-18, 1e-36)])
def test_values_of_any_size(cuda, name, q, k, v, s):
    """Queries, keys, values and states far from 1: fp32's range, no scaling."""
    st = LinSetup(name, 23)
    d, kd = st.dims, st.dims.hk * st.dims.dk
    x = st.tokens(150).float()
    x[:, :kd] *= q
    x[:, kd:2 * kd] *= k
    x[:, 2 * kd:] *= v
    x = x.to(st.act)
    st.pool.ssm.mul_(s)
    st.opool = f64(st.pool.ssm)
    out = st.out(150)
    _call(st, st.pool, _i32([2]), _i32([0, 150]), _i64([40]), x.cuda(), out)
    ref = linear.prefill(st.od, st.opool, None, st.old, st.scale, [2], [0, 150], [40], np.zeros((1, 0), int), 64, f64(x))
    assert_out_close(out, ref, d.dv)
    _state_close(st.pool, st.opool)


@pytest.mark.parametrize("name", ["square", "tiny"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_not_finite(cuda, name, bad):
    """Around a sequence they reach nothing; inside it, its outputs and states
    from that block of 64 positions on, and no other sequence."""
    st = LinSetup(name, 24)
    x = st.tokens(400)
    clean = x.clone()
    clean[:10], clean[310:] = 0, 0
    x[:10], x[310:] = bad, bad
    cu, sp, ids = _i32([10, 90, 310]), _i64([30, 0]), _i32([4, 6])
    outs, pools = [], []
    for y in (clean, x):
        p = StatePool(st.pool.ssm.clone())
        o = st.out(400)
        _call(st, p, ids, cu, sp, y.cuda(), o)
        outs.append(o)
        pools.append(p.ssm)
    assert torch.equal(outs[0], outs[1]) and torch.equal(pools[0], pools[1])
    x = clean.clone()
    x[10 + 60, 3] = bad  # position 90 of the first sequence: block 64 .. 127
    p, o = StatePool(st.pool.ssm.clone()), st.out(400)
    ck, _ = st.ckpt(2)
    _call(st, p, ids, cu, sp, x.cuda(), o, ck, _i32([[0, -1, -1], [-1, -1, -1]]))
    first = 10 + 64 - 30
    assert torch.equal(o[:first], outs[0][:first]) and torch.equal(o[90:], outs[0][90:])
    assert torch.equal(p.ssm[6], pools[0][6]) and bool(ck.ssm[0].isfinite().all())
    assert not bool(o[70:90].isfinite().all())


@pytest.mark.parametrize("name", ["square", "narrow"])
def test_a_prompt_in_parts(cuda, name):
    """Three calls, the last from a checkpoint that was copied to another slot,
    then single tokens: the float64 recurrence over all of them."""
    st = LinSetup(name, 25)
    x = st.tokens(300 + 3)
    ref = linear.prefill(st.od, st.opool, None, st.old, st.scale, [1], [0, 303], [0], np.zeros((1, 0), int), 64, f64(x))
    xd, out = x.cuda(), st.out(303)
    ck, _ = st.ckpt(3)
    _call(st, st.pool, _i32([1]), _i32([0, 100]), _i64([0]), xd[:100], out[:100])
    _call(st, st.pool, _i32([1]), _i32([0, 120]), _i64([100]), xd[100:220], out[100:220], ck, _i32([[0, 2]]))
    assert_out_close(out[:220], ref[:220], st.dims.dv)
    gdn.slot_copy(st.dims, ck, st.pool, _i32([2]), _i32([5]))  # the state at position 192
    _call(st, st.pool, _i32([5]), _i32([0, 108]), _i64([192]), xd[192:300], out[192:300])
    for i in range(300, 303):
        gdn.lin_decode_step(st.dims, st.pool, st.ld, _i32([5]), xd[i:i + 1], out[i:i + 1], scale=st.scale)
    assert_out_close(out, ref, st.dims.dv)
    assert max_rel_l2(f64(st.pool.ssm[5:6]), st.opool[1:2], st.dims.dv * st.dims.dk) <= STATE_TOL


@pytest.mark.parametrize("name", ["square", "tiny"])
def test_captured_calls(cuda, name):
    """One graph of a cut prefill with checkpoints and of a decode step, replayed
    on other inputs, against eager calls, bit for bit; two graphs at once."""
    lens, starts, total = [1500, 700], [10, 64], 2200
    xs = []
    graphs, held = [], []
    for seed in (26, 27):
        st = LinSetup(name, seed)
        table, n_ck = ckpt_table(lens, starts, 256, st.gen)
        ck, _ = st.ckpt(n_ck)
        x, out, tok = st.tokens(total).cuda(), st.out(total), st.out(2)
        ids, cu, sp = _i32([0, 3]), _i32([0, 1500, 2200]), _i64(starts)
        t, ws = torch.from_numpy(table).cuda(), _ws(st, 2, total)
        assert ws is not None
        first = st.pool.ssm.clone()

        def step(st=st, ck=ck, x=x, out=out, tok=tok, ids=ids, cu=cu, sp=sp, t=t, ws=ws):
            _call(st, st.pool, ids, cu, sp, x, out, ck, t, 256, ws)
            gdn.lin_decode_step(st.dims, st.pool, st.ld, ids, x[:2], tok, scale=st.scale)

        step()  # loads the kernels
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
        held.append((st, first, step, x, out, tok, ck))
    streams = [torch.cuda.Stream() for _ in graphs]
    for round_ in range(2):
        for st, first, step, x, out, tok, ck in held:
            st.pool.ssm.copy_(first)
            x.copy_(st.tokens(total).cuda())
            xs.append(x.clone())
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in (out, tok, st.pool.ssm, ck.ssm)] for st, _, _, _, out, tok, ck in held]
        for (st, first, step, x, out, tok, ck), want in zip(held, got):
            st.pool.ssm.copy_(first)
            step()
            assert all(torch.equal(a, b) for a, b in zip((out, tok, st.pool.ssm, ck.ssm), want))


@pytest.mark.parametrize("total", [900, 2600])
def test_threads_on_their_own_streams(cuda, total):
    """Whole sequences, and one that is cut (pieces of one call wait for others of it)."""
    base = LinSetup("square", 28)
    x = base.tokens(total).cuda()
    first = base.pool.ssm.clone()
    cu, sp, ids = _i32([0, total - 200, total]), _i64([0, 70]), _i32([2, 5])

    def work(stream, res):
        with torch.cuda.stream(stream):
            pool, out = StatePool(first.clone()), base.out(total)
            tok, ws = base.out(2), _ws(base, 2, total)
            for _ in range(20):
                _call(base, pool, ids, cu, sp, x, out, ws=ws)
                gdn.lin_decode_step(base.dims, pool, base.ld, ids, x[:2], tok, scale=base.scale)
        stream.synchronize()
        res.extend([out, tok, pool.ssm])

    torch.cuda.synchronize()
    streams, results = [torch.cuda.Stream() for _ in range(5)], [[] for _ in range(5)]
    jobs = [threading.Thread(target=work, args=a) for a in zip(streams, results)]
    for j in jobs:
        j.start()
    for j in jobs:
        j.join()
    ref = []
    work(torch.cuda.Stream(), ref)
    for r in results:
        assert len(r) == 3 and all(torch.equal(a, b) for a, b in zip(r, ref))


@pytest.mark.parametrize("name", ["square", "tiny"])
@pytest.mark.parametrize("seed", range(3))
def test_many_short_sequences(cuda, name, seed):
    rng = np.random.default_rng(seed)
    lens = rng.choice([0, 1, 2, 3, 63, 64, 65, 130], 60).tolist()
    starts = rng.choice([0, 1, 62, 63, 64, 127, 200], 60).tolist()
    st = LinSetup(name, 29 + seed, num_slots=60)
    run_prefill(st, lens, starts, gaps=(seed, 3 * seed))


def test_one_sequence_among_many_padded_ones(cuda):
    """The rule for segments counts padded and empty sequences; all are walked right."""
    st = LinSetup("square", 31, num_slots=40)
    lens = [0] * 12 + [1700] + [1] * 12
    slots = [-1] * 12 + [7] + list(range(8, 20))
    run_prefill(st, lens, [0] * 25, block=512, slots=slots)


def test_slots_and_rows_beyond_32_bits(cuda):
    st = LinSetup("square", 32)
    d = st.dims
    slots = 2 ** 31 // (d.hv * d.dv * d.dk) + 60
    rows = 2 ** 31 // d.channels + 100
    far = StatePool.empty(d, slots, "cuda")
    x = st.tokens(90).cuda()
    big = torch.zeros((rows, d.channels), dtype=st.act, device="cuda")
    big_o = torch.zeros((rows, d.hv, d.dv), dtype=st.act, device="cuda")
    big[-90:] = x
    for s in (slots - 1, slots - 2):
        far.ssm[s] = st.pool.ssm[slots - s]
    sp = _i64([60, 0])

    def run(pool, ids, lo, q, out):
        ck, _ = st.ckpt(4)
        _call(st, pool, _i32(ids), _i32([lo, lo + 50, lo + 90]), sp, q, out, ck, _i32([[1], [2]]))
        o, t = out[-90:].clone(), st.out(2)
        gdn.lin_decode_step(d, pool, st.ld, _i32(ids), q[-2:].contiguous(), t, scale=st.scale)
        return o, t, ck.ssm, pool.ssm[ids]

    want = run(st.pool, [1, 2], 0, x, st.out(90))
    got = run(far, [slots - 1, slots - 2], rows - 90, big, big_o)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("name", ["square", "own_keys"])
@pytest.mark.parametrize("lens,starts", [
    ([2100, 5, 64], [0, 3, 0]),           # one long sequence: cut
    ([5, 900, 5, 1], [62, 127, 0, 9]),
    ([720] * 3, [0, 64, 1]),              # of one length: whole
    ([0, 3000, 0], [5, 70, 64]),
    ([2000] + [7] * 31, [1] * 32),        # the most that are cut
    ([2000] + [7] * 32, [1] * 33),        # one more: whole
])
def test_cut_or_whole_by_the_longest(cuda, name, lens, starts):
    run_prefill(LinSetup(name, 33, num_slots=len(lens) + 3), lens, starts, block=256, gaps=(1, 2))


def test_bad_offsets_beside_a_cut_sequence(cuda):
    """A sequence whose rows are inconsistent is left out, the others run."""
    st = LinSetup("square", 34)
    x = st.tokens(2300)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = st.out(2300)
    _call(st, st.pool, _i32([1, 2, 5]), _i32([0, 2000, 2300, 2200]), _i64([0, 0, 0]), x.cuda(), out, err=err)
    ref = linear.prefill(st.od, st.opool, None, st.old, st.scale, [1, 2], [0, 2000, 2300], [0, 0], np.zeros((2, 0), int),
                         64, f64(x))
    assert_out_close(out, ref, 128)
    _state_close(st.pool, st.opool)
    assert int(err) == gdn.binding.DEV_ERR_SEQLENS


def test_a_verified_draft_is_committed(cuda):
    """spec_commit of slots without a conv history."""
    st = LinSetup("tiny", 35)
    spec = StatePool(torch.randn((6, *st.pool.ssm.shape[1:]), generator=st.gen).cuda())
    want = st.pool.ssm.clone()
    gdn.spec_commit(st.dims, spec, st.pool, _i32([[0, 1, 2], [3, 4, 5], [1, 2, 3]]), _i32([2, 0, 3]), _i32([4, 5, 0]))
    want[4], want[0] = spec.ssm[1], spec.ssm[3]
    assert torch.equal(st.pool.ssm, want)
