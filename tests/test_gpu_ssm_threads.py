"""State space calls from several host threads at once, each on its own
stream, pool and workspace: the results of one thread."""
import threading

import torch
import pytest

import hybrid_linear_attention_gdn_gb300 as gdn
from ssm_helpers import SsmSetup, shape

pytestmark = pytest.mark.gpu


def _steps(st, qkv, a, stream, res):
    sh, n = st.shape, qkv.shape[0]
    with torch.cuda.stream(stream):
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        ids, cu, sp = i32([2, 5]), i32([0, n - 30, n]), torch.tensor([0, 63], device="cuda")
        ws = torch.empty(gdn.ssm_prefill_workspace_size(st.dims, 2, n), dtype=torch.uint8, device="cuda")
        out = torch.zeros((n, sh.hv, sh.dv), dtype=sh.act_dtype, device="cuda")
        tok = torch.zeros((2, sh.hv, sh.dv), dtype=sh.act_dtype, device="cuda")
        q8 = torch.empty((n, sh.channels), dtype=torch.float8_e4m3fn, device="cuda")
        w = torch.ones(sh.channels, device="cuda")
        for _ in range(20):
            gdn.ssm_prefill(st.dims, st.pool, None, st.params, ids, cu, sp, n, None, 64, qkv, a, out, ws)
            gdn.ssm_decode_step(st.dims, st.pool, st.params, ids, qkv[:2], a[:2], tok)
            gdn.add_rmsnorm(qkv, None, w, q8=q8)
    stream.synchronize()
    res.extend([out, tok, q8.view(torch.uint8), st.pool.ssm, st.pool.conv])


def test_threads(cuda):
    sh = shape("wide")
    base = SsmSetup(sh, seed=95)
    qkv, a = (t.cuda() for t in base.tokens(1700))
    setups = [SsmSetup(sh, seed=95) for _ in range(5)]
    streams = [torch.cuda.Stream() for _ in setups]
    results = [[] for _ in setups]
    torch.cuda.synchronize()
    jobs = [threading.Thread(target=_steps, args=(st, qkv, a, s, r)) for st, s, r in zip(setups, streams, results)]
    for j in jobs:
        j.start()
    for j in jobs:
        j.join()
    ref = []
    _steps(base, qkv, a, torch.cuda.Stream(), ref)
    for r in results:
        assert len(r) == len(ref)
        for x, y in zip(r, ref):
            assert torch.equal(x, y)
