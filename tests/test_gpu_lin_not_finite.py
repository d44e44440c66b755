"""A NaN or an infinity in one query, key or value of a prompt: what it reaches
(its own heads' outputs and states from its block of 64 positions on) and what
it must not (anything before that block, other heads, columns, rows and
sequences), whole and cut, against the same call without it, bit for bit."""
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from hybrid_linear_attention_gdn_gb300 import StatePool
from lin_helpers import LinSetup
from test_gpu_lin_paths import _call, _i32, _i64

pytestmark = pytest.mark.gpu

# lens, starts, sequence and token of the bad value, checkpoint block
CASES = {
    "whole": ([80, 220], [30, 0], 0, 60, 64),
    "last_token": ([5, 70], [0, 60], 1, 69, 64),
    "first_token": ([64, 130], [0, 0], 1, 0, 64),
    "first_segment": ([64, 2100, 5], [0, 20, 7], 1, 200, 256),
    "middle_segment": ([2100, 64, 5], [0, 3, 9], 0, 1200, 256),
    "last_segment": ([7, 2100], [3, 100], 1, 2090, 256),
}


@pytest.mark.parametrize("name", ["square", "narrow", "tiny"])
@pytest.mark.parametrize("case", sorted(CASES))
@pytest.mark.parametrize("what", ["q", "k", "v"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_it_reaches(cuda, name, case, what, bad):
    lens, starts, seq, tok, block = CASES[case]
    st = LinSetup(name, 41 + tok)
    d, n, total = st.dims, len(lens), sum(lens)
    G, dk, dv = d.hv // d.hk, d.dk, d.dv
    cu = [sum(lens[:i]) for i in range(n + 1)]
    x = st.tokens(total)
    qk_head, col, head, row = d.hk - 1, dk // 2 + 1, d.hv - 1, dv // 2
    at = {"q": qk_head * dk + col, "k": (d.hk + qk_head) * dk + col, "v": 2 * d.hk * dk + head * dv + row}[what]
    heads = list(range(qk_head * G, (qk_head + 1) * G)) if what != "v" else [head]
    others = [h for h in range(d.hv) if h not in heads]
    counts = [(p + v) // block - p // block for v, p in zip(lens, starts)]
    table = torch.full((n, max(max(counts), 1)), -1, dtype=torch.int32)
    for r, c in enumerate(counts):
        table[r, :c] = torch.arange(c, dtype=torch.int32) + sum(counts[:r])
    res = []
    for y in (x, x.clone()):
        if res:
            y[cu[seq] + tok, at] = bad
        pool, out = StatePool(st.pool.ssm.clone()), st.out(total)
        ck, _ = st.ckpt(sum(counts) + 1)
        _call(st, pool, _i32([4, 6, 1][:n]), _i32(cu), _i64(starts), y.cuda(), out, ck, table.cuda(), block)
        res.append((out, pool.ssm, ck.ssm))
    (out, ssm, ck), (out2, ssm2, ck2) = res
    first = cu[seq] + max(0, (starts[seq] + tok) // 64 * 64 - starts[seq])  # the block's first row
    hit, end = cu[seq] + tok, cu[seq + 1]
    # what it must not reach
    assert torch.equal(out[:first], out2[:first]) and torch.equal(out[end:], out2[end:])
    assert torch.equal(out[:, others], out2[:, others]) and torch.equal(ssm[:, others], ssm2[:, others])
    slot = [4, 6, 1][seq]
    keep = [s for s in range(ssm.shape[0]) if s != slot]
    assert torch.equal(ssm[keep], ssm2[keep]) and torch.equal(ck[:, others], ck2[:, others])
    early = [int(table[r, i]) for r, c in enumerate(counts) for i in range(c)
             if r != seq or (starts[r] // block + i + 1) * block <= starts[r] + tok]
    late = [int(table[seq, i]) for i in range(counts[seq]) if (starts[seq] // block + i + 1) * block > starts[seq] + tok]
    assert torch.equal(ck[early], ck2[early])
    # what it reaches
    if what == "q":
        assert torch.equal(ssm, ssm2) and torch.equal(ck, ck2)
        assert not bool(out2[hit][heads].isfinite().any())
        return
    gone, rest = (torch.zeros(dv, dk, dtype=torch.bool, device="cuda") for _ in range(2))
    gone[(slice(None), col) if what == "k" else row] = True
    rest = ~gone
    for s, s2 in [(ssm[slot], ssm2[slot])] + [(ck[i], ck2[i]) for i in late]:
        assert not bool(s2[heads][:, gone].isfinite().any())
        assert torch.equal(s[heads][:, rest], s2[heads][:, rest])
    o = out2[hit:end][:, heads]
    assert not bool((o if what == "k" else o[..., row]).isfinite().any())
    if what == "v":
        sel = [r for r in range(dv) if r != row]
        assert torch.equal(out[..., sel], out2[..., sel])
