"""The batch maps against a plain Python construction; whole numbers, so exact."""
import numpy as np
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from hybrid_linear_attention_gdn_gb300 import binding

pytestmark = pytest.mark.gpu


def plain(lens, starts, block, table, free, n_free, mc, rows):
    """The definition, one request and one row at a time."""
    n, mb, err = len(lens), table.shape[1], 0
    table, n_free = table.copy(), max(0, min(n_free, len(free)))
    cu, ck = [0], np.full((n, mc), -1)
    seq, pos, slot = np.full(rows, -1), np.zeros(rows, np.int64), np.full(rows, -1, np.int64)
    for r in range(n):
        l, p = int(lens[r]), int(starts[r])
        if l < 0 or p < 0 or p + l > mb * block:
            err |= binding.DEV_ERR_SEQLENS
            l, p = 0, 0
        if cu[-1] + l > rows:
            err |= binding.DEV_ERR_SEQLENS
            l = rows - cu[-1]
        for i in range(-(-p // block), -(-(p + l) // block)):
            if n_free:
                n_free -= 1
                table[r, i] = free[n_free]
            else:
                table[r, i] = -1
                err |= binding.DEV_ERR_BLOCKS
        for k, i in enumerate(range(p // block, (p + l) // block)):
            if k < mc:
                ck[r, k] = max(-1, table[r, i])
        for j in range(l):
            t, i = cu[-1] + j, (p + j) // block
            seq[t], pos[t] = r, p + j
            slot[t] = table[r, i] * block + (p + j) % block if table[r, i] >= 0 else -1
            if table[r, i] < 0 and i < -(-p // block):
                err |= binding.DEV_ERR_SLOT_OOB
        cu.append(cu[-1] + l)
    return dict(cu=cu, table=table, ck=ck, seq=seq, pos=pos, slot=slot, n_free=n_free, err=err)


def run(lens, starts, block, mb, n_free=None, cap=None, mc=3, rows=None, seed=0, bad_held=False, in_place=True):
    rng = np.random.default_rng(seed)
    n = len(lens)
    ids = rng.permutation(n * mb + 64 + sum(max(0, v) for v in lens) // block + n)
    table = np.full((n, mb), -1, np.int64)
    for r in range(n):
        held = min(mb, max(0, -(-int(starts[r]) // block)))
        table[r, :held] = ids[r * mb:r * mb + held]
    if bad_held:
        table[0, 0] = -1
    free = ids[n * mb:][:cap] if cap is not None else ids[n * mb:]
    n_free = len(free) if n_free is None else n_free
    rows = sum(max(0, int(v)) for v in lens) + 5 if rows is None else rows
    ref = plain(lens, starts, block, table, free, n_free, mc, rows)
    d = lambda v, t=torch.int32: torch.tensor(np.asarray(v), dtype=t, device="cuda")
    tb, nf, cu = d(table), d([n_free]), torch.full((n + 1,), 77, dtype=torch.int32, device="cuda")
    nfo = nf if in_place else torch.full((1,), 77, dtype=torch.int32, device="cuda")
    ck = torch.full((n, mc), 77, dtype=torch.int32, device="cuda")
    seq = torch.full((rows,), 77, dtype=torch.int32, device="cuda")
    pos, slot = (torch.full((rows,), 77, dtype=torch.int64, device="cuda") for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    n0 = binding.launch_count(binding.K_BATCH_MAPS)
    gdn.batch_maps(d(lens), d(starts, torch.int64), block, tb, d(free), nf, cu, ck, seq, pos, slot,
                   n_free_out=None if in_place else nfo, dev_err=err)
    assert binding.launch_count(binding.K_BATCH_MAPS) == n0 + 1
    got = dict(cu=cu, table=tb, ck=ck, seq=seq, pos=pos, slot=slot, n_free=nfo, err=err)
    for k, v in ref.items():
        assert np.array_equal(got[k].cpu().numpy().reshape(-1), np.asarray(v).reshape(-1)), k
    if not in_place:
        assert int(nf.item()) == n_free
    return ref


@pytest.mark.parametrize("block", [1, 16, 64, 256])
@pytest.mark.parametrize("n", [1, 2, 33, 300])
def test_mixed_lengths(cuda, n, block):
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 3 * block + 2, n)
    starts = rng.integers(0, 5 * block + 1, n)
    ref = run(lens, starts, block, 9, seed=n, in_place=bool(n % 2))
    assert ref["err"] == 0


def test_many_requests(cuda):
    """More requests than one pass of the scan, most of them decode rows."""
    rng = np.random.default_rng(5)
    lens = np.where(rng.random(2500) < 0.9, 1, rng.integers(0, 20, 2500))
    run(lens, rng.integers(0, 200, 2500), 64, 4, seed=6)


def test_no_requests_and_no_tokens(cuda):
    assert run([], [], 64, 0, rows=3)["n_free"] > 0
    run([0, 0], [0, 130], 64, 4)


def test_aligned_decode_row_completes_a_block(cuda):
    """The row at position 63 fills a held block; the one at 64 takes a new
    one and completes none."""
    ref = run([1, 1], [63, 64], 64, 4, mc=1)
    assert ref["ck"][0, 0] == ref["table"][0, 0] and ref["ck"][1, 0] == -1


def test_problems_are_reported(cuda):
    assert run([10, 70, 5], [0, 100, 64], 64, 4, n_free=2)["err"] == binding.DEV_ERR_BLOCKS
    assert run([10, 70], [0, 100], 64, 4, n_free=0)["n_free"] == 0
    assert run([10, 3], [0, 4], 64, 4, n_free=-7)["err"] == binding.DEV_ERR_BLOCKS
    assert run([10, 3], [0, 4], 64, 4, n_free=10 ** 6, cap=8)["err"] == 0     # more than the list holds
    assert run([-1, 5, 5, 300], [0, -3, 0, 0], 64, 4)["err"] == binding.DEV_ERR_SEQLENS
    assert run([40, 40, 40], [0, 0, 0], 64, 4, rows=70)["err"] == binding.DEV_ERR_SEQLENS
    assert run([3, 5], [10, 0], 64, 4, bad_held=True)["err"] == binding.DEV_ERR_SLOT_OOB


def test_optional_outputs(cuda):
    d = lambda v, t=torch.int32: torch.tensor(v, dtype=t, device="cuda")
    cu, nf, table = d([9, 9, 9]), d([4]), d([[-1, -1], [-1, -1]])
    gdn.batch_maps(d([3, 65]), d([0, 0], torch.int64), 64, table, d([4, 5, 6, 7]), nf, cu)
    assert cu.tolist() == [0, 3, 68] and nf.tolist() == [1] and table.tolist() == [[7, -1], [6, 5]]
