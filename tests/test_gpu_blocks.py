"""Fork, release, compact and page copies against plain Python, exactly."""
import numpy as np
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from hybrid_linear_attention_gdn_gb300 import binding

pytestmark = pytest.mark.gpu


class Pool:
    """Block tables, counts and stack on the device and as plain lists."""

    def __init__(self, seed, num_blocks, rows, max_blocks, block, cap=None):
        self.rng = np.random.default_rng(seed)
        self.N, self.block = num_blocks, block
        self.cap = num_blocks if cap is None else cap
        self.free = self.rng.permutation(num_blocks).tolist()
        self.refs = [0] * num_blocks
        self.table = np.full((rows, max_blocks), -1, np.int64)
        self.lens = [0] * rows

    def hold(self, row, tokens):
        for j in range(-(-tokens // self.block)):
            self.table[row, j] = self.free.pop()
        self.lens[row] = tokens

    def device(self):
        i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")
        self.d_table, self.d_refs = i32(self.table), i32(self.refs)
        self.d_free = i32(self.free + [-9] * (self.cap - len(self.free)))
        self.d_n = i32([len(self.free)])
        return self

    def fork(self, src, dst, lens):
        cs, cd = [], []
        for s, d, n in zip(src, dst, lens):
            a = b = -1
            if s >= 0 and d >= 0:
                for j in range(n // self.block):
                    self.table[d, j] = self.table[s, j]
                    self.refs[self.table[s, j]] += 1
                if n % self.block:
                    if self.free:
                        a, b = self.table[s, n // self.block], self.free.pop()
                    self.table[d, n // self.block] = b
            cs.append(a)
            cd.append(b)
        return cs, cd

    def release(self, rows, old, new):
        gone = set()
        for r, o, n in zip(rows, old, new):
            if r < 0:
                continue
            for j in range(-(-n // self.block), -(-o // self.block)):
                id = self.table[r, j]
                self.table[r, j] = -1
                self.refs[id] -= 1
                if self.refs[id] < 0:
                    self.refs[id] = 0
                    gone.add(int(id))
        self.free += sorted(gone)

    def check(self):
        assert self.d_table.tolist() == self.table.tolist()
        assert self.d_refs.tolist() == self.refs
        assert int(self.d_n) == len(self.free)
        assert self.d_free.tolist()[:len(self.free)] == self.free


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda").reshape(-1)


def _i64(v):
    return torch.tensor(v, dtype=torch.int64, device="cuda").reshape(-1)


def _word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _fork(p, src, dst, lens, err=None):
    cs, cd = _i32([5] * len(src)), _i32([5] * len(src))
    gdn.block_fork(_i32(src), _i32(dst), _i64(lens), p.block, p.d_table, p.d_refs, p.d_free, p.d_n, cs, cd, dev_err=err)
    return cs.tolist(), cd.tolist()


def _release(p, rows, old, new, err=None):
    gdn.block_release(_i32(rows), _i64(old), _i64(new), p.block, p.d_table, p.d_refs, p.d_free, p.d_n, dev_err=err)


@pytest.mark.parametrize("parents,children,longest,block", [
    (1, 1, 1, 1), (1, 4, 100, 16), (3, 2, 64, 64), (40, 3, 700, 16), (700, 2, 40, 16),
])
def test_branches_come_and_go(cuda, parents, children, longest, block):
    n = parents * children
    mb = -(-longest // block) + 1
    p = Pool(n + longest, parents * mb + n + 3, parents + n, mb, block)
    for r in range(parents):
        p.hold(r, int(p.rng.integers(0, longest + 1)))
    p.device()
    src = [r for r in range(parents) for _ in range(children)]
    dst = list(range(parents, parents + n))
    lens = [p.lens[s] for s in src]
    if n > 5:
        src[2] = -1
    err = _word()
    assert _fork(p, src, dst, lens, err) == p.fork(src, dst, lens)
    p.check()
    # some branches end, some are cut back, then everything else goes: the last holder gives a block back
    live = [d for s, d in zip(src, dst) if s >= 0]
    lens = {d: n for s, d, n in zip(src, dst, lens) if s >= 0}
    rows = live[::2] + [-1]
    new = [0 if i % 2 else int(p.rng.integers(0, lens[r] + 1)) for i, r in enumerate(live[::2])] + [0]
    old = [lens[r] for r in live[::2]] + [3]
    _release(p, rows, old, new, err)
    p.release(rows, old, new)
    p.check()
    lens.update(zip(rows, new))
    rows = list(range(parents)) + live
    old = p.lens[:parents] + [lens[r] for r in live]
    _release(p, rows, old, [0] * len(rows), err)
    p.release(rows, old, [0] * len(rows))
    p.check()
    assert sorted(p.free) == list(range(p.N)) and int(err) == 0


def test_fork_refusals_on_the_device(cuda):
    p = Pool(1, 12, 6, 3, 4)
    p.hold(0, 10)  # 3 blocks
    p.hold(1, 9)
    p.device()
    err = _word()
    # a row out of range, its own branch, a negative and a too long length; the others run
    src, dst, lens = [9, 1, 0, 0, 0], [2, 1, 3, 4, 2], [4, 4, -1, 13, 8]
    assert _fork(p, src, dst, lens, err) == ([-1] * 5, [-1] * 5)
    p.fork([0], [2], [8])
    p.check()
    assert int(err) == binding.DEV_ERR_SLOT_OOB | binding.DEV_ERR_SEQLENS
    # a held entry that is no block: it stays -1 in the branch
    err.zero_()
    p.d_table[1, 0] = -1
    p.d_table[1, 2] = 55
    assert _fork(p, [1], [5], [9], err) == ([-1], [-1])
    assert p.d_table[5].tolist() == [-1, p.table[1, 1], -1] and int(err) == binding.DEV_ERR_SLOT_OOB


def test_the_stack_runs_out(cuda):
    p = Pool(2, 4, 5, 2, 8)
    p.hold(0, 9)
    p.device()  # two blocks are free
    err = _word()
    got = _fork(p, [0, 0, 0], [1, 2, 3], [9, 9, 9], err)
    assert got == p.fork([0, 0, 0], [1, 2, 3], [9, 9, 9])
    p.check()
    assert int(err) == binding.DEV_ERR_BLOCKS and int(p.d_n) == 0


def test_release_refusals_on_the_device(cuda):
    p = Pool(3, 12, 4, 3, 4)
    p.hold(0, 12)
    p.hold(1, 5)
    p.device()
    err = _word()
    _release(p, [7, 0, 1], [4, 4, 13], [0, 5, 0], err)  # out of range, longer than before, beyond the table
    p.check()
    assert int(err) == binding.DEV_ERR_SLOT_OOB | binding.DEV_ERR_SEQLENS
    # a block given up by a row that never shared it goes back once
    err.zero_()
    p.d_table[2, 0] = int(p.table[0, 0])
    p.table[2, 0] = p.table[0, 0]
    _release(p, [0, 2], [12, 4], [0, 0], err)
    p.release([0], [12], [0])
    p.table[2, 0] = -1
    p.check()
    assert int(err) == binding.DEV_ERR_SLOT_OOB
    # a stack that is too short keeps the lowest
    err.zero_()
    q = Pool(4, 10, 1, 8, 1)
    q.hold(0, 8)
    q.cap = 5
    q.device()
    _release(q, [0], [8], [0], err)
    assert int(err) == binding.DEV_ERR_BLOCKS and int(q.d_n) == 5
    assert q.d_free.tolist() == (q.free + sorted(q.table[0].tolist()))[:5]


def test_nothing_to_do(cuda):
    p = Pool(5, 3, 1, 1, 4).device()
    _fork(p, [], [], [])
    _release(p, [], [], [])
    p.check()


def compact(p, max_moves):
    live = p.N - len(p.free)
    free = set(p.free)
    movers = sorted((b for b in range(live, p.N) if b not in free), reverse=True)[:max_moves]
    holes = sorted(b for b in free if b < live)[:len(movers)]
    to = dict(zip(movers, holes))
    p.table = np.vectorize(lambda b: to.get(b, b))(p.table) if p.table.size else p.table
    refs = list(p.refs)
    for s, d in to.items():
        refs[d], refs[s] = p.refs[s], 0
    p.refs = refs
    p.free = sorted((free - set(holes)) | set(movers), reverse=True)
    return movers, holes


@pytest.mark.parametrize("N,used,max_moves,in_place", [
    (1, 0.0, 1, True), (1, 1.0, 1, False), (31, 0.5, 31, True), (64, 0.3, 40, False), (1000, 0.6, 1000, True),
    (1000, 0.6, 17, False), (1000, 0.6, 0, True), (5000, 0.97, 300, True), (300000, 0.4, 150000, False),
])
def test_compact(cuda, N, used, max_moves, in_place):
    rows = 7
    p = Pool(N, N, rows, N // rows + 2, 16)
    for _ in range(int(N * used)):
        r = int(p.rng.integers(rows))
        if p.lens[r] < p.table.shape[1]:
            p.table[r, p.lens[r]] = p.free.pop()
            p.refs[p.table[r, p.lens[r]]] = int(p.rng.integers(3))
            p.lens[r] += 1
    if p.table.shape[1] > p.lens[0]:
        p.table[0, p.lens[0]] = N + 5  # not a block: stays
    p.device()
    err, nm = _word(), _word() + 77
    src, dst = _i32([5] * max_moves), _i32([5] * max_moves)
    ws = torch.full((gdn.block_compact_workspace_size(N),), 255, dtype=torch.uint8, device="cuda")
    outs = {}
    if not in_place:
        old = p.d_table.clone(), p.d_refs.clone(), p.d_free.clone()
        outs = dict(table_out=torch.full_like(p.d_table, 3), refs_out=torch.full_like(p.d_refs, 3),
                    free_out=torch.full_like(p.d_free, 3))
    gdn.block_compact(p.d_table, p.d_refs, p.d_free, p.d_n, src, dst, nm, ws, dev_err=err, **outs)
    if not in_place:
        assert all(torch.equal(a, b) for a, b in zip(old, (p.d_table, p.d_refs, p.d_free)))
        assert outs["free_out"].tolist()[len(p.free):] == p.d_free.tolist()[len(p.free):]
        p.d_table, p.d_refs, p.d_free = outs["table_out"], outs["refs_out"], outs["free_out"]
    movers, holes = compact(p, max_moves)
    p.check()
    pad = [-1] * (max_moves - len(movers))
    assert int(nm) == len(movers) and src.tolist() == movers + pad and dst.tolist() == holes + pad and int(err) == 0


@pytest.mark.parametrize("N,used,rows,max_blocks,max_moves", [
    (8192, 0.5, 64, 128, 8192), (8192, 0.5, 64, 129, 5000), (8191, 0.9, 3, 3000, 8191), (8193, 0.5, 64, 128, 8193),
    (40, 0.5, 90, 100, 40), (9000, 0.7, 100, 100, 100), (1024, 1.0, 8, 128, 5), (1025, 0.001, 8, 200, 1025),
])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact_at_the_limits_of_one_cta(cuda, N, used, rows, max_blocks, max_moves, in_place):
    p = Pool(N + rows, N, rows, max_blocks, 16)
    for i in range(min(int(N * used), rows * max_blocks)):
        p.table[i % rows, i // rows] = p.free.pop()
        p.refs[p.table[i % rows, i // rows]] = int(p.rng.integers(3))
    p.table[-1, -1] = p.table[0, 0]  # shared
    p.device()
    err, nm, src, dst = _word(), _word(), _i32([5] * max_moves), _i32([5] * max_moves)
    ws = torch.full((gdn.block_compact_workspace_size(N),), 255, dtype=torch.uint8, device="cuda")
    outs = {} if in_place else dict(table_out=torch.full_like(p.d_table, 3), refs_out=torch.full_like(p.d_refs, 3),
                                    free_out=torch.full_like(p.d_free, 3))
    gdn.block_compact(p.d_table, p.d_refs, p.d_free, p.d_n, src, dst, nm, ws, dev_err=err, **outs)
    if not in_place:
        p.d_table, p.d_refs, p.d_free = outs.values()
    movers, holes = compact(p, max_moves)
    p.check()
    pad = [-1] * (max_moves - len(movers))
    assert int(nm) == len(movers) and src.tolist() == movers + pad and dst.tolist() == holes + pad and int(err) == 0


@pytest.mark.parametrize("wrong,bit", [("twice", binding.DEV_ERR_SLOT_OOB), ("outside", binding.DEV_ERR_SLOT_OOB),
                                       ("count", binding.DEV_ERR_BLOCKS), ("negative", binding.DEV_ERR_BLOCKS)])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact_of_an_inconsistent_stack(cuda, wrong, bit, in_place):
    p = Pool(6, 50, 2, 20, 4)
    p.hold(0, 70)
    p.device()
    n = len(p.free)
    if wrong == "twice":
        p.d_free[1] = p.d_free[0]
    if wrong == "outside":
        p.d_free[n - 1] = 50
    if wrong == "count":
        p.d_n.fill_(51)
    if wrong == "negative":
        p.d_n.fill_(-1)
    old = [t.clone() for t in (p.d_table, p.d_refs, p.d_free)]
    outs = {} if in_place else dict(table_out=torch.full_like(p.d_table, 3), refs_out=torch.full_like(p.d_refs, 3),
                                    free_out=torch.full_like(p.d_free, 3))
    err, nm, src, dst = _word(), _word() + 7, _i32([5] * 30), _i32([5] * 30)
    ws = torch.empty(gdn.block_compact_workspace_size(50), dtype=torch.uint8, device="cuda")
    gdn.block_compact(p.d_table, p.d_refs, p.d_free, p.d_n, src, dst, nm, ws, dev_err=err, **outs)
    now = list(outs.values()) or [p.d_table, p.d_refs, p.d_free]
    assert int(err) == bit and int(nm) == 0 and src.tolist() == [-1] * 30 == dst.tolist()
    assert all(torch.equal(a, b) for a, b in zip(old, now))


@pytest.mark.parametrize("shape,dtype", [((5, 8), torch.float32), ((9, 4, 2, 64), torch.bfloat16),
                                         ((70, 3, 5000), torch.bfloat16), ((4, 70000), torch.uint8)])
@pytest.mark.parametrize("n_planes", [1, 5])
def test_page_copy(cuda, shape, dtype, n_planes):
    g = torch.Generator().manual_seed(shape[0] + n_planes)
    whole = torch.randint(0, 255, (n_planes, *shape), generator=g, dtype=torch.uint8).to(dtype).cuda()
    planes = list(whole)
    ids = torch.randperm(shape[0], generator=g)
    k = shape[0] // 2
    src, dst = ids[:k].clone(), ids[k:2 * k].clone()
    src[-1] = src[0]  # one page to several
    want = whole.clone()
    want[:, dst.cuda()] = whole[:, src.cuda()]
    pad = torch.full((3,), -1)
    err = _word()
    s = torch.cat([pad, src, pad[:1], torch.tensor([0])]).to(torch.int32).cuda()
    d = torch.cat([torch.tensor([0, 1, -1]), dst, torch.tensor([2]), pad[:1]]).to(torch.int32).cuda()
    gdn.page_copy(gdn.PagePlanes(planes), s, d, dev_err=err)
    assert torch.equal(whole, want) and int(err) == 0


def test_page_copy_of_strided_planes_and_bad_ids(cuda):
    """Keys and values of a page side by side; ids outside the pool."""
    kv = torch.arange(6 * 2 * 32, dtype=torch.float32, device="cuda").reshape(6, 2, 32)
    want, err = kv.clone(), _word()
    want[4, 0] = kv[1, 0]
    gdn.page_copy(gdn.PagePlanes([kv[:, 0]]), _i32([1, 6, 0, -2]), _i32([4, 0, 6, 3]), dev_err=err)
    assert torch.equal(kv, want) and int(err) == binding.DEV_ERR_SLOT_OOB


def test_page_copy_of_many_padded_pairs(cuda):
    g = torch.Generator().manual_seed(9)
    x = torch.randn((4000, 64), generator=g).cuda()
    want = x.clone()
    src = torch.full((10000,), -1, dtype=torch.int32)
    dst = src.clone()
    at = torch.randperm(10000, generator=g)[:1500]
    ids = torch.randperm(4000, generator=g)
    src[at], dst[at] = ids[:1500].int(), ids[2000:3500].int()
    want[ids[2000:3500].cuda()] = x[ids[:1500].cuda()]
    gdn.page_copy(gdn.PagePlanes([x]), src.cuda(), dst.cuda())
    assert torch.equal(x, want)
