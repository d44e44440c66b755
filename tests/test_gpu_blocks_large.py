"""Releases of more entries than one cluster walks (two launches): many calls
behind one another, on several streams at once, captured and replayed.  Copies
of pages that lie beyond 2^32 bytes."""
import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from test_gpu_blocks import Pool, _i32, _i64, _word

pytestmark = pytest.mark.gpu
ROWS, BLOCKS_PER_ROW, BLOCK = 300, 40, 16


class Held:
    """A pool whose rows all hold blocks, and what their release leaves."""

    def __init__(self, seed, extra=0):
        p = self.p = Pool(seed, ROWS * BLOCKS_PER_ROW + extra, ROWS, BLOCKS_PER_ROW, BLOCK)
        for r in range(ROWS):
            p.hold(r, int(p.rng.integers(0, BLOCKS_PER_ROW * BLOCK + 1)))
        p.device()
        self.was = [t.clone() for t in (p.d_table, p.d_refs, p.d_free, p.d_n)]
        self.rows, self.old = list(range(ROWS)), list(p.lens)
        self.new = [int(p.rng.integers(0, n + 1)) for n in self.old]
        self.args = _i32(self.rows), _i64(self.old), _i64(self.new)
        self.err = _word()
        p.release(self.rows, self.old, self.new)

    def again(self):
        for t, w in zip((self.p.d_table, self.p.d_refs, self.p.d_free, self.p.d_n), self.was):
            t.copy_(w)
        p = self.p
        gdn.block_release(*self.args, BLOCK, p.d_table, p.d_refs, p.d_free, p.d_n, dev_err=self.err)

    def check(self):
        self.p.check()
        assert int(self.err) == 0


@pytest.mark.parametrize("extra", [0, 1, 40000])
def test_again_and_again(cuda, extra):
    h = Held(extra, extra)
    for _ in range(30):
        h.again()
    h.check()


def test_on_several_streams_and_replayed(cuda):
    held = [Held(seed) for seed in range(4)]
    streams = [torch.cuda.Stream() for _ in held]
    graphs = []
    for h in held:
        h.again()
    torch.cuda.synchronize()
    for h in held:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            h.again()
        graphs.append(g)
    for _ in range(5):
        for h, s, g in zip(held, streams, graphs):
            with torch.cuda.stream(s):
                h.again()
                g.replay()
    torch.cuda.synchronize()
    for h in held:
        h.check()


def test_pages_beyond_32_bits(cuda):
    """Three pages of 6000 bytes and more, 2^31 bytes apart, in two planes."""
    far, page = 2 ** 31 + 4096, 6016
    buf = torch.zeros(2 * far + 2 * page + 64, dtype=torch.uint8, device="cuda")
    planes = [buf[i * page:].as_strided((3, page), (far, 1)) for i in range(2)]
    for i, p in enumerate(planes):
        for j in range(3):
            p[j] = 1 + 3 * i + j
    err = _word()
    gdn.page_copy(gdn.PagePlanes(planes), _i32([2, -1]), _i32([0, 1]), dev_err=err)
    assert int(err) == 0
    for i, p in enumerate(planes):
        assert [sorted(set(p[j].tolist())) for j in range(3)] == [[3 + 3 * i], [2 + 3 * i], [3 + 3 * i]]
