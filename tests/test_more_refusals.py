"""Refusals of the rotation, block and page calls, without a GPU."""
import ctypes
import math

import pytest
import torch

import hybrid_linear_attention_gdn_gb300 as gdn
from hybrid_linear_attention_gdn_gb300 import _build, binding
from hybrid_linear_attention_gdn_gb300.binding import ERR_INVALID_ARG, ERR_UNSUPPORTED, OK, CPages, CRows


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gdn.load()


ROWS, PAGES, NONE, NO_PAGES = CRows(0x1000, 512, 64), CPages(0x2000, 4096, 256, 64), CRows(None, 0, 0), CPages(None, 0, 0, 0)


def _rope(lib, act=1, hq=8, hk=4, d=64, hv=4, dv=64, n=3, q=ROWS, k=ROWS, v=ROWS, qw=0x100, kw=0x200, eps=1e-6, cs=0x300,
          mp=10, rot=64, inter=0, pos=0x400, qo=ROWS, ko=NONE, kc=PAGES, vc=PAGES, pages=5, block=16, slots=0x500):
    return lib.gdn_qk_norm_rope(act, hq, hk, d, hv, dv, n, q, k, v, qw, kw, eps, cs, mp, rot, inter, pos, qo, ko, kc, vc,
                                pages, block, slots, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(act=2), ERR_INVALID_ARG),
    (dict(hq=-1), ERR_INVALID_ARG),
    (dict(hq=0, hk=0), ERR_INVALID_ARG),
    (dict(d=0), ERR_INVALID_ARG),
    (dict(d=1026, rot=64), ERR_UNSUPPORTED),
    (dict(dv=1025), ERR_UNSUPPORTED),
    (dict(dv=0), ERR_INVALID_ARG),
    (dict(n=-1), ERR_INVALID_ARG),
    (dict(n=1 << 31), ERR_UNSUPPORTED),
    (dict(q=NONE), ERR_INVALID_ARG),
    (dict(qo=NONE), ERR_INVALID_ARG),
    (dict(k=NONE), ERR_INVALID_ARG),
    (dict(v=NONE), ERR_INVALID_ARG),
    (dict(kc=NO_PAGES), ERR_INVALID_ARG),
    (dict(vc=NO_PAGES), ERR_INVALID_ARG),
    (dict(slots=None), ERR_INVALID_ARG),            # neither k_out nor a cache
    (dict(q=CRows(0x1001, 512, 64)), ERR_INVALID_ARG),
    (dict(q=CRows(0x1000, -512, 64)), ERR_INVALID_ARG),
    (dict(kc=CPages(0x2000, 4096, -1, 64)), ERR_INVALID_ARG),
    (dict(eps=-1e-6), ERR_INVALID_ARG),
    (dict(eps=math.nan), ERR_INVALID_ARG),
    (dict(cs=None), ERR_INVALID_ARG),
    (dict(cs=0x302), ERR_INVALID_ARG),
    (dict(pos=None), ERR_INVALID_ARG),
    (dict(rot=63), ERR_INVALID_ARG),
    (dict(rot=66), ERR_INVALID_ARG),
    (dict(rot=-2), ERR_INVALID_ARG),
    (dict(mp=-1), ERR_INVALID_ARG),
    (dict(inter=2), ERR_UNSUPPORTED),
    (dict(block=0), ERR_INVALID_ARG),
    (dict(block=12), ERR_INVALID_ARG),
    (dict(pages=-1), ERR_INVALID_ARG),
    (dict(n=0, q=NONE, pos=None), OK),
])
def test_rope_refusals(lib, kw, status):
    n0 = lib.gdn_launch_count(binding.K_QK_NORM_ROPE)
    assert _rope(lib, **kw) == status
    assert lib.gdn_launch_count(binding.K_QK_NORM_ROPE) == n0


def _fork(lib, src=0x100, dst=0x200, lens=0x300, n=2, block=16, table=0x400, rows=8, mb=4, refs=0x500, nb=32, free=0x600,
          cap=32, nf=0x700, nfo=0x700, cs=0x800, cd=0x900):
    return lib.gdn_block_fork(src, dst, lens, n, block, table, rows, mb, refs, nb, free, cap, nf, nfo, cs, cd, None, None)


def _release(lib, rows=0x100, old=0x200, new=0x300, n=2, block=16, table=0x400, nr=8, mb=4, refs=0x500, nb=32, free=0x600,
             cap=32, nf=0x700, nfo=0x700):
    return lib.gdn_block_release(rows, old, new, n, block, table, nr, mb, refs, nb, free, cap, nf, nfo, None, None)


@pytest.mark.parametrize("kw", [dict(n=-1), dict(block=0), dict(block=24), dict(mb=-1), dict(nb=-1), dict(cap=-1),
                                dict(nf=None), dict(nfo=None), dict(free=None), dict(table=None), dict(refs=None)])
def test_fork_and_release_refusals(lib, kw):
    n0 = [lib.gdn_launch_count(k) for k in (binding.K_BLOCK_FORK, binding.K_BLOCK_RELEASE)]
    assert _fork(lib, **kw) == ERR_INVALID_ARG and _release(lib, **kw) == ERR_INVALID_ARG
    for more in (dict(src=None), dict(dst=None), dict(lens=None), dict(cs=None), dict(cd=None), dict(rows=-1)):
        assert _fork(lib, **more) == ERR_INVALID_ARG
    for more in (dict(rows=None), dict(old=None), dict(new=None), dict(nr=-1)):
        assert _release(lib, **more) == ERR_INVALID_ARG
    assert [lib.gdn_launch_count(k) for k in (binding.K_BLOCK_FORK, binding.K_BLOCK_RELEASE)] == n0


def _compact(lib, t=0x100, to=0x100, n=8, refs=0x200, ro=0x200, nb=32, free=0x300, fo=0x300, cap=32, nf=0x400, ms=0x500,
             md=0x600, mm=4, nm=0x700, ws=0x1000, wsb=1 << 20):
    return lib.gdn_block_compact(t, to, n, refs, ro, nb, free, fo, cap, nf, ms, md, mm, nm, ws, wsb, None, None)


@pytest.mark.parametrize("kw", [dict(n=-1), dict(nb=-1), dict(cap=-1), dict(mm=-1), dict(t=None), dict(to=None),
                                dict(refs=None), dict(ro=None), dict(free=None), dict(fo=None), dict(nf=None),
                                dict(nm=None), dict(ms=None), dict(md=None), dict(ws=None), dict(ws=0x1010), dict(wsb=100)])
def test_compact_refusals(lib, kw):
    n0 = lib.gdn_launch_count(binding.K_BLOCK_COMPACT)
    assert _compact(lib, **kw) == ERR_INVALID_ARG
    assert lib.gdn_launch_count(binding.K_BLOCK_COMPACT) == n0


def test_compact_workspace_size(lib):
    size = lib.gdn_block_compact_workspace_size
    assert size(0) >= 16 and size(-5) >= 16
    for n in (1, 31, 33, 100000):
        assert size(n) >= 4 * n + 4 * ((n + 31) // 32) + 4 and size(n) % 256 == 0


def _copy(lib, planes=0x100, np_=2, pb=1024, ps=1024, n_pages=8, src=0x200, dst=0x300, n=4):
    return lib.gdn_page_copy(planes, np_, pb, ps, n_pages, src, dst, n, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(np_=-1), ERR_INVALID_ARG), (dict(n=-1), ERR_INVALID_ARG), (dict(n_pages=-1), ERR_INVALID_ARG),
    (dict(pb=0), ERR_INVALID_ARG), (dict(ps=512), ERR_INVALID_ARG), (dict(pb=1000), ERR_UNSUPPORTED),
    (dict(ps=1032), ERR_UNSUPPORTED), (dict(planes=None), ERR_INVALID_ARG), (dict(src=None), ERR_INVALID_ARG),
    (dict(dst=None), ERR_INVALID_ARG), (dict(n=0, src=None), OK), (dict(np_=0, planes=None), OK),
])
def test_page_copy_refusals(lib, kw, status):
    n0 = lib.gdn_launch_count(binding.K_PAGE_COPY)
    assert _copy(lib, **kw) == status
    assert lib.gdn_launch_count(binding.K_PAGE_COPY) == n0


def test_planes_on_the_host_are_refused(lib):
    with pytest.raises(gdn.GdnError):
        gdn.PagePlanes([])
    with pytest.raises(gdn.GdnError):
        gdn.PagePlanes([torch.zeros(4, 64)])


def test_tensors_on_the_host_are_refused(lib):
    i32, i64 = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    one, table = torch.zeros(1, dtype=torch.int32), torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(gdn.GdnError):
        gdn.block_fork(i32, i32, i64, 16, table, i32, i32, one, i32, i32)
    with pytest.raises(gdn.GdnError):
        gdn.block_release(i32, i64, i64, 16, table, i32, i32, one)
    with pytest.raises(gdn.GdnError):
        gdn.block_compact(table, i32, i32, one, i32, i32, one, torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(gdn.GdnError):
        gdn.qk_norm_rope(torch.zeros(2, 1, 8), None, None, None, torch.zeros(4, 8), i64)
