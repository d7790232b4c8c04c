"""The oracles of the page calls and of rotary positions on examples worked by hand; refusals of the
calls on the host (CPU only: nothing here reaches a GPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import pagedattention_kvc_store_gb300 as kvc
from oracle import rope as orope
from oracle.pages import Rows
from pagedattention_kvc_store_gb300.kvc import PageArray, PoolDesc, RopeDesc, lib
from workloads import PageAllocator

FAKE = ctypes.c_void_p(0x10000)      # never dereferenced: checks fail before any launch
FAR = ctypes.c_void_p(0x10000000)
POOL = PoolDesc(32, 16, 2, 64)


def _held(refs, pages, lens, P):
    r = Rows(refs, P)
    r.pages, r.lens = [list(p) for p in pages], list(lens)
    return r


def test_reserve_takes_the_lowest_free_pages_in_row_order():
    refs = np.array([0, 1, 0, 1, 0, 0])
    r = _held(refs, [[1], [3]], [4, 4], 4)
    assert r.reserve([5, 1], 8) == 0
    assert r.pages == [[1, 0, 2], [3, 4]] and r.lens == [9, 5]
    assert refs.tolist() == [1, 1, 1, 1, 1, 0]


def test_reserve_copies_shared_last_pages_but_for_the_last_sharer():
    pool = np.arange(6)
    refs = np.array([3, 0, 0, 0, 0, 0])
    r = _held(refs, [[0], [0], [0]], [3, 3, 3], 4)
    r.pools = [pool]
    assert r.reserve([1, 1, 1], 8) == 0
    assert r.pages == [[1], [2], [0]] and refs.tolist() == [1, 1, 1, 0, 0, 0]
    assert pool.tolist() == [0, 0, 0, 3, 4, 5]
    # held by somebody else too: all copy
    refs = np.array([3, 0, 0, 0])
    r = _held(refs, [[0], [0]], [3, 3], 4)
    assert r.reserve([1, 1], 8) == 0 and r.pages == [[1], [2]] and refs.tolist() == [1, 1, 1, 0]


def test_reserve_says_how_many_are_missing_and_changes_nothing():
    refs = np.array([2, 0, 0])
    r = _held(refs, [[0], [0]], [2, 2], 4)
    assert r.reserve([8, 1], 8) == 1     # a copy, two more pages; the second row keeps page 0
    assert r.pages == [[0], [0]] and r.lens == [2, 2] and refs.tolist() == [2, 0, 0]


def test_the_oracle_goes_as_the_host_allocator_does():
    """Random forks and growth: as many pages as the repository's host allocator uses, shared alike."""
    rng = np.random.default_rng(3)
    P, refs = 4, np.zeros(200, dtype=np.int64)
    host, rows = PageAllocator(200, P, range(200)), Rows(refs, P)
    lens = rng.integers(0, 30, 5)
    for s, n in enumerate(lens):
        host.reserve(s, int(n))
    rows.pages, rows.lens = [[] for _ in lens], [0] * 5
    assert rows.reserve(lens, 50) == 0
    for i, p in enumerate([0, 0, 3, 4, 4]):
        host.fork(5 + i, p)
    forks = rows.new_rows([0, 0, 3, 4, 4])
    grow = [3, 0, 1, 9, 2]
    for i, n in enumerate(grow):
        host.reserve(5 + i, n)
    assert forks.reserve(grow, 50) == 0
    both = rows.pages + forks.pages
    assert [len(p) for p in both] == [len(host.pages[s]) for s in range(10)]
    assert sorted(refs[refs > 0].tolist()) == sorted(host.refcount[host.refcount > 0].tolist())
    for a in range(10):
        for b in range(10):   # the same pages shared, whatever their ids
            assert [x == y for x, y in zip(both[a], both[b])] == \
                [x == y for x, y in zip(host.pages[a], host.pages[b])]


def test_compact_moves_the_upper_pages_into_the_holes():
    pool = np.arange(8) * 10
    refs = np.array([0, 2, 0, 1, 0, 0, 1, 1])
    r = _held(refs, [[7, 1, 3], [6, 1]], [12, 8], 4)
    r.pools = [pool]
    where, live = r.compact()
    assert live == 4 and where == [-1, 1, -1, 3, -1, -1, 0, 2]
    assert r.pages == [[2, 1, 3], [0, 1]] and refs.tolist() == [1, 2, 1, 1, 0, 0, 0, 0]
    assert pool.tolist() == [60, 10, 70, 30, 40, 50, 60, 70]


def test_rope_oracle_by_hand():
    x = np.zeros((2, 1, 64))
    x[:, 0, 0], x[:, 0, 1], x[:, 0, 2] = 1.0, 2.0, 3.0
    pos = np.array([[0, 1], [0, 3]])
    y = orope.rotate(x, pos, [math.pi / 2, math.pi / 3], [0, 1], adjacent=True)
    assert np.allclose(y[0], x[0])
    want = [-2.0, 1.0, -3.0, 0.0]      # a quarter turn of (1, 2), a half turn of (3, 0)
    assert np.allclose(y[1, 0, :4], want, atol=1e-12) and np.array_equal(y[1, 0, 4:], x[1, 0, 4:])
    z = orope.rotate(x, pos, [math.pi / 2, 0.0], [0, 0], adjacent=False)
    assert np.allclose(z[1, 0, :3], [-3.0, 2.0, 1.0], atol=1e-12)


def _rope(**changed):
    d = kvc.rope_desc([1.0] * 16, [0] * 8 + [1] * 8)
    for k, v in changed.items():
        setattr(d, k, v)
    return d


def _call_rope(rope, q_out=FAR, k_out=ctypes.c_void_p(0x20000000), q=FAKE, k=ctypes.c_void_p(0x30000000),
               q_stride=256, k_stride=128, q_out_stride=256, k_out_stride=128, T=3, positions=FAKE,
               D=64, heads=(4, 2)):
    return lib().kvc_rope(q_out, q_out_stride, k_out, k_out_stride, q, q_stride, k, k_stride, heads[0],
                          heads[1], D, rope, positions, T, None)


@pytest.mark.parametrize("change,status", [
    (dict(num_axes=0), 1), (dict(num_axes=9), 1), (dict(num_axes=1), 1),     # axis 1 of one
    (dict(rotary_dim=0), 1), (dict(rotary_dim=80), 1), (dict(rotary_dim=24), 2), (dict(pairing=2), 1),
])
def test_rope_descriptions_are_checked(change, status):
    assert _call_rope(_rope(**change)) == status and lib().kvc_last_error()


@pytest.mark.parametrize("bad", [math.nan, math.inf, 1e7])
def test_rope_frequencies_are_checked(bad):
    assert _call_rope(kvc.rope_desc([1.0] * 15 + [bad], [0] * 8 + [1] * 8)) == 1
    empty = RopeDesc(1, 32, 0, None, None)
    assert _call_rope(empty) == 1


@pytest.mark.parametrize("change,status", [
    (dict(D=96), 2), (dict(T=-1), 1), (dict(heads=(-1, 2)), 1), (dict(positions=None), 1),
    (dict(q=None), 1), (dict(q_stride=248), 1), (dict(q_stride=100), 1), (dict(q_out_stride=-8), 1),
    (dict(k=ctypes.c_void_p(0x30000008)), 1),
    (dict(q_out=FAKE, q_out_stride=264), 1),                     # q itself with another stride
    (dict(q_out=ctypes.c_void_p(0x10000 + 512)), 1),             # q's next token
    (dict(q_out=ctypes.c_void_p(0x30000000)), 1),                # over k
    (dict(k_out=FAR), 1),                                        # over q_out
])
def test_rope_rows_are_checked(change, status):
    assert _call_rope(_rope(), **change) == status and lib().kvc_last_error()


def test_rope_calls_with_nothing_to_do():
    assert _call_rope(_rope(), T=0) == 0
    assert _call_rope(_rope(), heads=(0, 0)) == 0
    assert lib().kvc_rope_store(None, FAKE, FAKE, POOL, None, 0, FAKE, 128, FAKE, 128, 0, _rope(), FAKE,
                                FAKE, 0, None) == 0


@pytest.mark.parametrize("pool,status", [(PoolDesc(32, 16, 2, 96), 2), (PoolDesc(32, 8, 2, 64), 2),
                                         (PoolDesc(32, 16, 2, 64, 5), 1)])
def test_rope_store_checks_its_pool(pool, status):
    assert lib().kvc_rope_store(FAR, FAKE, FAKE, pool, FAKE, 256, FAKE, 128, FAKE, 128, 4, _rope(), FAKE,
                                FAKE, 3, None) == status


def test_rope_store_checks_its_rows():
    def call(q_out=FAR, k_pool=FAKE, q=FAKE, q_stride=256, k=FAKE, v=FAKE, slots=FAKE):
        return lib().kvc_rope_store(q_out, k_pool, FAKE, POOL, q, q_stride, k, 128, v, 128, 4, _rope(),
                                    FAKE, slots, 3, None)
    assert call(k_pool=None) == 1 and call(q=None) == 1 and call(v=None) == 1 and call(slots=None) == 1
    assert call(k_pool=ctypes.c_void_p(0x10004)) == 1
    assert call(q_out=FAKE, q_stride=264) == 1     # in place, but q's rows are not contiguous
    assert call(q_out=ctypes.c_void_p(0x40000000), q=ctypes.c_void_p(0x40000100)) == 1


def _pages(call, **change):
    a = dict(table=FAKE, stride=8, lens=FAKE, seqs=4, refs=FAKE, pages=100, P=16)
    a.update(change)
    ws = ctypes.c_void_p(0x50000000)
    arrays = (PageArray * 1)(PageArray(0x10000, 64))
    n = 1
    if "arrays" in change:
        arrays, n = change["arrays"]
    if call == "truncate":
        return lib().kvc_truncate(a["table"], a["stride"], a["lens"], None, a["seqs"], a["refs"],
                                  a["pages"], a["P"], None)
    if call == "fork":
        return lib().kvc_fork(a.get("out", FAR), a.get("out_stride", 8), a.get("out_lens",
                              ctypes.c_void_p(0x20000000)), a.get("parents", FAKE), None,
                              a.get("num_out", 4), a["table"], a["stride"], a["lens"], a["seqs"],
                              a["refs"], a["pages"], a["P"], None)
    if call == "reserve":
        return lib().kvc_reserve(arrays, n, a["table"], a["stride"], a["lens"], a.get("grow"),
                                 a["seqs"], a["refs"], a["pages"], a["P"], a.get("missing", FAKE),
                                 a.get("ws", ws), a.get("ws_bytes", 1 << 20), None)
    return lib().kvc_compact(arrays, n, a["table"], a["stride"], a["lens"], a["seqs"], a["refs"],
                             a["pages"], a["P"], a.get("map", FAR), a.get("live", FAKE),
                             a.get("ws", ws), a.get("ws_bytes", 1 << 20), None)


@pytest.mark.parametrize("call", ["truncate", "fork", "reserve", "compact"])
@pytest.mark.parametrize("change,status", [
    (dict(pages=0), 1), (dict(P=0), 1), (dict(stride=0), 1), (dict(seqs=-1), 1), (dict(seqs=65536), 1),
    (dict(refs=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(pages=1 << 28), 2),
    (dict(stride=(1 << 26) + 1), 2),
])
def test_page_calls_check_their_table(call, change, status):
    assert _pages(call, **change) == status and lib().kvc_last_error()


@pytest.mark.parametrize("change", [dict(out=None), dict(out_lens=None), dict(parents=None),
                                    dict(out_stride=0), dict(num_out=65536), dict(out=FAKE),
                                    dict(out_lens=FAKE)])
def test_fork_checks_its_new_rows(change):
    assert _pages("fork", **change) == 1


@pytest.mark.parametrize("call", ["reserve", "compact"])
@pytest.mark.parametrize("change,status", [
    (dict(ws=None), 3), (dict(ws_bytes=100), 3), (dict(ws=ctypes.c_void_p(0x50000004)), 1),
    (dict(arrays=(None, 1)), 1), (dict(arrays=(None, -1)), 1),
    (dict(arrays=((PageArray * 1)(PageArray(0x10004, 64)), 1)), 1),
    (dict(arrays=((PageArray * 1)(PageArray(0x10000, 24)), 1)), 2),
    (dict(arrays=((PageArray * 1)(PageArray(0x10000, 0)), 1)), 2),
])
def test_reserve_and_compact_check_arrays_and_workspace(call, change, status):
    assert _pages(call, **change) == status


def test_outputs_of_reserve_and_compact_are_checked():
    assert _pages("reserve", missing=None) == 1 and _pages("reserve", grow=FAKE) == 1
    assert _pages("compact", map=None) == 1 and _pages("compact", live=None) == 1
    assert _pages("compact", map=FAKE) == 1
    with pytest.raises(kvc.KvcError):
        kvc.kvc_reserve_plan(70000, 10)
    with pytest.raises(kvc.KvcError):
        kvc.kvc_compact_plan(0)
    assert kvc.kvc_reserve_plan(0, 1) > 0 and kvc.kvc_compact_plan(1) > 0


CROSS_POOL = PoolDesc(2000, 16, 8, 128)


def _cross(pool=CROSS_POOL, out=FAKE, dtype=0, lse=None, q=FAKE, table=FAKE, stride=256, indptr=FAKE, lens=FAKE,
           S=4, T=8, most=2, src=4096, heads=32, splits=0, ws=None, ws_bytes=0):
    return lib().kvc_cross(out, dtype, lse, q, FAKE, FAKE, pool, table, stride, indptr, lens, S, T, most, src,
                           heads, 0.0, splits, ws, ws_bytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(pool=PoolDesc(32, 16, 2, 96)), 2), (dict(pool=PoolDesc(32, 8, 2, 64)), 2), (dict(heads=31), 1),
    (dict(heads=128), 2), (dict(S=-1), 1), (dict(S=65536), 1), (dict(T=-1), 1), (dict(most=-1), 1),
    (dict(src=-1), 1), (dict(splits=-1), 1), (dict(stride=10), 1), (dict(dtype=2), 1), (dict(out=None), 1),
    (dict(q=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(indptr=None), 1),
    (dict(lse=ctypes.c_void_p(0x10002)), 1), (dict(out=ctypes.c_void_p(0x10008)), 1),
    (dict(), 3), (dict(ws=FAKE, ws_bytes=16), 3), (dict(T=1 << 24), 2), (dict(most=1 << 29), 2),
])
def test_cross_checks_its_arguments(change, status):
    assert _cross(**change) == status and lib().kvc_last_error()


def test_cross_calls_with_nothing_to_do_and_their_plan():
    assert _cross(T=0) == 0 and _cross(S=0) == 0 and _cross(most=0) == 0
    for most in (1, 8, 9, 400):
        for n in (0, 1, 3, 50):
            splits, chunk, ws = kvc.kvc_cross_plan(4, 4 * most, 32, CROSS_POOL, most, 4096, n)
            assert splits * chunk >= 4096 > (splits - 1) * chunk and chunk % 64 == 0
            rows = 4 * most * 32
            assert ws == (0 if splits == 1 else -(-rows * splits * 128 * 4 // 256) * 256 + rows * splits * 4)
            assert n == 0 or splits <= n
    assert kvc.kvc_cross_plan(4, 4, 32, CROSS_POOL, 1, 0)[0] == 1


def test_bindings_refuse_cpu_tensors_and_odd_descriptions():
    t = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    rope = kvc.rope_desc([1.0] * 32)
    assert (rope.num_axes, rope.rotary_dim) == (1, 64)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.kvc_rope(t, None, t, None, i, rope)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.kvc_truncate(i.view(4, 1), i, None, i, 16)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.page_arrays([t])
    with pytest.raises(ValueError):
        kvc.rope_desc([1.0] * 8, [0] * 7)
    with pytest.raises(ValueError):
        kvc.rope_desc([1.0] * 8, pairing="thirds")
