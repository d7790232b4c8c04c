"""kvc_truncate, kvc_fork, kvc_reserve and kvc_compact on the GPU: whole numbers and raw copies, equal to
an allocator on the host that goes row after row."""
import numpy as np
import pytest
import torch

import pagedattention_kvc_store_gb300 as kvc
from oracle.pages import Rows
from workloads.device import i32_tensor

pytestmark = pytest.mark.gpu


class Device:
    """Tables, references and pools on the GPU beside the oracle's."""

    def __init__(self, pages, P, width, arrays=((64,), (2, 8)), seed=0):
        self.P, self.width, self.n = P, width, pages
        rng = np.random.default_rng(seed)
        pools = [rng.integers(0, 256, size=(pages, *shape), dtype=np.uint8) for shape in arrays]
        self.refs_h = np.zeros(pages, dtype=np.int64)
        self.pools_h = pools
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.pools = [torch.from_numpy(p).cuda() for p in pools]
        self.arrays = kvc.page_arrays(self.pools)
        self.missing = torch.full((1,), -7, dtype=torch.int32, device="cuda")

    def empty(self, rows, width=None):
        h = Rows(self.refs_h, self.P, self.pools_h)
        h.pages, h.lens = [[] for _ in range(rows)], [0] * rows
        w = self.width if width is None else width
        return h, torch.zeros(rows, w, dtype=torch.int32, device="cuda"), \
            torch.zeros(rows, dtype=torch.int32, device="cuda")

    def reserve(self, t, grow):
        h, table, lens = t
        ws = torch.empty(kvc.kvc_reserve_plan(len(h.lens), self.n), dtype=torch.uint8, device="cuda")
        ws.fill_(0xA5)
        g = None if grow is None else i32_tensor(np.array(grow), "cuda")
        kvc.kvc_reserve(table, lens, g, self.refs, self.missing, self.P, self.arrays, workspace=ws)
        short = h.reserve([1] * len(h.lens) if grow is None else grow, table.shape[1])
        assert self.missing.item() == short
        self.same(t)
        return short

    def fork(self, t, parents, share=None, width=None):
        h, table, lens = t
        new = self.empty(len(parents), width)
        s = None if share is None else i32_tensor(np.array(share), "cuda")
        kvc.kvc_fork(new[1], new[2], i32_tensor(np.array(parents), "cuda"), table, lens, self.refs,
                     self.P, share_lens=s)
        new = (h.new_rows(parents, share), new[1], new[2])
        self.same(new)
        return new

    def truncate(self, t, new_lens):
        h, table, lens = t
        g = None if new_lens is None else i32_tensor(np.array(new_lens), "cuda")
        kvc.kvc_truncate(table, lens, g, self.refs, self.P)
        h.truncate(new_lens)
        self.same(t)

    def compact(self, t, others=()):
        h, table, lens = t
        ws = torch.full((kvc.kvc_compact_plan(self.n),), 0xA5, dtype=torch.uint8, device="cuda")
        where = torch.full((self.n,), -9, dtype=torch.int32, device="cuda")
        live = torch.full((1,), -9, dtype=torch.int32, device="cuda")
        kvc.kvc_compact(table, lens, self.refs, where, live, self.P, self.arrays, workspace=ws)
        to, n = h.compact()
        assert live.item() == n and where.tolist() == to
        for o, o_table, o_lens in others:      # tables that the call was not given follow the map
            o.pages = [[to[p] for p in row] for row in o.pages]
            o_table.copy_(where[o_table.long()].clamp(min=0))
        self.same(t)

    def same(self, t):
        h, table, lens = t
        assert lens.tolist() == list(h.lens)
        for row, pages in zip(table.tolist(), h.pages):
            assert row[:len(pages)] == pages
        assert self.refs.tolist() == self.refs_h.tolist()
        for a, b in zip(self.pools, self.pools_h):
            assert np.array_equal(a.cpu().numpy(), b)
        assert kvc.kvc_device_errors() == 0


@pytest.mark.parametrize("pages,P,rows", [(40, 4, 3), (700, 16, 20), (9000, 16, 60), (5000, 3, 40)])
def test_a_run_of_all_calls(pages, P, rows):
    rng = np.random.default_rng(pages)
    d = Device(pages, P, width=64)
    t = d.empty(rows)
    most = max(1, min(20 * P, pages * P // (3 * rows)))
    assert d.reserve(t, rng.integers(0, most, rows)) == 0
    for turn in range(4):
        parents = rng.integers(-1, rows, size=rows + 3)
        share = None if turn % 2 else rng.integers(0, most, size=rows + 3)
        new = d.fork(t, parents, share, width=80)
        d.reserve(new, None if turn == 1 else rng.integers(-1, 2 * P, rows + 3))
        if turn == 2:
            d.compact(new, others=[t])
        d.truncate(t, None if turn == 3 else rng.integers(0, most, rows))
        if turn % 2:
            d.compact(t, others=[new])
        d.truncate(new, None)
        d.reserve(t, rng.integers(0, P + 2, rows))
    d.truncate(t, None)
    assert int(d.refs.sum()) == 0


def test_sharers_of_one_page():
    """Beams of one sequence grow: the last keeps the page once nobody else holds it."""
    d = Device(50, 4, width=8)
    t = d.empty(1)
    d.reserve(t, [6])
    beams = d.fork(t, [0, 0, 0, 0])
    d.reserve(beams, [1, 0, 1, 1])             # t and beam 1 hold the page: all three copy
    assert len({p[1] for p in beams[0].pages}) == 4
    d.truncate(t, None)
    d.truncate(beams, [0, 6, 0, 0])
    again = d.fork(beams, [1, 1, 1])
    d.truncate(beams, None)
    d.reserve(again, None)                     # nobody else: the last of the three keeps it
    assert again[0].pages[2][1] == 1 and again[0].pages[0][1] != 1


def test_a_shortage_changes_nothing():
    d = Device(10, 4, width=16)
    t = d.empty(3)
    assert d.reserve(t, [13, 10, 5]) == 0
    assert d.reserve(t, [9, 12, 0]) == 4      # five pages wanted, one free
    assert d.reserve(t, [3, 2, 0]) == 0


def test_more_rows_than_a_block_and_more_pages_than_a_segment():
    rng = np.random.default_rng(0)
    d = Device(20000, 16, width=16, arrays=((16,),))
    t = d.empty(2500)
    assert d.reserve(t, rng.integers(0, 100, 2500)) == 0
    new = d.fork(t, rng.integers(-1, 2500, 1100))
    assert d.reserve(new, None) == 0
    d.truncate(t, np.where(rng.random(2500) < 0.6, 0, 200))
    d.compact(new, others=[t])
    d.reserve(new, rng.integers(0, 40, 1100))


def test_most_of_a_pool_at_once():
    """More new pages than one block lists at a time, in the largest pool that one block takes and the next."""
    for pages in (16384, 16385):
        d = Device(pages, 2, width=96, arrays=((16,),))
        t = d.empty(200)
        assert d.reserve(t, np.full(200, 140)) == 0
        assert d.reserve(t, np.full(200, 40)) == 200 * 20 - (pages - 14000)
        d.truncate(t, np.arange(200) % 3)
        d.compact(t)


def test_more_arrays_than_a_launch_takes():
    d = Device(30, 4, width=8, arrays=[(16 * (1 + i % 3),) for i in range(131)] + [(40000,)])
    t = d.empty(3)
    d.reserve(t, [7, 5, 9])
    new = d.fork(t, [2, 0, 0])
    d.reserve(new, None)
    d.truncate(t, None)
    d.compact(new)


@pytest.mark.parametrize("pages,page_bytes", [(60, 400000), (60, 48), (17000, 48)])
def test_large_and_small_copies(pages, page_bytes):
    """Copies that are left to the deciding launch, that have one of their own, and a pool past one block's."""
    rng = np.random.default_rng(pages)
    d = Device(pages, 4, width=8, arrays=((page_bytes,), (16,)))
    t = d.empty(12)
    d.reserve(t, rng.integers(1, 10, 12))
    new = d.fork(t, rng.integers(0, 12, 12))
    d.reserve(new, rng.integers(0, 4, 12))
    d.truncate(t, None)
    d.compact(new)
    d.reserve(new, None)


@pytest.mark.parametrize("rows", [1023, 1024, 1025])
def test_row_counts_about_a_block(rows):
    d = Device(4000, 2, width=4, arrays=((16,),))
    t = d.empty(rows)
    d.reserve(t, np.arange(rows) % 4)
    new = d.fork(t, np.arange(rows) // 2)
    d.truncate(t, np.zeros(rows, dtype=np.int64))
    d.reserve(new, None)


def test_no_arrays_and_no_rows():
    d = Device(12, 16, width=4)
    d.arrays = None
    t = d.empty(2)
    d.pools_h.clear(), d.pools.clear()
    d.reserve(t, [20, 33])
    none = d.empty(0)
    d.reserve(none, [])
    d.truncate(none, None)
    d.truncate(t, [1, 40])
    d.compact(t)


def test_bad_contents_are_flagged():
    d = Device(8, 4, width=4)
    t = d.empty(2)
    d.reserve(t, [5, 5])
    h, table, lens = t
    # a row that has no room stays as it is
    g = torch.tensor([12, 1], dtype=torch.int32, device="cuda")
    ws = torch.empty(kvc.kvc_reserve_plan(2, 8), dtype=torch.uint8, device="cuda")
    kvc.kvc_reserve(table, lens, g, d.refs, d.missing, 4, workspace=ws)
    assert kvc.kvc_device_errors() == 1 << 7 and lens.tolist() == [5, 6]
    # parents past the table are empty rows; the others are right
    out, out_lens = torch.zeros(2, 4, dtype=torch.int32, device="cuda"), torch.zeros_like(lens)
    kvc.kvc_fork(out, out_lens, torch.tensor([2, 1], dtype=torch.int32, device="cuda"), table, lens,
                 d.refs, 4)
    assert kvc.kvc_device_errors() == 1 << 15 and out_lens.tolist() == [0, 6]
    # a new row that is too short is cut
    short, short_lens = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros_like(lens[:1])
    kvc.kvc_fork(short, short_lens, torch.tensor([0], dtype=torch.int32, device="cuda"), table, lens,
                 d.refs, 4)
    assert kvc.kvc_device_errors() == 1 << 7 and short_lens.tolist() == [4]
    refs = d.refs.clone()
    # a page outside the pool: the rest of the row is given back
    table[0, 1] = 99
    kvc.kvc_truncate(table, lens, torch.tensor([0, 6], dtype=torch.int32, device="cuda"), d.refs, 4)
    assert kvc.kvc_device_errors() == 1 << 10
    assert lens.tolist() == [0, 6] and d.refs[0].item() == refs[0].item() - 1
    # a page given back once too often is flagged and stays at nothing
    free = torch.nonzero(d.refs == 0)[0].item()
    table[0, 0] = free
    lens[0] = 3
    kvc.kvc_truncate(table, lens, torch.tensor([0, 6], dtype=torch.int32, device="cuda"), d.refs, 4)
    assert kvc.kvc_device_errors() == 1 << 14 and d.refs[free].item() == 0


def test_a_captured_step_grows_and_branches():
    """A beam step (branches let go, forked again, grown) captured once and replayed."""
    d = Device(400, 4, width=32, arrays=((32,),))
    t = d.empty(6)
    d.reserve(t, [9, 30, 4, 17, 1, 12])
    h, table, lens = t
    beams = d.empty(12)
    _, b_table, b_lens = beams
    parents = i32_tensor(np.arange(12) // 2, "cuda")
    grow = i32_tensor(np.ones(12), "cuda")
    ws = torch.empty(kvc.kvc_reserve_plan(12, 400), dtype=torch.uint8, device="cuda")

    def step():
        kvc.kvc_truncate(b_table, b_lens, None, d.refs, 4)
        kvc.kvc_fork(b_table, b_lens, parents, table, lens, d.refs, 4)
        kvc.kvc_reserve(b_table, b_lens, grow, d.refs, d.missing, 4, d.arrays, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng = np.random.default_rng(1)
    b = beams[0]
    for turn in range(3):
        p, g = rng.integers(0, 6, 12), rng.integers(0, 9, 12)
        parents.copy_(i32_tensor(p, "cuda"))
        grow.copy_(i32_tensor(g, "cuda"))
        graph.replay()
        b.truncate(None)
        b = h.new_rows(p)
        assert b.reserve(g, 32) == 0 == d.missing.item()
        d.same((b, b_table, b_lens))
