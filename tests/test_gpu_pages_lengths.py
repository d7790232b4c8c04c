"""Lengths that are no lengths in the page calls: a negative one counts as none, whichever kernels make the
decision (up to 1,024 rows and 16,384 pages one block, several past either)."""
import numpy as np
import pytest
import torch

import pagedattention_kvc_store_gb300 as kvc
from test_gpu_pages import Device
from workloads.device import i32_tensor

pytestmark = pytest.mark.gpu

NEGATIVE = [-1, -15, -16, -17, -100, -2 ** 31]
SIZES = [(4000, 60), (20000, 60), (4000, 1100), (20000, 1100)]   # pages, rows


def grown(pages, rows):
    """A table in which every seventh row is empty, by a negative length."""
    d = Device(pages, 16, width=8, arrays=((16,),))
    t = d.empty(rows)
    t[1].fill_(-5)
    d.reserve(t, np.where(np.arange(rows) % 7 == 3, 0, 5 + np.arange(rows) % 30))
    bad = np.flatnonzero(np.arange(rows) % 7 == 3)
    t[2][torch.from_numpy(bad).cuda()] = i32_tensor(np.resize(NEGATIVE, len(bad)), "cuda")
    return d, t, bad


def unused_entries_are_untouched(t):
    for row, pages in zip(t[1].tolist(), t[0].pages):
        assert all(x == -5 for x in row[len(pages):])


@pytest.mark.parametrize("pages,rows", SIZES)
def test_a_negative_length_grows_from_none(pages, rows):
    d, t, bad = grown(pages, rows)
    grow = 1 + np.arange(rows) % 40
    assert d.reserve(t, grow) == 0
    unused_entries_are_untouched(t)


@pytest.mark.parametrize("pages,rows", SIZES)
def test_a_negative_length_that_does_not_grow_needs_no_page(pages, rows):
    d, t, bad = grown(pages, rows)
    h, table, lens = t
    lens_before = lens.clone()
    grow = np.where(np.isin(np.arange(rows), bad), -(np.arange(rows) % 2), 1)
    neg = lens < 0
    # the oracle's rows hold 0 positions there, the device's lengths are still negative
    ws = torch.empty(kvc.kvc_reserve_plan(rows, pages), dtype=torch.uint8, device="cuda")
    kvc.kvc_reserve(table, lens, i32_tensor(grow, "cuda"), d.refs, d.missing, 16, d.arrays, workspace=ws)
    assert h.reserve(grow, 8) == 0 == d.missing.item()
    assert torch.equal(lens[neg].clamp(min=0), torch.zeros_like(lens[neg]))
    assert torch.equal(lens[~neg], lens_before[~neg] + 1)
    lens.clamp_(min=0)
    d.same(t)
    unused_entries_are_untouched(t)


@pytest.mark.parametrize("pages,rows", SIZES)
def test_a_negative_length_is_shared_given_back_and_moved_as_none(pages, rows):
    d, t, bad = grown(pages, rows)
    new = d.fork(t, (np.arange(rows) * 5) % rows)              # their branches have none either
    kept = d.fork(t, np.resize(bad, 7), np.resize([3, -4, 0, -2 ** 31, 2 ** 31 - 1], 7))
    assert kept[2].tolist() == [0] * 7
    negative = t[2].clone()
    t[2].clamp_(min=0)                                         # d.same compares lengths
    d.same(t)
    t[2].copy_(negative)
    d.truncate(t, np.resize([4, 0, -7, -2 ** 31, 40, 2 ** 31 - 1], rows))
    assert (t[2] >= 0).all()
    new[2][new[2] == 0] = -33
    h = new[0]
    d.truncate(t, None)
    before = new[2].clone()
    new[2].clamp_(min=0)
    d.same(new)
    new[2].copy_(before)
    # compaction reads lengths and leaves them
    ws = torch.empty(kvc.kvc_compact_plan(pages), dtype=torch.uint8, device="cuda")
    where = torch.empty(pages, dtype=torch.int32, device="cuda")
    live = torch.empty(1, dtype=torch.int32, device="cuda")
    kvc.kvc_compact(new[1], new[2], d.refs, where, live, 16, d.arrays, workspace=ws)
    to, n = h.compact()
    assert live.item() == n and where.tolist() == to and torch.equal(new[2], before)
    new[2].clamp_(min=0)
    d.same(new)


def test_the_largest_pool():
    """2^31 - 1 pages (of one position): the last ones are handed out, counted and moved like any other."""
    n = 2 ** 31 - 1
    free = [5, 2 ** 30, n - 4096, n - 2, n - 1]
    at = torch.tensor(free, device="cuda")
    refs = torch.ones(n, dtype=torch.int32, device="cuda")
    refs[at] = 0
    table = torch.full((2, 8), -5, dtype=torch.int32, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    missing = torch.full((1,), -7, dtype=torch.int32, device="cuda")
    ws = torch.empty(kvc.kvc_reserve_plan(2, n), dtype=torch.uint8, device="cuda")
    for grow, want in (([3, 3], 1), ([3, 2], 0), ([0, 1], 1)):
        kvc.kvc_reserve(table, lens, i32_tensor(np.array(grow), "cuda"), refs, missing, 1, workspace=ws)
        assert missing.item() == want
    assert table.tolist() == [free[:3] + [-5] * 5, free[3:] + [-5] * 6] and lens.tolist() == [3, 2]
    assert int(refs.sum()) == n
    del ws
    refs.zero_()
    refs[at] = torch.arange(1, 6, dtype=torch.int32, device="cuda")
    ws = torch.empty(kvc.kvc_compact_plan(n), dtype=torch.uint8, device="cuda")
    where = torch.empty(n, dtype=torch.int32, device="cuda")
    live = torch.empty(1, dtype=torch.int32, device="cuda")
    kvc.kvc_compact(table, lens, refs, where, live, 1, workspace=ws)
    assert live.item() == 5
    assert table.tolist() == [[0, 1, 2] + [-5] * 5, [3, 4] + [-5] * 6]
    assert refs[:6].tolist() == [1, 2, 3, 4, 5, 0] and int(refs.sum()) == 15
    assert where[at].tolist() == [0, 1, 2, 3, 4] and int((where >= 0).sum()) == 5
    kvc.kvc_truncate(table, lens, None, refs, 1)
    assert refs[:6].tolist() == [0, 1, 2, 3, 4, 0] and kvc.kvc_device_errors() == 0
