"""Workspaces of the page calls for pools up to the largest (2^31 - 1 pages)."""
import pytest

import pagedattention_kvc_store_gb300 as kvc

LARGEST = 2 ** 31 - 1


@pytest.mark.parametrize("pages", [1, 4095, 4096, 4097, 2 ** 30, LARGEST - 4096, LARGEST - 4095, LARGEST])
def test_a_workspace_holds_what_its_pages_need(pages):
    """reserve: two numbers of each page; compact: the source and the destination of a move of half of them.
    Both: a count of every 4,096 pages."""
    counts = 4 * (-(-pages // 4096))
    assert 8 * pages + counts <= kvc.kvc_reserve_plan(0, pages) <= 8 * pages + counts + 4096
    assert 4 * pages + counts <= kvc.kvc_compact_plan(pages) <= 4 * pages + counts + 4096
