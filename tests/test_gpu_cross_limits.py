"""kvc_cross at the limits of what its device arrays may say: both kernels, one and several splits."""
import numpy as np
import pytest
import torch

import pagedattention_kvc_store_gb300 as kvc
from test_gpu_cross import Case, check
from workloads.device import bf16_tensor, i32_tensor

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("most", [4, 60, 200])
def test_a_negative_length_is_no_position(most, D, splits):
    c = Case([0, 300, 0, 700, 0], [most, most, 2, most, most], 2, 2, D, 16)
    kvc.kvc_device_errors()
    c.lens = [-1, 300, -2 ** 31, 700, -2 ** 31 + 1]
    out, lse = c.run(splits=splits)
    assert kvc.kvc_device_errors() == 0
    c.lens = [0, 300, 0, 700, 0]
    check(c, out, lse)
    for s in (0, 2, 4):
        none = slice(int(c.indptr[s]), int(c.indptr[s + 1]))
        assert (out[none] == 0).all() and torch.isneginf(lse[none]).all()


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("most", [6, 60, 200])
@pytest.mark.parametrize("first,last", [(0, 9), (-5, 0), (0, 2 ** 31 - 1), (-2 ** 31, 0)])
def test_tokens_outside_of_the_call_are_flagged_and_not_written(first, last, most, D, splits):
    """Before the first token, or behind the last: the other sources' rows are right, and what lies around
    out and lse_out is left alone."""
    c = Case([300, 129, 700], [most, most, most], 2, 2, D, 16)
    q = c.q.cuda()
    around = torch.full((c.T + 40, 4, D), 7.25, device="cuda")
    logs = torch.full((c.T + 40, 4), 7.25, device="cuda")
    out, lse = around[20:c.T + 20], logs[20:c.T + 20]
    kd, vd = bf16_tensor(c.k, "cuda"), bf16_tensor(c.v, "cuda")
    indptr = c.indptr.copy()
    if first < 0:
        indptr[0] = first
    if last > 0:
        indptr[3] = min(c.T + last, 2 ** 31 - 1)
    most_given = most + 9     # what a caller would pass for the tokens that the array names
    ws = kvc.kvc_cross_plan(3, c.T, 4, kvc.pool_desc(kd), most_given, 700, splits)[2]
    work = torch.full((max(ws, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    kvc.kvc_device_errors()
    kvc.kvc_cross(out, q, kd, vd, i32_tensor(c.table, "cuda"), i32_tensor(indptr, "cuda"),
                  i32_tensor(np.array(c.lens), "cuda"), most_given, 700, lse_out=lse, num_splits=splits,
                  workspace=work)
    assert kvc.kvc_device_errors() == 1 << 7
    assert (around[:20] == 7.25).all() and (around[c.T + 20:] == 7.25).all()
    assert (logs[:20] == 7.25).all() and (logs[c.T + 20:] == 7.25).all()
    right = np.ones(c.T, dtype=bool)
    right[c.indptr[0 if first < 0 else 2]:c.indptr[1 if first < 0 else 3]] = False
    want, want_lse, weighed = c.exact()
    err = np.abs(out.cpu().numpy() - want)[right]
    assert (err <= 2.0 ** -7 * weighed[right] + 1e-6).all()
    assert (np.abs(lse.cpu().numpy() - want_lse)[right] <= 2.0 ** -14 + 2.0 ** -20 * np.abs(want_lse[right])).all()
