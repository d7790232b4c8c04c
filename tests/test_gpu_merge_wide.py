"""kvc_merge over few and many splits against a 64-bit merge.  |lse - M| stays below 32, so the
difference and its product with log2(e) are off by 2^-18 at most and a weight by that much of itself;
sums and products of up to 150 terms add 150 * 2^-24: below 2^-16 of the largest partial together."""
import numpy as np
import pytest
import torch

import pagedattention_kvc_store_gb300 as kvc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("splits", [1, 4, 16, 17, 31, 33, 48, 150])
def test_merge_of_many_splits(splits, D):
    rows = 37
    rng = np.random.default_rng(splits + D)
    o = rng.standard_normal((rows, splits, D)).astype(np.float32)
    lse = (3 * rng.standard_normal((rows, splits))).astype(np.float32)
    empty = rng.random((rows, splits)) < 0.3
    empty[0], empty[1] = True, False
    lse[empty] = -np.inf
    o[empty] = np.nan                       # an empty split's partial is never used
    out = torch.full((rows, D), 7.0, device="cuda")
    back = torch.zeros(rows, device="cuda")
    kvc.kvc_merge(out, torch.from_numpy(o).cuda(), torch.from_numpy(lse).cuda(), lse_out=back)
    w = np.exp(lse.astype(np.float64) - np.where(empty.all(1), 0.0, lse.max(1))[:, None])
    total = w.sum(1)
    ref = (w[:, :, None] * np.where(empty[:, :, None], 0.0, o.astype(np.float64))).sum(1)
    ref = np.where(total[:, None] > 0, ref / np.maximum(total, 1e-300)[:, None], 0.0)
    got = out.double().cpu().numpy()
    assert np.abs(got - ref).max() <= 2.0 ** -16 * np.nanmax(np.abs(o))
    live = ~empty.all(1)
    want = lse.max(1)[live] + np.log(total[live])
    assert np.abs(back.double().cpu().numpy()[live] - want).max() <= 2.0 ** -18
    assert (back.cpu().numpy()[~live] == -np.inf).all()
