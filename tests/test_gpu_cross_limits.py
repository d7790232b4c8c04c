"""kvc_cross at the limits of what its device arrays may say: both kernels, one and several splits."""
import pytest
import torch

import pagedattention_kvc_store_gb300 as kvc
from test_gpu_cross import Case, check

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
