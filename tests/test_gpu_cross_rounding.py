"""kvc_cross's one rounding to fewer bits, P to bf16 for the product with V, held to what it is.

The kernels sum the unrounded probabilities, so only the numerator has it: each p is off by at most 2^-8 of itself,
and the mean over them by 2^-8 * sum(w |v|).  What else there is, relative to sum(w |v|), for scores whose
sum |q k| scale is at most A, n positions and D dims:
  * a score is an fp32 sum of D products (2^-23 each, as tensor cores may cut), times scale * log2(e), itself two
    roundings, minus the maximum in one: (D + 4) 2^-23 A of the exponent, and 2^x 2^-22: e of each weight, in the
    numerator and in the sum, 2 e
  * the sum of p: a thread adds every fourth pair of columns, pairs first, n / 8 additions of 2^-24 at most
    behind each other; O: a matrix instruction adds 16 positions, n / 16 of them of 2^-22 (16 products and the sum
    before, cut); together below n / 4 of 2^-23.  Rescaling, joins of splits and halves, the division: below 64 of 2^-23.
bf16 outputs are rounded once more, 2^-8 of themselves."""
import math

import numpy as np
import pytest
import torch

import pagedattention_kvc_store_gb300 as kvc
from test_gpu_cross import RAGGED, Case
from workloads import f32_from_bf16

pytestmark = pytest.mark.gpu


def rest(c, n):
    """Everything but P's rounding, relative to sum(w |v|)."""
    q = np.abs(c.q[:c.T].float().numpy().astype(np.float64))
    reach = 0.0
    for s, m in enumerate(c.lens):
        t = slice(c.indptr[s], c.indptr[s + 1])
        p = np.arange(m)
        k = np.abs(f32_from_bf16(c.k[c.table[s][p // c.P], p % c.P]).astype(np.float64))
        for h in range(c.Hkv * c.G):
            if m and t.stop > t.start:
                reach = max(reach, (q[t, h] @ k[:, h // c.G].T).max() / math.sqrt(c.D))
    e = (c.D + 4) * 2.0 ** -23 * reach + 2.0 ** -22
    return 2 * e + (n / 4 + 64) * 2.0 ** -23


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("Hkv,G,D,P,layout,most", [(2, 4, 128, 16, "nhd", 5), (3, 1, 64, 32, "hnd", 9),
                                                   (2, 4, 128, 16, "nhd", 70), (4, 2, 64, 64, "hnd", 150)])
def test_only_the_numerator_s_probabilities_are_rounded(Hkv, G, D, P, layout, most, splits):
    q_lens = [most, 0, 1, 2, most - 1, 1, 3, most, 2, most]
    c = Case(RAGGED, q_lens, Hkv, G, D, P, layout, seed=most)
    want, _, weighed = c.exact()
    bound = (2.0 ** -8 + 1.01 * rest(c, max(RAGGED))) * weighed
    out, _ = c.run(splits=splits)
    assert (np.abs(out.cpu().numpy() - want) <= bound).all()
    out, _ = c.run(torch.bfloat16, splits, lse=False)
    assert (np.abs(out.float().cpu().numpy() - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound)).all()


@pytest.mark.parametrize("splits", [1, 4])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("most", [3, 50, 200])
def test_probabilities_are_rounded_to_the_nearest(most, D, splits):
    """Values of one: the output is the sum of the rounded p over that of p.  The roundings are independent, each
    within 2^-8 of its weight w, so but for one row in 10^12 the sum is off by less than 2^-8 sqrt(2 ln(2e12)
    sum(w^2)); cut off instead, p would be short by 2^-8 / m on average, m its mantissa: more than half of 2^-8."""
    c = Case([4000], [most], 2, 2, D, 16)
    p = np.arange(4000)
    at = c.table[0][p // 16], p % 16
    c.v[at] = 0x3F80
    out, _ = c.run(splits=splits)
    q = c.q.float().numpy().astype(np.float64)
    k = f32_from_bf16(c.k[at]).astype(np.float64)
    bound = np.empty((most, 4, 1))
    for h in range(4):
        x = np.exp(q[:, h] @ k[:, h // 2].T / math.sqrt(D))
        w = x / x.sum(1, keepdims=True)
        bound[:, h, 0] = 2.0 ** -8 * np.sqrt(2 * math.log(2e12) * (w ** 2).sum(1)) + rest(c, 4000)
    assert bound.max() < 0.5 * 2.0 ** -8      # or the test would tell nothing
    assert (np.abs(out.cpu().numpy() - 1.0) <= bound).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("most", [4, 300])
def test_the_same_call_gives_the_same_bits(most, D):
    """Whichever block takes an item over."""
    rng = np.random.default_rng(3)
    c = Case([int(n) for n in rng.integers(1, 900, 60)], [int(n) for n in rng.integers(0, most + 1, 60)],
             4, 2, D, 16)
    first = c.run(torch.bfloat16, splits=1, max_q=most)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(first, c.run(torch.bfloat16, splits=1, max_q=most)))
    assert kvc.kvc_device_errors() == 0
