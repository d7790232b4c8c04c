"""Calls over many sets of pools in turn (a model has pools for each layer; more sets here than the
library keeps tensor maps for): each call reads its own.  Values are constants that the formats hold
exactly, so the attention over any number of positions is that constant."""
import pytest
import torch

import pagedattention_kvc_store_gb300 as kvc

pytestmark = pytest.mark.gpu

P, H, G, D = 16, 1, 1, 64


def test_4_bit_and_bf16_pools_in_turn():
    n = 700                                 # three maps a set (K and V are the same here): 2,100
    value = torch.arange(n, device="cuda").remainder(251).float()
    codes = torch.zeros(n, 2, P, H, D // 2, dtype=torch.uint8, device="cuda")
    params = torch.zeros(n, 2, H, P, D // 64, 2, dtype=torch.bfloat16, device="cuda")
    params[..., 1] = value.view(-1, 1, 1, 1, 1).bfloat16()        # scale 0, minimum = value
    pools = (value + 1).view(-1, 1, 1, 1, 1).expand(n, 2, P, H, D).bfloat16().contiguous()
    q = torch.ones(2, H * G, D, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[0, 1], [1, 0]], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([20, 7], dtype=torch.int32, device="cuda")
    a, b = (torch.zeros(n, *q.shape, device="cuda") for _ in range(2))
    for _ in range(2):
        a.zero_(), b.zero_()
        for i in range(n):
            kvc.kvc_decode_int4(a[i], q, codes[i], codes[i], params[i], params[i], table, ctx, 32,
                                num_splits=1)
            kvc.kvc_decode(b[i], q, pools[i], pools[i], table, ctx, 32, num_splits=1)
        # equal scores: every weight is the same power of two times 1 / sum, so a few roundings
        for got, want in ((a, value), (b, value + 1)):
            assert ((got - want.view(-1, 1, 1, 1)).abs() <= 2.0 ** -18 * want.view(-1, 1, 1, 1)).all()
    assert kvc.kvc_device_errors() == 0
