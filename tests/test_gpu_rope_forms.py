"""kvc_rope_store without queries and in place, and kvc_rope in front of the stores that quantise."""
import numpy as np
import pytest
import torch

import pagedattention_kvc_store_gb300 as kvc
from oracle import int4, oracle
from test_gpu_int4 import assert_pools_equal, device_pools, empty_pools
from test_gpu_rope import _check, _inputs
from workloads import BF16_NAN
from workloads.device import bf16_bits_of, bf16_tensor, i32_tensor

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pairing", ["halves", "adjacent"])
@pytest.mark.parametrize("T,Hkv,D,P,layout", [(1, 2, 64, 16, "nhd"), (77, 3, 128, 32, "hnd")])
def test_a_store_without_queries(T, Hkv, D, P, layout, pairing):
    x, positions, inv_freq, axis = _inputs(T, T, 0, Hkv, D, D // 2, 2, 131072)
    pages = -(-T // P) + 1
    slots = np.random.default_rng(T).permutation(pages * P)[:T].astype(np.int32)
    slots[3::5] = -1
    kp = np.full((pages, P, Hkv, D) if layout == "nhd" else (pages, Hkv, P, D), BF16_NAN, dtype=np.uint16)
    kd, vd, d = bf16_tensor(kp, "cuda"), bf16_tensor(kp, "cuda"), bf16_tensor(x, "cuda")
    rope = kvc.rope_desc(inv_freq, axis, pairing=pairing, num_axes=2)
    pos = i32_tensor(positions, "cuda")
    kvc.kvc_rope_store(None, kd, vd, None, d[:, :Hkv], d[:, Hkv:], pos, i32_tensor(slots, "cuda"), rope,
                       layout=layout)
    rows = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
    kvc.kvc_rope(None, rows, None, d[:, :Hkv], pos, rope)
    _check(bf16_bits_of(rows), x[:, :Hkv], positions, inv_freq, axis, pairing == "adjacent", "k")
    vp = kp.copy()
    oracle.store(kp, vp, bf16_bits_of(rows), np.ascontiguousarray(x[:, Hkv:]), slots, layout=layout)
    assert np.array_equal(bf16_bits_of(kd), kp) and np.array_equal(bf16_bits_of(vd), vp)
    assert np.array_equal(bf16_bits_of(d), x) and kvc.kvc_device_errors() == 0


@pytest.mark.parametrize("T,Hq,Hkv,D", [(1, 8, 2, 64), (130, 4, 4, 128)])
def test_queries_turned_where_they_are(T, Hq, Hkv, D):
    """q_out is q: contiguous rows."""
    x, positions, inv_freq, axis = _inputs(T + 1, T, Hq, Hkv, D, D, 3, 131072)
    q = bf16_tensor(np.ascontiguousarray(x[:, :Hq]), "cuda")
    d, pos = bf16_tensor(x, "cuda"), i32_tensor(positions, "cuda")
    kd = torch.zeros(-(-T // 16), 16, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vd = torch.zeros_like(kd)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    kvc.kvc_rope_store(q, kd, vd, q, d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], pos, slots,
                       kvc.rope_desc(inv_freq, axis))
    _check(bf16_bits_of(q), x[:, :Hq], positions, inv_freq, axis, False, "q")
    _check(bf16_bits_of(kd.flatten(0, 1)[:T]), x[:, Hq:Hq + Hkv], positions, inv_freq, axis, False, "k")
    assert np.array_equal(bf16_bits_of(vd.flatten(0, 1)[:T]), x[:, Hq + Hkv:])
    assert kvc.kvc_device_errors() == 0


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("T,Hq,Hkv,D,P", [(5, 4, 2, 128, 16), (70, 6, 3, 64, 32)])
def test_turned_keys_into_quantised_pages(T, Hq, Hkv, D, P, bits):
    """kvc_rope on a projection's output, then the store that quantises: codes and parameters of the turned keys."""
    x, positions, inv_freq, axis = _inputs(T + 2, T, Hq, Hkv, D, D, 1, 131072)
    d = bf16_tensor(x, "cuda")
    q = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    k = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = d[:, Hq + Hkv:].contiguous()
    kvc.kvc_rope(q, k, d[:, :Hq], d[:, Hq:Hq + Hkv], i32_tensor(positions, "cuda"), kvc.rope_desc(inv_freq, axis))
    _check(bf16_bits_of(q), x[:, :Hq], positions, inv_freq, axis, False, "q")
    _check(bf16_bits_of(k), x[:, Hq:Hq + Hkv], positions, inv_freq, axis, False, "k")
    pages = -(-T // P) + 1
    slots = np.random.default_rng(T).permutation(pages * P)[:T].astype(np.int32)
    slots[1::6] = -1
    ds, new = i32_tensor(slots, "cuda"), (bf16_bits_of(k), bf16_bits_of(v))
    if bits == 4:
        pools = empty_pools(pages, P, Hkv, D, "nhd")
        dev = device_pools(pools)
        kvc.kvc_store_int4(*dev, k, v, ds)
        int4.store(*pools, *new, slots, "nhd")
        assert_pools_equal(dev, pools)
    else:
        rng = np.random.default_rng(0)
        pools = [rng.integers(-128, 128, size=(pages, P, Hkv, D)).astype(np.int8) for _ in "kv"]
        pools += [np.full((pages, Hkv, P), 0.5, np.float32) for _ in "kv"]
        dev = [torch.from_numpy(a).cuda() for a in pools]
        kvc.kvc_store_int8(*dev, k, v, ds)
        oracle.store_int8(*pools, *new, slots.astype(np.int64))
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(dev, pools))
    assert kvc.kvc_device_errors() == 0
