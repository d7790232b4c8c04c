"""The plain 4-bit pages (oracle/int4.py) against hand-worked values and their own definition; the
argument checks of the 4-bit entry points.  CPU only."""
import ctypes

import numpy as np
import pytest
import torch

import pagedattention_kvc_store_gb300 as kvc
from oracle import int4
from pagedattention_kvc_store_gb300.kvc import PoolDesc, lib


def bits_of(x):
    return torch.as_tensor(x).bfloat16().view(torch.int16).numpy().view(np.uint16)


def test_integers_0_to_15_are_exact():
    x = np.arange(64) % 16 - 3.0
    codes, params = int4.quantise(bits_of(x))
    assert int4.bf16_value(params).tolist() == [[1.0, -3.0]]
    assert codes[:4].tolist() == [0x10, 0x32, 0x54, 0x76]   # dim 0 in the low four bits
    np.testing.assert_array_equal(int4.values(codes, params), x)


def test_ties_go_to_the_even_code():
    x = np.zeros(64)
    x[:6] = [0.0, 30.0, 1.0, 3.0, 5.0, 29.0]   # step 2: quotients 0.5, 1.5, 2.5, 14.5
    codes, params = int4.quantise(bits_of(x))
    u = np.stack([codes & 15, codes >> 4], -1).ravel()
    assert u[:6].tolist() == [0, 15, 0, 2, 2, 14]


def test_constant_zero_and_non_finite_groups():
    x = np.full(192, 1.25, dtype=np.float32)
    x[64:128] = 0.0
    x[130] = np.inf
    codes, params = int4.quantise(bits_of(x))
    v = int4.values(codes, params)
    assert (v[:64] == 1.25).all() and (v[64:128] == 0).all() and np.isnan(v[128:]).all()
    assert not codes.any()


@pytest.mark.parametrize("power", [-130, -100, 0, 100, 126])
def test_error_is_half_a_step(power):
    """Against the definition in exact arithmetic, over bf16's exponents: within half a step (and
    the 0.03 steps that scale's own rounding moves the largest value by)."""
    rng = np.random.default_rng(power + 200)
    x = rng.standard_normal((50, 128)).astype(np.float32)
    b = bits_of(x * np.float32(2.0 ** (power / 2)) * np.float32(2.0 ** (power / 2)))
    codes, params = int4.quantise(b)
    exact = int4.bf16_value(b).astype(np.float64)
    step = np.repeat(int4.bf16_value(params[..., 0]).astype(np.float64), 64, axis=-1)
    if power > -120:   # below, the scale itself is subnormal and coarser
        assert (np.abs(int4.values(codes, params) - exact) <= 0.54 * step).all()
        assert (step > 0).all()


def test_store_load_and_layouts_agree():
    rng = np.random.default_rng(3)
    pages, P, H, D = 3, 16, 2, 64
    k, v = (bits_of(rng.standard_normal((20, H, D))) for _ in range(2))
    slots = rng.permutation(pages * P)[:20]
    slots[5] = -1
    got = {}
    for layout, shape in (("nhd", (pages, P, H, D // 2)), ("hnd", (pages, H, P, D // 2))):
        pools = [np.zeros(shape, np.uint8) for _ in range(2)] + \
                [np.zeros((pages, H, P, 1, 2), np.uint16) for _ in range(2)]
        int4.store(*pools, k, v, slots, layout)
        got[layout] = int4.load(pools[0], pools[2], slots, layout)
    np.testing.assert_array_equal(got["nhd"], got["hnd"])
    want = int4.values(*int4.quantise(k))
    want[5] = 0.0
    np.testing.assert_array_equal(got["nhd"], want)


def test_attention_matches_torch_softmax():
    rng = np.random.default_rng(4)
    P, H, G, D, n = 16, 2, 2, 64, 37
    k, v = (bits_of(rng.standard_normal((n, H, D))) for _ in range(2))
    pools = [np.zeros((4, P, H, D // 2), np.uint8) for _ in range(2)] + \
            [np.zeros((4, H, P, 1, 2), np.uint16) for _ in range(2)]
    table = np.array([[2, 0, 3]])
    p = np.arange(n)
    int4.store(*pools, k, v, table[0][p // P] * P + p % P)
    q = bits_of(rng.standard_normal((1, H * G, D)))
    got = int4.attention(q, *pools, table, np.array([n]))
    kd, vd = (torch.from_numpy(int4.values(*int4.quantise(x))).transpose(0, 1) for x in (k, v))
    qd = torch.from_numpy(int4.bf16_value(q).astype(np.float64)).view(H, G, D)
    want = torch.nn.functional.scaled_dot_product_attention(qd, kd, vd).reshape(1, H * G, D)
    np.testing.assert_allclose(got, want.numpy(), atol=1e-12)
    assert not int4.attention(q, *pools, table, np.array([0])).any()


# --------------------------------------------------------------------- argument checks
POOL = PoolDesc(32, 16, 2, 64)
FAKE = ctypes.c_void_p(0x10000)   # never dereferenced: checks fail before any launch
ODD = ctypes.c_void_p(0x10004)


def decode(pool=POOL, q_heads=4, out=FAKE, kp=FAKE, bt=8, max_ctx=100, splits=1, ws=None,
           nbytes=0, dtype=0, seqs=4):
    return lib().kvc_decode_int4(out, dtype, FAKE, FAKE, FAKE, kp, FAKE, pool, FAKE, bt, FAKE,
                                 seqs, max_ctx, q_heads, 0.0, splits, ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(pool=PoolDesc(32, 16, 2, 96)), 2), (dict(pool=PoolDesc(32, 8, 2, 64)), 2),
    (dict(pool=PoolDesc(32, 16, 2, 64, 5)), 1), (dict(q_heads=3), 1), (dict(q_heads=32), 2),
    (dict(out=ODD), 1), (dict(kp=ODD), 1), (dict(kp=None), 1), (dict(bt=4), 1),
    (dict(splits=-1), 1), (dict(splits=0, bt=16, max_ctx=200), 3), (dict(splits=2, ws=FAKE, nbytes=16), 3),
    (dict(dtype=7), 1), (dict(seqs=-1), 1), (dict(seqs=70000), 1), (dict(seqs=0), 0),
])
def test_decode_int4_refusals(kw, code):
    assert decode(**kw) == code


def test_store_and_load_int4_refusals():
    L = lib()

    def store(pool=POOL, new=FAKE, par=FAKE, slots=FAKE, n=4):
        return L.kvc_store_int4(FAKE, FAKE, par, FAKE, pool, new, FAKE, slots, n, None)

    def load(pool=POOL, out=FAKE, dtype=0, slots=FAKE, n=4):
        return L.kvc_load_int4(out, FAKE, dtype, FAKE, FAKE, FAKE, FAKE, pool, slots, n, None)

    assert store(n=0) == 0 and load(n=0) == 0
    for call in (store, load):
        assert call(n=-1) == 1 and call(slots=None) == 1
        assert call(pool=PoolDesc(32, 16, 2, 80)) == 2 and call(pool=PoolDesc(0, 16, 2, 64)) == 1
    assert store(new=ODD) == 1 and store(par=ODD) == 1 and store(par=None) == 1
    assert load(out=ODD) == 1 and load(out=None) == 1 and load(dtype=3) == 1


def test_decode_int4_plan():
    pool = PoolDesc(100, 16, 8, 128)
    assert kvc.kvc_decode_int4_plan(64, 32, pool, 4096, 1) == (64 * 8, 64, 0)
    warps, block, ws = kvc.kvc_decode_int4_plan(64, 32, pool, 4096, 0)
    assert block == 64 and warps % 8 == 0 and 0 < warps <= 64 * 128 * 8
    slots = 8 * (64 + warps // 8)
    assert ws >= slots * 4 * 129 * 4 + 64 * 8 * 8
    assert kvc.kvc_decode_int4_plan(1, 32, pool, 129, 0)[0] == 3 * 8   # one run per block
    assert kvc.kvc_decode_int4_plan(5, 32, pool, 128, 0) == (5 * 8, 64, 0)   # short: whole units
    assert kvc.kvc_decode_int4_plan(0, 32, pool, 0, 0)[0] == 8


def test_binding_checks_shapes_before_the_library():
    t = torch.zeros(2, 16, 2, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.kvc_store_int4(t, t, t, t, t, t, t)
    with pytest.raises(ValueError, match="uint8"):
        kvc.int4_pool_desc(t.float())
    assert kvc.int4_pool_desc(t).head_dim == 64 and kvc.int4_pool_desc(t, "hnd").page_size == 2
