"""The plain accumulated weights and eviction (oracle/evict.py) on hand-worked rows; the argument
checks of their entry points.  CPU only."""
import ctypes

import numpy as np
import pytest
import torch

import pagedattention_kvc_store_gb300 as kvc
from oracle import evict, oracle
from pagedattention_kvc_store_gb300.kvc import PoolDesc, lib
from workloads import config_case


def test_kept_slots_by_hand():
    w = np.array([5.0, 1.0, 3.0, 3.0, 0.0, 9.0, 0.0, 0.1])
    pos = np.arange(8)
    # the two newest, then 9, 5, and the lower of the two 3s
    assert np.flatnonzero(evict.kept(w, pos, 5, 2)).tolist() == [0, 2, 5, 6, 7]
    assert np.flatnonzero(evict.kept(w, pos, 5, 0)).tolist() == [0, 1, 2, 3, 5]
    assert evict.kept(w, pos, 8, 3).all() and evict.kept(w, pos, 100, 3).all()
    assert np.flatnonzero(evict.kept(w, pos, 3, 3)).tolist() == [5, 6, 7]
    # the newest by position, wherever they lie
    assert np.flatnonzero(evict.kept(w, np.array([7, 1, 8, 3, 4, 5, 6, 9]), 3, 3)).tolist() == [0, 2, 7]
    nan = np.array([np.nan, -1.0, -np.inf, 0.0, -0.0])
    assert np.flatnonzero(evict.kept(nan, np.arange(5), 3, 0)).tolist() == [1, 3, 4]
    assert np.flatnonzero(evict.kept(nan, np.arange(5), 4, 0)).tolist() == [0, 1, 3, 4]
    assert not evict.kept(w[:0], pos[:0], 3, 1).any()


def test_moves_by_hand():
    """Budget 3 of 6 slots on pages of 2: slots 1 and 2 are given up, slots 4 and 5 fill them."""
    kp = np.arange(8, dtype=np.uint16).reshape(4, 2, 1, 1)
    vp = kp + 100
    w = np.array([[[9.0, 0, 1, 2, 8, 3, 0]]])
    pos = np.array([[[0, 4, 2, 3, 11, 12, 99]]])
    table = np.array([[2, 0, 3]])
    lens = evict.evict(kp, vp, w, pos, table, np.array([6]), 3, 1)
    assert lens.tolist() == [3]
    assert kp[2].ravel().tolist() == [4, 6] and kp[0].ravel().tolist() == [7, 1]
    assert vp[2].ravel().tolist() == [104, 106]
    assert kp[3].ravel().tolist() == [6, 7]            # what is behind the end stays
    assert w[0, 0].tolist() == [9, 8, 3, 0, 0, 0, 0]
    assert pos[0, 0].tolist() == [0, 11, 12, 13, 14, 15, 16]


def test_weights_against_the_attention_oracle():
    """With one-hot values the attention output is the weights themselves."""
    case = config_case(1, poison=False)
    got = evict.weights(case.q, case.k_pool, case.block_table, case.context_lens)
    D = case.head_dim
    for s, n in enumerate(case.context_lens):
        n = min(int(n), D)
        onehot = np.zeros_like(case.v_pool)
        p = np.arange(n)
        onehot[case.block_table[s][p // case.page_size], p % case.page_size, :, p] = 0x3F80
        ref, _ = oracle.attention(case.q, case.k_pool, onehot, case.block_table,
                                  case.context_lens, case.q_indptr)
        want = ref[s].reshape(case.kv_heads, -1, D).sum(1)
        np.testing.assert_allclose(got[s][:, :n], want[:, :n], atol=1e-12)
        np.testing.assert_allclose(got[s].sum(-1), case.q_heads // case.kv_heads)


def test_a_row_that_is_cut_twice():
    """A cut may leave an old token in the last slot: the newest position is then given."""
    table = np.arange(2)[None]
    kp, vp = (np.arange(2 * 16 * 64, dtype=np.uint16).reshape(2, 16, 1, 64) + i for i in (0, 9))
    w = np.zeros((1, 1, 30), np.float32)
    w[0, 0, 7] = 1.0
    pos = np.arange(30, dtype=np.int32)[None, None].copy()
    assert evict.evict(kp, vp, w, pos, table, [20], 8, 3).tolist() == [8]
    # 17 .. 19 are the newest, 7 the heaviest, 0 .. 3 the first of equal weight
    assert pos[0, 0, :9].tolist() == [0, 1, 2, 3, 17, 18, 19, 7, 20]
    before = pos.copy()
    assert evict.evict(kp, vp, w, pos, table, [8], 8, 3, newest=[19]).tolist() == [8]
    assert np.array_equal(pos, before)
    assert evict.evict(kp, vp, w, pos, table, [8], 4, 3, newest=[19]).tolist() == [4]
    assert sorted(pos[0, 0, :4]) == [7, 17, 18, 19]
    assert pos[0, 0, 4:].tolist() == list(range(20, 46))


# --------------------------------------------------------------------- argument checks
POOL = PoolDesc(32, 16, 2, 64)
FAKE = ctypes.c_void_p(0x10000)   # never dereferenced: checks fail before any launch
FAKE2 = ctypes.c_void_p(0x20000)
FAKE3 = ctypes.c_void_p(0x30000)
ODD = ctypes.c_void_p(0x10004)


@pytest.mark.parametrize("kw,code", [
    (dict(pool=PoolDesc(32, 16, 2, 96)), 2), (dict(q_heads=3), 1), (dict(out=ODD), 1),
    (dict(weights=None), 1), (dict(num_rows=3), 1), (dict(num_rows=-1, rows=FAKE), 1),
    (dict(stride=99), 1), (dict(splits=-1), 1), (dict(splits=1), 3), (dict(ws=FAKE, nbytes=16), 3),
    (dict(ws=ODD, nbytes=1 << 30), 1), (dict(bt=4), 1), (dict(seqs=0), 0), (dict(seqs=-1), 1),
    (dict(bt=1 << 27), 2),
])
def test_decode_weights_refusals(kw, code):
    a = dict(pool=POOL, q_heads=4, out=FAKE, weights=FAKE, rows=None, num_rows=4, stride=100, bt=8,
             splits=0, ws=None, nbytes=0, seqs=4)
    a.update(kw)
    assert lib().kvc_decode_weights(a["out"], 0, a["weights"], a["rows"], a["num_rows"],
                                    a["stride"], FAKE, FAKE, FAKE, a["pool"], FAKE, a["bt"], FAKE,
                                    a["seqs"], 100, a["q_heads"], 0.0, a["splits"], a["ws"],
                                    a["nbytes"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(pool=PoolDesc(32, 8, 2, 64)), 2), (dict(k=ODD), 1), (dict(k=None), 1),
    (dict(weights=None), 1), (dict(positions=None), 1), (dict(budget=0), 1), (dict(recent=-1), 1),
    (dict(recent=51), 1), (dict(new=FAKE), 1), (dict(new=None), 1), (dict(stride=99), 1),
    (dict(num_rows=3), 1), (dict(bt=4), 1), (dict(), 3), (dict(ws=FAKE, nbytes=100), 3),
    (dict(ws=ODD, nbytes=1 << 30), 1), (dict(seqs=0), 0), (dict(seqs=-1), 1), (dict(seqs=70000), 1),
    (dict(bt=1 << 27), 2), (dict(new=ctypes.c_void_p(0x10008)), 1),
    (dict(wout=ctypes.c_void_p(0x10010)), 1), (dict(pout=ctypes.c_void_p(0xff00)), 1),
    (dict(wout=FAKE2, pout=FAKE3), 3),
])
def test_evict_refusals(kw, code):
    a = dict(pool=POOL, k=FAKE, weights=FAKE, positions=FAKE, budget=50, recent=10, new=FAKE2,
             stride=100, num_rows=4, bt=8, ws=None, nbytes=0, seqs=4, wout=FAKE, pout=FAKE)
    a.update(kw)
    assert lib().kvc_evict(a["k"], FAKE, a["pool"], FAKE, a["bt"], FAKE, a["seqs"], 100,
                           a["weights"], a["positions"], a["wout"], a["pout"], None, a["num_rows"],
                           a["stride"], a["budget"], a["recent"], a["new"], a["ws"], a["nbytes"],
                           None) == code


def test_plans():
    pool = PoolDesc(2000, 16, 8, 128)
    assert kvc.kvc_evict_plan(64, pool, 4096, 2048) == 64 * 8 * (2 * 2048 + 2) * 4
    assert kvc.kvc_evict_plan(64, pool, 4096, 4000) == 64 * 8 * (2 * 96 + 2) * 4
    assert kvc.kvc_evict_plan(64, pool, 4096, 5000) == 0
    s, c, ws = kvc.kvc_decode_weights_plan(64, 32, pool, 4096)
    assert (s, c) == kvc.kvc_decode_plan(64, 32, pool, 4096)[:2]
    assert ws >= 64 * 32 * (s * 130 + s * c) * 4
    assert kvc.kvc_decode_weights_plan(4, 32, pool, 10, 1)[2] > 0
    for most, call in ((22, lambda n: kvc.kvc_evict_plan(1, pool, n, 5)),
                       (30, lambda n: kvc.kvc_decode_weights_plan(1, 8, pool, n, 0)),
                       (30, lambda n: kvc.kvc_decode_int4_plan(1, 8, pool, n, 0))):
        call(1 << most)
        with pytest.raises(RuntimeError, match=f"2\\^{most}"):
            call((1 << most) + 1)


def test_binding_refuses_cpu_tensors():
    t = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.kvc_evict(t, t, i, i, i, i, i, i, i, 10, 5)
    with pytest.raises(ValueError, match="pinned"):
        kvc.kvc_decode_weights(t, i, t, t, t, i, i, 10)
