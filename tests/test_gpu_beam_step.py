"""A decoder with beams over sources, step by step as a server runs it: branch, give back, reserve, slot mapping,
rotate and store, attend over its own pages and over its source's.  Two captured graphs (the tables of the
beams change places from step to step), nothing read back in between; against plain attention in 64 bits."""
import math

import numpy as np
import pytest
import torch

import pagedattention_kvc_store_gb300 as kvc
from harness import assert_attention_close
from oracle import rope as orope
from workloads import BF16_NAN, f32_from_bf16, normal_bf16
from workloads.device import bf16_tensor, i32_tensor

pytestmark = pytest.mark.gpu

HQ, HKV, D, P, SOURCES, BEAMS, STEPS, WIDTH = 4, 2, 64, 16, 3, 4, 40, 16
ROWS = SOURCES * BEAMS
LENS = [37, 200, 0]          # of the sources; the last has no state


def _softmax_attend(q, k, v):
    """q [Hq, D], k and v [n, Hkv, D] -> [Hq, D]."""
    out = np.zeros_like(q)
    for h in range(HQ if len(k) else 0):
        x = k[:, h // (HQ // HKV)] @ q[h] / math.sqrt(D)
        w = np.exp(x - x.max())
        out[h] = (w / w.sum()) @ v[:, h // (HQ // HKV)]
    return out


def _bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).bfloat16().double().numpy()


def test_beams_over_sources():
    ss = np.random.SeedSequence(99)
    rng = np.random.default_rng(99)
    # the sources' states, stored once
    need = [-(-n // P) for n in LENS]
    src_pool = torch.full((sum(need) + 2, P, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    src_v = src_pool.clone()
    src_table = np.zeros((SOURCES, 16), dtype=np.int32)
    order = rng.permutation(sum(need) + 2)
    states, at = [], 0
    for s, n in enumerate(LENS):
        src_table[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
        kv = normal_bf16(ss.spawn(1)[0], (2, n, HKV, D))
        states.append(f32_from_bf16(kv).astype(np.float64))
        if n:
            p = np.arange(n)
            slots = i32_tensor(src_table[s][p // P] * P + p % P, "cuda")
            kvc.kvc_store(src_pool, src_v, bf16_tensor(kv[0], "cuda"), bf16_tensor(kv[1], "cuda"), slots)
    src_table, src_lens = i32_tensor(src_table, "cuda"), i32_tensor(np.array(LENS), "cuda")
    q_indptr = torch.arange(0, ROWS + 1, BEAMS, dtype=torch.int32, device="cuda")
    # the beams: one table in use, one for the next step
    pages = ROWS * 6
    kp = torch.full((pages, P, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    tables = [torch.zeros(ROWS, WIDTH, dtype=torch.int32, device="cuda") for _ in range(2)]
    lens = [torch.zeros(ROWS, dtype=torch.int32, device="cuda") for _ in range(2)]
    arrays = kvc.page_arrays([kp, vp])
    parents = torch.arange(ROWS, dtype=torch.int32, device="cuda")
    grow = torch.ones(ROWS, dtype=torch.int32, device="cuda")
    missing = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.zeros(ROWS, dtype=torch.int32, device="cuda")
    qkv = torch.zeros(ROWS, HQ + 2 * HKV, D, dtype=torch.bfloat16, device="cuda")
    positions = torch.zeros(3, ROWS, dtype=torch.int32, device="cuda")
    q_rot = torch.zeros(ROWS, HQ, D, dtype=torch.bfloat16, device="cuda")
    own, cross = torch.zeros_like(q_rot), torch.zeros_like(q_rot)
    inv_freq, axis = [0.7 ** i for i in range(24)], [i // 8 for i in range(24)]
    rope = kvc.rope_desc(inv_freq, axis)
    ws = torch.empty(max(kvc.kvc_reserve_plan(ROWS, pages), 16), dtype=torch.uint8, device="cuda")
    max_ctx = WIDTH * P
    dec = torch.empty(max(16, kvc.kvc_decode_plan(ROWS, HQ, kvc.pool_desc(kp), max_ctx)[2]),
                      dtype=torch.uint8, device="cuda")
    crs = torch.empty(max(16, kvc.kvc_cross_plan(SOURCES, ROWS, HQ, kvc.pool_desc(src_pool), BEAMS,
                                                 256)[2]), dtype=torch.uint8, device="cuda")

    def step(old, new):
        kvc.kvc_fork(tables[new], lens[new], parents, tables[old], lens[old], refs, P)
        kvc.kvc_truncate(tables[old], lens[old], None, refs, P)
        kvc.kvc_reserve(tables[new], lens[new], grow, refs, missing, P, arrays, workspace=ws)
        kvc.kvc_slot_mapping(slots, tables[new], lens[new], None, P)
        kvc.kvc_rope_store(q_rot, kp, vp, qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:],
                           positions, slots, rope)
        kvc.kvc_decode(own, q_rot, kp, vp, tables[new], lens[new], max_ctx, workspace=dec)
        kvc.kvc_cross(cross, q_rot, src_pool, src_v, src_table, q_indptr, src_lens, BEAMS, 256,
                      workspace=crs)

    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(i, 1 - i)
        graphs.append(g)

    beams = [[] for _ in range(ROWS)]           # (key, value) of every position, in 64 bits
    for n in range(STEPS):
        # beams of one source continue any of its beams
        p = np.concatenate([s * BEAMS + rng.integers(0, BEAMS, BEAMS) for s in range(SOURCES)])
        if n == 0:
            p[:] = np.arange(ROWS)
        bits = normal_bf16(ss.spawn(1)[0], (ROWS, HQ + 2 * HKV, D))
        pos = np.stack([np.full(ROWS, n), rng.integers(0, 50, ROWS), rng.integers(0, 50, ROWS)])
        parents.copy_(i32_tensor(p, "cuda"))
        qkv.copy_(bf16_tensor(bits, "cuda"))
        positions.copy_(i32_tensor(pos, "cuda"))
        graphs[n % 2].replay()
        torch.cuda.synchronize()
        x = f32_from_bf16(bits).astype(np.float64)
        y = _bf16(orope.rotate(x[:, :HQ + HKV], pos, inv_freq, axis, adjacent=False))
        beams = [list(beams[i]) for i in p]
        for r in range(ROWS):
            beams[r].append((y[r, HQ:], x[r, HQ + HKV:]))
        assert missing.item() == 0 and lens[1 - n % 2].tolist() == [n + 1] * ROWS
        want = np.stack([_softmax_attend(y[r, :HQ], np.stack([k for k, _ in b]),
                                         np.stack([v for _, v in b])) for r, b in enumerate(beams)])
        assert_attention_close(own.float().cpu().numpy().astype(np.float64), want, f"own, step {n}")
        want = np.stack([_softmax_attend(y[r, :HQ], *states[r // BEAMS]) for r in range(ROWS)])
        assert_attention_close(cross.float().cpu().numpy().astype(np.float64), want, f"cross, step {n}")
    # pages are shared and given back: as many in use as the beams' own positions take
    table = tables[STEPS % 2].cpu().numpy()
    held = {int(x) for row in table for x in row[:-(-STEPS // P)]}
    assert int((refs > 0).sum()) == len(held) and int(refs.sum()) == ROWS * -(-STEPS // P)
    # closed up, the same attention
    where = torch.zeros(pages, dtype=torch.int32, device="cuda")
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    cws = torch.empty(kvc.kvc_compact_plan(pages), dtype=torch.uint8, device="cuda")
    i = STEPS % 2
    kvc.kvc_compact(tables[i], lens[i], refs, where, live, P, arrays, workspace=cws)
    again = torch.zeros_like(own)
    kvc.kvc_decode(again, q_rot, kp, vp, tables[i], lens[i], max_ctx, workspace=dec)
    assert live.item() == len(held) and torch.equal(again, own)
    assert int(tables[i].max()) < len(held)
    assert kvc.kvc_device_errors() == 0
