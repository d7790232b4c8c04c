"""kvc_rope and kvc_rope_store on the GPU against the definition in 64 bits.

Bound: a result is rounded once to bf16 (2^-8 of its value) from fp32 terms whose cosines and sines are
off by at most 2^-21 each (2^-25 half turns in the argument, pi 2^-25 < 2^-23; two units of sincospif,
2^-22; the angle's 64-bit fraction, below 2^-23 for positions up to 2^20 as for all others but for 2^-53
of position * inv_freq), with two further fp32 roundings: 2^-20 (|x0| + |x1|) covers those."""
import numpy as np
import pytest
import torch

import pagedattention_kvc_store_gb300 as kvc
from oracle import oracle
from oracle import rope as orope
from workloads import BF16_NAN, f32_from_bf16, normal_bf16
from workloads.device import bf16_bits_of, bf16_tensor, i32_tensor

pytestmark = pytest.mark.gpu


def _inputs(seed, T, Hq, Hkv, D, rotary, axes, far, low=0):
    ss = np.random.SeedSequence(seed)
    qkv = normal_bf16(ss.spawn(1)[0], (T, Hq + 2 * Hkv, D))
    rng = np.random.default_rng(seed)
    positions = rng.integers(low, far, size=(axes, T)).astype(np.int32)
    n = rotary // 2
    inv_freq = [10000.0 ** (-i / n) for i in range(n)]
    axis = [i * axes // n for i in range(n)]
    return qkv, positions, inv_freq, axis


def _check(got_bits, x_bits, positions, inv_freq, axis, adjacent, what):
    x = f32_from_bf16(x_bits).astype(np.float64)
    got = f32_from_bf16(got_bits).astype(np.float64)
    ref = orope.rotate(x, positions, inv_freq, axis, adjacent)
    bound = 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * orope.magnitude(x, len(inv_freq), adjacent)
    over = np.abs(got - ref) > bound
    assert not over.any(), f"{what}: {over.sum()} values past the bound, first {np.argwhere(over)[0]}"
    rest = 2 * len(inv_freq)
    assert np.array_equal(got_bits[..., rest:], x_bits[..., rest:]), f"{what}: dims that do not turn"


@pytest.mark.parametrize("T,Hq,Hkv,D,P,layout,rotary,pairing,axes", [
    (1, 4, 2, 64, 16, "nhd", 64, "halves", 1),
    (64, 32, 8, 128, 16, "nhd", 128, "halves", 3),
    (77, 8, 8, 128, 64, "hnd", 64, "adjacent", 2),
    (133, 5, 5, 64, 32, "hnd", 48, "halves", 3),
    (29, 24, 3, 128, 16, "nhd", 16, "adjacent", 4),
    (1030, 8, 1, 64, 64, "nhd", 16, "halves", 8),
    (3, 64, 8, 128, 32, "hnd", 112, "halves", 2),
])
def test_rope_store(T, Hq, Hkv, D, P, layout, rotary, pairing, axes):
    qkv, positions, inv_freq, axis = _inputs(T * 7 + D, T, Hq, Hkv, D, rotary, axes, 131072)
    qkv[0, -1, :3] = [0x7FC1, 0xFF81, 0x8000]      # a value's NaN payloads and -0 go through
    rng = np.random.default_rng(T)
    pages = -(-T // P) + 2
    slots = rng.permutation(pages * P)[:T].astype(np.int32)
    slots[2::7] = -1
    shape = (pages, P, Hkv, D) if layout == "nhd" else (pages, Hkv, P, D)
    kp = np.full(shape, BF16_NAN, dtype=np.uint16)
    kd, vd = bf16_tensor(kp, "cuda"), bf16_tensor(kp, "cuda")
    d = bf16_tensor(qkv, "cuda")
    rope = kvc.rope_desc(inv_freq, axis, pairing=pairing, num_axes=axes)
    q_out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    k_out = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
    pos = i32_tensor(positions, "cuda")
    q, k, v = d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:]
    kvc.kvc_rope_store(q_out, kd, vd, q, k, v, pos, i32_tensor(slots, "cuda"), rope, layout=layout)
    _check(bf16_bits_of(q_out), qkv[:, :Hq], positions, inv_freq, axis, pairing == "adjacent", "q")
    # the rows of kvc_rope have the same bits, and the store is kvc_store's
    q2 = torch.empty_like(q_out)
    kvc.kvc_rope(q2, k_out, q, k, pos, rope)
    assert torch.equal(q2, q_out)
    rows = bf16_bits_of(k_out)
    _check(rows, qkv[:, Hq:Hq + Hkv], positions, inv_freq, axis, pairing == "adjacent", "k")
    vp = kp.copy()
    oracle.store(kp, vp, rows, np.ascontiguousarray(qkv[:, Hq + Hkv:]), slots, layout=layout)
    assert np.array_equal(bf16_bits_of(kd), kp) and np.array_equal(bf16_bits_of(vd), vp)
    assert np.array_equal(bf16_bits_of(d), qkv)     # inputs untouched
    assert kvc.kvc_device_errors() == 0
    # in place, in the projection's output itself
    kvc.kvc_rope(q, k, q, k, pos, rope)
    now = bf16_bits_of(d)
    assert np.array_equal(now[:, :Hq], bf16_bits_of(q_out))
    assert np.array_equal(now[:, Hq:Hq + Hkv], rows)
    assert np.array_equal(now[:, Hq + Hkv:], qkv[:, Hq + Hkv:])


@pytest.mark.parametrize("low,far", [(-131072, 0), (2 ** 31 - 50, 2 ** 31 - 1), (-2 ** 31, -2 ** 31 + 40)])
def test_far_and_negative_positions(low, far):
    """The oracle's own angle is off by 2^-53 of itself (2^-22 at 2^31), as the call's: 2^-20 more."""
    T, H, D = 50, 3, 64
    x, positions, inv_freq, axis = _inputs(5, T, H, 0, D, 64, 2, far, low)
    d = bf16_tensor(x, "cuda")
    out = torch.empty_like(d)
    kvc.kvc_rope(None, out, None, d, i32_tensor(positions, "cuda"), kvc.rope_desc(inv_freq, axis))
    f = f32_from_bf16(x).astype(np.float64)
    ref = orope.rotate(f, positions, inv_freq, axis, False)
    got = f32_from_bf16(bf16_bits_of(out)).astype(np.float64)
    bound = 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * orope.magnitude(f, 32, False)
    assert (np.abs(got - ref) <= bound).all()


def test_position_zero_changes_nothing_and_quarter_turns_are_exact():
    x = normal_bf16(np.random.SeedSequence(1), (6, 2, 64))
    d = bf16_tensor(x, "cuda")
    out = torch.empty_like(d)
    kvc.kvc_rope(out, None, d, None, torch.zeros(6, dtype=torch.int32, device="cuda"),
                 kvc.rope_desc([1.0] * 32))
    assert torch.equal(out, d)
    # inverse: position -p after p, to two roundings of the result
    p = torch.arange(6, dtype=torch.int32, device="cuda") * 1000
    rope = kvc.rope_desc([-(0.9 ** i) for i in range(32)])
    back = torch.empty_like(d)
    kvc.kvc_rope(out, None, d, None, p, rope)
    kvc.kvc_rope(back, None, out, None, -p, rope)
    pair = orope.magnitude(f32_from_bf16(x).astype(np.float64), 32, False)
    err = np.abs(f32_from_bf16(bf16_bits_of(back)).astype(np.float64) - f32_from_bf16(x))
    assert (err <= 2.0 ** -8 * 1.01 * (2 * pair)).all()


def test_slots_past_the_pool_are_skipped_and_flagged():
    T, H, D, P = 5, 2, 64, 16
    x, positions, inv_freq, axis = _inputs(9, T, H, H, D, 64, 1, 100)
    d = bf16_tensor(x, "cuda")
    kd = torch.zeros(2, P, H, D, dtype=torch.bfloat16, device="cuda")
    vd = kd.clone()
    q_out = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([3, 2 * P, -1, 31, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    kvc.kvc_device_errors()
    kvc.kvc_rope_store(q_out, kd, vd, d[:, :H], d[:, H:2 * H], d[:, 2 * H:], i32_tensor(positions, "cuda"),
                       slots, kvc.rope_desc(inv_freq, axis))
    assert kvc.kvc_device_errors() == 1 << 6
    written = vd.flatten(0, 1).abs().sum((1, 2)) > 0
    assert torch.nonzero(written)[:, 0].tolist() == [3, 31]
    _check(bf16_bits_of(q_out), x[:, :H], positions, inv_freq, axis, False, "q")


def test_captured_step_follows_its_positions_and_slots():
    T, Hq, H, D, P = 9, 4, 2, 64, 16
    x, positions, inv_freq, axis = _inputs(13, T, Hq, H, D, 64, 2, 1000)
    d, pos = bf16_tensor(x, "cuda"), i32_tensor(positions, "cuda")
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    kd = torch.zeros(3, P, H, D, dtype=torch.bfloat16, device="cuda")
    vd, q_out = kd.clone(), torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    rope = kvc.rope_desc(inv_freq, axis)

    def step():
        kvc.kvc_rope_store(q_out, kd, vd, d[:, :Hq], d[:, Hq:Hq + H], d[:, Hq + H:], pos, slots, rope)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    del rope                                   # its arrays are read during the call only
    positions = positions[:, ::-1].copy()
    pos.copy_(i32_tensor(positions, "cuda"))
    slots.add_(P)
    kd.zero_(), vd.zero_()
    graph.replay()
    torch.cuda.synchronize()
    _check(bf16_bits_of(q_out), x[:, :Hq], positions, inv_freq, axis, False, "q")
    _check(bf16_bits_of(kd.flatten(0, 1)[P:P + T]), x[:, Hq:Hq + H], positions, inv_freq, axis, False, "k")
    assert kd[0].abs().sum() == 0
