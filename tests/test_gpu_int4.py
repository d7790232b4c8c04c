"""4-bit pages on the GPU against oracle/int4.py.

Slots that hold no position keep random codes and NaN parameters, so a masked position that
reached a sum would show.  Store: codes and parameters bit for bit.  Decode, fp32 output, against fp64
attention over what the pages hold.  Its roundings, with R = the largest 15 scale and V the largest
|value| of the case's V, Q the largest sum of |q| over a row, K the largest |value| + 15 scale of K:
  * a probability times a value scale is rounded to fp16, half a step 2^-11 of the product: the
    output is off by at most 2^-11 R (the products' weighted mean);
  * a score is a sum of D products and a few terms in fp32 (tensor-core accumulation may truncate:
    2^-23 each): off by at most d = (D + 8) 2^-23 scale Q K, and the output by 2 d V;
  * 2^x and the division: below 2^-20 V.
Their sum bounds the largest error; the fp16 roundings are independent, so the mean error is held
to 2^-12 R, half of what a single one may give.  bf16 output: plus half a bf16 step, 2^-8 |x|."""
import math

import numpy as np
import pytest
import torch

import pagedattention_kvc_store_gb300 as kvc
from oracle import int4, oracle
from workloads import build_case, config_case
from workloads.device import bf16_bits_of, bf16_tensor, i32_tensor

pytestmark = pytest.mark.gpu


def u16_tensor(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def to_layout(codes, layout):
    return codes if layout == "nhd" else np.ascontiguousarray(codes.transpose(0, 2, 1, 3))


def empty_pools(pages, P, H, D, layout, seed=0):
    """Pools of random codes and NaN parameters."""
    rng = np.random.default_rng(seed)
    codes = [to_layout(rng.integers(0, 256, (pages, P, H, D // 2), dtype=np.uint8), layout)
             for _ in range(2)]
    params = [np.full((pages, H, P, D // 64, 2), int4.NAN_BITS, np.uint16) for _ in range(2)]
    return codes + params


def device_pools(pools):
    return [torch.from_numpy(pools[0]).cuda(), torch.from_numpy(pools[1]).cuda(),
            u16_tensor(pools[2]), u16_tensor(pools[3])]


def assert_pools_equal(dev, ref):
    for i, name in enumerate(("K codes", "V codes", "K parameters", "V parameters")):
        got = dev[i].cpu().numpy() if i < 2 else bf16_bits_of(dev[i])
        assert np.array_equal(got, ref[i]), f"{name} differ"


def filled(case, layout="nhd"):
    """The case's cached positions (the new tokens' too) in 4-bit pages, by the oracle."""
    pages, P, H, D = case.k_pool.shape
    pools = empty_pools(pages, P, H, D, layout)
    slots = np.concatenate([
        case.block_table[s][np.arange(n) // P].astype(np.int64) * P + np.arange(n) % P
        for s, n in enumerate(case.context_lens - 1)])
    flat = [x.reshape(pages * P, H, D)[slots] for x in (case.k_pool, case.v_pool)]
    int4.store(*pools, *flat, slots, layout)
    int4.store(*pools, case.k_new, case.v_new,
               oracle.slot_mapping(case.block_table, case.context_lens, case.q_indptr, P), layout)
    return pools


def run_decode(q, pools, table, ctx, max_ctx, num_splits=0, dtype=torch.float32, layout="nhd",
               scale=0.0):
    dev = pools if isinstance(pools[0], torch.Tensor) else device_pools(pools)
    q = q if isinstance(q, torch.Tensor) else bf16_tensor(q, "cuda")
    out = torch.full(q.shape, float("nan"), dtype=dtype, device="cuda")
    pool = kvc.int4_pool_desc(dev[0], layout)
    _, _, ws = kvc.kvc_decode_int4_plan(q.shape[0], q.shape[1], pool, max_ctx, num_splits)
    work = torch.full((max(ws, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    kvc.kvc_decode_int4(out, q, *dev, i32_tensor(table, "cuda"), i32_tensor(ctx, "cuda"), max_ctx,
                        scale=scale, num_splits=num_splits, workspace=work, layout=layout)
    torch.cuda.synchronize()
    assert kvc.kvc_device_errors() == 0
    return out.double().cpu().numpy()


def bounds(case, pools, scale=None):
    D = case.head_dim
    kp, vp = (int4.bf16_value(p).astype(np.float64) for p in pools[2:])
    R = np.nanmax(15 * vp[..., 0])
    V = np.nanmax(np.abs(vp[..., 1]) + 15 * vp[..., 0])
    K = np.nanmax(np.abs(kp[..., 1]) + 15 * kp[..., 0])
    Q = np.abs(int4.bf16_value(case.q)).sum(-1).max()
    d = (D + 8) * 2.0 ** -23 * (scale or 1 / math.sqrt(D)) * Q * K
    return 2.0 ** -11 * R + 2 * d * V + 2.0 ** -20 * V, 2.0 ** -12 * R


def check(case, got, ref, pools, what, bf16=False, scale=None):
    worst, mean = bounds(case, pools, scale)
    assert np.isfinite(got).all(), what
    err = np.abs(got - ref) - (2.0 ** -8 * np.abs(ref) if bf16 else 0.0)
    assert err.max() <= worst, f"{what}: {err.max():.3e} > {worst:.3e}"
    assert np.maximum(err, 0).mean() <= mean, f"{what}: mean {err.mean():.3e} > {mean:.3e}"


def ragged(seed, P, Hkv, G, D, ctx):
    return build_case(seed, name="int4", page_size=P, q_heads=Hkv * G, kv_heads=Hkv, head_dim=D,
                      context_lens=lambda rng: np.asarray(ctx) if not callable(ctx) else ctx(rng),
                      q_lens=lambda c: np.ones_like(c))


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("P,H,D", [(16, 2, 128), (32, 3, 64), (64, 1, 128), (16, 8, 64)])
def test_store_and_load(P, H, D, layout):
    rng = np.random.default_rng(P + H + D)
    pages, T = 5, 2 * P + 3
    x = [(rng.standard_normal((T, H, D)) * np.exp(2 * rng.standard_normal((T, H, 1)))) for _ in "kv"]
    new = [torch.from_numpy(a).bfloat16().cuda() for a in x]
    new[0][0] = 0.0                          # a vector of zeros
    new[0][1] = 7.0                          # equal values
    new[1][2, :, 3] = float("nan")
    new[1][3, :, D - 1] = float("-inf")
    new[0][4] *= 2.0 ** 120                  # hi - lo past fp32's largest value's half
    new[0][5, :, 0], new[0][5, :, 1] = 3e38, -3e38
    new[1][6] *= 2.0 ** -126                 # subnormal scales
    new[1][7] = torch.arange(D).cuda().bfloat16()   # quotients on ties
    slots = rng.permutation(pages * P)[:T].astype(np.int32)
    slots[9::7] = -1
    pools = empty_pools(pages, P, H, D, layout)
    dev, ds = device_pools(pools), i32_tensor(slots, "cuda")
    kvc.kvc_store_int4(*dev, *new, ds, layout=layout)
    int4.store(*pools, *(bf16_bits_of(t) for t in new), slots, layout)
    torch.cuda.synchronize()
    assert_pools_equal(dev, pools)
    for dtype in (torch.float32, torch.bfloat16):
        out = [torch.full((T, H, D), 9.0, dtype=dtype, device="cuda") for _ in "kv"]
        kvc.kvc_load_int4(*out, *dev, ds, layout=layout)
        torch.cuda.synchronize()
        for o, codes, params in zip(out, pools[:2], pools[2:]):
            ref = int4.load(codes, params, slots, layout)
            with np.errstate(over="ignore"):
                ref = torch.from_numpy(ref.astype(np.float32)).to(dtype).float().numpy()
            assert np.array_equal(o.float().cpu().numpy(), ref, equal_nan=True)
    assert kvc.kvc_device_errors() == 0


def test_store_rounds_every_quotient_as_the_division_does():
    """4 million values whose quotients crowd around ties."""
    rng = np.random.default_rng(8)
    T, H, D = 8192, 4, 128
    x = rng.integers(-300, 300, (T, H, D)) * 2.0 ** rng.integers(-6, 3, (T, H, 1))
    new = torch.from_numpy(x).bfloat16().cuda()
    slots = np.arange(T, dtype=np.int32)
    pools = empty_pools(T // 64, 64, H, D, "nhd")
    dev = device_pools(pools)
    kvc.kvc_store_int4(*dev, new, new, i32_tensor(slots, "cuda"))
    bits = bf16_bits_of(new)
    int4.store(*pools, bits, bits, slots)
    assert_pools_equal(dev, pools)


def test_slots_past_the_pool_are_flagged_and_skipped():
    pools = empty_pools(2, 16, 2, 64, "nhd")
    dev = device_pools(pools)
    x = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([32, -5, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    kvc.kvc_store_int4(*dev, x, x, slots)
    assert kvc.kvc_device_errors() == 1 << 6
    assert_pools_equal(dev, pools)
    out = torch.full((3, 2, 64), 5.0, device="cuda")
    kvc.kvc_load_int4(out, out.clone(), *dev, slots)
    assert kvc.kvc_device_errors() == 1 << 6 and not out.any()


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("H,G,D", [(2, 1, 128), (3, 2, 64), (8, 4, 128), (1, 8, 128), (5, 8, 64)])
def test_decode_ragged(H, G, D, P, layout):
    case = ragged(40 + P + G, P, H, G, D, lambda rng: rng.integers(1, 700, size=13))
    pools = filled(case, layout)
    ref = int4.attention(case.q, *pools, case.block_table, case.context_lens, layout=layout)
    for splits in (1, 3, 0):
        got = run_decode(case.q, pools, case.block_table, case.context_lens, case.max_ctx, splits,
                         layout=layout)
        check(case, got, ref, pools, f"splits={splits}")
    got = run_decode(case.q, pools, case.block_table, case.context_lens, case.max_ctx,
                     dtype=torch.bfloat16, layout=layout)
    check(case, got, ref, pools, "bf16", bf16=True)


@pytest.mark.parametrize("H,G,D,P", [(6, 2, 128, 16), (7, 1, 64, 32), (9, 4, 64, 16), (11, 1, 64, 16),
                                     (12, 2, 128, 64), (16, 1, 128, 16), (10, 8, 64, 32)])
def test_decode_head_counts(H, G, D, P):
    """Numbers of kv heads that one group of warps does not take: several groups share a sequence, or
    leave warps of a CTA idle."""
    case = ragged(140 + H, P, H, G, D, lambda rng: rng.integers(1, 400, size=7))
    layout = "hnd" if H % 2 else "nhd"
    pools = filled(case, layout)
    ref = int4.attention(case.q, *pools, case.block_table, case.context_lens, layout=layout)
    for splits in (0, 1, 2):
        got = run_decode(case.q, pools, case.block_table, case.context_lens, case.max_ctx, splits,
                         layout=layout)
        check(case, got, ref, pools, f"splits={splits}")


def test_more_sequences_than_threads():
    """700 sequences: each thread that cuts the runs counts several."""
    case = ragged(150, 16, 1, 2, 64, lambda rng: rng.integers(1, 200, size=700))
    pools = filled(case)
    ref = int4.attention(case.q, *pools, case.block_table, case.context_lens)
    for splits in (0, 7):
        got = run_decode(case.q, pools, case.block_table, case.context_lens, case.max_ctx, splits)
        check(case, got, ref, pools, f"splits={splits}")


@pytest.mark.parametrize("max_ctx", [100, 129])
def test_contexts_past_max_ctx(max_ctx):
    """max_ctx only sizes the launch: what the block-table row holds is attended all the same."""
    case = ragged(151, 16, 2, 4, 128, [700, 40, 129])
    pools = filled(case)
    ref = int4.attention(case.q, *pools, case.block_table, case.context_lens)
    got = run_decode(case.q, pools, case.block_table, case.context_lens, max_ctx)
    check(case, got, ref, pools, f"max_ctx={max_ctx}")


@pytest.mark.parametrize("D", [64, 128])
def test_every_position_counts_once(D):
    """A query of zeros weighs every position the same, and then no product is rounded (a bf16
    scale is exact in fp16): the output is the mean of V to fp32 accuracy, so one position lost,
    doubled or taken from another sequence would show.  The sum of n terms of at most V carries
    n 2^-23 V / n at worst, here and in the minimum's part."""
    ctx = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 511, 512, 513, 1030, 2500]
    case = ragged(7, 16, 2, 4, D, ctx)
    pools = filled(case)
    q = np.zeros_like(case.q)
    ref = int4.attention(q, *pools, case.block_table, case.context_lens)
    V = bounds(case, pools)[0] * 2 ** 11
    for splits in (0, 1, 2, 5):
        got = run_decode(q, pools, case.block_table, case.context_lens, case.max_ctx, splits)
        assert np.abs(got - ref).max() <= 2.0 ** -20 * V + 2.0 ** -23 * V * max(1, 32)


@pytest.mark.parametrize("splits", [0, 1, 4])
def test_empty_sequences_and_many_short_ones(splits):
    rng = np.random.default_rng(2)
    ctx = rng.integers(1, 90, size=300)
    case = ragged(91, 16, 2, 2, 64, ctx)
    pools = filled(case)
    ctx0 = ctx.copy()
    ctx0[::3] = 0
    ref = int4.attention(case.q, *pools, case.block_table, ctx0)
    got = run_decode(case.q, pools, case.block_table, ctx0, case.max_ctx, splits)
    assert not got[::3].any()
    check(case, got, ref, pools, "empty")
    none = run_decode(case.q, pools, case.block_table, 0 * ctx, case.max_ctx, splits)
    assert not none.any()


def test_values_of_any_exponent():
    """Value scales from 2^-100 to 2^100 in one batch: each row is right in its own measure, and
    a large value appearing late does not lose what came before."""
    case = ragged(17, 16, 2, 2, 128, [200, 200, 200, 333])
    pools = filled(case)
    for s, power in enumerate((-100, 100, 0)):
        for page in case.block_table[s][:13]:
            p = pools[3][page]
            v = int4.bf16_value(p) * np.float32(2.0 ** power)
            pools[3][page] = np.where(p == int4.NAN_BITS, p, int4.bf16_round(np.nan_to_num(v)))
    last = case.block_table[3][20]          # positions 320 .. 332 of sequence 3
    p = pools[3][last]
    grown = int4.bf16_round(np.nan_to_num(int4.bf16_value(p) * np.float32(4096.0)))
    pools[3][last] = np.where(p == int4.NAN_BITS, p, grown)
    ref = int4.attention(case.q, *pools, case.block_table, case.context_lens)
    d = bounds(ragged(17, 16, 2, 2, 128, [200, 200, 200, 333]), filled(case))[0]
    for splits in (1, 0):
        got = run_decode(case.q, pools, case.block_table, case.context_lens, case.max_ctx, splits)
        for s, power in enumerate((-100, 100, 0, 12)):
            assert np.abs(got[s] - ref[s]).max() <= d * 2.0 ** power


def test_query_rows_of_any_size():
    """Rows of one group with very different magnitudes, one of them zero."""
    case = ragged(18, 16, 1, 4, 128, [300, 70])
    q = int4.bf16_value(case.q).copy()
    q[:, 0] *= 2.0 ** -60
    q[:, 1] = 0
    q[:, 2] *= 8
    case.q = int4.bf16_round(q)
    pools = filled(case)
    ref = int4.attention(case.q, *pools, case.block_table, case.context_lens)
    got = run_decode(case.q, pools, case.block_table, case.context_lens, case.max_ctx)
    check(case, got, ref, pools, "query sizes")


def test_a_nan_position_reaches_only_its_rows():
    case = ragged(19, 16, 2, 2, 64, [50, 60])
    pools = filled(case)
    pools[2][case.block_table[0][1], 1, 3] = int4.NAN_BITS   # position 19, kv head 1, K
    for splits in (0, 1):
        out = torch.from_numpy(run_decode(case.q, pools, case.block_table, case.context_lens,
                                          case.max_ctx, splits))
        assert torch.isnan(out[0, 2:]).all()
        assert torch.isfinite(out[0, :2]).all() and torch.isfinite(out[1]).all()


def test_scale_argument_and_batched_workload():
    case = config_case(2, num_seqs=12)
    pools = filled(case)
    for scale in (None, 0.25):
        ref = int4.attention(case.q, *pools, case.block_table, case.context_lens, scale)
        got = run_decode(case.q, pools, case.block_table, case.context_lens, case.max_ctx,
                         scale=scale or 0.0)
        check(case, got, ref, pools, f"scale {scale}", scale=scale)


def test_long_context_few_sequences():
    case = ragged(23, 64, 1, 8, 128, [40001, 3])
    pools = filled(case)
    ref = int4.attention(case.q, *pools, case.block_table, case.context_lens)
    for splits in (0, 9, 100, 300):
        got = run_decode(case.q, pools, case.block_table, case.context_lens, case.max_ctx, splits)
        check(case, got, ref, pools, f"long {splits}")


@pytest.mark.parametrize("D,splits", [(64, 1), (64, 0), (128, 1)])
def test_long_sums_are_rounded_not_cut(D, splits):
    """A query of zeros over 100,000 positions: the output is the mean of V, a small remainder of
    sum(u) scale and the minima.  No probability is rounded (scales are exact in fp16).  A block's
    products are cut at most 4 times, 2^-23 each, and add 2^-21 R to the mean; the sums over blocks and
    the minima's over the positions of a thread (an eighth of all) are rounded, errors that grow with
    the root of their number: 2^-24 sqrt(N / 8) of R and V; the division and the rest 2^-22 V."""
    case = ragged(24, 64, 1, 2, D, [100001])
    pools = filled(case)
    q = np.zeros_like(case.q)
    ref = int4.attention(q, *pools, case.block_table, case.context_lens)
    got = run_decode(q, pools, case.block_table, case.context_lens, case.max_ctx, splits)
    vp = int4.bf16_value(pools[3]).astype(np.float64)
    R, V = np.nanmax(15 * vp[..., 0]), np.nanmax(np.abs(vp[..., 1]))
    rms = np.sqrt(((got - ref) ** 2).mean())
    assert rms <= 2.0 ** -21 * R + 2.0 ** -24 * math.sqrt(100001 / 8) * (R + V) + 2.0 ** -22 * V


def test_the_result_is_the_same_every_time():
    case = ragged(29, 16, 8, 4, 128, lambda rng: rng.integers(1, 3000, size=20))
    pools = device_pools(filled(case))
    runs = [run_decode(case.q, pools, case.block_table, case.context_lens, case.max_ctx)
            for _ in range(3)]
    assert np.array_equal(runs[0], runs[1]) and np.array_equal(runs[0], runs[2])


def test_bad_pages_and_long_contexts_are_flagged():
    """A page id outside the pool is flagged and spoils its own sequence only; a context past its
    block-table row attends over what the row holds."""
    case = ragged(31, 16, 2, 2, 64, [40, 40])
    pools = filled(case)
    table = case.block_table[:, :3].copy()
    good = run_decode(case.q, pools, table, case.context_lens, 48)
    bad = table.copy()
    bad[0, 1] = case.k_pool.shape[0]
    bad[0, 2] = -1
    dev, q = device_pools(pools), bf16_tensor(case.q, "cuda")
    out = torch.empty(q.shape, device="cuda")
    work = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    kvc.kvc_decode_int4(out, q, *dev, i32_tensor(bad, "cuda"), i32_tensor(case.context_lens, "cuda"),
                        48, workspace=work)
    assert kvc.kvc_device_errors() == 1 << 10
    assert np.array_equal(out[1].double().cpu().numpy(), good[1])
    # positions past the row's 48 do not exist: position 40 .. 47 hold NaN parameters here
    kvc.kvc_decode_int4(out, q, *dev, i32_tensor(table[:, :2].copy(), "cuda"),
                        i32_tensor(case.context_lens, "cuda"), 32, workspace=work)
    assert kvc.kvc_device_errors() == 1 << 7
    ref = int4.attention(case.q, *pools, table, np.array([32, 32]))
    assert np.abs(out.double().cpu().numpy() - ref).max() <= bounds(case, pools)[0]


def test_step_in_a_graph_with_growing_contexts_and_pinned_inputs():
    """Slot mapping, store and decode captured once and replayed as the sequences grow; then the
    same step with its small inputs and its output in pinned host memory."""
    case = ragged(37, 16, 2, 4, 128, [30, 61, 1])
    pools = filled(case)
    S, steps = 3, 4
    pages, P, H, D = case.k_pool.shape
    width = 8
    table = np.arange(S * width, dtype=np.int32).reshape(S, width)
    big = empty_pools(S * width, P, H, D, "nhd")
    slots = [table[s][np.arange(n - 1) // P] * P + np.arange(n - 1) % P
             for s, n in enumerate(case.context_lens)]
    rng = np.random.default_rng(1)
    n_old = sum(len(x) for x in slots)
    old = [bf16_bits_of(torch.from_numpy(rng.standard_normal((n_old, H, D))).bfloat16()) for _ in "kv"]
    int4.store(*big, *old, np.concatenate(slots))
    dev = device_pools(big)
    ctx, dt = i32_tensor(case.context_lens, "cuda"), i32_tensor(table, "cuda")
    q = torch.zeros(S, H * 4, D, dtype=torch.bfloat16, device="cuda")
    kn, vn = (torch.zeros(S, H, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    out = torch.empty(q.shape, device="cuda")
    slot = torch.empty(S, dtype=torch.int32, device="cuda")
    pool = kvc.int4_pool_desc(dev[0])
    work = torch.empty(kvc.kvc_decode_int4_plan(S, H * 4, pool, 128)[2], dtype=torch.uint8,
                       device="cuda")

    def step():
        kvc.kvc_slot_mapping(slot, dt, ctx, None, P)
        kvc.kvc_store_int4(*dev, kn, vn, slot)
        kvc.kvc_decode_int4(out, q, *dev, dt, ctx, 128, workspace=work)

    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens = case.context_lens.copy()
    for i in range(steps):
        new = [torch.from_numpy(rng.standard_normal((S, H, D))).bfloat16() for _ in "kv"]
        qn = torch.from_numpy(rng.standard_normal(tuple(q.shape))).bfloat16()
        kn.copy_(new[0]), vn.copy_(new[1]), q.copy_(qn)
        ctx.copy_(i32_tensor(lens, "cuda"))
        graph.replay()
        torch.cuda.synchronize()
        at = table[np.arange(S), (lens - 1) // P] * P + (lens - 1) % P
        int4.store(*big, *(bf16_bits_of(t) for t in new), at)
        ref = int4.attention(bf16_bits_of(qn), *big, table, lens)
        case.q = bf16_bits_of(qn)
        check(case, out.double().cpu().numpy(), ref, big, f"replay {i}")
        lens = lens + 1
    pin = [t.cpu().pin_memory() for t in (q, dt, ctx)]
    pout = torch.empty(q.shape, pin_memory=True)
    kvc.kvc_decode_int4(pout, pin[0], *dev, pin[1], pin[2], 128, workspace=work)
    torch.cuda.synchronize()
    assert torch.equal(pout, out.cpu()) and kvc.kvc_device_errors() == 0


def test_two_streams_with_a_workspace_each():
    cases = [ragged(50 + i, 16, 2, 4, 128, lambda rng: rng.integers(1, 900, size=9)) for i in (0, 1)]
    pools = [filled(c) for c in cases]
    dev = [device_pools(p) for p in pools]
    outs, works, streams = [], [], [torch.cuda.Stream() for _ in cases]
    args = []
    for c, d in zip(cases, dev):
        q = bf16_tensor(c.q, "cuda")
        n = kvc.kvc_decode_int4_plan(c.num_seqs, c.q_heads, kvc.int4_pool_desc(d[0]), c.max_ctx)[2]
        works.append(torch.empty(n, dtype=torch.uint8, device="cuda"))
        outs.append(torch.empty(q.shape, device="cuda"))
        args.append((q, i32_tensor(c.block_table, "cuda"), i32_tensor(c.context_lens, "cuda")))
    torch.cuda.synchronize()
    for _ in range(5):
        for i, c in enumerate(cases):
            q, t, n = args[i]
            kvc.kvc_decode_int4(outs[i], q, *dev[i], t, n, c.max_ctx, workspace=works[i],
                                stream=streams[i])
    torch.cuda.synchronize()
    for c, p, o in zip(cases, pools, outs):
        ref = int4.attention(c.q, *p, c.block_table, c.context_lens)
        check(c, o.double().cpu().numpy(), ref, p, "streams")


def test_load_brings_a_prefix_back_for_append():
    """A cached prefix leaves 4-bit pages for bf16 ones and kvc_append goes on over it: the same
    output, bit for bit, as over bf16 pages holding the values the 4-bit pages stand for."""
    case = build_case(61, name="int4-append", page_size=16, q_heads=8, kv_heads=2, head_dim=128,
                      context_lens=lambda rng: np.array([40, 77]), q_lens=lambda c: np.array([9, 20]))
    pages, P, H, D = case.k_pool.shape
    slots = np.concatenate([case.block_table[s][np.arange(n) // P] * P + np.arange(n) % P
                            for s, n in enumerate(case.context_lens - np.array([9, 20]))])
    pools = empty_pools(pages, P, H, D, "nhd")
    flat = [x.reshape(pages * P, H, D)[slots] for x in (case.k_pool, case.v_pool)]
    int4.store(*pools, *flat, slots)
    dev, ds = device_pools(pools), i32_tensor(slots, "cuda")
    k, v = (torch.empty(len(slots), H, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    kvc.kvc_load_int4(k, v, *dev, ds)
    kp, vp = (torch.zeros(pages, P, H, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    kvc.kvc_store(kp, vp, k, v, ds)
    new = torch.empty(case.num_tokens, dtype=torch.int32, device="cuda")
    bt, ctx = i32_tensor(case.block_table, "cuda"), i32_tensor(case.context_lens, "cuda")
    ind = i32_tensor(case.q_indptr, "cuda")
    kvc.kvc_slot_mapping(new, bt, ctx, ind, P, max_q_len=case.max_q_len)
    kvc.kvc_store(kp, vp, bf16_tensor(case.k_new, "cuda"), bf16_tensor(case.v_new, "cuda"), new)
    out = torch.empty(case.num_tokens, 8, D, device="cuda")
    kvc.kvc_append(out, bf16_tensor(case.q, "cuda"), kp, vp, bt, ind, ctx, case.max_q_len,
                   case.max_ctx)
    ref, _ = oracle.attention(case.q, bf16_bits_of(kp), bf16_bits_of(vp), case.block_table,
                              case.context_lens, case.q_indptr)
    assert np.abs(out.double().cpu().numpy() - ref).max() <= 1e-2
    want = int4.load(pools[0], pools[2], slots).astype(np.float32)
    assert torch.equal(k.cpu(), torch.from_numpy(want).bfloat16())


def test_groups_of_any_exponent():
    """Value scales of a vector's two groups 2^60 apart, either way round: each group of dims is right in
    its own measure, also after one of them grows late."""
    case = ragged(63, 16, 2, 4, 128, [300, 77, 500])
    pools = filled(case)
    powers = np.zeros((case.num_seqs, 2))
    powers[0], powers[1], powers[2] = (30, -30), (-30, 30), (-30, 12)
    for s in range(case.num_seqs):
        for i, page in enumerate(case.block_table[s][:-(-int(case.context_lens[s]) // 16)]):
            p = pools[3][page]
            up = powers[s].copy()
            if s == 2 and i < 20:
                up[1] = 0                    # group 1 of sequence 2 grows at position 320
            v = int4.bf16_value(p) * (2.0 ** up[:, None]).astype(np.float32)
            pools[3][page] = np.where(p == int4.NAN_BITS, p, int4.bf16_round(np.nan_to_num(v)))
    ref = int4.attention(case.q, *pools, case.block_table, case.context_lens)
    same = ragged(63, 16, 2, 4, 128, [300, 77, 500])
    d = bounds(same, filled(same))[0]        # of the pools before they were scaled
    for splits in (1, 0, 3):
        got = run_decode(case.q, pools, case.block_table, case.context_lens, case.max_ctx, splits)
        for s in range(case.num_seqs):
            for g in range(2):
                err = np.abs(got[s] - ref[s])[:, 64 * g:64 * g + 64].max()
                assert err <= d * 2.0 ** powers[s, g], (splits, s, g)


@pytest.mark.parametrize("D", [64, 128])
def test_every_position_counts_once_to_the_derived_bound(D):
    """A query of zeros, so the output is the mean of V; held for every sequence of n positions to what
    its own sums can lose.  V the largest |minimum|, R the largest 15 scale.  No probability and no
    product is rounded (probabilities are 1, a bf16 scale is exact in fp16).
      * minima: a thread adds n / 8 of them one after the other, the j-th sum up to j V is off by half a
        step, 2^-24 j V: n^2 / 128 2^-24 V a thread, n^2 / 16 for the eight, n / 16 2^-24 V of the mean;
        three more sums join the threads: 3 2^-24 V;
      * codes: a block of 64 positions is four products whose sums the tensor cores cut, 2^-23 each:
        2^-21 R of the mean; the n / 64 blocks are added one after the other: n / 128 2^-24 R;
      * joining the pieces: a log-sum-exp up to 8 in base e, rounded three times (2^-21 each, the
        logarithm included), 2^x (2^-22): a weight is off by 2^-19, numerator and sum 2^-18 (V + R);
        the division and the last product are below 2^-22 (V + R).
    A position lost, doubled or of another sequence moves the mean by about |v| / n, above the bound
    for all but the smallest |v| at the longest sequence."""
    ctx = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 511, 512, 513, 1030, 2500]
    case = ragged(7, 16, 2, 4, D, ctx)
    pools = filled(case)
    q = np.zeros_like(case.q)
    ref = int4.attention(q, *pools, case.block_table, case.context_lens)
    vp = int4.bf16_value(pools[3]).astype(np.float64)
    V, R = np.nanmax(np.abs(vp[..., 1])), np.nanmax(15 * vp[..., 0])
    n = case.context_lens.astype(np.float64)
    bound = ((n / 16 + 3) * V + n / 128 * R) * 2.0 ** -24 + 2.0 ** -21 * R
    for splits in (0, 1, 2, 5):
        got = run_decode(q, pools, case.block_table, case.context_lens, case.max_ctx, splits)
        joined = (2.0 ** -18 + 2.0 ** -22) * (V + R)
        err = np.abs(got - ref).max((1, 2))
        assert (err <= bound + joined).all(), (splits, (err / (bound + joined)).max())


def test_append_over_a_loaded_prefix_is_append_over_its_values():
    """kvc_append over pages that kvc_load_int4 filled, and over pages that the oracle's values (rounded
    to bf16) were put into without the GPU: the same bits."""
    case = build_case(61, name="int4-append", page_size=16, q_heads=8, kv_heads=2, head_dim=128,
                      context_lens=lambda rng: np.array([40, 77]), q_lens=lambda c: np.array([9, 20]))
    pages, P, H, D = case.k_pool.shape
    slots = np.concatenate([case.block_table[s][np.arange(n) // P] * P + np.arange(n) % P
                            for s, n in enumerate(case.context_lens - np.array([9, 20]))])
    pools = empty_pools(pages, P, H, D, "nhd")
    flat = [x.reshape(pages * P, H, D)[slots] for x in (case.k_pool, case.v_pool)]
    int4.store(*pools, *flat, slots)
    dev, ds = device_pools(pools), i32_tensor(slots, "cuda")
    loaded = [torch.empty(len(slots), H, D, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    kvc.kvc_load_int4(*loaded, *dev, ds)
    first = [torch.zeros(pages, P, H, D, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    kvc.kvc_store(*first, *loaded, ds)
    second = []
    for codes, params in zip(pools[:2], pools[2:]):
        bits = np.zeros((pages * P, H, D), np.uint16)
        bits[slots] = int4.bf16_round(int4.load(codes, params, slots).astype(np.float32))
        second.append(bf16_tensor(bits.reshape(pages, P, H, D), "cuda"))
    bt, ctx = i32_tensor(case.block_table, "cuda"), i32_tensor(case.context_lens, "cuda")
    ind = i32_tensor(case.q_indptr, "cuda")
    new = torch.empty(case.num_tokens, dtype=torch.int32, device="cuda")
    kvc.kvc_slot_mapping(new, bt, ctx, ind, P, max_q_len=case.max_q_len)
    outs = []
    for kp, vp in (first, second):
        kvc.kvc_store(kp, vp, bf16_tensor(case.k_new, "cuda"), bf16_tensor(case.v_new, "cuda"), new)
        outs.append(torch.full((case.num_tokens, 8, D), float("nan"), device="cuda"))
        kvc.kvc_append(outs[-1], bf16_tensor(case.q, "cuda"), kp, vp, bt, ind, ctx, case.max_q_len,
                       case.max_ctx)
    assert torch.isfinite(outs[0]).all() and torch.equal(*outs)
    assert all(torch.equal(a, b) for a, b in zip(first, second))
