"""Attention weights and eviction on the GPU against oracle/evict.py.

Weights (fp32).  A score is a sum of D exact products in fp32 (tensor-core accumulation may truncate:
2^-23 each) and two roundings: off by at most d = (D + 8) 2^-23 scale Q K, Q the largest sum of |q|
of a row and K the largest |k|.  The weight exp(x - lse) moves by 2 d relatively (its own score's
error and the sum's), by 2^-24 (|x| + |lse|) / ln 2 each for the roundings of x, lse and their
difference, and by 2^-20 for 2^x, the logarithm and the sums; accumulating a step adds 2^-24.
Their sum bounds every weight; the errors are independent, so the norm of all of them together is
held to 1 / sqrt(D) of it.
Eviction moves bits: everything is equal."""
import math

import numpy as np
import pytest
import torch

import pagedattention_kvc_store_gb300 as kvc
from oracle import evict, int4
from workloads import build_case, config_case
from workloads.device import bf16_bits_of, bf16_tensor, i32_tensor

pytestmark = pytest.mark.gpu


def decode_case(seed, P, H, G, D, ctx, **kw):
    return build_case(seed, name="weights", page_size=P, q_heads=H * G, kv_heads=H, head_dim=D,
                      context_lens=lambda rng: ctx(rng) if callable(ctx) else np.asarray(ctx),
                      q_lens=lambda c: np.ones_like(c), **kw)


def full_pools(case, layout="nhd"):
    """The case's pools with the new tokens stored: K and V bits."""
    from oracle import oracle
    kp, vp = case.k_pool.copy(), case.v_pool.copy()
    oracle.store(kp, vp, case.k_new, case.v_new,
                 oracle.slot_mapping(case.block_table, case.context_lens, case.q_indptr,
                                     case.page_size))
    if layout == "hnd":
        kp, vp = (np.ascontiguousarray(x.transpose(0, 2, 1, 3)) for x in (kp, vp))
    return kp, vp


class Run:
    def __init__(self, case, layout="nhd", stride=None, rows=None, num_rows=None):
        self.case, self.layout = case, layout
        self.kp, self.vp = full_pools(case, layout)
        self.k, self.v = bf16_tensor(self.kp, "cuda"), bf16_tensor(self.vp, "cuda")
        self.table = i32_tensor(case.block_table, "cuda")
        self.ctx = i32_tensor(case.context_lens, "cuda")
        self.pool = kvc.pool_desc(self.k, layout)
        self.stride = stride or case.max_ctx
        self.max_ctx = case.max_ctx
        self.rows = rows
        self.drows = None if rows is None else i32_tensor(rows, "cuda")
        self.weights = torch.zeros(num_rows or case.num_seqs, case.kv_heads, self.stride,
                                   device="cuda")
        self.q = bf16_tensor(case.q, "cuda")

    def decode(self, splits=0, ctx=None, dtype=torch.bfloat16, scale=0.0, stream=None):
        c = self.case
        out = torch.full(self.q.shape, float("nan"), dtype=dtype, device="cuda")
        n = kvc.kvc_decode_weights_plan(c.num_seqs, c.q_heads, self.pool, self.max_ctx, splits)[2]
        self.work = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")
        kvc.kvc_decode_weights(out, self.weights, self.q, self.k, self.v, self.table,
                               self.ctx if ctx is None else i32_tensor(ctx, "cuda"), self.max_ctx,
                               scale=scale, num_splits=splits, workspace=self.work,
                               weight_rows=self.drows, layout=self.layout, stream=stream)
        return out

    def plain_decode(self, splits=0, ctx=None, dtype=torch.bfloat16, scale=0.0):
        c = self.case
        out = torch.full(self.q.shape, float("nan"), dtype=dtype, device="cuda")
        n = kvc.kvc_decode_plan(c.num_seqs, c.q_heads, self.pool, self.max_ctx, splits)[2]
        work = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        kvc.kvc_decode(out, self.q, self.k, self.v, self.table,
                       self.ctx if ctx is None else i32_tensor(ctx, "cuda"), self.max_ctx,
                       scale=scale, num_splits=splits, workspace=work, layout=self.layout)
        return out

    def relative_bound(self, scale=None, steps=1):
        c = self.case
        scale = scale or 1 / math.sqrt(c.head_dim)
        q = np.abs(int4.bf16_value(c.q)).astype(np.float64)
        K = np.nanmax(np.abs(int4.bf16_value(self.kp)))
        qk = scale * q.sum(-1).max() * K
        # |x| and |lse| are at most the norms' product and the logarithm of the context more
        X = scale * np.sqrt((q ** 2).sum(-1).max() * c.head_dim) * K + math.log(c.max_ctx + 1)
        rho = 2 * (c.head_dim + 8) * 2.0 ** -23 * qk + 6 * 2.0 ** -24 * X / math.log(2) + 2.0 ** -20
        return rho + steps * 2.0 ** -24

    def check(self, ref_rows, steps=1, scale=None):
        got = self.weights.double().cpu().numpy()
        rho = self.relative_bound(scale, steps)
        err = np.abs(got - ref_rows)
        assert np.isfinite(got).all()
        assert (err <= rho * ref_rows + 1e-37).all(), (err / (ref_rows + 1e-30)).max()
        assert np.linalg.norm(err) <= rho / math.sqrt(self.case.head_dim) * np.linalg.norm(ref_rows)


def rows_of(run, per_seq, into=None):
    ref = np.zeros(tuple(run.weights.shape)) if into is None else into
    for s, w in enumerate(per_seq):
        row = s if run.rows is None else run.rows[s]
        if row >= 0:
            ref[row, :, :w.shape[1]] += w
    return ref


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("P,H,G,D", [(16, 2, 1, 128), (32, 3, 2, 64), (64, 2, 4, 128), (16, 1, 8, 64)])
def test_weights_ragged(P, H, G, D, layout):
    case = decode_case(11 + G, P, H, G, D, lambda rng: rng.integers(1, 1500, size=9))
    run = Run(case, layout, stride=case.max_ctx + 3)
    per_seq = evict.weights(case.q, run.kp, case.block_table, case.context_lens, layout=layout)
    for splits in (0, 1, 3, 20):
        run.weights.zero_()
        out = run.decode(splits)
        assert torch.equal(out, run.plain_decode(splits)), "the output is kvc_decode's"
        run.check(rows_of(run, per_seq))
    torch.cuda.synchronize()
    assert kvc.kvc_device_errors() == 0


def test_weights_of_the_batched_workload_accumulate():
    case = config_case(2, num_seqs=10)
    run = Run(case)
    ctx = [case.context_lens - 2, case.context_lens - 1, case.context_lens]
    ref = np.zeros(tuple(run.weights.shape))
    for n in ctx:
        run.decode(ctx=n)
        rows_of(run, evict.weights(case.q, run.kp, case.block_table, n), ref)
    run.check(ref, steps=3)
    sums = run.weights.double().sum(-1).cpu().numpy()
    assert np.abs(sums - 3 * 4).max() <= 12 * run.relative_bound(steps=3)


def test_short_and_empty_contexts_and_rows():
    """Contexts from 0; rows given out of order, one left out; nothing else in the array moves."""
    ctx = np.array([0, 1, 2, 63, 64, 65, 0, 200])
    case = decode_case(5, 16, 2, 4, 64, np.maximum(ctx, 1))
    rows = np.array([3, 9, 0, -1, 7, 2, 5, 8])
    run = Run(case, rows=rows, num_rows=10, stride=256)
    run.weights.fill_(0.25)
    out = run.decode(ctx=ctx)
    assert torch.equal(out, run.plain_decode(ctx=ctx))
    assert not out[0].any() and not out[6].any()
    ref = np.full(tuple(run.weights.shape), 0.25)
    rows_of(run, evict.weights(case.q, run.kp, case.block_table, ctx), ref)
    got = run.weights.double().cpu().numpy()
    assert np.abs(got - ref).max() <= 4.25 * run.relative_bound()
    untouched = np.ones(ref.shape, bool)
    for s, n in enumerate(ctx):
        if rows[s] >= 0:
            untouched[rows[s], :, :n] = False
    assert (got[untouched] == 0.25).all()
    assert kvc.kvc_device_errors() == 0


def test_rows_past_the_array_are_flagged():
    case = decode_case(6, 16, 2, 2, 64, [40, 50])
    run = Run(case, rows=np.array([0, 2]), num_rows=2)
    run.decode()
    assert kvc.kvc_device_errors() == 1 << 6
    assert not run.weights[1].any()


def test_contexts_past_max_ctx_are_flagged():
    """The scores of the launch hold max_ctx positions (here a chunk of 256): weights past it stay as
    they are, in rows that could hold them."""
    case = decode_case(9, 16, 2, 2, 64, [90, 700])
    run = Run(case, stride=800)
    run.weights.fill_(0.5)
    run.max_ctx = 200
    out = run.decode()
    assert kvc.kvc_device_errors() == 1 << 7
    assert torch.equal(out, run.plain_decode())
    assert (run.weights[1, :, 200:] == 0.5).all() and (run.weights[0, :, 90:] == 0.5).all()
    got = run.weights[0, :, :90].double().cpu().numpy() - 0.5
    ref = evict.weights(case.q[:1], run.kp, case.block_table[:1], np.array([90]))[0]
    assert np.abs(got - ref).max() <= 2.5 * run.relative_bound()


def test_a_custom_scale_and_sharp_rows():
    """Scores over a range of about 200: weights down to exact zeros."""
    case = decode_case(7, 16, 2, 2, 128, [700, 33])
    run = Run(case)
    ref = evict.weights(case.q, run.kp, case.block_table, case.context_lens, scale=1.5)
    run.decode(scale=1.5)
    got = run.weights.double().cpu().numpy()
    want = rows_of(run, ref)
    rho = run.relative_bound(scale=1.5)
    assert (np.abs(got - want) <= rho * want + 1e-37).all()


def test_weights_repeat_and_share_pages():
    """Two sequences over the same pages, each with its own row; the same bits every time."""
    case = decode_case(8, 16, 2, 4, 128, [300, 300, 900])
    case.block_table[1] = case.block_table[0]
    run = Run(case)
    run.q[1] = run.q[0]
    run.decode()
    first = run.weights.clone()
    assert torch.equal(first[0], first[1])
    run.weights.zero_()
    run.decode()
    assert torch.equal(run.weights, first)


def state(case, budget, seed, earlier=True, values="normal"):
    """Weights and positions as a serving loop would hold them: sequences over the budget have
    been evicted before."""
    rng = np.random.default_rng(seed)
    S, H, L = case.num_seqs, case.kv_heads, case.max_ctx + 5
    w = np.exp(1.5 * rng.standard_normal((S, H, L))).astype(np.float32)
    if values == "ties":
        w = rng.integers(0, 3, (S, H, L)).astype(np.float32)
    elif values == "zero":
        w[:] = 0
    elif values == "odd":
        w = rng.choice(np.array([0.0, -0.0, np.nan, np.inf, -np.inf, 1e-40, -2.0, 3.0], np.float32),
                       (S, H, L))
    pos = np.tile(np.arange(L, dtype=np.int32), (S, H, 1))
    for s, n in enumerate(case.context_lens):
        kept = min(budget, int(n) // 2)
        if earlier and kept and n > budget:
            gone = int(rng.integers(1, 1000))
            for h in range(H):
                pos[s, h, kept:] += gone
                pos[s, h, :kept] = rng.permutation(kept + gone)[:kept]
    return w, pos


def run_evict(case, budget, recent, w, pos, layout="nhd", rows=None, in_place=False, ctx=None,
              max_ctx=None):
    kp, vp = full_pools(case, layout)
    ctx = case.context_lens if ctx is None else ctx
    max_ctx = max_ctx or case.max_ctx
    k, v = bf16_tensor(kp, "cuda"), bf16_tensor(vp, "cuda")
    dw, dp = torch.from_numpy(w).cuda(), torch.from_numpy(pos).cuda()
    ow = dw if in_place else torch.full_like(dw, 77.0)
    op = dp if in_place else torch.full_like(dp, -7)
    new = torch.full((len(ctx),), -1, dtype=torch.int32, device="cuda")
    pool = kvc.pool_desc(k, layout)
    n = kvc.kvc_evict_plan(len(ctx), pool, max_ctx, budget)
    work = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    kvc.kvc_evict(k, v, ow, op, new, dw, dp, i32_tensor(case.block_table, "cuda"),
                  i32_tensor(ctx, "cuda"), max_ctx, budget, recent, workspace=work,
                  weight_rows=None if rows is None else i32_tensor(rows, "cuda"), layout=layout)
    torch.cuda.synchronize()
    rw, rp = w.copy(), pos.copy()
    lens = evict.evict(kp, vp, rw, rp, case.block_table, ctx, budget, recent, rows, layout)
    assert np.array_equal(new.cpu().numpy(), lens)
    assert np.array_equal(bf16_bits_of(k), kp), "K"
    assert np.array_equal(bf16_bits_of(v), vp), "V"
    gw, gp = ow.cpu().numpy(), op.cpu().numpy()
    if not in_place:   # rows and slots that the call does not write
        for s in range(len(ctx)):
            row = s if rows is None else rows[s]
            if row >= 0:
                assert (gw[row, :, ctx[s]:] == 77.0).all()
                gw[row, :, ctx[s]:] = rw[row, :, ctx[s]:]
        written = np.zeros(len(w), bool)
        written[[r for r in (range(len(ctx)) if rows is None else rows) if r >= 0]] = True
        assert (gw[~written] == 77.0).all() and (gp[~written] == -7).all()
        gw[~written], gp[~written] = rw[~written], rp[~written]
    assert np.array_equal(gp, rp), "positions"
    assert np.array_equal(gw.view(np.uint32), rw.view(np.uint32)), "weights"
    return lens


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("P,H,D,budget,recent", [
    (16, 2, 64, 100, 16), (32, 3, 128, 1, 1), (64, 1, 128, 333, 0), (16, 5, 64, 512, 512),
    (16, 2, 128, 600, 31)])
def test_evict_ragged(P, H, D, budget, recent, layout):
    case = decode_case(60 + P + budget, P, H, 1, D, lambda rng: np.concatenate(
        [[1, budget, budget + 1], rng.integers(1, 900, size=8)]))
    for in_place in (False, True):
        w, pos = state(case, budget, budget)
        run_evict(case, budget, recent, w, pos, layout, in_place=in_place)
    assert kvc.kvc_device_errors() == 0


@pytest.mark.parametrize("values", ["ties", "zero", "odd"])
def test_evict_equal_and_odd_weights(values):
    case = decode_case(80, 16, 2, 1, 64, [500, 33, 700, 256])
    w, pos = state(case, 100, 3, values=values)
    run_evict(case, 100, 10, w, pos)
    run_evict(case, 100, 100, w, pos)
    run_evict(case, 499, 0, w, pos)


def test_evict_rows_and_empty_sequences():
    case = decode_case(81, 16, 2, 1, 64, [300, 20, 40, 100, 64])
    w, pos = state(decode_case(81, 16, 2, 1, 64, [300] * 9), 50, 4, earlier=False)
    rows = np.array([8, 1, -1, 0, 5])
    ctx = np.array([300, 0, 40, 100, 64])
    lens = run_evict(case, 50, 7, w, pos, rows=rows, ctx=ctx)
    assert lens.tolist() == [50, 0, 40, 50, 50]


@pytest.mark.parametrize("S,n,budget", [(1, 5000, 1000), (2, 20000, 7777), (1, 70000, 3), (40, 3000, 2990)])
def test_evict_clusters(S, n, budget):
    """Few long rows: several CTAs share one; ranks run on across them."""
    case = decode_case(82 + S, 64, 1, 1, 64, lambda rng: rng.integers(n // 2, n + 1, size=S))
    w, pos = state(case, budget, 5)
    run_evict(case, budget, min(budget, 200), w, pos)
    w, pos = state(case, budget, 6, values="ties")
    run_evict(case, budget, 1, w, pos, in_place=True)


def test_evict_clusters_in_quick_succession():
    """Rows shared by 8 CTAs, 300 calls with nothing waited for in between: CTAs of a cluster drift
    apart by whole passes, and every call gives the same bits."""
    S, H, L, budget = 4, 2, 40000, 9000
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    w = torch.exp(torch.randn(S, H, L, generator=gen, device="cuda"))
    pos = torch.arange(L, dtype=torch.int32, device="cuda").repeat(S, H, 1)
    pages = S * (L // 64)
    k = torch.randn(pages, 64, H, 64, generator=gen, device="cuda").bfloat16()
    v = k.clone()
    table = torch.randperm(pages, generator=gen, device="cuda").int().view(S, -1)
    ctx = torch.tensor([L, L - 777, L // 2 + 1, L], dtype=torch.int32, device="cuda")
    pool = kvc.pool_desc(k)
    n = kvc.kvc_evict_plan(S, pool, L, budget)
    outs = []
    for i in range(300):
        kk, vv = (k.clone(), v.clone()) if i in (0, 299) else (k, v)
        o = [torch.zeros_like(w), torch.zeros_like(pos),
             torch.zeros(S, dtype=torch.int32, device="cuda")]
        work = torch.empty(n, dtype=torch.uint8, device="cuda")
        if i == 299:
            kk, vv = first_k.clone(), first_v.clone()
        kvc.kvc_evict(kk, vv, *o, w, pos, table, ctx, L, budget, 100, workspace=work)
        if i == 0:
            first_k, first_v = kk, vv
        outs.append(o)
    torch.cuda.synchronize()
    assert torch.equal(kk, first_k) and torch.equal(vv, first_v)   # moving again moves the same
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))
    assert kvc.kvc_device_errors() == 0


@pytest.mark.parametrize("n", [400000, 1200000])
def test_evict_more_slots_than_the_cache_of_keys(n):
    """Rows over 8 CTAs that hold more slots than these keep in shared memory."""
    P = 64
    S = 1
    pages = n // P + 1
    rng = np.random.default_rng(9)
    kp = rng.integers(0, 2 ** 16, (pages, P, 1, 64), dtype=np.uint16) & 0xBFFF
    table = rng.permutation(pages)[None].astype(np.int32)
    w = np.exp(rng.standard_normal((S, 1, n))).astype(np.float32)
    pos = np.arange(n, dtype=np.int32)[None, None].copy()
    budget, recent = 5000, 100
    k, v = bf16_tensor(kp, "cuda"), bf16_tensor(kp, "cuda")
    dw, dp = torch.from_numpy(w).cuda(), torch.from_numpy(pos).cuda()
    new = torch.zeros(1, dtype=torch.int32, device="cuda")
    need = kvc.kvc_evict_plan(1, kvc.pool_desc(k), n, budget)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    kvc.kvc_evict(k, v, dw, dp, new, dw, dp, i32_tensor(table, "cuda"),
                  i32_tensor(np.array([n]), "cuda"), n, budget, recent, workspace=work)
    torch.cuda.synchronize()
    ref = kp.copy()
    lens = evict.evict(ref, ref.copy(), w, pos, table, np.array([n]), budget, recent)
    assert new.item() == lens[0]
    assert np.array_equal(bf16_bits_of(k), ref) and np.array_equal(bf16_bits_of(v), ref)
    assert np.array_equal(dw.cpu().numpy(), w) and np.array_equal(dp.cpu().numpy(), pos)


def test_evict_flags_bad_pages_rows_and_lengths():
    case = decode_case(83, 16, 2, 1, 64, [100, 100])
    w, pos = state(case, 30, 7, earlier=False)
    table = case.block_table.copy()
    table[0, 5] = case.k_pool.shape[0]     # slots 80 .. 95: kept ones there cannot move
    kp, vp = full_pools(case)
    k, v = bf16_tensor(kp, "cuda"), bf16_tensor(vp, "cuda")
    dw, dp = torch.from_numpy(w).cuda(), torch.from_numpy(pos).cuda()
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    work = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")

    def call(t, ctx, max_ctx, rows=None):
        kvc.kvc_evict(k, v, dw.clone(), dp.clone(), new, dw, dp, i32_tensor(t, "cuda"),
                      i32_tensor(ctx, "cuda"), max_ctx, 30, 20, workspace=work,
                      weight_rows=None if rows is None else i32_tensor(rows, "cuda"))
        return kvc.kvc_device_errors()

    assert call(table, case.context_lens, 100) == 1 << 10
    want, wv = kp.copy(), vp.copy()
    lens = evict.evict(want, wv, w.copy(), pos.copy(), case.block_table[1:], case.context_lens[1:],
                       30, 20)
    mine = case.block_table[1][:7]
    # (sequence 1 with the weights of row 1)
    want, wv = kp.copy(), vp.copy()
    evict.evict(want, wv, w[1:].copy(), pos[1:].copy(), case.block_table[1:], case.context_lens[1:],
                30, 20)
    assert np.array_equal(bf16_bits_of(k)[mine], want[mine]) and lens[0] == 30
    assert call(case.block_table, np.array([100, 101]), 100) == 1 << 7
    assert call(case.block_table, case.context_lens, 100, np.array([0, 2])) == 1 << 6
    assert new.cpu().tolist() == [30, 100]


def test_rows_whose_last_slot_is_not_the_newest_are_flagged():
    """An eviction straight after another one, and the same with a token in between."""
    case = decode_case(84, 16, 2, 1, 64, [100, 90])
    w, pos = state(case, 30, 8, earlier=False)
    w[:, :, 29] = 1e6                    # stays, so the last slot of 30 is an old one
    k, v = (bf16_tensor(x, "cuda") for x in full_pools(case))
    dw, dp = torch.from_numpy(w).cuda(), torch.from_numpy(pos).cuda()
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    work = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    rows = torch.tensor([0, 1], dtype=torch.int32, device="cuda")

    def call(ctx, budget):
        kvc.kvc_evict(k, v, dw, dp, new, dw, dp, i32_tensor(case.block_table, "cuda"),
                      i32_tensor(np.array(ctx), "cuda"), 100, budget, 5, workspace=work,
                      weight_rows=rows)
        return kvc.kvc_device_errors()

    assert call([100, 90], 30) == 0
    assert (dp[:, :, 29] == 29).all()
    assert call([31, 31], 30) == 0
    before = dp.clone()
    rows[1] = -1
    assert call([30, 31], 20) == 1 << 13
    assert torch.equal(dp[1], before[1])


def test_evictions_on_two_streams():
    """Different sequences of the same pools, a workspace each."""
    case = decode_case(85, 16, 3, 1, 128, lambda rng: rng.integers(1500, 3000, size=8))
    budget, recent = 1000, 100
    w, pos = state(case, budget, 9)
    kp, vp = full_pools(case)
    k, v = bf16_tensor(kp, "cuda"), bf16_tensor(vp, "cuda")
    dw, dp = torch.from_numpy(w).cuda(), torch.from_numpy(pos).cuda()
    table, ctx = i32_tensor(case.block_table, "cuda"), i32_tensor(case.context_lens, "cuda")
    new = torch.zeros(8, dtype=torch.int32, device="cuda")
    need = kvc.kvc_evict_plan(4, kvc.pool_desc(k), case.max_ctx, budget)
    streams = [torch.cuda.Stream() for _ in "ab"]
    works = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in "ab"]
    torch.cuda.synchronize()
    for i, s in enumerate(streams):
        at = slice(4 * i, 4 * i + 4)
        kvc.kvc_evict(k, v, dw[at], dp[at], new[at], dw[at], dp[at], table[at], ctx[at],
                      case.max_ctx, budget, recent, workspace=works[i], stream=s)
    torch.cuda.synchronize()
    lens = evict.evict(kp, vp, w, pos, case.block_table, case.context_lens, budget, recent)
    assert np.array_equal(new.cpu().numpy(), lens)
    assert np.array_equal(bf16_bits_of(k), kp) and np.array_equal(bf16_bits_of(v), vp)
    assert np.array_equal(dp.cpu().numpy(), pos)
    assert np.array_equal(dw.cpu().numpy().view(np.uint32), w.view(np.uint32))
    assert kvc.kvc_device_errors() == 0


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_serving_loop_with_eviction(layout):
    """Store, decode with weights and, when the cache is full, evict: several rounds in a captured
    graph per step, against the oracle doing the same in 64 bits on its own copy.  Positions are
    checked to stay distinct, newest last."""
    S, H, G, D, P, width = 2, 2, 4, 64, 16, 4
    budget, recent, cap = 40, 8, 64
    rng = np.random.default_rng(12)
    table = rng.permutation(S * width).reshape(S, width).astype(np.int32)
    shape = (S * width, P, H, D) if layout == "nhd" else (S * width, H, P, D)
    kp, vp = np.zeros(shape, np.uint16), np.zeros(shape, np.uint16)
    k, v = bf16_tensor(kp, "cuda"), bf16_tensor(vp, "cuda")
    w = torch.zeros(S, H, cap, device="cuda")
    pos = torch.arange(cap, dtype=torch.int32, device="cuda").repeat(S, H, 1)
    rpos = pos.cpu().numpy().copy()
    dt = i32_tensor(table, "cuda")
    ctx, slot, new = (torch.zeros(S, dtype=torch.int32, device="cuda") for _ in range(3))
    q = torch.zeros(S, H * G, D, dtype=torch.bfloat16, device="cuda")
    kn, vn = (torch.zeros(S, H, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    out = torch.empty(q.shape, device="cuda")
    pool = kvc.pool_desc(k, layout)
    wd = torch.empty(kvc.kvc_decode_weights_plan(S, H * G, pool, cap)[2], dtype=torch.uint8,
                     device="cuda")
    we = torch.empty(kvc.kvc_evict_plan(S, pool, cap, budget), dtype=torch.uint8, device="cuda")

    def step():
        kvc.kvc_slot_mapping(slot, dt, ctx, None, P)
        kvc.kvc_store(k, v, kn, vn, slot, layout=layout)
        kvc.kvc_decode_weights(out, w, q, k, v, dt, ctx, cap, workspace=wd, layout=layout)

    def cut():
        kvc.kvc_evict(k, v, w, pos, new, w, pos, dt, ctx, cap, budget, recent, workspace=we,
                      layout=layout)
        ctx.copy_(new)

    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        step()
        cut()
    torch.cuda.synchronize()
    w.zero_()
    pos.copy_(torch.arange(cap, dtype=torch.int32, device="cuda").expand_as(pos))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, f in zip(graphs, (step, cut)):
        with torch.cuda.graph(g):
            f()
    k.zero_(), v.zero_(), w.zero_()
    pos.copy_(torch.arange(cap, dtype=torch.int32, device="cuda").expand_as(pos))
    lens = np.zeros(S, np.int64)
    ref_w = np.zeros((S, H, cap))
    for t in range(150):
        lens = lens + 1
        if t == 100:
            lens[1] = 1   # sequence 1 begins anew
            w[1].zero_()
            pos[1] = torch.arange(cap, dtype=torch.int32, device="cuda")
            ref_w[1], rpos[1] = 0, np.arange(cap)
        new_kv = [torch.from_numpy(rng.standard_normal((S, H, D))).bfloat16() for _ in "kv"]
        qn = torch.from_numpy(2 * rng.standard_normal(tuple(q.shape))).bfloat16()
        kn.copy_(new_kv[0]), vn.copy_(new_kv[1]), q.copy_(qn)
        ctx.copy_(i32_tensor(lens, "cuda"))
        graphs[0].replay()
        p = lens - 1
        for pl, x in zip((kp, vp), new_kv):
            at = pl if layout == "nhd" else pl.transpose(0, 2, 1, 3)
            at[table[np.arange(S), p // P], p % P] = bf16_bits_of(x)
        for s, x in enumerate(evict.weights(bf16_bits_of(qn), kp, table, lens, layout=layout)):
            ref_w[s, :, :lens[s]] += x
        got = w.double().cpu().numpy()
        assert np.abs(got - ref_w).max() <= 2e-3 * max(1.0, ref_w.max())
        if lens.max() == cap:
            w32 = w.cpu().numpy()        # the device's own weights decide, so ties of rounding agree
            graphs[1].replay()
            lens = evict.evict(kp, vp, w32, rpos, table, lens, budget, recent, layout=layout).astype(np.int64)
            assert np.array_equal(pos.cpu().numpy(), rpos)
            assert np.array_equal(w.cpu().numpy(), w32)
            assert np.array_equal(bf16_bits_of(k), kp) and np.array_equal(bf16_bits_of(v), vp)
            assert ctx.cpu().tolist() == lens.tolist()
            ref_w = w32.astype(np.float64)
            for s in range(S):
                for h in range(H):
                    held = rpos[s, h, :lens[s]]
                    assert len(set(held)) == len(held)
    torch.cuda.synchronize()
    assert kvc.kvc_device_errors() == 0
