"""kvc_cross on the GPU against plain softmax attention in 64 bits.

Bound of an fp32 output, for values |v| <= vmax and scores from fp32 sums: probabilities are rounded to
bf16 (2^-8 of themselves) and normalised by the sum of the rounded ones, so the mean over them is off by
at most 2 * 2^-8 * sum(w |v|) / sum(w) <= 2^-7 * sum(w |v|); the scores' own error, 2^-24 * sqrt(D) of
sum |q k| scale (below 2^-15 here), and ex2's 2^-22 disappear in that.  bf16 outputs: 2^-8 of themselves
more.  A log-sum-exp is off by the scores' error and fp32's of the sum: 2^-14 + 2^-20 |lse|."""
import math

import numpy as np
import pytest
import torch

import pagedattention_kvc_store_gb300 as kvc
from oracle import oracle
from workloads import BF16_NAN, PageAllocator, f32_from_bf16, normal_bf16
from workloads.device import bf16_tensor, i32_tensor
from workloads.gen import round_up

pytestmark = pytest.mark.gpu


class Case:
    """Sources in scattered pages, NaN everywhere else; queries for each."""

    def __init__(self, lens, q_lens, Hkv, G, D, P, layout="nhd", seed=0, sharp=1.0, pad=0):
        self.lens, self.q_lens, self.Hkv, self.G, self.D, self.P = lens, q_lens, Hkv, G, D, P
        self.layout = layout
        ss = np.random.SeedSequence(seed + 77)
        pages = sum(-(-n // P) for n in lens) + 3
        a = PageAllocator(pages, P, np.random.default_rng(seed).permutation(pages))
        for s, n in enumerate(lens):
            a.reserve(s, n)
        width = round_up(max(1, max(len(a.pages[s]) for s in range(len(lens)))), 16)
        self.table = a.table(range(len(lens)), width)
        self.T = sum(q_lens)
        self.k = np.full((pages, P, Hkv, D), BF16_NAN, dtype=np.uint16)
        self.v = self.k.copy()
        for s, n in enumerate(lens):
            p = np.arange(n)
            at = self.table[s][p // P], p % P
            self.k[at] = normal_bf16(ss.spawn(1)[0], (n, Hkv, D))
            self.v[at] = normal_bf16(ss.spawn(1)[0], (n, Hkv, D))
        q = f32_from_bf16(normal_bf16(ss.spawn(1)[0], (self.T + pad, Hkv * G, D))) * sharp
        self.q = torch.from_numpy(q).bfloat16()
        self.indptr = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)

    def run(self, dtype=torch.float32, splits=0, lse=True, scale=0.0, q=None, max_q=None, max_src=None):
        pool = (lambda b: oracle.nhd_to_hnd(b)) if self.layout == "hnd" else (lambda b: b)
        kd, vd = bf16_tensor(pool(self.k), "cuda"), bf16_tensor(pool(self.v), "cuda")
        q = (self.q if q is None else q).cuda()
        out = torch.full(q.shape, 7.25, dtype=dtype, device="cuda")
        logs = torch.full(q.shape[:2], 7.25, device="cuda") if lse else None
        max_q = max(self.q_lens) if max_q is None else max_q
        max_src = max(self.lens) if max_src is None else max_src
        desc = kvc.pool_desc(kd, self.layout)
        n, chunk, ws = kvc.kvc_cross_plan(len(self.lens), q.shape[0], q.shape[1], desc, max_q, max_src,
                                          splits)
        work = torch.full((max(ws, 16),), 0xFF, dtype=torch.uint8, device="cuda")
        kvc.kvc_cross(out, q, kd, vd, i32_tensor(self.table, "cuda"), i32_tensor(self.indptr, "cuda"),
                      i32_tensor(np.array(self.lens), "cuda"), max_q, max_src, lse_out=logs,
                      scale=scale, num_splits=splits, workspace=work, layout=self.layout)
        torch.cuda.synchronize()
        return out, logs

    def exact(self, scale=0.0, q=None):
        """(out, lse, sum of w |v|) in 64 bits."""
        q = (self.q if q is None else q).float().numpy().astype(np.float64)
        scale = scale or 1.0 / math.sqrt(self.D)
        out, lse, weighed = np.zeros(q.shape), np.full(q.shape[:2], -np.inf), np.zeros(q.shape)
        for s, n in enumerate(self.lens):
            t = slice(self.indptr[s], self.indptr[s + 1])
            if n == 0 or t.start == t.stop:
                continue
            p = np.arange(n)
            at = self.table[s][p // self.P], p % self.P
            k, v = (f32_from_bf16(x[at]).astype(np.float64) for x in (self.k, self.v))
            for h in range(self.Hkv * self.G):
                x = q[t, h] @ k[:, h // self.G].T * scale
                m = x.max(1, keepdims=True)
                e = np.exp(x - m)
                w = e / e.sum(1, keepdims=True)
                lse[t, h] = m[:, 0] + np.log(e.sum(1))
                out[t, h] = w @ v[:, h // self.G]
                weighed[t, h] = w @ np.abs(v[:, h // self.G])
        return out, lse, weighed


def check(c, got, logs, scale=0.0, bf16=False):
    out, lse, weighed = c.exact(scale)
    x = got.float().cpu().numpy().astype(np.float64)
    T = c.T
    assert np.isfinite(x[:T]).all()
    bound = 2.0 ** -7 * weighed + (2.0 ** -8 * np.abs(out) if bf16 else 0.0) + 1e-6
    over = np.abs(x - out)[:T] > bound[:T]
    assert not over.any(), f"{over.sum()} values past the bound, first {np.argwhere(over)[0]}"
    if logs is not None:
        y = logs.cpu().numpy().astype(np.float64)[:T]
        e = lse[:T]
        assert np.array_equal(np.isinf(y), np.isinf(e))
        f = np.isfinite(e)
        assert (np.abs(y[f] - e[f]) <= 2.0 ** -14 + 2.0 ** -20 * np.abs(e[f])).all()


RAGGED = [1, 15, 16, 17, 127, 128, 129, 300, 0, 1000]


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("Hkv,G,D,P,layout", [(2, 4, 128, 16, "nhd"), (3, 1, 64, 32, "hnd"),
                                              (1, 8, 128, 64, "hnd"), (4, 2, 64, 64, "nhd")])
def test_ragged_sources_and_queries(Hkv, G, D, P, layout, splits):
    q_lens = [3, 0, 1, 40, 70, 129, 64, 5, 4, 33]
    c = Case(RAGGED, q_lens, Hkv, G, D, P, layout, seed=Hkv)
    out, lse = c.run(splits=splits)
    check(c, out, lse)
    assert kvc.kvc_device_errors() == 0
    # a source without positions: zeros and -inf
    none = slice(c.indptr[8], c.indptr[9])
    assert (out[none] == 0).all() and torch.isinf(lse[none]).all()
    b, _ = c.run(torch.bfloat16, splits, lse=False)
    check(c, b, None, bf16=True)


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("Hkv,G,D,P,layout,most", [(2, 4, 128, 16, "nhd", 4), (3, 1, 64, 32, "hnd", 9),
                                                   (1, 8, 128, 64, "hnd", 4), (4, 2, 64, 16, "nhd", 16),
                                                   (2, 8, 64, 64, "nhd", 3), (2, 2, 128, 32, "hnd", 17)])
def test_ragged_sources_and_few_queries(Hkv, G, D, P, layout, most, splits):
    """Up to 16, up to 32 and just over 32 rows a kv head."""
    q_lens = [most, 0, 1, 2, most - 1, 1, 3, most, 2, most]
    c = Case(RAGGED, q_lens, Hkv, G, D, P, layout, seed=most, pad=2)
    out, lse = c.run(splits=splits)
    check(c, out, lse)
    assert (out[c.T:] == 7.25).all() and (lse[c.T:] == 7.25).all()
    assert kvc.kvc_device_errors() == 0
    none = slice(c.indptr[8], c.indptr[9])
    assert (out[none] == 0).all() and torch.isinf(lse[none]).all()
    b, _ = c.run(torch.bfloat16, splits, lse=False)
    check(c, b, None, bf16=True)


@pytest.mark.parametrize("splits", [0, 1, 2, 9])
@pytest.mark.parametrize("rows", [1, 4, 8, 10])
def test_beams_over_long_sources(rows, splits):
    c = Case([5000, 2049, 4096], [rows] * 3, 8, 4, 128, 16, seed=rows)
    out, lse = c.run(splits=splits)
    check(c, out, lse)


def test_prompts_of_many_tiles():
    c = Case([700, 1500], [600, 259], 2, 4, 128, 64)
    out, lse = c.run()
    check(c, out, lse)
    one, _ = c.run(splits=1, lse=False)
    check(c, one, None)


@pytest.mark.parametrize("splits", [1, 4])
def test_one_token_is_the_decode(splits):
    """A source of n positions and one query: kvc_decode over it, to both calls' rounding."""
    c = Case([1, 64, 777, 1025], [1] * 4, 2, 4, 64, 16)
    out, _ = c.run(splits=splits)
    kd, vd = bf16_tensor(c.k, "cuda"), bf16_tensor(c.v, "cuda")
    ref = torch.empty_like(out)
    kvc.kvc_decode(ref, c.q.cuda(), kd, vd, i32_tensor(c.table, "cuda"),
                   i32_tensor(np.array(c.lens), "cuda"), 1025, num_splits=1)
    _, _, weighed = c.exact()
    assert (np.abs((out - ref).cpu().numpy()) <= 2.0 ** -6 * weighed + 1e-6).all()


def test_rows_of_no_source_are_left_alone():
    c = Case([40, 300], [2, 3], 2, 2, 64, 16, pad=6)
    c.indptr = np.array([2, 4, 7], dtype=np.int32)
    for splits in (1, 2):
        out, lse = c.run(splits=splits)
        rest = [0, 1, 7, 8, 9, 10]
        assert (out[rest] == 7.25).all() and (lse[rest] == 7.25).all()
        want, logs, weighed = c.exact()
        err = np.abs(out.cpu().numpy() - want)[2:7]
        assert (err <= 2.0 ** -7 * weighed[2:7] + 1e-6).all()


@pytest.mark.parametrize("splits", [1, 3])
def test_large_scores_and_a_growing_maximum(splits):
    """Sharp softmaxes whose maximum moves from block to block by more than the lazy rescale's 2^8."""
    c = Case([900], [5], 2, 2, 128, 16, sharp=8.0)
    p = np.arange(900)
    at = c.table[0][p // 16], p % 16
    k = f32_from_bf16(c.k[at]) * np.linspace(0.1, 3.0, 900, dtype=np.float32)[:, None, None]
    c.k[at] = torch.from_numpy(k).bfloat16().view(torch.int16).numpy().view(np.uint16)
    out, lse = c.run(splits=splits)
    # scores reach 300: fp32 sums of 128 products are off by up to 2^-24 * 128 * sum |q k| scale, 2^-7
    # at the very most of a score of 2^9; measured against that
    want, logs, weighed = c.exact()
    q = c.q.float().numpy().astype(np.float64)
    reach = np.abs(q).max() * np.abs(k).max() * 128 / math.sqrt(128) * 2.0 ** -20
    assert (np.abs(out.cpu().numpy() - want) <= (2.0 ** -7 + 2 * reach) * weighed + 1e-6).all()
    assert (np.abs(lse.cpu().numpy() - logs) <= reach + 2.0 ** -14 + 2.0 ** -20 * np.abs(logs)).all()


def test_scale_and_lse_join_two_sources():
    """Two halves of a source, joined by kvc_merge, are the whole."""
    c = Case([256, 256], [4, 4], 2, 4, 64, 16)
    c.q[4:] = c.q[:4]
    out, lse = c.run(scale=0.3)
    whole = Case([512], [4], 2, 4, 64, 16)
    whole.q[:] = c.q[:4]
    p = np.arange(256)
    for s in range(2):
        src = c.table[s][p // 16], p % 16
        dst = whole.table[0][(p + 256 * s) // 16], p % 16
        whole.k[dst], whole.v[dst] = c.k[src], c.v[src]
    want, logs, weighed = whole.exact(scale=0.3)
    parts = torch.stack([out[:4], out[4:]], 2).flatten(0, 1)
    parts_lse = torch.stack([lse[:4], lse[4:]], 2).flatten(0, 1)
    joined, joined_lse = torch.empty(32, 64, device="cuda"), torch.empty(32, device="cuda")
    kvc.kvc_merge(joined, parts, parts_lse, joined_lse)
    err = np.abs(joined.cpu().numpy().reshape(4, 8, 64) - want)
    assert (err <= 2.0 ** -7 * weighed + 2.0 ** -12).all()
    assert (np.abs(joined_lse.cpu().numpy().reshape(4, 8) - logs) <= 2.0 ** -12).all()


@pytest.mark.parametrize("splits", [1, 2])
def test_nan_and_inf_stay_with_their_rows(splits):
    c = Case([400, 200], [3, 3], 2, 2, 64, 16)
    q = c.q.clone()
    q[1, 2, 5] = math.nan
    out, lse = c.run(splits=splits, q=q)
    bad = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
    bad[1, 2] = True
    assert torch.isnan(out[bad]).all() and torch.isfinite(out[~bad]).all()
    assert torch.isnan(lse[bad]).all() and torch.isfinite(lse[~bad]).all()
    # a NaN value reaches its kv head's rows of its source, in its dim
    c.v[c.table[1][0], 3, 1, 9] = BF16_NAN
    out, _ = c.run(splits=splits)
    hit = torch.isnan(out)
    assert hit[3:, 2:, 9].all() and hit.sum() == 3 * 2


def test_lengths_past_the_bounds_are_flagged():
    c = Case([300, 40], [3, 2], 1, 2, 64, 16)
    kvc.kvc_device_errors()
    out, _ = c.run(max_src=256, splits=1)
    assert kvc.kvc_device_errors() == 1 << 7
    c.lens = [256, 40]
    check(c, out, None)
    c.run(max_q=2, splits=1)
    assert kvc.kvc_device_errors() == 1 << 7


@pytest.mark.parametrize("most", [4, 100])
def test_captured_call_follows_its_lengths_and_two_graphs_with_workspaces_of_their_own(most):
    c = Case([1500, 800], [most, most], 2, 4, 128, 16)
    kd, vd = bf16_tensor(c.k, "cuda"), bf16_tensor(c.v, "cuda")
    q, table = c.q.cuda(), i32_tensor(c.table, "cuda")
    indptr, lens = i32_tensor(c.indptr, "cuda"), i32_tensor(np.array(c.lens), "cuda")
    pool = kvc.pool_desc(kd)
    graphs = []
    for splits in (3, 5):
        ws = kvc.kvc_cross_plan(2, c.T, 8, pool, most, 1500, splits)[2]
        work = torch.empty(ws, dtype=torch.uint8, device="cuda")
        out = torch.zeros(c.T, 8, 128, device="cuda")
        call = lambda: kvc.kvc_cross(out, q, kd, vd, table, indptr, lens, most, 1500,   # noqa: E731
                                     num_splits=splits, workspace=work)
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append((g, out, work))
    c.lens = [700, 800]
    lens.copy_(i32_tensor(np.array(c.lens), "cuda"))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for (g, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, out, _ in graphs:
        check(c, out, None)


@pytest.mark.parametrize("most", [4, 200])
def test_sources_without_positions_alone(most):
    """Nothing to attend to anywhere: zeros and -inf, both kernels, one and several splits."""
    c = Case([0, 0], [most, 1], 2, 4, 128, 16)
    for splits, src in ((1, 0), (1, 256), (2, 256)):
        c.table = np.zeros((2, 16), dtype=np.int32)
        out, lse = c.run(splits=splits, max_src=src)
        assert (out == 0).all() and torch.isinf(lse).all() and (lse < 0).all()


@pytest.mark.parametrize("most", [4, 200])
def test_two_calls_at_once_on_two_streams(most):
    """Each with its workspace; results as one after the other, bit for bit."""
    cases = [Case([1200, 700], [most, most // 2], 2, 4, 128, 16, seed=s) for s in range(2)]
    alone = [c.run(splits=3) for c in cases]
    args = []
    for c in cases:
        kd, vd = bf16_tensor(c.k, "cuda"), bf16_tensor(c.v, "cuda")
        ws = kvc.kvc_cross_plan(2, c.T, 8, kvc.pool_desc(kd), most, 1200, 3)[2]
        args.append((torch.empty(c.T, 8, 128, device="cuda"), c.q.cuda(), kd, vd,
                     i32_tensor(c.table, "cuda"), i32_tensor(c.indptr, "cuda"),
                     i32_tensor(np.array(c.lens), "cuda"), most, 1200,
                     torch.empty(ws, dtype=torch.uint8, device="cuda")))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for a, s in zip(args, streams):
            kvc.kvc_cross(*a[:9], num_splits=3, workspace=a[9], stream=s)
    torch.cuda.synchronize()
    for a, (out, _) in zip(args, alone):
        assert torch.equal(a[0], out)


@pytest.mark.parametrize("most", [4, 200])
def test_results_do_not_depend_on_where_pages_lie(most):
    a, b = (Case([500, 300], [most, 3], 2, 4, 64, 32, seed=1) for _ in range(2))
    perm = np.random.default_rng(5).permutation(b.k.shape[0])
    b.k[perm], b.v[perm], b.table = a.k, a.v, perm[a.table].astype(np.int32)
    for splits in (1, 2):
        assert all(torch.equal(x, y) for x, y in zip(a.run(splits=splits), b.run(splits=splits)))


# q_len * G rows of a kv head: 100 in one tile, 400 in two pairs of tiles (the last without its second), 340
# with a last tile of 84 rows
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("D,P,layout", [(64, 32, "hnd"), (128, 16, "nhd")])
@pytest.mark.parametrize("most,sharp,top", [(50, 8.0, 3.0), (200, 8.0, 3.0), (170, 30.0, 1.0)])
def test_a_growing_maximum_under_many_rows(most, sharp, top, D, P, layout, splits):
    """Maxima that move by more than 2^8 from block to block, at different blocks for different rows, while
    products of earlier blocks are in flight."""
    c = Case([900, 129], [most, most // 2], 2, 2, D, P, layout, sharp=sharp)
    k_max = 0.0
    for s, n in enumerate(c.lens):
        p = np.arange(n)
        at = c.table[s][p // P], p % P
        k = f32_from_bf16(c.k[at]) * np.linspace(0.1, top, n, dtype=np.float32)[:, None, None]
        c.k[at] = torch.from_numpy(k).bfloat16().view(torch.int16).numpy().view(np.uint16)
        k_max = max(k_max, np.abs(k).max())
    out, lse = c.run(splits=splits)
    want, logs, weighed = c.exact()
    # fp32 sums of D products are off by up to D 2^-24 sum |q k| scale <= D 2^-24 D q k scale (2^-10 D q k scale
    # 2^-20 with D <= 128: below `reach`)
    reach = np.abs(c.q.float().numpy()).max() * k_max * D / math.sqrt(D) * 2.0 ** -20
    assert np.isfinite(out.cpu().numpy()).all()
    assert (np.abs(out.cpu().numpy() - want) <= (2.0 ** -7 + 2 * reach) * weighed + 1e-6).all()
    assert (np.abs(lse.cpu().numpy() - logs) <= reach + 2.0 ** -14 + 2.0 ** -20 * np.abs(logs)).all()
    assert kvc.kvc_device_errors() == 0


@pytest.mark.parametrize("splits", [1, 4])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("most", [3, 60, 200])
def test_scores_of_minus_infinity_before_the_first_finite_one(most, D, splits):
    """Positions whose keys make every score -inf weigh nothing, be they whole blocks at the start, some
    inside a block or the end; a source of nothing else gives zeros and -inf."""
    c = Case([900, 140, 300], [most, most, most], 2, 2, D, 16)
    c.q[..., 0] = c.q[..., 0].abs() + 0.25
    minus = torch.tensor([-math.inf]).bfloat16().view(torch.int16).numpy().view(np.uint16)[0]
    for s, gone in enumerate((list(range(0, 300)) + [301, 500, 899], [139], list(range(300)))):
        p = np.array(gone)
        c.k[c.table[s][p // 16], p % 16, :, 0] = minus
    out, lse = c.run(splits=splits)
    seen = slice(0, int(c.indptr[2]))
    c.lens = c.lens[:2]
    want, logs, weighed = c.exact()
    x, y = out.cpu().numpy(), lse.cpu().numpy()
    assert (np.abs(x - want) <= 2.0 ** -7 * weighed + 1e-6)[seen].all()
    assert (np.abs(y[seen] - logs[seen]) <= 2.0 ** -14 + 2.0 ** -20 * np.abs(logs[seen])).all()
    assert (x[c.indptr[2]:] == 0).all() and np.isneginf(y[c.indptr[2]:]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("splits", [1, 2])
def test_nan_stays_with_its_row_among_many(splits, D):
    c = Case([400, 700], [40, 200], 2, 2, D, 16)
    q = c.q.clone()
    q[1, 2, 5] = math.nan      # one tile
    q[45, 1, 0] = math.nan     # two
    out, lse = c.run(splits=splits, q=q)
    bad = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
    bad[1, 2] = bad[45, 1] = True
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    want, logs, weighed = c.exact()
    err = np.abs(out.cpu().numpy() - want)
    good = ~bad.cpu().numpy()
    assert (err <= 2.0 ** -7 * weighed + 1e-6)[good].all()
    assert (np.abs(lse.cpu().numpy() - logs) <= 2.0 ** -14 + 2.0 ** -20 * np.abs(logs))[good].all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S", [2, 33, 255, 256, 257])
def test_many_sources_of_any_length_in_any_order(S, D):
    """More items than SMs: whatever order they are worked off in, every source gets its rows."""
    rng = np.random.default_rng(S)
    lens = [int(n) for n in rng.choice([0, 1, 17, 128, 300, 640, 1100], S)]
    lens[0], lens[-1] = 1100, 1500
    q_lens = [int(n) for n in rng.choice([0, 1, 20, 40], S)]
    q_lens[0], q_lens[1] = 40, 40
    if S == 2:
        q_lens = [3000, 2100]
    c = Case(lens, q_lens, 2, 2, D, 16, seed=S)
    for max_src in (1500, 1536):   # the longest, and what the table's rows hold
        out, lse = c.run(splits=1, max_src=max_src)
        check(c, out, lse)
        assert kvc.kvc_device_errors() == 0
