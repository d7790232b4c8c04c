"""NaN and infinity in queries, keys and values.

The reference is the definition in 64 bits, where a score of NaN or +infinity makes its row NaN, one
of -infinity weighs nothing, and an infinite value reaches its dim.  Finite outputs (fp32): a
probability is rounded to bf16, half a step 2^-8 of itself, in the numerator and in the sum, so the
weighted mean of values up to V moves by 2^-7 V (1 + 2^-8); a score, a sum of D products in fp32
(2^-23 each, tensor cores may cut), by d = (D + 8) 2^-23 scale Q K and the mean by 2 d V; 2^x, the sums
and the division by 2^-18 V."""
import math

import numpy as np
import pytest
import torch

import pagedattention_kvc_store_gb300 as kvc
from oracle import int4
from workloads.device import bf16_tensor, i32_tensor

pytestmark = pytest.mark.gpu

NAN, INF, NEG_INF = 0x7FC0, 0x7F80, 0xFF80
P, H, G = 16, 2, 2
CTX = np.array([50, 2500, 300, 40, 200, 0, 33])


class Case:
    """Sequences over pages of their own; nothing below holds a position past its context."""

    def __init__(self, D, seed=1):
        rng = np.random.default_rng(seed)
        width = -(-int(CTX.max()) // P)
        self.D, self.S = D, len(CTX)
        self.max_ctx = int(CTX.max())
        self.table = rng.permutation(self.S * width).reshape(self.S, width).astype(np.int32)
        shape = (self.S * width, P, H, D)
        self.k, self.v = (int4.bf16_round(rng.standard_normal(shape).astype(np.float32))
                          for _ in "kv")
        self.q = int4.bf16_round(rng.standard_normal((self.S, H * G, D)).astype(np.float32))

    def at(self, pool, s, p):
        return pool[self.table[s, p // P], p % P]   # [H, D], a view

    def reference(self):
        q, k, v = (int4.bf16_value(x).astype(np.float64) for x in (self.q, self.k, self.v))
        out = np.zeros(self.q.shape)
        with np.errstate(invalid="ignore"):
            for s, n in enumerate(CTX):
                pos = np.arange(n)
                page = self.table[s][pos // P], pos % P
                for h in range(H * G if n else 0):
                    x = k[page][:, h // G] @ q[s, h] / math.sqrt(self.D)
                    w = np.exp(x - x.max())
                    out[s, h] = w @ v[page][:, h // G] / w.sum()
        return out

    def check(self, got):
        ref = self.reference()
        got = got.double().cpu().numpy()
        finite = np.isfinite(ref)
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        assert np.array_equal(got[np.isinf(ref)], ref[np.isinf(ref)])
        q, k, v = (np.abs(int4.bf16_value(x).astype(np.float64)) for x in (self.q, self.k, self.v))
        Q, K, V = (x[np.isfinite(x)].max() for x in (q.sum(-1), k, v))
        d = (self.D + 8) * 2.0 ** -23 / math.sqrt(self.D) * Q * K
        bound = (2.0 ** -7 * (1 + 2.0 ** -8) + 2 * d + 2.0 ** -18) * V
        assert np.abs(got[finite] - ref[finite]).max() <= bound

    def upload(self):
        self.dk, self.dv = bf16_tensor(self.k, "cuda"), bf16_tensor(self.v, "cuda")
        self.dq, self.dt = bf16_tensor(self.q, "cuda"), i32_tensor(self.table, "cuda")
        self.dc = i32_tensor(CTX, "cuda")
        self.pool = kvc.pool_desc(self.dk)

    def decode(self, splits, dtype=torch.float32):
        out = torch.full(self.q.shape, 9.0, dtype=dtype, device="cuda")
        n, _, ws = kvc.kvc_decode_plan(self.S, H * G, self.pool, self.max_ctx, splits)
        work = torch.empty(max(ws, 16), dtype=torch.uint8, device="cuda")
        kvc.kvc_decode(out, self.dq, self.dk, self.dv, self.dt, self.dc, self.max_ctx,
                       num_splits=splits, workspace=work)
        return out, n


def spoiled(D):
    """Rows of every kind, in a sequence of one chunk and of many; and which rows must be NaN."""
    c = Case(D)
    c.at(c.k, 0, 19)[1, 3] = NAN              # sequence 0 (50 positions), kv head 1
    c.at(c.k, 1, 700)[0, 0] = NAN             # sequence 1 (2,500), kv head 0
    c.q[2, 3, 5] = NAN                        # one query head
    c.at(c.k, 3, 5)[1, 0] = INF               # scores of both infinities, by the query's sign
    c.q[3, 2, 0], c.q[3, 3, 0] = int4.bf16_round(np.array([1.5, -1.5], np.float32))
    c.at(c.v, 4, 100)[0, 7] = INF             # one dim
    c.at(c.v, 6, 32)[1, 1] = NAN
    return c


@pytest.mark.parametrize("D", [64, 128])
def test_the_reference_says_what_the_cases_are_for(D):
    ref = spoiled(D).reference()
    nan = np.isnan(ref).all(-1)
    assert nan.nonzero()[0].tolist() == [0, 0, 1, 1, 2, 3] and nan[3, 2] and not nan[3, 3]
    assert np.isinf(ref[4, :2, 7]).all() and np.isnan(ref[6, 2:, 1]).all()


@pytest.mark.parametrize("D", [64, 128])
def test_merge_of_nan_partials(D):
    """Rows whose only non-empty splits are NaN are NaN, like rows with numbers beside them; rows of
    empty splits are 0 as before."""
    for splits in (1, 3, 5, 40):              # both forms of the merge
        rows = 6
        lse = np.full((rows, splits), -np.inf, np.float32)
        o = np.full((rows, splits, D), 2.0, np.float32)
        lse[0, splits // 2] = np.nan          # the only one
        lse[1] = np.nan
        lse[2] = np.log(np.float32(1.0))      # all numbers
        lse[3, 0], lse[3, -1] = 0.5, np.nan   # (the same split where there is one)
        lse[4, -1] = 3.0
        out = torch.full((rows, D), 7.0, device="cuda")
        back = torch.zeros(rows, device="cuda")
        kvc.kvc_merge(out, torch.from_numpy(o).cuda(), torch.from_numpy(lse).cuda(), lse_out=back)
        out, back = out.cpu().numpy(), back.cpu().numpy()
        for row in (0, 1, 3):
            assert np.isnan(out[row]).all() and np.isnan(back[row]), (splits, row)
        assert np.abs(out[[2, 4]] - 2.0).max() <= 40 * 2.0 ** -22
        assert not out[5].any() and back[5] == -np.inf


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("splits", [1, 3, 0, 20])
def test_decode(D, splits):
    c = spoiled(D)
    c.upload()
    out, n = c.decode(splits)
    assert splits == 0 or n == splits         # 20: the wide merge
    c.check(out)
    assert kvc.kvc_device_errors() == 0


def decode_weights(c, splits, dtype=torch.float32):
    out = torch.full(c.q.shape, 9.0, dtype=dtype, device="cuda")
    weights = torch.zeros(c.S, H, c.max_ctx, device="cuda")
    ws = kvc.kvc_decode_weights_plan(c.S, H * G, c.pool, c.max_ctx, splits)[2]
    work = torch.full((ws,), 0xFF, dtype=torch.uint8, device="cuda")
    kvc.kvc_decode_weights(out, weights, c.dq, c.dk, c.dv, c.dt, c.dc, c.max_ctx,
                           num_splits=splits, workspace=work)
    return out, weights.double().cpu().numpy()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("splits", [1, 3, 0, 20])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_decode_weights_is_decode(D, splits, dtype):
    """The same output wherever it is not NaN, and NaN in the same places; among them rows whose
    scores are all -infinity, whose softmax is 0 / 0."""
    c = spoiled(D)
    for p in range(CTX[6]):
        c.at(c.k, 6, p)[0, 2] = NEG_INF
    c.q[6, :2, 2] = int4.bf16_round(np.array([0.5, 2.0], np.float32))
    c.upload()
    out, _ = decode_weights(c, splits, dtype)
    want, _ = c.decode(splits, dtype)
    assert torch.equal(out.isnan(), want.isnan())
    assert torch.equal(out.nan_to_num(nan=5.0), want.nan_to_num(nan=5.0))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("splits", [1, 0, 20])
def test_weights(D, splits):
    """A NaN softmax gives NaN weights to its kv head, for the sequence's positions alone; a score of
    -infinity gives 0.  Finite weights: relative error 2 d of the score and the sum, 2^-24 each for the
    six roundings of numbers up to X, 2^-20 for 2^x, the logarithm and the sums."""
    c = spoiled(D)
    c.q[3, 2, 0] = int4.bf16_round(np.array([-0.5], np.float32))[0]   # both -infinity now
    c.upload()
    out, got = decode_weights(c, splits)
    q, k = (int4.bf16_value(x).astype(np.float64) for x in (c.q, c.k))
    want = np.zeros(got.shape)
    with np.errstate(invalid="ignore"):
        for s, n in enumerate(CTX):
            pos = np.arange(n)
            for h in range(H * G if n else 0):
                x = k[c.table[s][pos // P], pos % P][:, h // G] @ q[s, h] / math.sqrt(D)
                w = np.exp(x - x.max())
                want[s, h // G, :n] += w / w.sum()
    assert np.isnan(want[0, 1, :50]).all() and want[3, 1, 5] == 0 and np.isfinite(want[3]).all()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    Q = np.abs(q)[np.isfinite(q).all(-1)].sum(-1).max()
    K = np.abs(k[np.isfinite(k)]).max()
    d = (D + 8) * 2.0 ** -23 / math.sqrt(D) * Q * K
    X = Q * K / math.sqrt(D) + math.log(c.max_ctx)
    rho = 2 * d + 6 * 2.0 ** -24 * X / math.log(2) + 2.0 ** -20
    fine = np.isfinite(want)
    assert (np.abs(got[fine] - want[fine]) <= rho * want[fine] + 1e-37).all()
    assert kvc.kvc_device_errors() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("splits", [1, 2, 0, 9])
def test_decode_int8(D, splits):
    """A NaN scale makes NaN of the rows that attend over its position, in a sequence of one piece and of
    many, and of no other; a NaN in the query makes NaN of its row, all of whose pieces are NaN."""
    c = Case(D)
    rng = np.random.default_rng(3)
    shape = (len(c.k), P, H, D)
    codes = [torch.from_numpy(rng.integers(-127, 128, shape, dtype=np.int8)).cuda() for _ in "kv"]
    scales = [np.full((len(c.k), H, P), 0.01, np.float32) for _ in "kv"]
    scales[0][c.table[0, 19 // P], 1, 19 % P] = np.nan        # sequence 0 (50), K of kv head 1
    scales[0][c.table[1, 700 // P], 0, 700 % P] = np.nan      # sequence 1 (2,500), K of kv head 0
    scales[1][c.table[2, 250 // P], 1, 250 % P] = np.nan      # sequence 2 (300), V of kv head 1
    c.q[1, 3, 5] = NAN                                        # every piece of one query head
    nan_rows = np.zeros((c.S, H * G), bool)
    nan_rows[0, 2:] = nan_rows[1, :2] = nan_rows[1, 3] = nan_rows[2, 2:] = True
    dev = codes + [torch.from_numpy(x).cuda() for x in scales]
    c.upload()
    out = torch.full(c.q.shape, 9.0, device="cuda")
    ws = kvc.kvc_decode_int8_plan(c.S, H * G, kvc.int8_pool_desc(dev[0]), c.max_ctx, splits)[2]
    work = torch.empty(max(ws, 16), dtype=torch.uint8, device="cuda")
    kvc.kvc_decode_int8(out, c.dq, *dev, c.dt, c.dc, c.max_ctx, num_splits=splits, workspace=work)
    got = out.cpu().numpy()
    assert np.isnan(got[nan_rows]).all() and np.isfinite(got[~nan_rows]).all()
    assert not got[CTX == 0].any() and kvc.kvc_device_errors() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_decode_shared_prefix(D):
    """A NaN key in pages that a group shares reaches every member's rows of that kv head, in positions
    of its own those of one member; a NaN query one row.  Groups of 2 and 1, 96 and 16 shared."""
    c = Case(D)
    c.table[2, :6] = c.table[1, :6]           # sequences 1 and 2 share 96 positions
    c.at(c.k, 1, 30)[0, 4] = NAN
    c.at(c.k, 2, 200)[1, 0] = NAN
    c.at(c.k, 4, 3)[0, 9] = NAN               # sequence 4, alone in its group
    c.q[1, 3, 5] = NAN
    c.upload()
    i32 = lambda x: i32_tensor(np.array(x), "cuda")
    ws = kvc.kvc_decode_shared_prefix_plan(c.S, H * G, c.pool, c.max_ctx, 2, 96)
    work = torch.full((ws,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full(c.q.shape, 9.0, device="cuda")
    kvc.kvc_decode_shared_prefix(out, c.dq, c.dk, c.dv, c.dt, c.dc, c.max_ctx, i32([0, 2, 3]),
                                 i32([1, 2, 4]), i32([96, 16]), 2, 96, work)
    c.check(out)
    nan = np.isnan(c.reference()).all(-1)
    assert nan.sum() == 2 + 1 + 2 + 2 + 2 and kvc.kvc_device_errors() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("splits", [1, 2, 0, 9])
def test_decode_int4(D, splits):
    """NaN parameters (a group that held a NaN or an infinity) reach the rows that attend over them, V's
    only the group's dims; a NaN in the query its row, all of whose pieces are NaN."""
    c = Case(D)
    rng = np.random.default_rng(4)
    codes = [torch.from_numpy(rng.integers(0, 256, (len(c.k), P, H, D // 2), dtype=np.uint8)).cuda()
             for _ in "kv"]
    params = [np.empty((len(c.k), H, P, D // 64, 2), np.uint16) for _ in "kv"]
    for x in params:
        x[..., 0] = int4.bf16_round(np.float32(0.25))
        x[..., 1] = int4.bf16_round(rng.standard_normal(x.shape[:-1]).astype(np.float32))
    params[0][c.table[0, 19 // P], 1, 19 % P, 0] = NAN        # sequence 0 (50), K of kv head 1
    params[0][c.table[1, 700 // P], 0, 700 % P, -1] = NAN     # sequence 1 (2,500), K of kv head 0
    params[1][c.table[2, 250 // P], 1, 250 % P, -1] = NAN     # sequence 2 (300), V of kv head 1, last group
    c.q[1, 3, 5] = NAN
    nan = np.zeros((c.S, H * G, D), bool)
    nan[0, 2:] = nan[1, :2] = nan[1, 3] = nan[2, 2:, D - 64:] = True
    dev = codes + [bf16_tensor(x, "cuda") for x in params]
    c.upload()
    out = torch.full(c.q.shape, 9.0, device="cuda")
    ws = kvc.kvc_decode_int4_plan(c.S, H * G, kvc.int4_pool_desc(dev[0]), c.max_ctx, splits)[2]
    work = torch.full((max(ws, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    kvc.kvc_decode_int4(out, c.dq, *dev, c.dt, c.dc, c.max_ctx, num_splits=splits, workspace=work)
    got = out.cpu().numpy()
    assert np.isnan(got[nan]).all() and np.isfinite(got[~nan]).all()
    assert not got[CTX == 0].any() and kvc.kvc_device_errors() == 0
