"""kvc_evict over batches in which sequences pause between a cut and their next token, against a
model that knows every sequence's length itself: eviction moves whole numbers, all is equal."""
import numpy as np
import pytest
import torch

import pagedattention_kvc_store_gb300 as kvc
from workloads.device import bf16_bits_of, bf16_tensor, i32_tensor

pytestmark = pytest.mark.gpu

P, H, D = 16, 2, 64


class Model:
    """The slots of every (sequence, kv head): position, weight and what K and V hold."""

    def __init__(self, S, stride):
        self.stride = stride
        self.tokens = np.zeros(S, int)          # that the sequence has had
        self.slots = [[[] for _ in range(H)] for _ in range(S)]

    def token(self, s, weight, tag):
        for h in range(H):
            self.slots[s][h].append((int(self.tokens[s]), weight[h], tag[h]))
        self.tokens[s] += 1

    def cut(self, s, budget, recent):
        for h in range(H):
            row = self.slots[s][h]
            n = min(len(row), budget)
            newest = [p >= self.tokens[s] - recent for p, _, _ in row]
            order = sorted(range(len(row)), key=lambda i: (not newest[i], 0 if newest[i] else -row[i][1], i))
            stay = set(order[:n])
            gaps = [i for i in range(n) if i not in stay]
            for g, m in zip(gaps, [i for i in range(n, len(row)) if i in stay]):
                row[g] = row[m]
            del row[n:]

    def positions(self, s, h):
        row = [p for p, _, _ in self.slots[s][h]]
        return row + list(range(self.tokens[s], self.tokens[s] + self.stride - len(row)))


@pytest.mark.parametrize("in_place", [(True, True), (False, False), (True, False), (False, True)])
@pytest.mark.parametrize("n,budget,recent", [(70, 40, 8), (5000, 2500, 100)])
def test_sequences_that_pause(n, budget, recent, in_place):
    """Three rounds: tokens to some sequences, then a cut of all of them.  Sequence 1 pauses after
    the first round and goes on in the third; sequence 2 never gets another token; 3 is empty.
    In place, apart, or one array of either kind."""
    rng = np.random.default_rng(n)
    S, stride = 4, n + 40
    width = -(-stride // P)
    table = rng.permutation(S * width).reshape(S, width).astype(np.int32)
    kp = rng.integers(0, 0x7F00, (S * width, P, H, D), dtype=np.uint16)
    k, v = bf16_tensor(kp, "cuda"), bf16_tensor(kp ^ 1, "cuda")
    model = Model(S, stride)
    w = np.zeros((S, H, stride), np.float32)
    pos = np.tile(np.arange(stride, dtype=np.int32), (S, H, 1))
    dw, dp = torch.from_numpy(w).cuda(), torch.from_numpy(pos).cuda()
    pool = kvc.pool_desc(k)
    work = torch.empty(kvc.kvc_evict_plan(S, pool, n + 30, budget), dtype=torch.uint8, device="cuda")
    dt = i32_tensor(table, "cuda")
    for grow in ([n, n - 3, n - 7, 0], [25, 0, 0, 0], [25, 12, 0, 0]):
        for s, more in enumerate(grow):
            for _ in range(more):
                at = len(model.slots[s][0])
                heavy = (rng.random(H) * 100).astype(np.float32)
                if at == budget - 1:
                    heavy[0] = 1e6          # stays: kv head 0's last slot is an old token after a cut
                model.token(s, heavy, [int(x) for x in
                                       bf16_bits_of(k[table[s, at // P], at % P, :, 0])]
                            if n < 100 else [0] * H)
            live = len(model.slots[s][0])
            dw[s, :, :live] = torch.from_numpy(
                np.array([[x[1] for x in model.slots[s][h]] for h in range(H)], np.float32).reshape(H, live))
        lens = [len(model.slots[s][0]) for s in range(S)]
        ow = dw if in_place[0] else torch.zeros_like(dw)
        op = dp if in_place[1] else torch.full_like(dp, -7)
        new = torch.full((S,), -1, dtype=torch.int32, device="cuda")
        kvc.kvc_evict(k, v, ow, op, new, dw, dp, dt, i32_tensor(np.array(lens), "cuda"), n + 30,
                      budget, recent, workspace=work)
        for s in range(S):
            model.cut(s, budget, recent)
        dw, dp = ow, op
        got_w, got_p = dw.cpu().numpy(), dp.cpu().numpy()
        for s in range(S):
            live = len(model.slots[s][0])
            assert new[s].item() == live
            for h in range(H):
                assert got_p[s, h].tolist() == model.positions(s, h), (grow, s, h)
                assert got_w[s, h, :live].tolist() == [x[1] for x in model.slots[s][h]]
                assert not got_w[s, h, live:lens[s]].any()
                if n < 100:
                    slots = np.arange(live)
                    held = bf16_bits_of(k)[table[s, slots // P], slots % P, h, 0]
                    assert held.tolist() == [x[2] for x in model.slots[s][h]]
        assert kvc.kvc_device_errors() == 0
    # a second cut to less with no token in between: right, and told
    new = torch.zeros(S, dtype=torch.int32, device="cuda")
    less = budget // 2
    lens = np.array([len(model.slots[s][0]) for s in range(S)])
    work = torch.empty(kvc.kvc_evict_plan(S, pool, n + 30, less), dtype=torch.uint8, device="cuda")
    kvc.kvc_evict(k, v, dw, dp, new, dw, dp, dt, i32_tensor(lens, "cuda"), n + 30, less, recent,
                  workspace=work)
    assert kvc.kvc_device_errors() == 1 << 13
    for s in range(S):
        model.cut(s, less, recent)
        for h in range(H):
            assert dp[s, h].tolist() == model.positions(s, h)
