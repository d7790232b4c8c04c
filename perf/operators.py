"""What the 4-bit pages and the eviction operators are measured on, with their plain forms.

Each case is one operator at one size: ``run`` makes the calls that a serving loop makes of the
library where ``own`` is true, and computes the same with elementary torch operations otherwise.
``exact`` gives the results from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

GROUP = 64   # values that share a scale and a minimum in 4-bit pages


def listed():
    return [
        # one decode step's new tokens quantised into 4-bit pages, and read back as bf16
        dict(name="int4 store+load step", op="pages", tokens=64, kv_heads=8, head_dim=128,
             page=16, layout="nhd", f32=False),
        # the new tokens of 1,000 rewound documents (50 each)
        dict(name="int4 store+load chunk", op="pages", tokens=50000, kv_heads=8, head_dim=128,
             page=16, layout="nhd", f32=False),
        # a handful of short sequences: latency
        dict(name="int4 decode tiny", op="int4", seqs=4, lo=1, hi=100, lens=1, empty=0, kv_heads=2,
             group=2, head_dim=64, page=16, layout="nhd"),
        # the batched decode step of a server
        dict(name="int4 decode batched", op="int4", seqs=64, lo=512, hi=4096, lens=2, empty=0,
             kv_heads=8, group=4, head_dim=128, page=16, layout="nhd"),
        # few sequences of long contexts
        dict(name="int4 decode long", op="int4", seqs=8, lo=32768, hi=131072, lens=3, empty=0,
             kv_heads=8, group=8, head_dim=128, page=64, layout="nhd"),
        # ragged, one query head per kv head, head-major pages, an idle sequence in the batch
        dict(name="int4 decode ragged", op="int4", seqs=19, lo=1, hi=2001, lens=4, empty=7,
             kv_heads=5, group=1, head_dim=64, page=32, layout="hnd"),
        # a decode step that also adds up the attention weights, for a later eviction
        dict(name="weights tiny", op="weights", seqs=4, lo=1, hi=100, lens=1, empty=0, kv_heads=2,
             group=2, head_dim=64, page=16, layout="nhd"),
        dict(name="weights batched", op="weights", seqs=64, lo=512, hi=4096, lens=2, empty=0,
             kv_heads=8, group=4, head_dim=128, page=16, layout="nhd"),
        dict(name="weights long", op="weights", seqs=8, lo=32768, hi=131072, lens=3, empty=0,
             kv_heads=8, group=8, head_dim=128, page=64, layout="nhd"),
        # one short sequence over its budget
        dict(name="evict small", op="evict", seqs=1, lo=300, hi=300, lens=1, empty=0, kv_heads=2,
             head_dim=64, page=16, layout="nhd", budget=256, recent=32),
        # a batch brought back to half its longest context
        dict(name="evict batched", op="evict", seqs=64, lo=512, hi=4096, lens=2, empty=0,
             kv_heads=8, head_dim=128, page=16, layout="nhd", budget=2048, recent=256),
        # long prompts cut to a budget once they are in the cache
        dict(name="evict long", op="evict", seqs=8, lo=32768, hi=131072, lens=3, empty=0,
             kv_heads=8, head_dim=128, page=64, layout="nhd", budget=16384, recent=1024),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "int4", "int4", "weights", "evict"])
    c = dict(op=op, kv_heads=rng.choice([1, 2, 3, 4, 5, 8]), head_dim=rng.choice([64, 128]),
             page=rng.choice([16, 32, 64]), layout=rng.choice(["nhd", "hnd"]))
    if op == "pages":
        f32 = rng.random() < 0.25
        c.update(tokens=_log_int(rng, 1, 25000 if f32 else 50000), f32=f32)
        return c
    hi = _log_int(rng, 1, 131072)
    c.update(hi=hi, lo=rng.choice([1, 1, max(1, hi // 8), max(1, hi // 2), hi]),
             lens=rng.randrange(1 << 20), empty=rng.choice([0, 0, 0, 5]),
             seqs=_log_int(rng, 1, max(1, min(256, (4 * 131072) // hi))))
    if op == "evict":
        c["budget"] = _log_int(rng, 1, hi)
        c["recent"] = min(c["budget"], rng.choice([0, 1, 32, c["budget"] // 4, c["budget"]]))
    else:
        c["group"] = rng.choice([1, 2, 4, 8])
    return c


def _lengths(case):
    """The case's context lengths (its own, whatever the seed of its values)."""
    r = random.Random(case["lens"])
    ctx = [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    ctx[0] = case["hi"]
    if case["empty"]:
        ctx = [0 if s % case["empty"] == case["empty"] - 1 else n for s, n in enumerate(ctx)]
    return ctx


def _vec_bytes4(d):
    return d // 2 + d // GROUP * 4


def work(case):
    H, D = case["kv_heads"], case["head_dim"]
    if case["op"] == "pages":
        vectors = 2 * case["tokens"] * H
        out = 4 if case["f32"] else 2
        return {"bytes": vectors * (2 * D + 2 * _vec_bytes4(D) + out * D) + 8 * case["tokens"],
                "flops": vectors * D * 8}
    ctx = _lengths(case)
    n = sum(ctx)
    if case["op"] == "evict":
        moved = 0.0
        for N in ctx:
            kept = min(N, case["budget"])
            tail = N - kept
            rec = min(case["recent"], N)
            rec_tail = min(rec, tail)   # the newest slots are the last ones
            other = (tail - rec_tail) * (kept - rec) / max(1, N - rec)
            moved += rec_tail + other
        return {"bytes": H * (16 * n + moved * 8 * D), "flops": H * n * 8}
    q = case["seqs"] * H * case["group"] * D
    vec = 2 * _vec_bytes4(D) if case["op"] == "int4" else 4 * D + 8
    return {"bytes": n * H * vec + q * 4, "flops": 4 * n * H * case["group"] * D}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def _quantise(x):
    """[..., D] values -> (uint8 codes [..., D / 2], bf16 (scale, minimum) [..., D / 64, 2])."""
    g = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    scale = ((hi * 0.5 - lo * 0.5) / 7.5).bfloat16().float()
    code = torch.where(scale > 0, ((g * 0.5 - lo * 0.5) / (scale * 0.5)).round(), 0.0).clamp(0, 15)
    code = code.to(torch.uint8).flatten(-2)
    params = torch.cat([scale, lo], -1).bfloat16()
    return code[..., 0::2] | (code[..., 1::2] << 4), params


def _dequantise(codes, params):
    """The fp32 values that codes [..., D / 2] and params [..., D / 64, 2] stand for."""
    u = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    return (u * params[..., 0:1].float() + params[..., 1:2].float()).flatten(-2)


def _values(gen, shape, channel, sharp=1.0):
    """bf16 values N(0, channel^2): keys have a few large channels, values are even."""
    return (torch.randn(shape, generator=gen, device="cuda") * channel * sharp).bfloat16()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    H, D, P, layout = case["kv_heads"], case["head_dim"], case["page"], case["layout"]
    state = {"case": case, "layout": layout}
    channel = torch.exp(0.4 * torch.randn(D, generator=gen, device="cuda"))

    def pool_shape(pages, last):
        return (pages, P, H, last) if layout == "nhd" else (pages, H, P, last)

    if case["op"] == "pages":
        T = case["tokens"]
        pages = -(-T // P) + max(1, T // (10 * P))
        slots = torch.randperm(pages * P, generator=gen, device="cuda")[:T].int()
        if T > 8:
            slots[3::11] = -1   # padding tokens of a captured step
        out = torch.float32 if case["f32"] else torch.bfloat16
        state.update(
            k_new=_values(gen, (T, H, D), channel), v_new=_values(gen, (T, H, D), 1.0),
            slots=slots,
            k_codes=torch.zeros(pool_shape(pages, D // 2), dtype=torch.uint8, device="cuda"),
            v_codes=torch.zeros(pool_shape(pages, D // 2), dtype=torch.uint8, device="cuda"),
            k_params=torch.zeros(pages, H, P, D // GROUP, 2, dtype=torch.bfloat16, device="cuda"),
            v_params=torch.zeros(pages, H, P, D // GROUP, 2, dtype=torch.bfloat16, device="cuda"),
            k_out=torch.empty(T, H, D, dtype=out, device="cuda"),
            v_out=torch.empty(T, H, D, dtype=out, device="cuda"))
        return state

    ctx = _lengths(case)
    S, max_ctx = len(ctx), max(1, max(ctx))
    need = [-(-n // P) for n in ctx]
    pages = sum(need) + max(1, sum(need) // 10)
    width = -(-max(max(need), 1) // 16) * 16
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    table = torch.zeros(S, width, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    state.update(table=table, ctx=torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                 max_ctx=max_ctx)
    chan_k = channel
    if case["op"] == "int4":
        for name, ch in (("k", chan_k), ("v", 1.0)):
            codes, params = _quantise(_values(gen, pool_shape(pages, D), ch))
            if layout == "nhd":
                params = params.transpose(1, 2)
            state[name + "_codes"], state[name + "_params"] = codes, params.contiguous()
    else:
        state["k_pool"] = _values(gen, pool_shape(pages, D), chan_k)
        state["v_pool"] = _values(gen, pool_shape(pages, D), 1.0)
    if case["op"] == "evict":
        w = torch.exp(1.5 * torch.randn(S, H, max_ctx, generator=gen, device="cuda"))
        w[torch.rand(S, H, max_ctx, generator=gen, device="cuda") < 0.05] = 0.0
        # an earlier eviction left `kept` slots of the longer sequences with scattered original
        # positions; later tokens follow in order
        kept = min(case["budget"], max(1, case["hi"] // 2))
        before = (state["ctx"] >= kept)[:, None, None]
        gone = case["hi"] // 4
        i = torch.arange(max_ctx, device="cuda", dtype=torch.int32)
        pos = torch.where(before, i + gone, i).repeat(1, H, 1)
        scattered = torch.rand(S, H, kept + gone, generator=gen, device="cuda").argsort(-1)
        pos[:, :, :kept] = torch.where(before, scattered[:, :, :kept].int(), pos[:, :, :kept])
        state.update(weights=w, positions=pos, weights_out=torch.zeros_like(w),
                     positions_out=torch.zeros_like(pos),
                     new_lens=torch.zeros(S, dtype=torch.int32, device="cuda"))
    else:
        G = case["group"]
        state["q"] = _values(gen, (S, H * G, D), 1.0, 1.5)
        state["out"] = torch.empty(S, H * G, D, dtype=torch.bfloat16, device="cuda")
    if case["op"] == "weights":
        state["weights"] = torch.zeros(S, H, max_ctx, device="cuda")
    return state


def _workspace(state, nbytes):
    """The caller's workspace, kept between steps as a serving loop keeps it."""
    if "work" not in state or state["work"].numel() < nbytes:
        state["work"] = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")
    return state["work"]


# ------------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------------
def _take(pool, page, off, layout):
    """Vectors [..., H, last] of the positions at (page, off)."""
    return pool[page, off] if layout == "nhd" else pool[page, :, off]


def _places(state):
    """(page, offset) of every position [S, L] and which of them exist."""
    P = state["case"]["page"]
    p = torch.arange(state["max_ctx"], device="cuda")
    page = state["table"][:, p // P].long()
    off = (p % P).expand_as(page)
    return page, off, p[None, :] < state["ctx"][:, None]


def _attend(q, k, v, live, scale):
    """q [S, H, G, D], k and v [S, L, H, D], live [S, L] -> (out, weights [S, H, G, L])."""
    x = torch.einsum("shgd,slhd->shgl", q, k) * scale
    x = torch.where(live[:, None, None, :], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = e.sum(-1, keepdim=True)
    w = e / torch.where(total > 0, total, 1.0)
    return torch.einsum("shgl,slhd->shgd", w, torch.where(live[:, :, None, None], v, 0.0)), w


def _plain_pages(st):
    case = st["case"]
    P, layout = case["page"], st["layout"]
    live = st["slots"] >= 0
    slot = st["slots"][live].long()
    page, off = slot // P, slot % P
    for name in ("k", "v"):
        codes, params = _quantise(st[name + "_new"][live])
        if layout == "nhd":
            st[name + "_codes"][page, off] = codes
        else:
            st[name + "_codes"][page, :, off] = codes
        st[name + "_params"][page, :, off] = params
    outs = []
    for name in ("k", "v"):
        x = _dequantise(_take(st[name + "_codes"], page, off, layout),
                        st[name + "_params"][page, :, off])
        out = torch.zeros_like(st[name + "_out"])
        out[live] = x.to(out.dtype)
        outs.append(out)
    return outs


def _plain_int4(st):
    case = st["case"]
    page, off, live = _places(st)
    k, v = (_dequantise(_take(st[n + "_codes"], page, off, st["layout"]),
                        st[n + "_params"][page, :, off]) for n in ("k", "v"))
    S, D = live.shape[0], case["head_dim"]
    q = st["q"].float().view(S, case["kv_heads"], case["group"], D)
    out, _ = _attend(q, k, v, live, 1.0 / math.sqrt(D))
    return out.reshape(S, -1, D).bfloat16()


def _plain_weights(st):
    case = st["case"]
    page, off, live = _places(st)
    k, v = (_take(st[n + "_pool"], page, off, st["layout"]).float() for n in ("k", "v"))
    S, D = live.shape[0], case["head_dim"]
    q = st["q"].float().view(S, case["kv_heads"], case["group"], D)
    out, w = _attend(q, k, v, live, 1.0 / math.sqrt(D))
    st["weights"] += w.sum(2)
    return [out.reshape(S, -1, D).bfloat16(), st["weights"]]


def _plain_evict(st):
    case = st["case"]
    w, pos, ctx = st["weights"], st["positions"], st["ctx"].long()
    S, H, L = w.shape
    P, layout = case["page"], st["layout"]
    i = torch.arange(L, device="cuda")
    live = (i < ctx[:, None])[:, None, :].expand(S, H, L)
    n = ctx.clamp(max=case["budget"])
    last = pos.gather(2, (ctx - 1).clamp(min=0)[:, None, None].expand(S, H, 1))
    newest = live & (pos > last - case["recent"])
    # largest weight first, then the newest before the others and what exists before the rest;
    # a stable sort leaves equal weights in slot order
    first = torch.sort(torch.where(torch.isnan(w), -math.inf, w), dim=-1, descending=True,
                       stable=True).indices
    rank = (newest.int() + live.int()).gather(2, first)
    order = first.gather(2, torch.sort(rank, dim=-1, descending=True, stable=True).indices)
    at = torch.empty_like(order).scatter_(2, order, i.expand(S, H, L))
    keep = at < n[:, None, None]
    low = (i < n[:, None])[:, None, :]
    hole, tail = torch.nonzero(low & ~keep), torch.nonzero(keep & ~low)   # as many of each
    s, h, dst, src = hole[:, 0], hole[:, 1], hole[:, 2], tail[:, 2]
    table = st["table"]
    dp, sp = table[s, dst // P].long(), table[s, src // P].long()
    for pool in (st["k_pool"], st["v_pool"]):
        if layout == "nhd":
            pool[dp, dst % P, h] = pool[sp, src % P, h]
        else:
            pool[dp, h, dst % P] = pool[sp, h, src % P]
    wo, po = st["weights_out"], st["positions_out"]
    wo.copy_(torch.where(keep & low, w, torch.where(live, 0.0, wo)))
    wo[s, h, dst] = w[s, h, src]
    total = torch.where(ctx[:, None, None] > 0, last + 1, 0)
    po.copy_(torch.where(low, pos, total + (i - n[:, None])[:, None, :]))
    po[s, h, dst] = pos[s, h, src]
    st["new_lens"].copy_(n)
    return [st["k_pool"], st["v_pool"], wo, po, st["new_lens"]]


# ------------------------------------------------------------------------------------------
# the library's calls
# ------------------------------------------------------------------------------------------
def _own_pages(st):
    import pagedattention_kvc_store_gb300 as kvc
    pools = (st["k_codes"], st["v_codes"], st["k_params"], st["v_params"])
    kvc.kvc_store_int4(*pools, st["k_new"], st["v_new"], st["slots"], layout=st["layout"])
    kvc.kvc_load_int4(st["k_out"], st["v_out"], *pools, st["slots"], layout=st["layout"])
    return [st["k_out"], st["v_out"]]


def _own_int4(st):
    import pagedattention_kvc_store_gb300 as kvc
    if "work" not in st:
        pool = kvc.int4_pool_desc(st["k_codes"], st["layout"])
        _workspace(st, kvc.kvc_decode_int4_plan(st["q"].shape[0], st["q"].shape[1], pool,
                                                st["max_ctx"])[2])
    kvc.kvc_decode_int4(st["out"], st["q"], st["k_codes"], st["v_codes"], st["k_params"],
                        st["v_params"], st["table"], st["ctx"], st["max_ctx"],
                        workspace=st["work"], layout=st["layout"])
    return st["out"]


def _own_weights(st):
    import pagedattention_kvc_store_gb300 as kvc
    if "work" not in st:
        pool = kvc.pool_desc(st["k_pool"], st["layout"])
        _workspace(st, kvc.kvc_decode_weights_plan(st["q"].shape[0], st["q"].shape[1], pool,
                                                   st["max_ctx"])[2])
    kvc.kvc_decode_weights(st["out"], st["weights"], st["q"], st["k_pool"], st["v_pool"],
                           st["table"], st["ctx"], st["max_ctx"], workspace=st["work"],
                           layout=st["layout"])
    return [st["out"], st["weights"]]


def _own_evict(st):
    import pagedattention_kvc_store_gb300 as kvc
    case = st["case"]
    if "work" not in st:
        pool = kvc.pool_desc(st["k_pool"], st["layout"])
        _workspace(st, kvc.kvc_evict_plan(st["ctx"].shape[0], pool, st["max_ctx"],
                                          case["budget"]))
    kvc.kvc_evict(st["k_pool"], st["v_pool"], st["weights_out"], st["positions_out"],
                  st["new_lens"], st["weights"], st["positions"], st["table"], st["ctx"],
                  st["max_ctx"], case["budget"], case["recent"], workspace=st["work"],
                  layout=st["layout"])
    return [st["k_pool"], st["v_pool"], st["weights_out"], st["positions_out"], st["new_lens"]]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"pages": _own_pages, "int4": _own_int4, "weights": _own_weights,
                "evict": _own_evict}[op](state)
    return {"pages": _plain_pages, "int4": _plain_int4, "weights": _plain_weights,
            "evict": _plain_evict}[op](state)


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------
def _exact_group(x):
    """What one group's values [..., 64] stand for once they are held in 4 bits."""
    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    step = ((hi - lo) / 15.0).to(torch.bfloat16).double()
    code = torch.floor((x - lo) / torch.where(step > 0, step, 1.0) + 0.5)
    half_up = ((x - lo) / torch.where(step > 0, step, 1.0) + 0.5 == code) & (code % 2 == 1)
    code = torch.where(half_up, code - 1, code).clamp(0.0, 15.0)   # ties to even
    return torch.where(step > 0, lo + step * code, lo)


def _exact_vectors(st, name, pages, offs):
    """[n, H, D] fp64 keys or values of the positions at (pages, offs)."""
    nhd = st["layout"] == "nhd"
    if name + "_pool" in st:
        pool = st[name + "_pool"]
        return (pool[pages, offs] if nhd else pool.transpose(1, 2)[pages, offs]).double()
    codes = st[name + "_codes"]
    codes = codes[pages, offs] if nhd else codes.transpose(1, 2)[pages, offs]
    par = st[name + "_params"].transpose(1, 2)[pages, offs].double()
    D = codes.shape[-1] * 2
    x = torch.empty(*codes.shape[:-1], D, dtype=torch.float64, device="cuda")
    x[..., 0::2] = (codes % 16).double()
    x[..., 1::2] = (codes // 16).double()
    for g in range(D // GROUP):
        part = x[..., g * GROUP:(g + 1) * GROUP]
        part.mul_(par[..., g, 0:1]).add_(par[..., g, 1:2])
    return x


def exact(case, seed):
    st = prepare(case, seed)
    H, D, P = case["kv_heads"], case["head_dim"], case["page"]
    if case["op"] == "pages":
        outs = []
        for name in ("k_new", "v_new"):
            x = st[name].double()
            y = torch.cat([_exact_group(x[..., g:g + GROUP]) for g in range(0, D, GROUP)], -1)
            y[st["slots"] < 0] = 0.0
            outs.append(y)
        return outs
    if case["op"] == "evict":
        return _exact_evict(case, st)
    G = case["group"]
    out = torch.zeros(case["seqs"], H * G, D, dtype=torch.float64, device="cuda")
    sums = torch.zeros(case["seqs"], H, st["max_ctx"], dtype=torch.float64, device="cuda")
    for s, n in enumerate(_lengths(case)):
        if n == 0:
            continue
        p = torch.arange(n, device="cuda")
        pages, offs = st["table"][s][p // P].long(), p % P
        k, v = _exact_vectors(st, "k", pages, offs), _exact_vectors(st, "v", pages, offs)
        for h in range(H):
            q = st["q"][s, h * G:(h + 1) * G].double()
            prob = torch.softmax(q @ k[:, h].T / math.sqrt(D), dim=1)
            out[s, h * G:(h + 1) * G] = prob @ v[:, h]
            sums[s, h, :n] = prob.sum(0)
    return out if case["op"] == "int4" else [out, sums]


def _exact_evict(case, st):
    """One (sequence, kv head) after another: the kept slots by a sort of (weight, slot)."""
    P, nhd = case["page"], st["layout"] == "nhd"
    kp, vp = (st[n] if nhd else st[n].transpose(1, 2) for n in ("k_pool", "v_pool"))
    wo, po = st["weights_out"].double(), st["positions_out"].clone()
    ctx = _lengths(case)
    for s, n_all in enumerate(ctx):
        n = min(n_all, case["budget"])
        for h in range(case["kv_heads"]):
            w, pos = st["weights"][s, h, :n_all].double(), st["positions"][s, h, :n_all].long()
            total = int(pos[-1]) + 1 if n_all else 0
            new = pos >= total - case["recent"]
            old = torch.nonzero(~new)[:, 0]
            best = old[torch.argsort(-w[old], stable=True)][:n - int(new.sum())]
            stay = new.clone()
            stay[best] = True
            holes, movers = torch.nonzero(~stay[:n])[:, 0], n + torch.nonzero(stay[n:])[:, 0]
            wo[s, h, :n_all] = 0.0
            wo[s, h, :n] = w[:n]
            wo[s, h, holes] = w[movers]
            po[s, h, n:] = total + torch.arange(po.shape[2] - n, device="cuda").int()
            po[s, h, :n] = pos[:n].int()
            po[s, h, holes] = pos[movers].int()
            d, m = st["table"][s][holes // P].long(), st["table"][s][movers // P].long()
            for pool in (kp, vp):
                pool[d, holes % P, h] = pool[m, movers % P, h]
    lens = torch.tensor([min(n, case["budget"]) for n in ctx], dtype=torch.int32, device="cuda")
    return [st["k_pool"], st["v_pool"], wo, po, lens]
