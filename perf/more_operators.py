"""What rotary positions, cross attention and the page operators are measured on, with their plain
forms.

Each case is one operator (for pages: a run of them) at one size: ``run`` makes the calls that a
serving loop makes of the library where ``own`` is true, and computes the same with elementary torch
operations otherwise.  ``exact`` gives the results from the definitions in 64 bits.
"""
import math
import random

import torch

own = False


def listed():
    return [
        # one decode step's new tokens, 64 sequences: latency
        dict(name="rope step", op="rope", tokens=64, q_heads=32, kv_heads=8, head_dim=128, page=16,
             layout="nhd", rotary=128, pairing="halves", axes=3, far=131072),
        # the new tokens of 1,000 rewound documents (50 each)
        dict(name="rope chunk", op="rope", tokens=50000, q_heads=32, kv_heads=8, head_dim=128,
             page=16, layout="nhd", rotary=128, pairing="halves", axes=3, far=131072),
        # an odd number of image patches; half of each head turns, adjacent dims, head-major pages
        dict(name="rope patches", op="rope", tokens=9973, q_heads=64, kv_heads=8, head_dim=128,
             page=64, layout="hnd", rotary=64, pairing="adjacent", axes=2, far=1000),
        # a handful of short sources, one to three queries each: latency
        dict(name="cross tiny", op="cross", sources=4, lo=1, hi=100, lens=1, empty=0, q_lo=1, q_hi=3,
             kv_heads=2, group=2, head_dim=64, page=16, layout="nhd", lse=True),
        # a decode step of 64 requests with 4 beams each over their sources
        dict(name="cross beams", op="cross", sources=64, lo=512, hi=4096, lens=2, empty=0, q_lo=4,
             q_hi=4, kv_heads=8, group=4, head_dim=128, page=16, layout="nhd", lse=False),
        # prompts of up to 400 tokens over the same sources
        dict(name="cross prompts", op="cross", sources=64, lo=512, hi=4096, lens=2, empty=0, q_lo=200,
             q_hi=400, kv_heads=8, group=4, head_dim=128, page=16, layout="nhd", lse=False),
        # few sources of long contexts, 16 tokens each, to be joined with others by their log-sum-exps
        dict(name="cross long", op="cross", sources=8, lo=32768, hi=131072, lens=3, empty=0, q_lo=16,
             q_hi=16, kv_heads=8, group=8, head_dim=128, page=64, layout="nhd", lse=True),
        # ragged: sources without a state, requests without a token, head-major pages
        dict(name="cross ragged", op="cross", sources=19, lo=1, hi=2001, lens=4, empty=7, q_lo=0,
             q_hi=201, kv_heads=5, group=1, head_dim=64, page=32, layout="hnd", lse=True),
        # two branches of each of four short sequences, one layer, one more token each
        dict(name="branches tiny", op="branch", seqs=4, lo=1, hi=100, lens=1, empty=0, branches=2,
             grow=1, layers=1, kv_heads=2, head_dim=64, page=16, layout="nhd"),
        # four branches of each of 64 sequences, four layers, up to 24 more tokens each
        dict(name="branches batched", op="branch", seqs=64, lo=512, hi=4096, lens=2, empty=0,
             branches=4, grow=24, layers=4, kv_heads=8, head_dim=128, page=16, layout="nhd"),
        # half of a few short sequences end, their pages are closed up, others take their place
        dict(name="compact small", op="compact", seqs=8, lo=20, hi=300, lens=5, empty=0, layers=1,
             kv_heads=2, head_dim=64, page=16, layout="nhd"),
        # the same with a server's batch
        dict(name="compact batched", op="compact", seqs=64, lo=512, hi=4096, lens=2, empty=0, layers=2,
             kv_heads=8, head_dim=128, page=16, layout="nhd"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "cross", "cross", "cross", "branch", "compact"])
    c = dict(op=op, kv_heads=rng.choice([1, 2, 3, 4, 5, 8]), head_dim=rng.choice([64, 128]),
             page=rng.choice([16, 32, 64]), layout=rng.choice(["nhd", "hnd"]))
    if op == "rope":
        c.update(tokens=_log_int(rng, 1, 40000), q_heads=c["kv_heads"] * rng.choice([1, 2, 4, 8]),
                 rotary=16 * rng.randint(1, c["head_dim"] // 16),
                 pairing=rng.choice(["halves", "adjacent"]), axes=rng.choice([1, 2, 3, 4]),
                 far=_log_int(rng, 8, 1 << 20))
        return c
    c.update(lens=rng.randrange(1 << 20), empty=rng.choice([0, 0, 0, 5]))
    if op == "cross":
        hi = _log_int(rng, 1, 131072)
        q_hi = _log_int(rng, 1, 1024)
        group = rng.choice([1, 2, 4, 8])
        # at most the scores and the keys of the largest listed cases
        room = min((1 << 23) // (hi * q_hi), (1 << 20) // hi)
        c.update(hi=hi, lo=rng.choice([1, max(1, hi // 8), max(1, hi // 2), hi]), group=group,
                 q_hi=q_hi, q_lo=rng.choice([0, 1, max(1, q_hi // 2), q_hi]),
                 sources=_log_int(rng, 1, max(1, min(256, room))), lse=rng.random() < 0.5)
        if hi * q_hi > (1 << 23):
            c["q_hi"] = max(1, (1 << 23) // hi)
            c["q_lo"] = min(c["q_lo"], c["q_hi"])
        return c
    hi = _log_int(rng, 8, 16384)
    c.update(hi=hi, lo=rng.choice([1, max(1, hi // 8), max(1, hi // 2), hi]),
             layers=rng.choice([1, 2, 4]),
             seqs=2 * _log_int(rng, 1, max(1, min(64, (1 << 16) // hi))))
    if op == "branch":
        c.update(branches=rng.choice([1, 2, 3, 4]), grow=_log_int(rng, 1, 64))
    return c


def _lengths(case):
    """The case's context lengths (its own, whatever the seed of its values)."""
    r = random.Random(case["lens"])
    n = case["sources"] if "sources" in case else case["seqs"]
    ctx = [r.randint(case["lo"], case["hi"]) for _ in range(n)]
    ctx[0] = case["hi"]
    if case["empty"]:
        ctx = [0 if s % case["empty"] == case["empty"] - 1 else x for s, x in enumerate(ctx)]
    return ctx


def _query_lens(case):
    r = random.Random(case["lens"] + 1)
    n = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["sources"])]
    n[0] = case["q_hi"]
    return n


def _branches(case):
    """Of each branch: the sequence that it starts from and the tokens that it grows by."""
    r = random.Random(case["lens"] + 2)
    parents = [s for s in range(case["seqs"]) for _ in range(case["branches"])]
    r.shuffle(parents)
    return parents, [r.randint(0 if case["grow"] > 1 else 1, case["grow"]) for _ in parents]


def _pages(n, P):
    return -(-n // P)


def work(case):
    H, D, P = case["kv_heads"], case["head_dim"], case["page"]
    if case["op"] == "rope":
        row = (2 * case["q_heads"] + 4 * H) * D * 2   # q, k and v read, q_out and pages written
        return {"bytes": case["tokens"] * (row + 4 + 4 * case["axes"]),
                "flops": case["tokens"] * (case["q_heads"] + H) * case["rotary"] * 3}
    if case["op"] == "cross":
        G = case["group"]
        pairs = list(zip(_lengths(case), _query_lens(case)))
        rows = sum(n for _, n in pairs) * H * G
        return {"bytes": sum(L for L, n in pairs if n) * H * D * 4 + rows * (4 * D + 4 * case["lse"]),
                "flops": 4 * D * H * G * sum(L * n for L, n in pairs)}
    arrays = 2 * case["layers"]
    page = P * H * D * 2
    ctx = _lengths(case)
    if case["op"] == "branch":
        parents, grow = _branches(case)
        # a partly filled last page is shared with the sequence itself: each branch that grows copies it
        copies = sum(1 for p, n in zip(parents, grow) if n and ctx[p] % P)
        entries = sum(_pages(ctx[p], P) for p in parents)
        return {"bytes": copies * arrays * 2 * page + entries * 16, "flops": 0}
    left = sum(_pages(n, P) for n in ctx[1::2])
    gone = sum(_pages(n, P) for n in ctx[0::2])
    return {"bytes": min(left, gone) * arrays * 2 * page + (left + gone) * 16, "flops": 0}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def _values(gen, shape, spread):
    """bf16 values N(0, spread^2)."""
    return (torch.randn(shape, generator=gen, device="cuda") * spread).bfloat16()


def _frequencies(case):
    """Angles per unit of position and the axis of each, in runs one axis after another."""
    n, axes = case["rotary"] // 2, case["axes"]
    return [10000.0 ** (-i / n) for i in range(n)], [i * axes // n for i in range(n)]


def _pool_shape(case, pages):
    H, D, P = case["kv_heads"], case["head_dim"], case["page"]
    return (pages, P, H, D) if case["layout"] == "nhd" else (pages, H, P, D)


def _table(case, ctx, gen, spare=0):
    """A block table whose rows list pages in random order, and the number of pages."""
    P = case["page"]
    need = [_pages(n, P) for n in ctx]
    pages = sum(need) + max(1, sum(need) // 10) + spare
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    return _rows(need, order), pages


def _rows(need, order, more=0):
    width = -(-max(max(need) + more, 1) // 16) * 16
    table = torch.zeros(len(need), width, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return table


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    H, D, P = case["kv_heads"], case["head_dim"], case["page"]
    st = {"case": case, "layout": case["layout"]}
    channel = torch.exp(0.4 * torch.randn(D, generator=gen, device="cuda"))

    if case["op"] == "rope":
        T, Hq = case["tokens"], case["q_heads"]
        pages = _pages(T, P) + max(1, T // (10 * P))
        slots = torch.randperm(pages * P, generator=gen, device="cuda")[:T].int()
        if T > 8:
            slots[3::11] = -1   # padding tokens of a captured step
        # q, k and v are parts of one projection's output, as a model has them
        qkv = _values(gen, (T, Hq + 2 * H, D), channel)
        st.update(
            q=qkv[:, :Hq], k_new=qkv[:, Hq:Hq + H], v_new=qkv[:, Hq + H:], slots=slots,
            positions=torch.randint(0, case["far"], (case["axes"], T), generator=gen,
                                    device="cuda").int(),
            q_out=torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda"),
            k_pool=torch.zeros(_pool_shape(case, pages), dtype=torch.bfloat16, device="cuda"),
            v_pool=torch.zeros(_pool_shape(case, pages), dtype=torch.bfloat16, device="cuda"))
        st["inv_freq"], st["axis"] = _frequencies(case)
        st["freq"] = torch.tensor(st["inv_freq"], dtype=torch.float64, device="cuda")
        st["axis_of"] = torch.tensor(st["axis"], device="cuda")
        return st

    ctx = _lengths(case)
    if case["op"] == "cross":
        st["table"], pages = _table(case, ctx, gen)
        n, G = _query_lens(case), case["group"]
        T = sum(n)
        starts = [0]
        for x in n:
            starts.append(starts[-1] + x)
        st.update(
            ctx=_i32(ctx), max_src=max(1, max(ctx)), max_q=max(n), q_indptr=_i32(starts),
            q=_values(gen, (T, H * G, D), 1.5),
            k_pool=_values(gen, _pool_shape(case, pages), channel),
            v_pool=_values(gen, _pool_shape(case, pages), 1.0),
            out=torch.empty(T, H * G, D, dtype=torch.bfloat16, device="cuda"),
            lse=torch.empty(T, H * G, device="cuda") if case["lse"] else None)
        # the query of each (source, index) pair, T where there is none
        i = torch.arange(max(n), device="cuda")
        first = torch.tensor(starts[:-1], device="cuda")[:, None]
        there = i < torch.tensor(n, device="cuda")[:, None]
        st.update(there=there, row=torch.where(there, first + i, T))
        return st

    shape = lambda pages: _pool_shape(case, pages)   # noqa: E731
    pages_of = [_pages(n, P) for n in ctx]
    if case["op"] == "branch":
        parents, grow = _branches(case)
        more = _pages(case["grow"], P) + 1
        st["table"], pages = _table(case, ctx, gen, spare=sum(_pages(n, P) + 1 for n in grow))
        st["table"] = torch.nn.functional.pad(st["table"], (0, -(-more // 16) * 16))
        st.update(parents=_i32(parents), grow=_i32(grow), lens=_i32(ctx),
                  new_table=torch.zeros(len(parents), st["table"].shape[1], dtype=torch.int32,
                                        device="cuda"),
                  new_lens=torch.zeros(len(parents), dtype=torch.int32, device="cuda"),
                  missing=torch.zeros(1, dtype=torch.int32, device="cuda"), most=more)
    else:
        # sequences 0, 2, 4, ... hold the lower pages and 1, 3, 5, ... the upper ones, each set in
        # random order: what is left after either set ends is moved down as far as there is room
        first, rest = sum(pages_of[0::2]), sum(pages_of[1::2])
        total = first + rest
        pages = total + max(1, total // 10)
        order = torch.cat([torch.randperm(first, generator=gen, device="cuda"),
                           first + torch.randperm(rest, generator=gen, device="cuda")]).int()
        table = _rows(pages_of[0::2] + pages_of[1::2], order)
        back = [s // 2 + (len(ctx) + 1) // 2 * (s % 2) for s in range(len(ctx))]
        st["table"] = table[torch.tensor(back, device="cuda")].contiguous()
        full = _i32(ctx)
        even = torch.arange(len(ctx), device="cuda") % 2 == 0
        zero = torch.zeros_like(full)
        st.update(lens=full, turn=0, most=max(pages_of),
                  keep=[torch.where(even, zero, full), torch.where(even, full, zero)],
                  grow=[torch.where(even, full, zero), torch.where(even, zero, full)],
                  page_map=torch.zeros(pages, dtype=torch.int32, device="cuda"),
                  num_live=torch.zeros(1, dtype=torch.int32, device="cuda"),
                  missing=torch.zeros(1, dtype=torch.int32, device="cuda"))
    live = torch.arange(st["table"].shape[1], device="cuda") < _i32(pages_of)[:, None]
    st["refs"] = torch.bincount(st["table"][live].long(), minlength=pages).int()
    st["pools"] = [_values(gen, shape(pages), 1.0) for _ in range(2 * case["layers"])]
    return st


def _workspace(st, nbytes):
    """The caller's workspace, kept between steps as a serving loop keeps it."""
    if "work" not in st or st["work"].numel() < nbytes:
        st["work"] = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")
    return st["work"]


# ------------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------------
def _turn(x, cos, sin, case):
    """The rotated values of x [T, H, D] (fp32), cos and sin [T, 1, rotary / 2]."""
    r, rest = x[..., :case["rotary"]], x[..., case["rotary"]:]
    if case["pairing"] == "halves":
        a, b = r.chunk(2, -1)
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, rest], -1)


def _plain_rope(st):
    case, P = st["case"], st["case"]["page"]
    angle = st["positions"][st["axis_of"]].T.double() * st["freq"]   # [T, rotary / 2]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    st["q_out"].copy_(_turn(st["q"].float(), cos, sin, case))
    k = _turn(st["k_new"].float(), cos, sin, case).bfloat16()
    live = st["slots"] >= 0
    slot = st["slots"][live].long()
    for pool, new in ((st["k_pool"], k), (st["v_pool"], st["v_new"])):
        if st["layout"] == "nhd":
            pool[slot // P, slot % P] = new[live]
        else:
            pool[slot // P, :, slot % P] = new[live]
    return [st["q_out"], st["k_pool"], st["v_pool"]]


def _plain_cross(st):
    case = st["case"]
    P, H, G, D = case["page"], case["kv_heads"], case["group"], case["head_dim"]
    p = torch.arange(st["max_src"], device="cuda")
    page, off = st["table"][:, p // P].long(), p % P
    live = p < st["ctx"][:, None]
    if st["layout"] == "nhd":
        k, v = (st[n][page, off].float() for n in ("k_pool", "v_pool"))
    else:
        k, v = (st[n][page, :, off].float() for n in ("k_pool", "v_pool"))
    T = st["q"].shape[0]
    q = torch.cat([st["q"], st["q"].new_zeros(1, H * G, D)])[st["row"]].float()
    q = q.unflatten(2, (H, G))                                  # [S, Q, H, G, D]
    x = torch.einsum("sqhgd,slhd->shgql", q, k) * (1.0 / math.sqrt(D))
    x.masked_fill_(~live[:, None, None, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp_(x.sub_(torch.where(m == -math.inf, 0.0, m)))
    total = e.sum(-1, keepdim=True)
    e.div_(torch.where(total > 0, total, 1.0))
    o = torch.einsum("shgql,slhd->sqhgd", e, v.masked_fill_(~live[:, :, None, None], 0.0))
    lse = (m + total.log()).squeeze(-1).permute(0, 3, 1, 2)     # [S, Q, H, G]
    # rows of no query go to one more row, which is left off
    out = o.new_empty(T + 1, H * G, D)
    out[st["row"]] = o.flatten(2, 3)
    logs = lse.new_empty(T + 1, H * G)
    logs[st["row"]] = lse.flatten(2)
    return [out[:T].bfloat16()] + ([logs[:T].contiguous()] if case["lse"] else [])


def _pages_of(lens, P):
    return (lens + (P - 1)) // P


def _add_refs(refs, table, first, last, n):
    """refs += n for entries first .. last - 1 of each row."""
    j = torch.arange(table.shape[1], device="cuda")
    at = (j >= first[:, None]) & (j < last[:, None])
    refs.index_add_(0, table.long().flatten(), torch.where(at, n, 0).int().flatten())


def _plain_truncate(table, lens, new_lens, refs, P):
    new = torch.minimum(lens, new_lens)
    _add_refs(refs, table, _pages_of(new, P), _pages_of(lens, P), -1)
    lens.copy_(new)


def _plain_reserve(table, lens, grow, refs, pools, missing, P, most):
    S = lens.shape[0]
    have, want = _pages_of(lens, P), _pages_of(lens + grow, P)
    row = torch.arange(S, device="cuda")
    open_ = (grow > 0) & (lens % P != 0)
    at = (have - 1).clamp(min=0).long()
    last = table[row, at].long()
    # of the rows that grow into one page, the last keeps it unless others hold it too
    last_row = torch.full_like(refs, -1, dtype=torch.long).scatter_reduce_(
        0, last, torch.where(open_, row, -1), "amax")
    sharers = torch.zeros_like(refs).index_add_(0, last, open_.int())
    copy = open_ & ~((sharers[last] == refs[last]) & (last_row[last] == row))
    need = copy.long() + want - have
    start = need.cumsum(0) - need
    free = torch.sort((refs != 0).int(), stable=True).indices   # free pages first, ascending
    short = (need.sum() - (refs == 0).sum()).clamp(min=0)
    missing.copy_(short)
    fits = short == 0
    j = torch.arange(most + 1, device="cuda")
    # page j of a row's new ones: the copy's first, then those of the following entries
    entry = torch.where(copy[:, None], at[:, None] + j, have[:, None] + j)
    ok = (j < need[:, None]) & fits
    page = free[(start[:, None] + j).clamp(max=free.numel() - 1)]
    who, which = torch.nonzero(ok, as_tuple=True)
    entry, page = entry[who, which], page[who, which]
    table[who, entry] = page.int()
    refs[page] = 1
    copied = torch.nonzero(copy & fits)[:, 0]
    src, dst = last[copied], table[copied, at[copied]].long()
    refs.index_add_(0, src, torch.full_like(src, -1, dtype=torch.int32))
    for pool in pools:
        pool[dst] = pool[src]
    lens.add_(torch.where(fits, grow, 0))


def _plain_branch(st):
    P, refs = st["case"]["page"], st["refs"]
    table, lens = st["new_table"], st["new_lens"]
    _plain_truncate(table, lens, torch.zeros_like(lens), refs, P)
    parents = st["parents"].long()
    lens.copy_(st["lens"][parents])
    have = _pages_of(lens, P)
    j = torch.arange(table.shape[1], device="cuda")
    table.copy_(torch.where(j < have[:, None], st["table"][parents], table))
    _add_refs(refs, table, torch.zeros_like(have), have, 1)
    _plain_reserve(table, lens, st["grow"], refs, st["pools"], st["missing"], P, st["most"])
    return [table, lens, refs, st["missing"]] + st["pools"]


def _plain_compact(st):
    P, refs, table, lens = st["case"]["page"], st["refs"], st["table"], st["lens"]
    turn = st["turn"]
    _plain_truncate(table, lens, st["keep"][turn], refs, P)
    live = refs > 0
    count = live.sum()
    page = torch.arange(refs.numel(), device="cuda")
    src, dst = torch.nonzero(live & (page >= count))[:, 0], torch.nonzero(~live & (page < count))[:, 0]
    to = torch.where(live, page, -1)
    to[src] = dst
    st["page_map"].copy_(to)
    st["num_live"].copy_(count)
    for pool in st["pools"]:
        pool[dst] = pool[src]
    refs[dst] = refs[src]
    refs[src] = 0
    j = torch.arange(table.shape[1], device="cuda")
    table.copy_(torch.where(j < _pages_of(lens, P)[:, None], to[table.long()].int(), table))
    _plain_reserve(table, lens, st["grow"][turn], refs, st["pools"], st["missing"], P, st["most"])
    st["turn"] = 1 - turn
    return [table, lens, refs, st["page_map"], st["num_live"], st["missing"]] + st["pools"]


# ------------------------------------------------------------------------------------------
# the library's calls
# ------------------------------------------------------------------------------------------
def _own_rope(st):
    import pagedattention_kvc_store_gb300 as kvc
    if "rope" not in st:
        st["rope"] = kvc.rope_desc(st["inv_freq"], st["axis"], pairing=st["case"]["pairing"])
    kvc.kvc_rope_store(st["q_out"], st["k_pool"], st["v_pool"], st["q"], st["k_new"], st["v_new"],
                       st["positions"], st["slots"], st["rope"], layout=st["layout"])
    return [st["q_out"], st["k_pool"], st["v_pool"]]


def _own_cross(st):
    import pagedattention_kvc_store_gb300 as kvc
    if "work" not in st:
        pool = kvc.pool_desc(st["k_pool"], st["layout"])
        _workspace(st, kvc.kvc_cross_plan(st["ctx"].shape[0], st["q"].shape[0], st["q"].shape[1],
                                          pool, st["max_q"], st["max_src"])[2])
    kvc.kvc_cross(st["out"], st["q"], st["k_pool"], st["v_pool"], st["table"], st["q_indptr"],
                  st["ctx"], st["max_q"], st["max_src"], lse_out=st["lse"], workspace=st["work"],
                  layout=st["layout"])
    return [st["out"]] + ([st["lse"]] if st["case"]["lse"] else [])


def _own_branch(st):
    import pagedattention_kvc_store_gb300 as kvc
    P, refs, table, lens = st["case"]["page"], st["refs"], st["new_table"], st["new_lens"]
    if "work" not in st:
        _workspace(st, kvc.kvc_reserve_plan(lens.shape[0], refs.shape[0]))
        st["arrays"] = kvc.page_arrays(st["pools"])
    kvc.kvc_truncate(table, lens, None, refs, P)
    kvc.kvc_fork(table, lens, st["parents"], st["table"], st["lens"], refs, P)
    kvc.kvc_reserve(table, lens, st["grow"], refs, st["missing"], P, st["arrays"],
                    workspace=st["work"])
    return [table, lens, refs, st["missing"]] + st["pools"]


def _own_compact(st):
    import pagedattention_kvc_store_gb300 as kvc
    P, refs, table, lens = st["case"]["page"], st["refs"], st["table"], st["lens"]
    if "work" not in st:
        _workspace(st, max(kvc.kvc_reserve_plan(lens.shape[0], refs.shape[0]),
                           kvc.kvc_compact_plan(refs.shape[0])))
        st["arrays"] = kvc.page_arrays(st["pools"])
    turn = st["turn"]
    kvc.kvc_truncate(table, lens, st["keep"][turn], refs, P)
    kvc.kvc_compact(table, lens, refs, st["page_map"], st["num_live"], P, st["arrays"],
                    workspace=st["work"])
    kvc.kvc_reserve(table, lens, st["grow"][turn], refs, st["missing"], P, st["arrays"],
                    workspace=st["work"])
    st["turn"] = 1 - turn
    return [table, lens, refs, st["page_map"], st["num_live"], st["missing"]] + st["pools"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "cross": _own_cross, "branch": _own_branch,
                "compact": _own_compact}[op](state)
    return {"rope": _plain_rope, "cross": _plain_cross, "branch": _plain_branch,
            "compact": _plain_compact}[op](state)


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------
def _exact_rope(case, st):
    P, n = case["page"], case["rotary"] // 2
    freq, axis = _frequencies(case)
    q, k, v = (st[x].double() for x in ("q", "k_new", "v_new"))
    lo = [f if case["pairing"] == "halves" else 2 * f for f in range(n)]
    hi = [f + n if case["pairing"] == "halves" else 2 * f + 1 for f in range(n)]
    for f in range(n):
        a = (st["positions"][axis[f]].double() * freq[f])[:, None]
        for x in (q, k):
            z = torch.complex(x[..., lo[f]], x[..., hi[f]]) * torch.polar(torch.ones_like(a), a)
            x[..., lo[f]], x[..., hi[f]] = z.real, z.imag
    pools = [st[x].double() for x in ("k_pool", "v_pool")]
    there = torch.nonzero(st["slots"] >= 0)[:, 0]
    slot = st["slots"][there].long()
    for pool, x in zip(pools, (k, v)):
        by_slot = pool if st["layout"] == "nhd" else pool.transpose(1, 2)
        by_slot[slot // P, slot % P] = x[there]
    return [q] + pools


def _exact_cross(case, st):
    P, H, G, D = case["page"], case["kv_heads"], case["group"], case["head_dim"]
    pools = [st[n] if st["layout"] == "nhd" else st[n].transpose(1, 2) for n in ("k_pool", "v_pool")]
    T = st["q"].shape[0]
    out = torch.zeros(T, H * G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, H * G), -math.inf, dtype=torch.float64, device="cuda")
    t = 0
    for s, (L, n) in enumerate(zip(_lengths(case), _query_lens(case))):
        if L and n:
            p = torch.arange(L, device="cuda")
            k, v = (pool[st["table"][s][p // P].long(), p % P].double() for pool in pools)
            for h in range(H * G):
                x = st["q"][t:t + n, h].double() @ k[:, h // G].T / math.sqrt(D)
                lse[t:t + n, h] = torch.logsumexp(x, 1)
                out[t:t + n, h] = torch.softmax(x, 1) @ v[:, h // G]
        t += n
    return [out] + ([lse] if case["lse"] else [])


def _exact_reserve(table, lens, grow, refs, pools, P):
    """Row after row, as an allocator on the host goes."""
    free = iter([p for p, n in enumerate(refs) if n == 0])
    moves = []
    for s, n in enumerate(grow):
        if n and lens[s] % P and refs[table[s][lens[s] // P]] > 1:
            old, new = table[s][lens[s] // P], next(free)
            refs[old] -= 1
            refs[new] = 1
            table[s][lens[s] // P] = new
            moves.append((old, new))
        for j in range(_pages(lens[s], P), _pages(lens[s] + n, P)):
            table[s][j] = next(free)
            refs[table[s][j]] = 1
        lens[s] += n
    _move(pools, moves)


def _move(pools, moves):
    if moves:
        src, dst = (torch.tensor(x, device="cuda") for x in zip(*moves))
        for pool in pools:
            pool[dst] = pool[src].clone()


def _exact_pages(case, st):
    P, refs, lens = case["page"], st["refs"].tolist(), st["lens"].tolist()
    table, pools = st["table"].tolist(), [p.clone() for p in st["pools"]]
    if case["op"] == "branch":
        width = len(table[0])
        rows, new_lens = [], []
        for p in st["parents"].tolist():
            held = table[p][:_pages(lens[p], P)]
            for page in held:
                refs[page] += 1
            rows.append(held + [0] * (width - len(held)))
            new_lens.append(lens[p])
        _exact_reserve(rows, new_lens, st["grow"].tolist(), refs, pools, P)
        return [_i32(rows), _i32(new_lens), _i32(refs), _i32([0])] + pools
    for s in range(0, len(lens), 2):   # the first pass lets go of the even sequences
        for page in table[s][:_pages(lens[s], P)]:
            refs[page] -= 1
    live = [p for p, n in enumerate(refs) if n > 0]
    free = [p for p in range(len(live)) if refs[p] == 0]
    to = {p: p for p in live}
    moves = list(zip([p for p in live if p >= len(live)], free))
    to.update(moves)
    _move(pools, moves)
    count = [0] * len(refs)
    for p in live:
        count[to[p]] = refs[p]
    page_map = _i32([to.get(p, -1) for p in range(len(refs))])
    full = list(lens)
    for s in range(len(lens)):
        if s % 2 == 0:
            lens[s] = 0
        for j in range(_pages(lens[s], P)):
            table[s][j] = to[table[s][j]]
    _exact_reserve(table, lens, [n if s % 2 == 0 else 0 for s, n in enumerate(full)], count, pools, P)
    return [_i32(table), _i32(lens), _i32(count), page_map, _i32([len(live)]), _i32([0])] + pools


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, st)
    return _exact_cross(case, st) if case["op"] == "cross" else _exact_pages(case, st)
