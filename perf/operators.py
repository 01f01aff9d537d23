"""What is measured of the paged 8-bit cache: its block plan, its store and load, the attention over
all of its keys and the attention over selected ones.

Every case is a call that a server of this framework makes: sequences of different lengths, pages
scattered over the cache, 64 or 128 head dimensions, up to 262,144 keys. The plain forms below are
elementary torch operations in 32 bits; with `own` true the calls are the framework's.
"""
import math
import random

import torch

own = False

TINY = 2.0 ** -100  # the smallest scale of a page
# the code that a page's largest value gets (e4m3: a power of two, so that the scale is exact), and
# the code at which values saturate
FULL = {"int8": 127.0, "e4m3": 256.0}
QMAX = {"int8": 127.0, "e4m3": 448.0}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
FLOAT = {"bf16": torch.bfloat16, "fp16": torch.float16, "int8": torch.int8}
DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # block plan of one decode step: 64 requests, one new token each
        dict(name="plan_decode_r64", op="plan", r=64, ctx_lo=1, ctx_hi=8191, new_lo=1, new_hi=1,
             long_every=0, bs=64, ls=1),
        # block plan of a large admission: 1500 requests, odd prompt lengths, small pages
        dict(name="plan_admit_r1500", op="plan", r=1500, ctx_lo=0, ctx_hi=300, new_lo=0, new_hi=67,
             long_every=0, bs=16, ls=2),
        # decode append: one token of 64 sequences into part-filled pages, read back for the tree
        dict(name="append_r64_int8", op="store", r=64, ctx_lo=1, ctx_hi=4000, new_lo=1, new_hi=1,
             long_every=0, hkv=8, d=128, bs=64, code="int8", src="bf16", ls=3),
        # prompts stored: ragged prompts, eight heads, e4m3 pages of 16
        dict(name="prompts_16k_e4m3", op="store", r=9, ctx_lo=0, ctx_hi=40, new_lo=700, new_hi=2900,
             long_every=0, hkv=8, d=128, bs=16, code="e4m3", src="bf16", ls=4),
        # the smallest call: one sequence of about a thousand keys, one token
        dict(name="decode_r1_n1024_d64", op="attend", r=1, ctx_lo=1023, ctx_hi=1023, new_lo=1,
             new_hi=1, long_every=0, hq=8, hkv=8, d=64, bs=16, code="int8", q="bf16", ls=5),
        # ordinary decode: 64 sequences, grouped heads, ragged lengths
        dict(name="decode_r64_gqa_int8", op="attend", r=64, ctx_lo=900, ctx_hi=16383, new_lo=1,
             new_hi=1, long_every=0, hq=32, hkv=8, d=128, bs=64, code="int8", q="bf16", ls=6),
        # long decode: 4 sequences of 262,144 keys, one query head for each key head
        dict(name="decode_r4_n262144_e4m3", op="attend", r=4, ctx_lo=262143, ctx_hi=262143, new_lo=1,
             new_hi=1, long_every=0, hq=8, hkv=8, d=128, bs=128, code="e4m3", q="bf16", ls=7),
        # a chunk of 2048 new tokens behind 14,336 cached ones, two sequences
        dict(name="chunk_2x2048_n16384", op="attend", r=2, ctx_lo=14336, ctx_hi=14336, new_lo=2048,
             new_hi=2048, long_every=0, hq=32, hkv=8, d=128, bs=64, code="int8", q="bf16", ls=8),
        # whole prompts of odd lengths, d = 64, heads not grouped, e4m3
        dict(name="prompts_r5_d64_e4m3", op="attend", r=5, ctx_lo=0, ctx_hi=0, new_lo=301,
             new_hi=4096, long_every=0, hq=16, hkv=16, d=64, bs=32, code="e4m3", q="fp16", ls=9),
        # a serving step: decode rows with a chunk of a few hundred tokens among them
        dict(name="mixed_r17_chunk511", op="attend", r=17, ctx_lo=100, ctx_hi=7600, new_lo=1,
             new_hi=1, long_every=17, chunk=511, hq=16, hkv=4, d=128, bs=32, code="int8", q="bf16",
             ls=10),
        # routed decode: 64 x 8 queries, up to 96 keys each of caches of 32,768 keys
        dict(name="selected_decode_b64h8", op="selected", r=64, n=32768, nq=1, h=8, hkv=8, d=128,
             bs=64, keys=96, code="int8", q="int8"),
        # routed prefill at 2 x 8 x 16,384, d = 64
        dict(name="selected_prefill_b2h8", op="selected", r=2, n=16384, nq=16384, h=8, hkv=8, d=64,
             bs=32, keys=96, code="int8", q="int8"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "store", "attend", "attend", "attend", "selected"])
    ls = rng.randrange(1 << 30)
    d = rng.choice([64, 128])
    bs = rng.choice([16, 32, 64, 128])
    code = rng.choice(["int8", "e4m3"])
    if op == "plan":
        return dict(op=op, r=_log(rng, 1, 1500), ctx_lo=0, ctx_hi=_log(rng, 10, 8000), new_lo=0,
                    new_hi=_log(rng, 1, 70), long_every=0, bs=bs, ls=ls)
    if op == "store":
        r = _log(rng, 1, 128)
        return dict(op=op, r=r, ctx_lo=0, ctx_hi=_log(rng, 10, 3000), new_lo=1,
                    new_hi=max(1, _log(rng, 1, 30000) // r), long_every=0, hkv=rng.choice([1, 2, 5, 8]),
                    d=d, bs=bs, code=code, src=rng.choice(["bf16", "fp16"]), ls=ls)
    if op == "selected":
        r, hkv = _log(rng, 1, 64), rng.choice([1, 2, 4, 8])
        g = rng.choice([1, 1, 2, 4])
        n = _log(rng, 40, 32768)
        nq = 1 if rng.random() < 0.5 else min(n, max(1, _log(rng, 2, 100000) // (r * hkv * g)))
        return dict(op=op, r=r, n=n, nq=nq, h=hkv * g, hkv=hkv, d=d, bs=bs,
                    keys=rng.choice([96, 96, 48, 33]), code=code, q=rng.choice(["int8", "bf16", "fp16"]))
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 8, 16])
    kind = rng.choice(["decode", "decode", "chunk", "mixed"])
    base = dict(op=op, hq=hq, hkv=hkv, d=d, bs=bs, code=code, q=rng.choice(["bf16", "fp16"]), ls=ls)
    if kind == "decode":  # single tokens, and a few tokens a sequence
        r = _log(rng, 1, 64)
        n = _log(rng, 16, min(120000, 2500000 // (r * hkv)))
        return dict(base, r=r, ctx_lo=max(0, n // 3), ctx_hi=n, new_lo=1,
                    new_hi=rng.choice([1, 1, 1, 4]), long_every=0)
    if kind == "chunk":
        r = rng.randint(1, 4)
        new = _log(rng, 17, 2048)
        ctx = rng.choice([0, _log(rng, 20, max(21, min(16000, 800000000 // (r * hq * new))))])
        return dict(base, r=r, ctx_lo=ctx // 2, ctx_hi=ctx, new_lo=max(1, new // 3), new_hi=new,
                    long_every=0)
    return dict(base, r=rng.randint(2, 20), ctx_lo=0, ctx_hi=_log(rng, 50, 4000), new_lo=1, new_hi=2,
                long_every=rng.randint(2, 9), chunk=_log(rng, 20, 400))


def lengths(case):
    """Tokens in the cache and new tokens of every request: of the case alone, not of the seed."""
    rng = random.Random(case["ls"])
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["r"])]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["r"])]
    if case["long_every"]:
        new = [case["chunk"] if (r + 1) % case["long_every"] == 0 else n for r, n in enumerate(new)]
    return ctx, new


def _ceil(a, b):
    return -(-a // b)


def counts(case):
    """Keys of each query row of a head in a case of selected keys."""
    n, nq, keys = case["n"], case["nq"], case["keys"]
    return [min(i + 1, keys) for i in range(n - nq, n)]


def work(case):
    if case["op"] == "plan":
        ctx, new = lengths(case)
        bs = case["bs"]
        need = sum(_ceil(c + n, bs) - _ceil(c, bs) for c, n in zip(ctx, new))
        return {"bytes": 16 * case["r"] + 8 * need + 12 * sum(new) + 16, "flops": 0}
    if case["op"] == "store":
        ctx, new = lengths(case)
        bs, row = case["bs"], 2 * case["hkv"] * case["d"]
        back = sum(c % bs + n for c, n in zip(ctx, new))  # tokens of the touched pages, read back
        pages = sum(_ceil(c + n, bs) - c // bs for c, n in zip(ctx, new))
        return {"bytes": sum(new) * (3 * row + 8) + back * (3 * row + 8) + pages * 16 * case["hkv"],
                "flops": 2 * row * (sum(new) + back)}
    if case["op"] == "attend":
        ctx, new = lengths(case)
        kv = sum(c + n for c, n in zip(ctx, new))
        pages = sum(_ceil(c + n, case["bs"]) for c, n in zip(ctx, new))
        seen = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
        t = sum(new)
        return {"bytes": kv * case["hkv"] * case["d"] * 2 + pages * (4 + 8 * case["hkv"])
                + t * case["hq"] * (4 * case["d"] + 4),
                "flops": 4 * case["d"] * case["hq"] * seen}
    rows = case["r"] * case["h"]
    per = rows * sum(counts(case))
    q = rows * case["nq"]
    # each cached key is read at least once, but no more than the selections name
    kv = min(per, case["r"] * case["hkv"] * case["n"])
    return {"bytes": kv * 2 * case["d"] + per * 4 + q * (4 + 6 * case["d"]),
            "flops": 4 * case["d"] * per}


# ---------------------------------------------------------------- inputs

def _codes(shape, code, g):
    out = torch.empty(shape, dtype=CODE[code], device=DEV)
    flat = out.view(-1)
    step = 1 << 27
    for a in range(0, flat.numel(), step):
        x = torch.randn(min(step, flat.numel() - a), generator=g, device=DEV)
        x = (x * 38).round_().clamp_(-127, 127) if code == "int8" else (x * 130).clamp_(-448, 448)
        flat[a:a + x.numel()] = x.to(CODE[code])
    return out


def _cache(blocks, hkv, bs, d, code, g):
    s = 1.0 if code == "int8" else 0.29
    scale = lambda: (0.026 * s * torch.exp(0.4 * torch.randn(blocks, hkv, generator=g, device=DEV)))  # noqa: E731
    return dict(k=_codes((blocks, hkv, bs, d), code, g), v=_codes((blocks, hkv, bs, d), code, g),
                k_scale=scale(), v_scale=scale())


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _table(held, width, blocks, g):
    """Scattered pages: request r has the next held[r] pages of a random order."""
    order = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    col = torch.arange(width, device=DEV)
    first = torch.tensor([sum(held[:r]) for r in range(len(held))], device=DEV)
    has = col[None] < torch.tensor(held, device=DEV)[:, None]
    at = (first[:, None] + col[None]).clamp(max=blocks - 1)
    return torch.where(has, order[at], torch.full_like(order[at], -1)).contiguous(), order


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "selected":
        r, n, nq, d, h, m = (case[x] for x in ("r", "n", "nq", "d", "h", "keys"))
        width = _ceil(n, case["bs"])
        s["table"], _ = _table([width] * r, width, r * width, g)
        s["cache"] = _cache(r * width, case["hkv"], case["bs"], d, case["code"], g)
        # the window's 16 keys and routed ones spread over the past, ascending, -1 behind them
        i = torch.arange(n - nq, n, device=DEV)
        cnt = torch.tensor(counts(case), device=DEV)
        win = cnt.clamp(max=16)
        routed = cnt - win
        j = torch.arange(m, device=DEV)
        u = torch.rand(r, h, nq, m, generator=g, device=DEV, dtype=torch.float64)
        past = (i + 1 - win)[:, None].double()
        far = ((j + u) * past / routed.clamp(min=1)[:, None]).floor().long()
        far = torch.minimum(far, (past - 1).clamp(min=0).long())
        near = (i + 1 - win)[:, None] + j[None] - routed[:, None]
        idx = torch.where(j[None] < routed[:, None], far, near.expand_as(far))
        s["idx"] = torch.where(j[None] < cnt[:, None], idx, -1).to(torch.int32).contiguous()
        s["count"] = cnt.to(torch.int32).expand(r, h, nq).contiguous()
        s["ctx"], s["len"] = _ints([n - nq] * r), _ints([n] * r)
        if case["q"] == "int8":
            s["q"] = torch.randint(-16, 17, (r, h, nq, d), generator=g, device=DEV, dtype=torch.int8)
            s["scale"] = 0.15 / math.sqrt(d)
        else:
            s["q"] = (1.5 * torch.randn(r, h, nq, d, generator=g, device=DEV)).to(FLOAT[case["q"]])
            s["scale"] = 1.0 / math.sqrt(d)
        return s
    ctx, new = lengths(case)
    bs, r, t = case["bs"], case["r"], sum(new)
    ends = [_ceil(c + n, bs) for c, n in zip(ctx, new)]
    s["ctx"], s["new"] = _ints(ctx), _ints(new)
    s["len"] = _ints([c + n for c, n in zip(ctx, new)])
    s["tokens"] = t
    if case["op"] == "plan":
        held = [_ceil(c, bs) for c in ctx]
        blocks = sum(ends) + 7
        s["table"], order = _table(held, max(ends) + 1, blocks, g)
        s["free"] = order[sum(held):].contiguous()
        s["first"] = _ints([0])
        return s
    blocks = sum(ends) + 3
    s["table"], _ = _table(ends, max(ends), blocks, g)
    s["cache"] = _cache(blocks, case["hkv"], bs, case["d"], case["code"], g)
    start = [sum(new[:i]) for i in range(r + 1)]
    s["q_start"] = _ints(start)
    if case["op"] == "store":
        pos = torch.cat([torch.arange(c, c + n) for c, n in zip(ctx, new)])
        row = torch.cat([torch.full((n,), i) for i, n in enumerate(new)])
        s["slots"] = _slots(s["table"], row.to(DEV), pos.to(DEV), bs)
        pos = torch.cat([torch.arange(c - c % bs, c + n) for c, n in zip(ctx, new)])
        row = torch.cat([torch.full((c % bs + n,), i) for i, (c, n) in enumerate(zip(ctx, new))])
        s["back"] = _slots(s["table"], row.to(DEV), pos.to(DEV), bs)
        # keys and values of a fused projection: one row holds both, with outlying channels
        x = torch.randn(t, 2, case["hkv"], case["d"], generator=g, device=DEV)
        x[..., ::37] *= 4
        s["kv"] = x.to(FLOAT[case["src"]])
        return s
    s["max_q"] = max(new)
    s["max_len"] = max(ends) * bs
    q = torch.randn(t, case["hq"], case["d"], generator=g, device=DEV)
    s["q"] = (2.0 * q).to(FLOAT[case["q"]])
    s["scale"] = 1.0 / math.sqrt(case["d"])
    return s


def _slots(table, row, pos, bs):
    return (table[row, pos // bs].long() * bs + pos % bs).contiguous()


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        from tree_routed_sparse_b200 import cache
        if op == "plan":
            got = cache.plan_blocks(state["ctx"], state["new"], state["table"], state["free"],
                                    state["first"], state["tokens"], state["case"]["bs"])
            return dict(got, table=state["table"])
        c = state["cache"]
        if op == "store":
            cache.store_cache(state["kv"][:, 0], state["kv"][:, 1], c, state["slots"])
            back = cache.load_cache(c, state["back"])
            return dict(back, k_scale=c["k_scale"], v_scale=c["v_scale"])
        if op == "attend":
            return cache.attend_cache(state["q"], c, state["table"], state["ctx"], state["len"],
                                      state["q_start"], max_q=state["max_q"], want_lse=True)
        return dict(out=cache.attend_cache_selected(
            state["q"], c, state["table"], state["ctx"], state["len"], state["idx"], state["count"],
            scale=state["scale"]))
    return {"plan": _plan, "store": _store, "attend": _attend, "selected": _selected}[op](state)


def _plan(s):
    bs, t = s["case"]["bs"], s["tokens"]
    ctx, new, table, free = s["ctx"].long(), s["new"].long(), s["table"], s["free"]
    start = torch.cat([new.new_zeros(1), new.cumsum(0)])
    held, total = (ctx + bs - 1) // bs, (ctx + new + bs - 1) // bs
    need = total - held
    base = s["first"].long() + need.cumsum(0) - need
    col = torch.arange(table.shape[1], device=table.device)
    at = base[:, None] + col[None] - held[:, None]
    mine = (col[None] >= held[:, None]) & (col[None] < total[:, None])
    table.copy_(torch.where(mine, free[at.clamp(0, free.numel() - 1)], table))
    tok = torch.arange(t, device=table.device)
    row = torch.searchsorted(start[1:], tok, right=True)
    pos = ctx[row] + tok - start[row]
    return dict(q_start=start.int(), seq_len=(ctx + new).int(), slots=_slots(table, row, pos, bs),
                positions=pos.int(), free_next=(s["first"] + need.sum()).int(), table=table)


def _encode(x, code):
    q = QMAX[code]
    return (x.round() if code == "int8" else x).clamp(-q, q).to(CODE[code])


def _store_one(x, codes, scale, slots, code):
    """x [T, H, d] float32 into codes [blocks, H, bs, d] with one scale for each block and head."""
    blocks, heads, bs, d = codes.shape
    page, off = slots // bs, slots % bs
    amax = x.new_zeros(blocks, heads)
    amax.scatter_reduce_(0, page[:, None].expand(-1, heads), x.abs().amax(-1), "amax")
    first = torch.full((blocks,), bs, device=x.device).scatter_reduce_(0, page, off, "amin")
    touched = (first < bs)[:, None]
    old = torch.where(first[:, None] == 0, torch.zeros_like(scale), scale)
    top = torch.maximum(torch.maximum(old, amax / FULL[code]), torch.full_like(old, TINY))
    factor = old / top
    back = (torch.arange(bs, device=x.device)[None] < first[:, None]) & touched
    again = _encode(codes.float() * factor[:, :, None, None], code)
    codes.copy_(torch.where(back[:, None, :, None], again.float(), codes.float()).to(codes.dtype))
    scale.copy_(torch.where(touched, top, scale))
    got = _encode(x / top[page][..., None], code)
    # 8-bit floats are moved as bytes: indexing is not there for them
    codes.view(torch.int8)[page, :, off] = got.view(torch.int8)


def _load_one(codes, scale, slots):
    bs = codes.shape[2]
    page, off = slots // bs, slots % bs
    got = codes.view(torch.int8)[page, :, off].view(codes.dtype)
    return (got.float() * scale[page][..., None]).to(torch.bfloat16)


def _store(s):
    c, code = s["cache"], s["case"]["code"]
    _store_one(s["kv"][:, 0].float(), c["k"], c["k_scale"], s["slots"], code)
    _store_one(s["kv"][:, 1].float(), c["v"], c["v_scale"], s["slots"], code)
    return dict(K=_load_one(c["k"], c["k_scale"], s["back"]),
                V=_load_one(c["v"], c["v_scale"], s["back"]),
                k_scale=c["k_scale"], v_scale=c["v_scale"])


def _pages(codes, scale, table):
    """The keys or values of every request, as numbers: [R, H, pages * bs, d]."""
    at = table.clamp(min=0).long()
    got = codes.view(torch.int8)[at].view(codes.dtype).float() * scale[at][..., None, None]
    r, p, h, bs, d = got.shape
    return got.transpose(1, 2).reshape(r, h, p * bs, d)


def _attend(s):
    q, c, table = s["q"], s["cache"], s["table"]
    t, hq, d = q.shape
    r, hkv, maxq = table.shape[0], c["k"].shape[1], s["max_q"]
    start, ctx = s["q_start"].long(), s["ctx"].long()
    tok = torch.arange(t, device=q.device)
    row = torch.searchsorted(start[1:], tok, right=True)
    at = tok - start[row]
    padded = q.new_zeros(r, maxq, hq, d, dtype=torch.float32)
    padded[row, at] = q.float()
    padded = padded.view(r, maxq, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    padded = padded.reshape(r, hkv, hq // hkv * maxq, d)
    k = _pages(c["k"], c["k_scale"], table)
    score = (padded @ k.transpose(-1, -2)) * s["scale"]
    del k
    score = score.view(r, hkv, hq // hkv, maxq, -1)
    seen = torch.minimum(ctx[:, None] + torch.arange(maxq, device=q.device) + 1, s["len"][:, None])
    key = torch.arange(score.shape[-1], device=q.device)
    hidden = key[None, None] >= seen[..., None]
    score.masked_fill_(hidden[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score = score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    lse = (total.log() + top).view(r, hq, maxq)
    v = _pages(c["v"], c["v_scale"], table)
    out = (score.view(r, hkv, hq // hkv * maxq, -1) @ v).view(r, hkv, hq // hkv, maxq, d) / total
    return dict(out=out.view(r, hq, maxq, d)[row, :, at].to(q.dtype), lse=lse[row, :, at])


def _selected(s):
    q, c, table, idx = s["q"], s["cache"], s["table"], s["idx"]
    r, h, nq, d = q.shape
    hkv, bs = c["k"].shape[1], c["k"].shape[2]
    at = idx.clamp(min=0).long()
    page = table.long()[torch.arange(r, device=q.device)[:, None, None, None], at // bs]
    head = (torch.arange(h, device=q.device) // (h // hkv))[None, :, None, None]
    off = at % bs
    take = lambda x, w: (x.view(torch.int8)[page, head, off].view(x.dtype).float()  # noqa: E731
                         * w[page, head][..., None])
    score = (take(c["k"], c["k_scale"]) @ q.float()[..., None])[..., 0] * s["scale"]
    seen = torch.arange(idx.shape[-1], device=q.device) < s["count"][..., None]
    score = score.masked_fill(~seen, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    return dict(out=(p[..., None, :] @ take(c["v"], c["v_scale"]))[..., 0, :])


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    if case["op"] == "plan":  # whole numbers
        return None
    s = prepare(case, seed)
    return {"store": _exact_store, "attend": _exact_attend, "selected": _exact_selected}[case["op"]](s)


def _values(codes):
    """The numbers that 8-bit codes stand for, by a table of all 256."""
    if codes.dtype == torch.int8:
        return codes.double()
    b = torch.arange(256, dtype=torch.float64)
    sign, e, m = b // 128, b % 128 // 8, b % 8
    mag = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7))
    lut = torch.where(sign > 0, -mag, mag).to(codes.device)
    return lut[codes.view(torch.uint8).int()]


def _nearest(x, code):
    """x rounded to the nearest code's number, ties to even, saturated; 64 bits."""
    if code == "int8":
        return torch.round(x).clamp(-127, 127)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30)))
    step = 2.0 ** (e.clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_store(s):
    c, case = s["cache"], s["case"]
    bs, full = case["bs"], FULL[case["code"]]
    ctx, new = lengths(case)
    out = {}
    for which, (name, codes, scale) in enumerate((("K", c["k"], c["k_scale"]), ("V", c["v"], c["v_scale"]))):
        x = s["kv"][:, which].double()
        scales = scale.double()
        table = s["table"].tolist()
        rows, t = [], 0
        for r, (lo, n) in enumerate(zip(ctx, new)):
            end = lo + n
            for p in range(lo // bs, _ceil(end, bs)):
                page, a, b = table[r][p], max(lo, p * bs), min(end, (p + 1) * bs)
                part = x[t:t + b - a]
                t += b - a
                kept = a - p * bs
                old = scales[page] if kept else torch.zeros_like(scales[page])
                top = torch.maximum(old, part.abs().amax((0, 2)) / full).clamp(min=TINY)
                if kept:
                    was = _values(codes[page, :, :kept]).transpose(0, 1)
                    rows.append(_nearest(was * (old / top)[None, :, None], case["code"]) * top[None, :, None])
                rows.append(_nearest(part / top[None, :, None], case["code"]) * top[None, :, None])
                scales[page] = top
        out[name] = torch.cat(rows)
        out["k_scale" if name == "K" else "v_scale"] = scales
    return out


def _exact_attend(s):
    q, c, table = s["q"].double(), s["cache"], s["table"].long()
    hq, hkv, bs = q.shape[1], c["k"].shape[1], c["k"].shape[2]
    ctx, new = lengths(s["case"])
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
    t = 0
    for r, (lo, n) in enumerate(zip(ctx, new)):
        pages = table[r, :_ceil(lo + n, bs)]
        gone = torch.arange(lo + n, device=q.device)[None] > torch.arange(lo, lo + n, device=q.device)[:, None]
        for h in range(hkv):
            k, v = ((_values(x[pages, h]) * w[pages, h].double()[:, None, None]).flatten(0, 1)[:lo + n]
                    for x, w in ((c["k"], c["k_scale"]), (c["v"], c["v_scale"])))
            for j in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                a = q[t:t + n, j] @ k.T * s["scale"]
                a = a.masked_fill(gone, -math.inf)
                lse[t:t + n, j] = torch.logsumexp(a, -1)
                out[t:t + n, j] = torch.softmax(a, -1) @ v
        t += n
    return dict(out=out, lse=lse)


def _exact_selected(s):
    q, c, table = s["q"].double(), s["cache"], s["table"].long()
    r, h, nq, d = q.shape
    hkv, bs = c["k"].shape[1], c["k"].shape[2]
    out = torch.empty_like(q)
    for b in range(r):
        for j in range(h):
            w = j // (h // hkv)
            k, v = ((_values(x[table[b], w]) * y[table[b], w].double()[:, None, None]).flatten(0, 1)
                    for x, y in ((c["k"], c["k_scale"]), (c["v"], c["v_scale"])))
            at, n = s["idx"][b, j].long(), s["count"][b, j]
            a = torch.einsum("qd,qmd->qm", q[b, j], k[at.clamp(min=0)]) * s["scale"]
            off = torch.arange(at.shape[1], device=q.device)[None] >= n[:, None]
            p = torch.softmax(a.masked_fill(off, -math.inf), -1)
            out[b, j] = torch.einsum("qm,qmd->qd", p, v[at.clamp(min=0)])
    return dict(out=out)
