"""The paged 8-bit cache against its definition in 64 bits (tests/cache_util.py)."""
import math
import os
import subprocess
import sys
import threading

import pytest
import torch

from cache_util import (SAT, attend_ref, ceil_div, numbers, plan_ref, random_cache, scattered_table,
                        score_error, store_ref)

pytestmark = pytest.mark.gpu
I8, E4 = torch.int8, torch.float8_e4m3fn
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def C():
    from tree_routed_sparse_b200 import build
    build.build()
    from tree_routed_sparse_b200 import cache
    return cache


def ints(v, dev="cuda"):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def bits(x):
    return x.view(torch.uint8) if x.element_size() == 1 else x


# ------------------------------------------------------------------ plan

PLANS = {
    "one_token": dict(ctx=[0], new=[1], width=1, free=[3], bs=16),
    "decode": dict(ctx=[15, 16, 17, 0, 31], new=[1] * 5, width=3, free=list(range(9, 0, -1)), bs=16),
    "zero_lengths": dict(ctx=[0, 0, 5, 0], new=[0, 0, 0, 7], width=2, free=[4, 2], bs=32),
    "negative": dict(ctx=[-3, 4], new=[5, -1], width=2, free=[4, 2], bs=32),
    "many_blocks": dict(ctx=[3, 100], new=[4000, 333], width=40, free=list(range(50)), bs=128),
    "padded": dict(ctx=[5, 9], new=[3, 20], width=4, free=[7, 8, 1], bs=16, pad=11),
    "capacity": dict(ctx=[30, 0, 64], new=[10, 3, 1], width=2, free=list(range(9)), bs=32),
    "list_ends": dict(ctx=[1, 16, 0, 3], new=[40, 1, 17, 2], width=4, free=[5, 6], bs=16),
    "list_empty": dict(ctx=[1, 16], new=[3, 1], width=4, free=[], bs=16),
    "rows_end": dict(ctx=[1, 16, 2], new=[3, 9, 4], width=4, free=[5, 6], bs=16, pad=-8),
    "bad_blocks": dict(ctx=[1, 17, 0], new=[3, 1, 40], width=4, free=[5, -7, 99], bs=16, spoil=True),
    "late_first": dict(ctx=[0, 0], new=[20, 20], width=4, free=[5, 6, 7, 8, 9], bs=16, first=2),
}


@pytest.mark.parametrize("name", sorted(PLANS))
def test_plan(C, name):
    c = dict(PLANS[name])
    r = len(c["ctx"])
    blocks, bs, first = 60, c["bs"], c.get("first", 0)
    tokens = max(0, sum(max(n, 0) for n in c["new"]) + c.get("pad", 0))
    table = [[(20 + 7 * i + j) if j < ceil_div(max(c["ctx"][i], 0), bs) else -5
              for j in range(c["width"])] for i in range(r)]
    if c.get("spoil"):
        table[1][1] = 77
    want = plan_ref(c["ctx"], c["new"], table, c["free"], first, tokens, bs, blocks)
    tab = ints(table)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = C.plan_blocks(ints(c["ctx"]), ints(c["new"]), tab, ints(c["free"]), ints([first]), tokens,
                        bs, blocks=blocks, dev_err=err)
    assert got["q_start"].tolist() == want[0]
    assert got["seq_len"].tolist() == want[1]
    assert got["slots"].tolist() == want[2]
    assert got["positions"].tolist() == want[3]
    assert got["free_next"].tolist() == [want[4]]
    assert tab.tolist() == want[5]
    assert err.item() == want[6]


@pytest.mark.parametrize("r,top", [(1, 70000), (513, 40), (8192, 9)])
def test_plan_many(C, r, top):
    g = torch.Generator().manual_seed(r)
    ctx = torch.randint(0, 300, (r,), generator=g).tolist()
    new = torch.randint(0, top, (r,), generator=g).tolist()
    bs = 16
    width = ceil_div(300 + top, bs)
    table = [[1000 + i + j if j < ceil_div(ctx[i], bs) else -1 for j in range(width)]
             for i in range(r)]
    free = list(range(200000, 200000 + sum(ceil_div(a + b, bs) - ceil_div(a, bs)
                                           for a, b in zip(ctx, new)) + 3))
    want = plan_ref(ctx, new, table, free, 0, sum(new) + 5, bs, 1 << 20)
    tab = ints(table)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = C.plan_blocks(ints(ctx), ints(new), tab, ints(free), ints([0]), sum(new) + 5, bs,
                        dev_err=err)
    for key, w in zip(("q_start", "seq_len", "slots", "positions"), want):
        assert got[key].tolist() == w, key
    assert tab.tolist() == want[5] and got["free_next"].item() == want[4] and err.item() == 0


@pytest.mark.parametrize("counts", [[6127, 6128, 6143, 6144, 8192, 6127], [6143], [8192, 6144]])
def test_plan_at_the_edge_of_the_default_shared_memory(counts):
    """Request counts whose sums fill what a kernel gets of shared memory without asking, in a
    process of their own: an earlier, larger call leaves the limit raised."""
    code = f"""
import sys
sys.path[:0] = ["tests", "."]
import torch
from tree_routed_sparse_b200 import cache as C
ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
for r in {counts}:
    got = C.plan_blocks(ints([0] * r), ints([1] * r), torch.full((r, 1), -1, dtype=torch.int32,
                        device="cuda"), ints(list(range(r))), ints([0]), r, 16)
    assert got["slots"].tolist() == [16 * i for i in range(r)], r
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                          timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_plan_from_two_threads(C):
    """Plans of different sizes from host threads with streams of their own: none changes what
    another one's kernel is launched with."""
    faults = []

    def work(r):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                args = (ints([0] * r), ints([1] * r),
                        torch.full((r, 1), -1, dtype=torch.int32, device="cuda"),
                        ints(list(range(r))), ints([0]))
                q, seq, nxt = ints([0] * (r + 1)), ints([0] * r), ints([0])
                slots, pos = torch.zeros(r, dtype=torch.int64, device="cuda"), ints([0] * r)
                torch.cuda.current_stream().synchronize()
                L, st = alhr.lib(), torch.cuda.current_stream().cuda_stream
                ptr = [x.data_ptr() for x in (*args, q, seq, slots, pos, nxt)]
                for _ in range(2000):
                    got = L.alhr_plan_blocks(r, 1, 16, r, r, r, *ptr, None, st)
                    assert got == 0, (r, got)
                torch.cuda.current_stream().synchronize()
                assert slots.tolist() == [16 * i for i in range(r)]
        except Exception as e:  # noqa: BLE001 - handed to the test
            faults.append(e)

    from tree_routed_sparse_b200 import alhr
    threads = [threading.Thread(target=work, args=(r,)) for r in (8192, 6200, 8192, 6200)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not faults, faults[0]


def test_plan_without_requests(C):
    got = C.plan_blocks(ints([]), ints([]), torch.empty(0, 3, dtype=torch.int32, device="cuda"),
                        ints([1]), ints([1]), 4, 16)
    assert got["q_start"].tolist() == [0] and got["slots"].tolist() == [-1] * 4
    assert got["positions"].tolist() == [-1] * 4 and got["free_next"].tolist() == [1]


# ------------------------------------------------------------------ store and load

def runs(spec, blocks, bs):
    """Slots of the listed (page, first offset, rows) pieces; page -1: rows without a slot."""
    out = []
    for page, off, n in spec:
        out += [-1] * n if page < 0 else [page * bs + off + i for i in range(n)]
    return torch.tensor(out, dtype=torch.int64)


STORES = {
    "one": [(2, 0, 1)],
    "append": [(1, 5, 1), (0, 15, 1), (3, 1, 2)],
    "whole": [(1, 0, 16), (2, 0, 16), (0, 0, 16)],
    "ragged": [(4, 3, 13), (5, 0, 16), (6, 0, 7), (-1, 0, 3), (2, 9, 4)],
    "ends": [(0, 15, 1), (1, 15, 1), (2, 0, 1), (7, 0, 5)],
}


@pytest.mark.parametrize("dtype", [I8, E4])
@pytest.mark.parametrize("src", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("name,d,bs,heads", [
    ("one", 64, 16, 1), ("append", 128, 16, 3), ("whole", 64, 16, 2), ("ragged", 128, 16, 5),
    ("ends", 64, 16, 8), ("ragged", 64, 128, 2), ("append", 128, 64, 8), ("whole", 128, 32, 1)])
def test_store_bits(C, dtype, src, name, d, bs, heads):
    """Codes and scales to the bit: rows before a run are rounded anew when the scale grew, rows
    behind it and other blocks keep what they held."""
    g = torch.Generator(device="cuda").manual_seed(5)
    blocks = 8
    cache = random_cache(blocks, heads, bs, d, dtype, g, "cuda")
    spec = [(p, off * bs // 16, n if n < 16 else bs) for p, off, n in STORES[name]]
    slots = runs(spec, blocks, bs)
    t = slots.numel()
    # a fused projection: keys and values are slices of one row; some runs raise the scale
    x = torch.randn(t, 2 * heads + 1, d, generator=g, device="cuda")
    x *= torch.where(torch.arange(t, device="cuda") % 3 == 0, 6.0, 1.5)[:, None, None]
    x = x.to(src)
    K, V = x[:, :heads], x[:, heads + 1:]
    ref = {}
    for key, y in (("k", K), ("v", V)):
        codes, scale = cache[key].cpu().clone(), cache[key + "_scale"].cpu().clone()
        store_ref(y.float().cpu(), codes, scale, slots)
        ref[key], ref[key + "_scale"] = codes, scale
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    C.store_cache(K, V, cache, slots.cuda(), dev_err=err)
    for key in ("k_scale", "v_scale", "k", "v"):
        assert torch.equal(bits(cache[key].cpu()), bits(ref[key])), key
    assert err.item() == 0
    # what is stored is within half a step of what was given (e4m3: half of 1/8 of the number's
    # power of two, at most x / 16, and half the smallest step); rows before a run carry the error
    # of two roundings, so only the run's own rows are held to it. By arithmetic: the quotient x / s
    # rounds at 2^-24 of itself before it is rounded to a code, which moves a number at the border
    # by 2^-24 |x|; code * s rounds at 2^-24 (|x| + half), and so does the difference taken here:
    # below 2^-22 |x| + 2^-20 half together
    back = C.load_cache(cache, slots.cuda(), dtype=torch.float32)
    for key, y in (("K", K), ("V", V)):
        s = cache[key.lower() + "_scale"][(slots.clamp(min=0) // bs).cuda()][..., None]
        on = (slots >= 0).cuda()[:, None, None]
        half = s * 0.5 if dtype == I8 else torch.maximum(y.float().abs() / 16, s * 2.0 ** -10)
        far = ((back[key] - y.float()).abs() - half * (1 + 2.0 ** -20)
               - y.float().abs() * 2.0 ** -22)
        assert float(torch.where(on, far, -1.0).max()) <= 0
        assert float(torch.where(on, 0.0, back[key]).abs().max()) == 0


def large_store(kind, bs, g):
    """(spec of runs, blocks) of a store whose warps look through 16 tokens each: prompts of ragged
    lengths behind part-filled blocks, or single tokens; rows without a slot among them."""
    spec, page = [], 0
    rand = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))
    while sum(n for *_, n in spec) < 1100:
        if rand(0, 9) == 0:
            spec.append((-1, 0, rand(1, 3 if kind == "single" else 40)))
        if kind == "single":
            spec.append((page, rand(0, bs - 1), 1))
        else:
            off, left = rand(0, bs - 1), rand(1, 5 * bs if kind == "long" else bs + 9)
            while left:
                n = min(left, bs - off)
                spec.append((page, off, n))
                page, off, left = page + 1, 0, left - n
        page += 1 + (rand(0, 3) == 0)
    # pages that follow one another in the call lie anywhere in the cache, some side by side
    order = torch.randperm(page // 2, generator=g).tolist()
    where = [2 * order[p // 2] + p % 2 if p // 2 < len(order) else p for p in range(page)]
    return [(p if p < 0 else where[p], o, n) for p, o, n in spec], page + 1


@pytest.mark.parametrize("kind,bs,d,dtype,src", [
    ("long", 128, 128, E4, torch.bfloat16), ("long", 64, 64, I8, torch.float32),
    ("long", 16, 128, I8, torch.float16), ("short", 32, 64, E4, torch.float32),
    ("short", 128, 64, I8, torch.bfloat16), ("single", 16, 64, E4, torch.float16),
    ("single", 128, 128, I8, torch.bfloat16)])
def test_store_bits_of_many_tokens(C, kind, bs, d, dtype, src):
    """Stores of more than 16,384 (token, head, keys or values) triples, of which a warp takes all
    runs that begin in 16 tokens: several of them, and runs that go on past its 32 lanes."""
    g = torch.Generator().manual_seed(len(kind) + bs + d)
    heads = 8
    spec, blocks = large_store(kind, bs, g)
    slots = runs(spec, blocks, bs)
    t = slots.numel()
    assert t * heads * 2 > 16384 and len({p for p, *_ in spec if p >= 0}) == sum(p >= 0 for p, *_ in spec)
    gg = torch.Generator(device="cuda").manual_seed(7)
    cache = random_cache(blocks, heads, bs, d, dtype, gg, "cuda")
    x = torch.randn(t, 2 * heads, d, generator=gg, device="cuda")
    x *= torch.where(torch.arange(t, device="cuda") % 5 == 0, 6.0, 1.0)[:, None, None]
    x = x.to(src)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref = {}
    for key, y in (("k", x[:, :heads]), ("v", x[:, heads:])):
        codes, scale = cache[key].cpu().clone(), cache[key + "_scale"].cpu().clone()
        store_ref(y.float().cpu(), codes, scale, slots)
        ref[key], ref[key + "_scale"] = codes, scale
    C.store_cache(x[:, :heads], x[:, heads:], cache, slots.cuda(), dev_err=err)
    for key in ("k_scale", "v_scale", "k", "v"):
        assert torch.equal(bits(cache[key].cpu()), bits(ref[key])), key
    assert err.item() == 0


@pytest.mark.parametrize("dtype", [I8, E4])
def test_store_special_values(C, dtype):
    """Zeros, tiny and huge numbers, infinities and NaN; NaN in rows without a slot is not read."""
    bs, d, heads = 16, 64, 1
    cache = C.alloc_cache(4, heads, bs, d, dtype)
    x = torch.zeros(6, heads, d)
    x[1] = 1e-44
    x[2] = 3e38
    x[2, 0, 3] = -3e38
    x[3, 0, :5] = torch.tensor([math.inf, -math.inf, math.nan, 1.0, -0.5])
    x[4] = math.nan
    x[5, 0, 7] = 2.0
    slots = torch.tensor([0, bs, 2 * bs, 3 * bs, -1, 3 * bs + 1])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    C.store_cache(x.cuda(), x.cuda(), cache, slots.cuda(), dev_err=err)
    assert err.item() == C.DEVERR_NONFINITE
    # the row without a slot parts block 3 in two runs of one call: what that block then holds is
    # not specified, the other blocks are; its runs in calls of their own are
    codes, scale = torch.zeros(4, heads, bs, d).to(dtype), torch.zeros(4, heads)
    store_ref(x, codes, scale, slots)
    assert torch.equal(bits(cache["k"].cpu())[:3], bits(codes)[:3])
    assert torch.equal(cache["v_scale"].cpu()[:3], scale[:3])
    for part in (slice(3, 4), slice(4, 6)):
        store_ref(x[part], codes, scale, slots[part])
        C.store_cache(x[part].cuda(), x[part].cuda(), cache, slots[part].cuda())
        if part.start == 3:
            top = cache["k"][3, 0, 0].float().cpu()
            assert top[0] == SAT[dtype] and top[1] == -SAT[dtype] and top[2] == 0
    assert torch.equal(bits(cache["k"].cpu()), bits(codes))
    assert torch.equal(cache["v_scale"].cpu(), scale)
    err.zero_()
    C.store_cache(x[4:].cuda(), x[4:].cuda(), cache, torch.tensor([-1, 5], device="cuda"),
                  dev_err=err)
    assert err.item() == 0


@pytest.mark.parametrize("dtype", [I8, E4])
@pytest.mark.parametrize("src", [torch.bfloat16, torch.float32])
def test_store_infinities_beside_the_largest_numbers(C, dtype, src):
    """Infinities and NaN in runs whose finite numbers reach the top of the type: the finite ones
    are stored as without them, the infinities saturated whatever the scale."""
    top = torch.finfo(src).max
    x = torch.linspace(-1, 1, 64).repeat(3, 1, 1)
    x[0] *= top
    x[0, 0, :3] = torch.tensor([math.inf, -math.inf, math.nan])
    x[1, 0, 5] = -top
    x[1, 0, 6] = math.inf
    x[2, 0, 7] = -math.inf  # the largest finite number of this run is 1
    x = x.to(src)
    slots = torch.tensor([0, 1, 16])
    cache = C.alloc_cache(2, 1, 16, 64, dtype)
    codes, scale = torch.zeros(2, 1, 16, 64).to(dtype), torch.zeros(2, 1)
    store_ref(x.float(), codes, scale, slots)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    C.store_cache(x.cuda(), x.cuda(), cache, slots.cuda(), dev_err=err)
    assert err.item() == C.DEVERR_NONFINITE
    for key in ("k", "v"):
        assert torch.equal(bits(cache[key].cpu()), bits(codes))
        assert torch.equal(cache[key + "_scale"].cpu(), scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("code", [I8, E4])
@pytest.mark.parametrize("d,bs", [(64, 128), (128, 16)])
def test_load(C, dtype, code, d, bs):
    g = torch.Generator(device="cuda").manual_seed(9)
    cache = random_cache(5, 3, bs, d, code, g, "cuda")
    slots = torch.tensor([0, 7, -1, 5 * bs - 1, 7, 2 * bs, 5 * bs, -9, 1 << 40], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = C.load_cache(cache, slots, dtype, dev_err=err)
    assert err.item() == C.DEVERR_BLOCK
    ok = ((slots >= 0) & (slots < 5 * bs))
    at = torch.where(ok, slots, 0)
    for key, name in (("K", "k"), ("V", "v")):
        want = cache[name].float() * cache[name + "_scale"][..., None, None]
        want = want.transpose(1, 2).reshape(-1, 3, d)[at] * ok[:, None, None]
        assert torch.equal(got[key], want.to(dtype))


def test_store_slot_outside(C):
    cache = C.alloc_cache(2, 1, 16, 64)
    x = torch.ones(3, 1, 64, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    C.store_cache(x, x, cache, torch.tensor([32, -2, 3], device="cuda"), dev_err=err)
    assert err.item() == C.DEVERR_BLOCK
    assert int((cache["k"] != 0).sum()) == 64 and int((cache["k"][0, 0, 3] == 127).sum()) == 64


# ------------------------------------------------------------------ attention over all keys

def make(ctx, new, hq, hkv, d, bs, code, qt, seed=1, spread=0.4, pad=0, strided=False, qs=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = [max(0, c + n) for c, n in zip(ctx, new)]
    width = max(1, max(ceil_div(n, bs) for n in lens))
    blocks = sum(ceil_div(n, bs) for n in lens) + 2
    cache = random_cache(blocks, hkv, bs, d, code, g, "cuda", spread)
    table = scattered_table(lens, bs, blocks, width, g, "cuda")
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    T = start[-1] + pad
    if strided:
        q = (qs * torch.randn(T, hq + 2 * hkv, d + 8, generator=g, device="cuda")).to(qt)[:, 1:hq + 1, :d]
    else:
        q = (qs * torch.randn(T, hq, d, generator=g, device="cuda")).to(qt)
    return dict(q=q, cache=cache, table=table, ctx=ints(ctx), seq=ints(lens), start=ints(start),
                max_q=max(new))


def check(C, s, scale=None, max_q="known", err_want=0, **kw):
    """attend_cache against the definition. Tolerance for one number of out: half a step of its
    type; 2^-11 for a weight that is rounded to a half and the error of the scores, both on the sum
    of p |v|; and 2^-25 for a weight below the smallest normal half, 2^-14 (its step is 2^-24),
    which moves at most what attend_ref calls small, since the largest weight is 1 or more."""
    c, q = s["cache"], s["q"]
    d = q.shape[2]
    sc = 1 / math.sqrt(d) if scale is None else scale
    ref, lse, weight, most, owned, small = attend_ref(q, c["k"], c["v"], c["k_scale"], c["v_scale"],
                                               s["table"], s["ctx"], s["seq"], s["start"], sc)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    got = C.attend_cache(q, c, s["table"], s["ctx"], s["seq"], s["start"],
                         max_q=s["max_q"] if max_q == "known" else max_q, scale=scale,
                         want_lse=True, out=out, dev_err=err, **kw)
    assert got["out"] is out and err.item() == err_want
    own = owned.cuda()
    assert bool((out[~own] == 7.0).all())  # rows behind the last sequence, left as they were
    e = score_error(d, most)
    half = torch.finfo(q.dtype).eps / 2
    # the smallest step of a half-precision output is 2^-24
    tol = half * ref.abs() + (2.0 ** -11 + 2 * e) * weight * (1 + half)
    tol = tol + 2.0 ** -25 * (small + 1)
    assert bool(torch.isfinite(out[own]).all())
    off = (out.double() - ref).abs()
    bad = (off > tol) & own[:, None, None]
    assert not bool(bad.any()), (
        f"{int(bad.sum())} of {int(own.sum()) * ref[0].numel()} off, worst "
        f"{float((off / tol)[bad].max()):.2f} x, first {bad.nonzero()[0].tolist()}")
    dead = lse.isinf() & own[:, None]
    assert bool((got["lse"][dead] == -math.inf).all()) and bool((out[dead] == 0).all())
    live = ~lse.isinf() & own[:, None]
    far = (got["lse"].double() - lse).abs()[live] - (2 * e + 2.0 ** -22 * lse.abs()[live])
    assert far.numel() == 0 or float(far.max()) <= 0
    return out, got["lse"]


DECODE = [
    # ctx, new, q heads, key heads, d, block, code, type
    ([0], [1], 1, 1, 64, 16, I8, torch.bfloat16),
    ([0, 1, 15, 16, 17], [1] * 5, 8, 8, 64, 16, I8, torch.bfloat16),
    ([127, 128, 129, 255, 1000], [1] * 5, 4, 1, 128, 128, E4, torch.float16),
    ([63, 64, 65, 4095], [1] * 4, 16, 2, 128, 64, I8, torch.float16),
    ([33, 700, 31, 32], [1] * 4, 15, 3, 64, 32, E4, torch.bfloat16),
    ([5, 0, 77], [4, 3, 2], 8, 2, 128, 16, I8, torch.bfloat16),
    ([500, 0, 12], [1, 0, 1], 32, 2, 64, 64, E4, torch.bfloat16),
    ([300], [1], 64, 1, 128, 32, I8, torch.bfloat16),
    ([40, 3000], [2, 1], 24, 2, 128, 16, E4, torch.bfloat16),
    ([9000, 20, 300] * 30, [1] * 90, 8, 8, 64, 16, I8, torch.float16),
]


@pytest.mark.parametrize("case", range(len(DECODE)))
def test_attend_few_rows(C, case):
    check(C, make(*DECODE[case]))


CHUNKS = [
    ([0], [17], 1, 1, 64, 16, I8, torch.bfloat16),
    ([0], [300], 2, 2, 128, 64, I8, torch.bfloat16),
    ([0, 0, 0], [1, 129, 257], 4, 4, 64, 32, E4, torch.float16),
    ([1000], [128], 8, 2, 128, 16, I8, torch.float16),
    ([77, 0, 512], [100, 200, 1], 16, 2, 128, 128, E4, torch.bfloat16),
    ([0, 2000, 30, 5], [700, 1, 0, 2], 12, 4, 64, 16, I8, torch.bfloat16),
    ([129], [33], 64, 1, 128, 32, E4, torch.bfloat16),
    ([3, 4, 5], [500, 511, 513], 5, 1, 64, 128, I8, torch.bfloat16),
    ([6000], [64], 8, 1, 128, 64, I8, torch.bfloat16),
]


@pytest.mark.parametrize("case", range(len(CHUNKS)))
def test_attend_chunks(C, case):
    check(C, make(*CHUNKS[case]))


@pytest.mark.parametrize("max_q", [None, 1, 5])
def test_attend_result_does_not_need_max_q(C, max_q):
    """max_q chooses kernels; a wrong or missing one does not change what is computed."""
    check(C, make([200, 7, 0], [40, 1, 150], 8, 2, 64, 32, I8, torch.bfloat16), max_q=max_q)


@pytest.mark.parametrize("new", [[1, 1, 1], [40, 30, 2]])
def test_attend_strides_padding_and_poison(C, new):
    """Sliced queries, rows behind the last request, NaN in every code, scale and table entry that
    no visible key needs."""
    s = make([70, 0, 130], new, 8, 2, 128, 32, E4, torch.bfloat16, pad=9, strided=True)
    c, bs = s["cache"], 32
    used = torch.zeros(c["k"].shape[0], dtype=torch.bool)
    for r, n in enumerate(s["seq"].tolist()):
        pages = s["table"][r, :ceil_div(n, bs)].long()
        used[pages.cpu()] = True
        if n % bs:
            for x in ("k", "v"):
                bits(c[x])[pages[-1], :, n % bs:] = 0x7f
    for x in ("k", "v"):
        bits(c[x])[~used] = 0x7f
        c[x + "_scale"][~used] = math.nan
    s["q"][-9:] = math.nan
    check(C, s)


@pytest.mark.parametrize("new", [[1, 1, 1, 1], [20, 60, 200, 33]])
def test_attend_rows_that_see_nothing(C, new):
    """A request without keys, one whose first rows stand before its first key, one cut at fewer
    keys than rows."""
    s = make([0, 10, 5, 64], new, 4, 2, 64, 16, I8, torch.bfloat16)
    s["seq"] = ints([0, 10 + new[1], 3, 64 + new[3]])
    s["ctx"] = ints([0, 10, 5, -7])
    check(C, s)


@pytest.mark.parametrize("new", [[1, 1], [70, 3]])
def test_attend_blocks_outside_are_left_out(C, new):
    s = make([100, 90], new, 4, 2, 64, 16, I8, torch.bfloat16)
    s["table"][0, 2] = -1
    s["table"][1, 0] = s["cache"]["k"].shape[0]
    s["table"][1, 5] = -2 ** 31
    check(C, s, err_want=C.DEVERR_BLOCK)


@pytest.mark.parametrize("new", [[1, 1, 1], [40, 30, 20]])
def test_attend_lengths_and_offsets_out_of_range(C, new):
    """Lengths up to the type's largest are cut at the table, offsets at the rows."""
    s = make([100, 90, 50], new, 4, 2, 64, 16, I8, torch.bfloat16)
    width, blocks = s["table"].shape[1], s["cache"]["k"].shape[0]
    s["table"] %= blocks  # every entry is a block, so that a request may see the whole row
    top = 2 ** 31 - 1
    s["ctx"] = ints([top, top - 5, -2 ** 31])
    s["seq"] = ints([top, 16 * width, top])
    check(C, s)
    s["ctx"], s["seq"] = ints([100, 90, 50]), ints([top, -4, 16 * width + 1])
    s["start"][0], s["start"][3] = -7, top
    check(C, s)


@pytest.mark.parametrize("new", [[1, 1], [70, 130]])
@pytest.mark.parametrize("code", [I8, E4])
def test_attend_scales_far_apart(C, new, code):
    """Blocks whose value scales differ by many powers of ten, and blocks of zeros."""
    s = make([200, 330], new, 4, 2, 64, 16, code, torch.bfloat16)
    c = s["cache"]
    c["v_scale"] *= 10.0 ** (torch.arange(c["v_scale"].numel(), device="cuda") % 13 - 6).view_as(c["v_scale"])
    c["v_scale"][3] = 2.0 ** -100
    c["v"][3] = 0
    check(C, s)
    check(C, s, scale=1.0)


@pytest.mark.parametrize("new", [[1], [150]])
@pytest.mark.parametrize("scale", [0.0, -0.125, 3.0])
def test_attend_scales_of_the_scores(C, new, scale):
    check(C, make([300], new, 4, 2, 64, 32, I8, torch.bfloat16, qs=1.0), scale=scale)


@pytest.mark.parametrize("qt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("new", [[1], [90]])
def test_attend_queries_large_and_small(C, qt, new):
    """Queries near the top and the bottom of their type (the other scales make up for it)."""
    for q, k in ((2.0 ** 13, 2.0 ** -13), (2.0 ** -12, 2.0 ** 12)):
        s = make([100], new, 2, 2, 64, 16, I8, qt, qs=q)
        s["cache"]["k_scale"] *= k
        check(C, s)
    if qt == torch.bfloat16:
        s = make([100], new, 2, 2, 64, 16, I8, qt, qs=2.0 ** 60)
        s["cache"]["k_scale"] *= 2.0 ** -60
        check(C, s)
    s = make([100], new, 2, 2, 64, 16, I8, qt)
    s["q"][0] = 0
    check(C, s)


@pytest.mark.parametrize("ctx,new", [
    ([3, 40], [1, 1]), ([20000, 40], [1, 1]), ([3, 40], [3, 2]),
    ([0, 100], [70, 40]), ([9000, 100], [70, 40])])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_attend_nan_stays_in_its_row(C, ctx, new, bad):
    """A NaN in a query gives NaN in that row's output (an infinity too: inf - inf in the softmax,
    and inf * 0), and touches no other row: whole units and those that are joined."""
    s = make(ctx, new, 8, 2, 64, 16, I8, torch.bfloat16)
    c = s["cache"]
    c["k"][..., 0] = 5  # a number that no product with an infinity loses
    run = lambda: C.attend_cache(s["q"], c, s["table"], s["ctx"], s["seq"], s["start"],
                                 max_q=s["max_q"], want_lse=True)
    want = run()
    row, head = s["q"].shape[0] // 2, 5
    s["q"][row, head, 0] = bad
    s["q"][0, 2, 0] = bad
    got = run()
    hit = torch.zeros(s["q"].shape[:2], dtype=torch.bool, device="cuda")
    hit[row, head] = hit[0, 2] = True
    assert bool(got["out"][hit].isnan().all()) and bool(got["lse"][hit].isnan().all())
    for key in ("out", "lse"):
        assert torch.equal(got[key][~hit], want[key][~hit])


def test_attend_codes_past_32_bits(C):
    """Blocks whose bytes lie behind 2^32."""
    d, bs, hkv = 128, 128, 8
    blocks = (1 << 32) // (d * bs * hkv) + 40
    cache = dict(k=torch.zeros(blocks, hkv, bs, d, dtype=I8, device="cuda"),
                 v=torch.zeros(blocks, hkv, bs, d, dtype=I8, device="cuda"),
                 k_scale=torch.ones(blocks, hkv, device="cuda"),
                 v_scale=torch.ones(blocks, hkv, device="cuda"))
    free = ints(list(range(blocks - 1, blocks - 12, -1)))
    table = torch.full((2, 8), -1, dtype=torch.int32, device="cuda")
    new = ints([600, 301])
    plan = C.plan_blocks(ints([0, 0]), new, table, free, ints([0]), 901, bs)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(901, 2, hkv, d, generator=g, device="cuda").bfloat16()
    C.store_cache(x[:, 0], x[:, 1], cache, plan["slots"])
    assert int(cache["k"][:blocks - 12].ne(0).sum(dtype=torch.int64)) == 0
    for n in (1, 40):
        q = torch.randn(2 * n, 16, d, generator=g, device="cuda").bfloat16()
        s = dict(q=q, cache=cache, table=table, ctx=ints([600 - n, 301 - n]), seq=plan["seq_len"],
                 start=ints([0, n, 2 * n]), max_q=n)
        check(C, s)
    back = C.load_cache(cache, plan["slots"], torch.float32)
    step = cache["k_scale"][(plan["slots"] // bs)][..., None]
    assert bool(((back["K"] - x[:, 0].float()).abs() <= step * 0.5001).all())


def test_attend_repeats_to_the_bit(C):
    """Two calls give the same bits, and a request's rows do not depend on the workspace."""
    for new in ([1] * 7, [50, 1, 1, 200, 3, 0, 9]):
        s = make([3000, 10, 900, 64, 2000, 5, 1], new, 8, 2, 64, 16, I8, torch.bfloat16)
        args = (s["q"], s["cache"], s["table"], s["ctx"], s["seq"], s["start"])
        a = C.attend_cache(*args, max_q=s["max_q"], want_lse=True)
        ws = torch.full((C.attend_cache_workspace(*args[:3]),), 255, dtype=torch.uint8, device="cuda")
        b = C.attend_cache(*args, max_q=s["max_q"], want_lse=True, workspace=ws)
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


def test_attend_two_streams_at_once(C):
    s = [make([4000, 300], n, 8, 2, 64, 16, I8, torch.bfloat16, seed=i)
         for i, n in enumerate(([1, 1], [60, 2]))]
    run = lambda x: C.attend_cache(x["q"], x["cache"], x["table"], x["ctx"], x["seq"], x["start"],
                                   max_q=x["max_q"])["out"]
    want = [run(x) for x in s]
    streams = [torch.cuda.Stream() for _ in s]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for x, st in zip(s, streams):
            with torch.cuda.stream(st):
                got.append(run(x))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_attend_refuses_what_it_cannot_use(C):
    from tree_routed_sparse_b200 import alhr
    s = make([10], [1], 4, 2, 64, 16, I8, torch.bfloat16)
    call = lambda **kw: C.attend_cache(*[dict(s, **kw)[k] for k in (
        "q", "cache", "table", "ctx", "seq", "start")], **{k: v for k, v in kw.items() if k in (
            "out", "workspace", "max_q", "scale")})
    with pytest.raises(ValueError, match="block_table"):
        call(table=s["table"].cpu())
    with pytest.raises(ValueError, match="q_start"):
        call(start=s["start"][:1])
    with pytest.raises(ValueError, match="Q"):
        call(q=s["q"].float())
    with pytest.raises(ValueError, match="Q"):
        call(q=torch.cat([s["q"], s["q"]], -1)[..., ::2])
    with pytest.raises(ValueError, match="out"):
        call(out=torch.empty(1, 4, 64, device="cuda"))
    with pytest.raises(ValueError, match="max_q"):
        call(max_q=0)
    with pytest.raises(alhr.AlhrError, match="INVALID_ARG"):
        call(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(alhr.AlhrError, match="INVALID_ARG"):
        call(scale=math.inf)
    with pytest.raises(alhr.AlhrError, match="INVALID_ARG"):
        call(q=s["q"][:, :3].contiguous())
    with pytest.raises(alhr.AlhrError, match="INVALID_ARG"):  # rows of an odd distance
        call(q=torch.empty(3, 4, 67, dtype=torch.bfloat16, device="cuda")[:1, :, :64])


# ------------------------------------------------------------------ selected keys

@pytest.mark.parametrize("qt", [torch.int8, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,hq,hkv,nq,n,m,d,bs,code", [
    (1, 1, 1, 1, 1, 1, 64, 16, I8), (2, 8, 8, 1, 500, 96, 128, 64, I8),
    (3, 4, 2, 7, 65, 17, 64, 16, E4), (2, 15, 3, 3, 300, 33, 128, 32, E4),
    (1, 4, 4, 200, 200, 96, 64, 128, I8)])
def test_selected(C, qt, B, hq, hkv, nq, n, m, d, bs, code):
    """Selections of any order and length (none too), entries outside what a row may see."""
    g = torch.Generator(device="cuda").manual_seed(n + m)
    width = ceil_div(n, bs)
    cache = random_cache(B * width + 1, hkv, bs, d, code, g, "cuda")
    table = scattered_table([n] * B, bs, B * width + 1, width, g, "cuda")
    idx = torch.randint(0, n, (B, hq, nq, m), generator=g, device="cuda").int()
    count = torch.randint(0, m + 1, (B, hq, nq), generator=g, device="cuda").int()
    count[0, 0, 0] = m
    if qt == torch.int8:
        q = torch.randint(-16, 17, (B, hq, nq, d), generator=g, device="cuda").to(qt)
        scale = 0.1 / math.sqrt(d)
    else:
        q = torch.randn(B, hq, nq, d, generator=g, device="cuda").to(qt)
        scale = None
    ctx, seq = ints([n - nq] * B), ints([n - (b % 2) for b in range(B)])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = C.attend_cache_selected(q, cache, table, ctx, seq, idx, count, scale=scale, dev_err=err)
    sc = 1 / math.sqrt(d) if scale is None else scale
    at = idx.long()
    page = table.long()[torch.arange(B, device="cuda")[:, None, None, None], at // bs]
    head = (torch.arange(hq, device="cuda") // (hq // hkv))[None, :, None, None]
    K, V = (numbers(cache[x], cache[x + "_scale"])[page, head, at % bs] for x in ("k", "v"))
    pos = torch.arange(n - nq, n, device="cuda")[None, None, :, None]
    named = torch.arange(m, device="cuda") < count[..., None]
    ok = named & (at <= pos) & (at < seq[:, None, None, None])
    assert err.item() == (4 if bool((named & ~ok).any()) else 0)
    s = torch.einsum("bhqd,bhqmd->bhqm", q.double(), K) * sc
    most = float(torch.einsum("bhqd,bhqmd->bhqm", q.double().abs(), K.abs()).max()) * sc
    s = s.masked_fill(~ok, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top.isinf(), torch.zeros_like(top), top))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
    want = torch.einsum("bhqm,bhqmd->bhqd", p, V)
    weight = torch.einsum("bhqm,bhqmd->bhqd", p, V.abs())
    # weights and sums in fp32 (a weight may be held as two 16-bit terms: 2^-21 of it)
    tol = (2 * score_error(d, most) + 2.0 ** -20 + (m + 4) * 2.0 ** -24) * weight + 1e-30
    assert bool(((out.double() - want).abs() <= tol).all())


def test_selected_blocks_outside(C):
    g = torch.Generator(device="cuda").manual_seed(3)
    cache = random_cache(4, 1, 16, 64, I8, g, "cuda")
    table = ints([[0, 9, -1, 2]])
    idx = ints([[[[0, 17, 33, 50, -1, 64]]]])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.randn(1, 1, 1, 64, generator=g, device="cuda").bfloat16()
    a = C.attend_cache_selected(q, cache, table, ints([63]), ints([64]), idx, ints([[[6]]]),
                                dev_err=err)
    assert err.item() == C.DEVERR_BLOCK | 4
    b = C.attend_cache_selected(q, cache, table, ints([63]), ints([64]), ints([[[[0, 50]]]]),
                                ints([[[2]]]))
    assert float((a - b).abs().max()) <= 2.0 ** -20 * float(b.abs().max())


@pytest.mark.parametrize("qt", [torch.bfloat16, torch.float16])
def test_selected_nan_stays_in_its_row(C, qt):
    g = torch.Generator(device="cuda").manual_seed(4)
    cache = random_cache(5, 2, 16, 64, I8, g, "cuda")
    table = scattered_table([80], 16, 5, 5, g, "cuda")
    q = torch.randn(1, 4, 3, 64, generator=g, device="cuda").to(qt)
    idx = torch.randint(0, 70, (1, 4, 3, 40), generator=g, device="cuda").int()
    count = torch.full((1, 4, 3), 40, dtype=torch.int32, device="cuda")
    run = lambda: C.attend_cache_selected(q, cache, table, ints([77]), ints([80]), idx, count)
    want = run()
    q[0, 1, 2, 7] = math.nan
    got = run()
    assert bool(got[0, 1, 2].isnan().all())
    got[0, 1, 2] = want[0, 1, 2]
    assert torch.equal(got, want)


@pytest.mark.parametrize("first", [31, 32, 64, 95])
def test_selected_pages_of_others_have_no_effect(C, first):
    """Entries that are skipped, more than a warp's worth of them before the first that is not, and
    NaN in every code of the pages that are not the request's (the first page among them)."""
    g = torch.Generator(device="cuda").manual_seed(6)
    cache = random_cache(6, 1, 16, 128, E4, g, "cuda")
    q = torch.randn(1, 1, 1, 128, generator=g, device="cuda").bfloat16()
    idx = torch.full((1, 1, 1, 96), -1, dtype=torch.int32, device="cuda")
    idx[0, 0, 0, first:] = torch.randint(0, 40, (96 - first,), generator=g, device="cuda").int()
    want = C.attend_cache_selected(q, cache, ints([[3, 5, 2]]), ints([47]), ints([48]), idx,
                                   ints([[[96]]]))
    for key in ("k", "v"):
        bits(cache[key])[[0, 1, 4]] = 0x7f
    got = C.attend_cache_selected(q, cache, ints([[3, 5, 2]]), ints([47]), ints([48]), idx,
                                  ints([[[96]]]))
    assert bool(want.isfinite().all()) and torch.equal(got, want)


# ------------------------------------------------------------------ the set together

@pytest.mark.parametrize("code", [I8, E4])
def test_serving_steps(C, code):
    """Prompts, then decode steps, of sequences that grow into new blocks: every step's attention
    equals the definition over what the cache holds, and that is near what was stored."""
    bs, d, hq, hkv = 16, 64, 4, 2
    g = torch.Generator(device="cuda").manual_seed(11)
    cache = C.alloc_cache(40, hkv, bs, d, code)
    table = torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(40, generator=g, device="cuda").int()
    first, ctx = ints([0]), ints([0, 0, 0])
    kept = [[], [], []]
    for step in range(20):
        new = ints([30, 1, 17] if step == 0 else [1, 1, 0] if step % 3 else [2, 0, 3])
        t = int(new.sum()) + 2
        plan = C.plan_blocks(ctx, new, table, free, first, t, bs)
        x = torch.randn(t, 2, hkv, d, generator=g, device="cuda").bfloat16()
        C.store_cache(x[:, 0], x[:, 1], cache, plan["slots"])
        q = torch.randn(t, hq, d, generator=g, device="cuda").bfloat16()
        check(C, dict(q=q, cache=cache, table=table, ctx=ctx, seq=plan["seq_len"],
                      start=plan["q_start"], max_q=30))
        for r in range(3):
            a, b = plan["q_start"][r:r + 2].tolist()
            kept[r].append(x[a:b, 0])
        first, ctx = plan["free_next"], plan["seq_len"]
    for r in range(3):
        want = torch.cat(kept[r]).float()
        n = want.shape[0]
        assert n == int(ctx[r])
        p = torch.arange(n, device="cuda")
        back = C.load_cache(cache, table[r, p // bs].long() * bs + p % bs, torch.float32)["K"]
        s = cache["k_scale"][table[r, p // bs].long()][..., None]
        # a number is rounded once when stored and once for each growth of its block's scale, at
        # most 16 times (a block's rows), each by half a step of the scale of that time, which is
        # no larger than the last one
        half = s * 0.5 if code == I8 else torch.maximum(want.abs() / 16, s * 2.0 ** -10) * 1.1
        assert float(((back - want).abs() - 16 * half).max()) <= 0


def test_routed_decode_over_the_cache(C):
    """The framework's routing picks the positions, the cache is read there: equal to alhr.attend
    on the numbers that the cache holds (values rounded to bf16 there: half a step, 2^-8)."""
    from tree_routed_sparse_b200 import alhr
    B, H, n, d, bs = 2, 4, 1024, 64, 32
    g = torch.Generator(device="cuda").manual_seed(21)
    Q = torch.randint(-16, 17, (B, H, 1, d), generator=g, device="cuda").to(torch.int8)
    K = torch.randint(-16, 17, (B, H, n, d), generator=g, device="cuda").to(torch.int8)
    V = torch.randn(B, H, n, d, generator=g, device="cuda").bfloat16()
    W = torch.randint(-4, 5, (32, 2 * d), generator=g, device="cuda").to(torch.int8)
    tree = alhr.build_tree(K)
    cache = C.alloc_cache(B * n // bs, H, bs, d)
    table = torch.full((B, n // bs), -1, dtype=torch.int32, device="cuda")
    plan = C.plan_blocks(ints([0] * B), ints([n] * B), table, torch.randperm(
        B * n // bs, generator=g, device="cuda").int(), ints([0]), B * n, bs)
    rows = lambda x: x.transpose(1, 2).reshape(B * n, H, d)
    C.store_cache(rows(K.bfloat16()), rows(V), cache, plan["slots"])
    # one scale that makes the codes the routing keys themselves: the scores are then alike
    cache["k"].copy_((cache["k"].float() * cache["k_scale"][..., None, None]).round().to(torch.int8))
    cache["k_scale"].fill_(1.0)
    budget = alhr.predict_budget(Q, K, tree, W, q_start=n - 1)
    sel = alhr.route(Q, K, tree, budget, q_start=n - 1)
    out = C.attend_cache_selected(Q, cache, table, ints([n - 1] * B), plan["seq_len"], sel["idx"],
                                  sel["count"])
    back = C.load_cache(cache, plan["slots"], torch.bfloat16)
    V8 = back["V"].view(B, n, H, d).transpose(1, 2).contiguous()
    K8 = back["K"].view(B, n, H, d).transpose(1, 2).to(torch.int8).contiguous()
    assert torch.equal(K8, K)
    want = alhr.attend(Q, K8, V8, sel["idx"], sel["count"], q_start=n - 1)
    assert float((out - want).abs().max()) <= 2.0 ** -8 * float(V8.float().abs().max())
    # with every key selected it is the attention over all keys
    few = torch.arange(96, device="cuda").int().expand(B, H, 1, 96).contiguous()
    a = C.attend_cache_selected(Q, cache, table, ints([95] * B), ints([96] * B), few,
                                ints([96]).expand(B, H, 1).contiguous())
    b = C.attend_cache(Q[:, :, 0].bfloat16(), cache, table, ints([95] * B), ints([96] * B),
                       ints([0, 1, 2]), max_q=1)["out"]
    top = float(cache["v_scale"].max()) * 127
    assert float((a[:, :, 0] - b.float()).abs().max()) <= (2.0 ** -8 + 2.0 ** -10) * top


def test_step_captured_and_replayed(C):
    """A captured step replays with other lengths, tables and free lists in the same tensors, two
    graphs side by side."""
    bs, d, hq, hkv, R, T = 16, 128, 8, 2, 3, 64
    g = torch.Generator(device="cuda").manual_seed(31)

    def state(seed):
        cache = random_cache(60, hkv, bs, d, I8, g, "cuda")
        order = torch.randperm(60, generator=g, device="cuda").int()
        return dict(cache=cache, ctx=ints([20, 0, 100]), new=ints([1, 5, 40]), free=order[30:].clone(),
                    first=ints([0]), table=order[:30].reshape(3, 10).contiguous(),
                    x=torch.randn(T, 2, hkv, d, generator=g, device="cuda").bfloat16(),
                    q=torch.randn(T, hq, d, generator=g, device="cuda").bfloat16())

    def step(s, out):
        plan = C.plan_blocks(s["ctx"], s["new"], s["table"], s["free"], s["first"], T, bs)
        C.store_cache(s["x"][:, 0], s["x"][:, 1], s["cache"], plan["slots"])
        C.attend_cache(s["q"], s["cache"], s["table"], s["ctx"], plan["seq_len"], plan["q_start"],
                       out=out, max_q=T)
        return plan

    clone = lambda s: {k: ({a: b.clone() for a, b in v.items()} if isinstance(v, dict) else v.clone())
                       for k, v in s.items()}
    a, b = state(1), state(2)
    outs = [torch.zeros(T, hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    step(clone(a), outs[0].clone())  # loads everything before the capture
    torch.cuda.synchronize()
    graphs = []
    for s, o in zip((a, b), outs):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(s, o)
        graphs.append(gr)
    for new in ([1, 5, 40], [1, 1, 1], [0, 60, 2]):
        for s in (a, b):
            s["new"].copy_(ints(new))
        want = []
        for s in (a, b):
            c, o = clone(s), torch.zeros_like(outs[0])
            step(c, o)
            want.append((c, o))
        for o in outs:
            o.zero_()
        side = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for gr, st in zip(graphs, side):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for s, o, (c, w) in zip((a, b), outs, want):
            assert torch.equal(o, w) and torch.equal(s["table"], c["table"])
            assert all(torch.equal(s["cache"][k], c["cache"][k]) for k in c["cache"])


# ------------------------------------------------------------------ value scales of any size

def spread_scales(s, powers):
    """Block i of the cache has the value scale 2^powers[i % len]; None: 0, with its codes kept."""
    c = s["cache"]
    n = c["v_scale"].shape[0]
    p = [powers[i % len(powers)] for i in range(n)]
    f = torch.tensor([0.0 if x is None else 2.0 ** x for x in p], device="cuda")
    c["v_scale"].copy_(f[:, None].expand_as(c["v_scale"]))
    # blocks in the order of their positions, so that the powers follow one another in a sequence
    for r in range(s["table"].shape[0]):
        row = s["table"][r]
        row.copy_(torch.where(row >= 0, row.masked_fill(row < 0, n).sort()[0], row))
    return s


@pytest.mark.parametrize("rows,keys,requests", [(1, 32768, 64), (4, 32768, 64), (300, 16384, 8)])
def test_attend_lse_of_zero_values(C, rows, keys, requests):
    """Heads whose values are all zero (a scale of 2^-100 as store_cache writes it, 0 as
    alloc_cache does), with scores that rise by nearly 8 powers of two behind the first keys: lse is
    that of the scores, out is zero. The requests share their pages."""
    hkv, d, bs = 8, 64, 128
    cache = C.alloc_cache(keys // bs, hkv, bs, d)
    cache["v_scale"].fill_(2.0 ** -100)
    cache["v_scale"][:, 0] = 0
    cache["k_scale"].fill_(1.0)
    cache["k"][..., 0] = 54
    cache["k"][0, :, :, 0] = 0
    q = torch.zeros(requests * rows, hkv, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    table = torch.arange(keys // bs, device="cuda").int().expand(requests, -1).contiguous()
    got = C.attend_cache(q, cache, table, ints([keys - rows] * requests), ints([keys] * requests),
                         ints([rows * i for i in range(requests + 1)]), max_q=rows, scale=0.1,
                         want_lse=True)
    seen = keys - rows + 1 + torch.arange(rows, device="cuda").double().repeat(requests)
    want = torch.log(128 + (seen - 128) * math.exp(5.4))[:, None]
    assert bool((got["out"] == 0).all())
    # terms of at most 5.4 and their sum: a few roundings of each, the sum's of `keys` numbers in
    # 32 bits at 2^-24 of it for each step of a lane's or thread's chain (at most keys / 16)
    assert float((got["lse"].double() - want).abs().max()) <= keys / 16 * 2.0 ** -24 + 2.0 ** -18


SPREADS = [
    [-100, 20], [-100, 40], [20, -100], [30, -100, None, 0], [0, 60, -60, 90, -99, 3],
    [-99, -60, -20, 20, 60, 100], [100, 60, 20, -20, -60, -99], [None, -6], [-6, None, -100],
    [110, -100], [-33, 0], [0, 33, -33], [None], [-100], [-70, -66],
]


@pytest.mark.parametrize("powers", SPREADS, ids=str)
@pytest.mark.parametrize("new,d,code", [([1, 1], 64, I8), ([3, 4], 128, E4), ([70, 130], 64, E4),
                                        ([300, 9], 128, I8)])
def test_attend_value_scales_of_any_size(C, powers, new, d, code):
    """Blocks whose value scales lie any number of powers of two apart, zeros among them: every
    key keeps its share of the softmax, whatever the scale of its value."""
    s = spread_scales(make([1800, 330], new, 4, 2, d, 16, code, torch.bfloat16, qs=0.5), powers)
    c, q = s["cache"], s["q"]
    for scale in (None, 0.0):
        check(C, s, scale=scale)
        # without the absolute term that check allows for half-precision outputs: tiny values too
        sc = 1 / math.sqrt(d) if scale is None else scale
        ref, _, weight, most, _, small = attend_ref(q, c["k"], c["v"], c["k_scale"], c["v_scale"],
                                                    s["table"], s["ctx"], s["seq"], s["start"], sc)
        out = C.attend_cache(q, c, s["table"], s["ctx"], s["seq"], s["start"], max_q=s["max_q"],
                             scale=scale)["out"]
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2 * score_error(d, most)) * weight * 1.01
        assert bool(((out.double() - ref).abs() <= tol + 2.0 ** -25 * small).all())


@pytest.mark.parametrize("new", [[1], [40]])
def test_attend_zeros_beside_large_values(C, new):
    """Every second block holds zeros, the other ones 2^30: equal scores, so out is their mean."""
    n, bs, d = 4096, 64, 128
    x = torch.zeros(n, 1, d, device="cuda")
    x.view(n // bs, bs, d)[1::2] = 2.0 ** 30
    cache = C.alloc_cache(n // bs, 1, bs, d)
    C.store_cache(torch.zeros_like(x), x, cache, torch.arange(n, device="cuda"))
    t = new[0]
    q = torch.ones(t, 2, d, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(n // bs, device="cuda").int()[None]
    got = C.attend_cache(q, cache, table, ints([n - 1] * 1), ints([n]), ints([0, t]), max_q=t,
                         want_lse=True)
    assert float((got["out"].double() / 2.0 ** 30 - 0.5).abs().max()) <= 2.0 ** -9
    assert float((got["lse"] - math.log(n)).abs().max()) <= 1e-5


@pytest.mark.parametrize("powers", [[-6, -6, -6, -100], [-50, 3, 40], [-100, 40, -6, None]], ids=str)
@pytest.mark.parametrize("requests,ctx,new,d", [(40, 3000, 1, 64), (6, 4000, 260, 128),
                                                (6, 4000, 260, 64)])
def test_attend_value_scales_of_many_units(C, powers, requests, ctx, new, d):
    """Warps and CTAs that go through several requests and heads: what one unit's value scales ask
    for ends with it."""
    s = make([ctx + 37 * i for i in range(requests)], [new] * requests, 8, 8, d, 64, I8,
             torch.bfloat16, qs=0.5)
    s = spread_scales(s, powers)
    s["cache"]["v_scale"][:, ::2] = 0.02  # every second head is an ordinary one
    check(C, s)


@pytest.mark.parametrize("requests,new", [(1500, [1]), (3000, [1, 0, 2, 40, 1])])
def test_attend_many_requests(C, requests, new):
    """More requests than threads of a CTA: each sums a run of them for the list of tiles."""
    g = torch.Generator().manual_seed(requests)
    ctx = torch.randint(0, 90, (requests,), generator=g).tolist()
    check(C, make(ctx, [new[i % len(new)] for i in range(requests)], 2, 1, 64, 16, I8,
                  torch.bfloat16, pad=3))


def test_attend_without_rows(C):
    """Requests without a row, and rows that belong to none: nothing is written."""
    s = make([20, 3], [0, 0], 4, 2, 64, 16, I8, torch.bfloat16, pad=50)
    check(C, s, max_q=None)
