"""The paged 8-bit cache without a GPU: host-side checks of the ABI and of the binding."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def C():
    from tree_routed_sparse_b200 import build
    build.build()
    from tree_routed_sparse_b200 import alhr, cache
    alhr.lib()
    return cache


P = 4096  # an aligned address that is never read: every call below is refused or has nothing to do


def cache_of(C, **kw):
    base = dict(k=P, v=P, k_scale=P, v_scale=P, blocks=10, heads=2, block_size=16, d=64, code=0)
    base.update(kw)
    return C.CacheStruct(*[base[f] for f, _ in C.CacheStruct._fields_])


INVALID, UNSUPPORTED = 1, 2
BAD_CACHES = [
    (dict(blocks=0), INVALID), (dict(heads=0), INVALID), (dict(code=2), INVALID),
    (dict(code=-1), INVALID), (dict(block_size=8), UNSUPPORTED), (dict(block_size=48), UNSUPPORTED),
    (dict(block_size=256), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED),
    (dict(blocks=1 << 27, heads=1, block_size=16), UNSUPPORTED), (dict(heads=65536), UNSUPPORTED),
    (dict(blocks=2 ** 31 - 1, heads=2 ** 31 - 1), UNSUPPORTED),
]
BAD_MEMORY = [dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(k=P + 8),
              dict(v=P + 1), dict(k_scale=P + 2), dict(v_scale=P + 1)]


def test_plan_refusals(C):
    from tree_routed_sparse_b200 import alhr
    L = alhr.lib()

    def call(**kw):
        a = dict(requests=2, max_blocks=4, block_size=16, blocks=9, tokens=5, free_count=3, ctx=P,
                 new=P, table=P, free=P, first=P, q_start=P, seq=2 * P, slots=P, positions=P,
                 nxt=2 * P)
        a.update(kw)
        return L.alhr_plan_blocks(*a.values(), None, None)

    for kw in (dict(requests=-1), dict(max_blocks=0), dict(blocks=0), dict(tokens=-1),
               dict(free_count=-1), dict(ctx=None), dict(new=None), dict(table=None),
               dict(free=None), dict(first=None), dict(q_start=None), dict(seq=None),
               dict(slots=None), dict(positions=None), dict(nxt=None),
               # outputs that are inputs: CTAs would read what others have written
               dict(nxt=P), dict(seq=P), dict(ctx=2 * P, seq=2 * P)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(block_size=0), dict(block_size=24), dict(requests=8193),
               dict(max_blocks=1 << 27), dict(max_blocks=(1 << 26) + 1)):
        assert call(**kw) == UNSUPPORTED, kw


def store(C, L, cache, **kw):
    a = dict(K=P, V=P, type=0, tokens=4, kt=128, kh=64, vt=128, vh=64, slots=P)
    a.update(kw)
    return L.alhr_store_cache(None if cache is None else ctypes.byref(cache), *a.values(), None, None)


def test_store_and_load_refusals(C):
    from tree_routed_sparse_b200 import alhr
    L = alhr.lib()
    load = lambda c, K=P, V=P, type=0, tokens=4, slots=P: L.alhr_load_cache(
        ctypes.byref(c), K, V, type, tokens, slots, None, None)
    assert store(C, L, None) == INVALID
    for kw, want in BAD_CACHES:
        assert store(C, L, cache_of(C, **kw)) == want, kw
        assert load(cache_of(C, **kw)) == want, kw
    for kw in BAD_MEMORY:
        assert store(C, L, cache_of(C, **kw)) == INVALID, kw
        assert load(cache_of(C, **kw)) == INVALID, kw
    for kw in (dict(K=None), dict(V=None), dict(slots=None), dict(K=P + 2), dict(V=P + 8),
               dict(type=3), dict(type=-1), dict(tokens=-1), dict(kt=4), dict(kh=7), dict(vt=1),
               dict(vh=12), dict(type=2, kt=130)):
        assert store(C, L, cache_of(C), **kw) == INVALID, kw
    for kw in (dict(K=None), dict(V=None), dict(slots=None), dict(K=P + 2), dict(type=3),
               dict(tokens=-1)):
        assert load(cache_of(C), **kw) == INVALID, kw
    # nothing to store or load: nothing is read
    assert store(C, L, cache_of(C, k=None), tokens=0, K=None) == 0
    assert load(cache_of(C), tokens=0, K=None) == 0


def test_attend_refusals(C):
    from tree_routed_sparse_b200 import alhr
    L = alhr.lib()

    def call(cache=None, ptrs=(), **kw):
        q = dict(requests=2, tokens=6, q_heads=4, max_blocks=5, max_q=0, type=0,
                 q_token_stride=256, q_head_stride=64, scale=0.125)
        q.update(kw)
        st = C.QueriesStruct(*[q[f] for f, _ in C.QueriesStruct._fields_])
        a = dict(Q=P, table=P, ctx=P, seq=P, start=P, out=P, lse=None, ws=P, size=1 << 40)
        a.update(ptrs)
        return L.alhr_attend_cache(ctypes.byref(cache or cache_of(C)), ctypes.byref(st),
                                   *a.values(), None, None)

    for kw, want in BAD_CACHES:
        assert call(cache_of(C, **kw)) == want, kw
    for kw in BAD_MEMORY:
        assert call(cache_of(C, **kw)) == INVALID, kw
    for kw in (dict(requests=-1), dict(tokens=-1), dict(q_heads=0), dict(q_heads=3),
               dict(max_blocks=0), dict(max_q=-1), dict(type=2), dict(type=3),
               dict(q_token_stride=12), dict(q_head_stride=1), dict(scale=math.nan),
               dict(scale=math.inf), dict(scale=3.4e38)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(requests=8193), dict(q_heads=130), dict(tokens=1 << 30),
               dict(max_blocks=1 << 27), dict(max_blocks=(1 << 26) + 1)):
        assert call(**kw) == UNSUPPORTED, kw
    for k in ("Q", "table", "ctx", "seq", "start", "out", "ws"):
        assert call(ptrs={k: None}) == INVALID, k
    for k in ("Q", "out", "ws"):
        assert call(ptrs={k: P + 4}) == INVALID, k
    assert call(tokens=0, ptrs=dict(Q=None)) == 0 and call(requests=0, ptrs=dict(out=None)) == 0


def test_selected_refusals(C):
    from tree_routed_sparse_b200 import alhr
    L = alhr.lib()

    def call(cache=None, ptrs=(), **kw):
        q = dict(batch=2, q_heads=4, nq=3, max_keys=96, max_blocks=5, type=3, scale=0.125)
        q.update(kw)
        st = C.SelectionStruct(*[q[f] for f, _ in C.SelectionStruct._fields_])
        a = dict(Q=P, table=P, ctx=P, seq=P, idx=P, count=P, out=P)
        a.update(ptrs)
        return L.alhr_attend_cache_selected(ctypes.byref(cache or cache_of(C)), ctypes.byref(st),
                                            *a.values(), None, None)

    for kw, want in BAD_CACHES:
        assert call(cache_of(C, **kw)) == want, kw
    for kw in BAD_MEMORY:
        assert call(cache_of(C, **kw)) == INVALID, kw
    for kw in (dict(batch=0), dict(q_heads=0), dict(q_heads=5), dict(nq=-1), dict(max_keys=0),
               dict(max_blocks=0), dict(type=2), dict(scale=math.nan)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(max_keys=97), dict(q_heads=130), dict(nq=1 << 30), dict(max_blocks=1 << 27)):
        assert call(**kw) == UNSUPPORTED, kw
    for k in ("Q", "table", "ctx", "seq", "idx", "count", "out"):
        assert call(ptrs={k: None}) == INVALID, k
    for k in ("Q", "out"):
        assert call(ptrs={k: P + 4}) == INVALID, k
    assert call(nq=0, ptrs=dict(Q=None)) == 0


def test_binding_refuses_what_it_cannot_pass_on(C):
    """Wrong types, shapes, devices and strides are named before anything is called."""
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError, match="block_table"):
        C.plan_blocks(i32(2), i32(2), i32(2, 3), i32(4), i32(1), 4, 16)  # not on a GPU
    with pytest.raises(ValueError, match="slots"):
        C.store_cache(torch.zeros(1, 1, 64), torch.zeros(1, 1, 64), {}, torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="block_size"):
        C.alloc_cache(2, 2, 24, 64, device="cpu")
    with pytest.raises(ValueError, match="dtype"):
        C.alloc_cache(2, 2, 16, 64, torch.float16, device="cpu")
    with pytest.raises(ValueError, match="d 96"):
        C.alloc_cache(2, 2, 16, 96, device="cpu")
    c = C.alloc_cache(3, 2, 16, 64, device="cpu")
    assert c["k"].shape == (3, 2, 16, 64) and c["v_scale"].shape == (3, 2)
    cpu = torch.device("cpu")
    st = C._struct(c, cpu)
    assert (st.blocks, st.heads, st.block_size, st.d, st.code) == (3, 2, 16, 64, 0)
    for key, bad in (("v", c["v"].transpose(0, 1)), ("v", c["v"][:2]), ("k", c["k"].float()),
                     ("k_scale", c["k_scale"].double()), ("v_scale", c["v_scale"][:, :1])):
        with pytest.raises(ValueError, match="cache"):
            C._struct(dict(c, **{key: bad}), cpu)
    with pytest.raises(ValueError, match="device|on meta|on cpu"):
        C._struct(c, torch.device("meta"))
    x = torch.zeros(4, 3, 2, 64)
    assert C._rows(x[:, 1], (4, 2, 64), torch.float32, "K", cpu) == (384, 64)
    one = torch.zeros(67)[3:].as_strided((1, 1, 64), (5, 7, 1))
    assert C._rows(one, (1, 1, 64), torch.float32, "K", cpu) == (0, 0)  # strides of nothing
    for bad in (x[:, 1].transpose(1, 2), x[:, 1, :, ::2], x[0, 1]):
        with pytest.raises(ValueError, match="K: expected"):
            C._rows(bad, (4, 2, 64), torch.float32, "K", cpu)


@pytest.mark.parametrize("tokens", [-1, 2 ** 31, 2 ** 32, 2 ** 32 + 4])
def test_plan_refuses_tokens_that_32_bits_do_not_hold(C, tokens):
    """The ABI's count is an int32: a larger one is named, not cut to its low bits."""
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError, match="tokens"):
        C.plan_blocks(i32(2), i32(2), i32(2, 3), i32(4), i32(1), tokens, 16)


def test_plan_by_hand():
    """The test oracle itself: two requests, pages of 4 written out by hand."""
    from cache_util import plan_ref
    got = plan_ref([3, 0], [2, 5], [[7, -1], [-1, -1]], [5, 2, 6], 0, 8, 4, 10)
    assert got == ([0, 2, 7], [5, 5], [31, 20, 8, 9, 10, 11, 24, -1],
                   [3, 4, 0, 1, 2, 3, 4, -1], 3, [[7, 5], [2, 6]], 0)


def test_attention_by_hand():
    """The test oracle itself: one row over three keys, a mask and a block that is left out."""
    from cache_util import attend_ref
    k = torch.zeros(3, 1, 16, 64, dtype=torch.int8)
    v = torch.zeros_like(k)
    k[1, 0, :3, 0] = torch.tensor([1, 2, 3], dtype=torch.int8)
    v[1, 0, :3, 5] = torch.tensor([10, 20, 90], dtype=torch.int8)
    one, half = torch.ones(3, 1), torch.full((3, 1), 0.5)
    q = torch.zeros(1, 1, 64)
    q[0, 0, 0] = 1.0
    i = lambda *x: torch.tensor(x, dtype=torch.int32)
    out, lse, _, _, owned, _ = attend_ref(q, k, v, one, half, i(1)[None], i(1), i(9), i(0, 1), 1.0)
    e1, e2 = math.exp(1), math.exp(2)
    assert abs(out[0, 0, 5].item() - 0.5 * (10 * e1 + 20 * e2) / (e1 + e2)) < 1e-12
    assert abs(lse.item() - math.log(e1 + e2)) < 1e-12 and owned.tolist() == [True]
    out, lse, *_ = attend_ref(q, k, v, one, half, i(-1)[None], i(1), i(9), i(0, 1), 1.0)
    assert out.abs().max() == 0 and lse.item() == -math.inf


def test_attend_ref_sees_planted_mistakes():
    """The tolerance of the GPU tests tells a wrong mask and a lost scale from rounding."""
    from cache_util import attend_ref, random_cache, score_error
    g = torch.Generator().manual_seed(0)
    c = random_cache(4, 1, 16, 64, torch.int8, g, "cpu")
    i = lambda *x: torch.tensor(x, dtype=torch.int32)
    q = 2 * torch.randn(1, 2, 64, generator=g)
    run = lambda ctx=40, ks=c["k_scale"], vs=c["v_scale"]: attend_ref(
        q, c["k"], c["v"], ks, vs, i(2, 0, 3)[None], i(ctx), i(48), i(0, 1), 0.125)
    ref, _, weight, most, *_ = run()
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2 * score_error(64, most)) * weight
    for other in (run(ctx=39), run(ctx=41), run(ks=c["k_scale"].mean().expand(4, 1)),
                  run(vs=c["v_scale"].mean().expand(4, 1))):
        assert bool(((other[0] - ref).abs() > tol).any())
