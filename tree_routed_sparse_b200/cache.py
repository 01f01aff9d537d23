"""The paged 8-bit key/value cache: thin binding of include/alhr_cache.h.

Argument marshalling only, like alhr.py: every step runs in the library's CUDA kernels. A cache is
a dict of tensors (alloc_cache makes one):

    k, v              int8 or float8_e4m3fn codes [blocks, heads, block_size, d]
    k_scale, v_scale  float32 [blocks, heads]; a number is code * scale

A serving step:

    plan = plan_blocks(ctx_len, new_len, block_table, free_blocks, free_first, tokens, block_size)
    store_cache(K, V, cache, plan["slots"])
    out = attend_cache(Q, cache, block_table, ctx_len, plan["seq_len"], plan["q_start"])["out"]

Lengths, tables and slots stay on the GPU; nothing here waits for it, so a step can be captured in
a CUDA graph and replayed with other lengths in the same tensors.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import alhr

DEVERR_CAPACITY = 0x10
DEVERR_BLOCK = 0x20
DEVERR_NONFINITE = 0x40

_CODES = {torch.int8: 0, torch.float8_e4m3fn: 1}
_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.int8: 3}
BLOCK_SIZES = (16, 32, 64, 128)


class CacheStruct(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_void_p) for f in ("k", "v", "k_scale", "v_scale")] +
                [(f, ctypes.c_int32) for f in ("blocks", "heads", "block_size", "d", "code")])


class QueriesStruct(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_int32) for f in
                 ("requests", "tokens", "q_heads", "max_blocks", "max_q", "type")] +
                [(f, ctypes.c_int64) for f in ("q_token_stride", "q_head_stride")] +
                [("scale", ctypes.c_float)])


class SelectionStruct(ctypes.Structure):
    _fields_ = ([(f, ctypes.c_int32) for f in
                 ("batch", "q_heads", "nq", "max_keys", "max_blocks", "type")] +
                [("scale", ctypes.c_float)])


# The checks below run before every launch of a few microseconds: they read each attribute once.

def _need(t, dtype, shape, name, device):
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if t.device != device:
        raise ValueError(f"{name}: expected a tensor on {device}, got {t.device}")
    raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)}, got "
                     f"{t.dtype} {tuple(t.shape)}, strides {t.stride()}")


def _cuda(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    return t.device


def _err(dev_err, device):
    if dev_err is None:
        return None
    if dev_err.dtype not in (torch.int32, torch.uint32) or dev_err.numel() < 1 \
            or dev_err.device != device:
        raise ValueError("dev_err: expected one int32 word on the tensors' device")
    return dev_err.data_ptr()


_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream  # the handle itself, without an object


def _call(name, device, *args):
    """The entry point on `device` and its current stream."""
    fn = getattr(alhr.lib(), name)
    index = device.index
    if _current_device() == index:
        status = fn(*args, _current_stream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _current_stream(index))
    if status != alhr.ALHR_OK:
        raise alhr.AlhrError(status, name)


def _struct(cache, device):
    """The C view of a cache dict on `device`."""
    k, v, ks, vs = cache["k"], cache["v"], cache["k_scale"], cache["v_scale"]
    if k.dim() != 4 or k.dtype not in _CODES:
        raise ValueError(f"cache k: expected int8 or float8_e4m3fn [blocks, heads, block_size, d],"
                         f" got {k.dtype} {tuple(k.shape)}")
    blocks, heads, bs, d = k.shape
    scales = (blocks, heads)
    return CacheStruct(_need(k, k.dtype, k.shape, "cache k", device),
                       _need(v, k.dtype, k.shape, "cache v", device),
                       _need(ks, torch.float32, scales, "cache k_scale", device),
                       _need(vs, torch.float32, scales, "cache v_scale", device),
                       blocks, heads, bs, d, _CODES[k.dtype])


def alloc_cache(blocks: int, heads: int, block_size: int, d: int, dtype=torch.int8,
                device="cuda") -> dict:
    """An empty cache of `blocks` blocks of `block_size` tokens."""
    if dtype not in _CODES:
        raise ValueError(f"cache dtype {dtype}: int8 or float8_e4m3fn")
    if block_size not in BLOCK_SIZES:
        raise ValueError(f"block_size {block_size}: one of {BLOCK_SIZES}")
    if d not in (64, 128):
        raise ValueError(f"d {d}: 64 or 128")
    codes = lambda: torch.zeros((blocks, heads, block_size, d), dtype=dtype, device=device)
    scale = lambda: torch.zeros((blocks, heads), dtype=torch.float32, device=device)
    return dict(k=codes(), v=codes(), k_scale=scale(), v_scale=scale())


def plan_blocks(ctx_len: torch.Tensor, new_len: torch.Tensor, block_table: torch.Tensor,
                free_blocks: torch.Tensor, free_first: torch.Tensor, tokens: int,
                block_size: int, blocks: int = 2**31 - 1,
                dev_err: torch.Tensor | None = None) -> dict:
    """Block table, slots and row offsets of a step (alhr_plan_blocks).

    ctx_len, new_len int32 [R]; block_table int32 [R, max_blocks], updated in place; free_blocks
    int32 [F]; free_first int32 [1]; tokens: rows of the step's tensors, at least the new tokens;
    blocks: the cache's (a larger block number is refused on the device). Returns q_start int32
    [R + 1], seq_len int32 [R], slots int64 [tokens], positions int32 [tokens] and free_next
    int32 [1], the next step's free_first."""
    tokens = int(tokens)
    if not 0 <= tokens < 2**31:  # an int32 of the ABI
        raise ValueError(f"tokens {tokens}: at least 0, below 2^31")
    dev = _cuda(block_table, "block_table")
    if block_table.dim() != 2 or free_blocks.dim() != 1:
        raise ValueError("block_table [requests, max_blocks] and free_blocks [free] expected")
    r, width = block_table.shape
    ctx = _need(ctx_len, torch.int32, (r,), "ctx_len", dev)
    new = _need(new_len, torch.int32, (r,), "new_len", dev)
    table = _need(block_table, torch.int32, (r, width), "block_table", dev)
    free = _need(free_blocks, torch.int32, free_blocks.shape, "free_blocks", dev)
    first = _need(free_first, torch.int32, (1,), "free_first", dev)
    slots = ctx_len.new_empty(tokens, dtype=torch.int64)
    # one allocation for what is 32 bits wide
    q_start, seq_len, positions, free_next = ctx_len.new_empty(2 * r + tokens + 2).split(
        (r + 1, r, tokens, 1))
    _call("alhr_plan_blocks", dev, r, width, block_size, min(blocks, (2**31 - 1) // block_size),
          tokens, free_blocks.numel(), ctx, new, table, free, first, q_start.data_ptr(),
          seq_len.data_ptr(), slots.data_ptr(), positions.data_ptr(), free_next.data_ptr(),
          _err(dev_err, dev))
    return dict(q_start=q_start, seq_len=seq_len, slots=slots, positions=positions,
                free_next=free_next)


def _rows(t, shape, dtype, name, device):
    """Token and head strides of [tokens, heads, d] rows whose numbers are contiguous."""
    if t.dtype != dtype or t.shape != shape or (shape[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} with contiguous rows, got "
                         f"{t.dtype} {tuple(t.shape)}, strides {t.stride()}")
    if t.device != device:
        raise ValueError(f"{name}: expected a tensor on {device}, got {t.device}")
    # the stride of a single token or head is never used, whatever it says
    return t.stride(0) if shape[0] > 1 else 0, t.stride(1) if shape[1] > 1 else 0


def store_cache(K: torch.Tensor, V: torch.Tensor, cache: dict, slots: torch.Tensor,
                dev_err: torch.Tensor | None = None) -> None:
    """Writes keys and values [tokens, heads, d] (bf16, fp16 or fp32; rows contiguous, token and
    head strides multiples of 16 bytes) into their slots (int64 [tokens], -1 for none). A block's
    scale grows with its tokens; the codes before them are rounded anew when it does
    (alhr_store_cache). The tokens of one block must be consecutive rows."""
    dev = _cuda(slots, "slots")
    c = _struct(cache, dev)
    if K.dtype not in (torch.bfloat16, torch.float16, torch.float32):
        raise ValueError(f"K: bf16, fp16 or fp32 expected, got {K.dtype}")
    if slots.dim() != 1:
        raise ValueError(f"slots: expected [tokens], got {tuple(slots.shape)}")
    t = slots.shape[0]
    _need(slots, torch.int64, (t,), "slots", dev)
    shape = (t, c.heads, c.d)
    kt, kh = _rows(K, shape, K.dtype, "K", dev)
    vt, vh = _rows(V, shape, K.dtype, "V", dev)
    _call("alhr_store_cache", dev, ctypes.byref(c), K.data_ptr(), V.data_ptr(), _TYPES[K.dtype], t,
          kt, kh, vt, vh, slots.data_ptr(), _err(dev_err, dev))


def load_cache(cache: dict, slots: torch.Tensor, dtype=torch.bfloat16,
               dev_err: torch.Tensor | None = None) -> dict:
    """The keys and values [tokens, heads, d] that the slots (int64 [tokens]) hold, as `dtype`
    (bf16, fp16 or fp32); zeros for slot -1 (alhr_load_cache)."""
    dev = _cuda(slots, "slots")
    c = _struct(cache, dev)
    if dtype not in (torch.bfloat16, torch.float16, torch.float32):
        raise ValueError(f"dtype: bf16, fp16 or fp32 expected, got {dtype}")
    if slots.dim() != 1:
        raise ValueError(f"slots: expected [tokens], got {tuple(slots.shape)}")
    t = slots.shape[0]
    _need(slots, torch.int64, (t,), "slots", dev)
    K = slots.new_empty((t, c.heads, c.d), dtype=dtype)
    V = slots.new_empty((t, c.heads, c.d), dtype=dtype)
    _call("alhr_load_cache", dev, ctypes.byref(c), K.data_ptr(), V.data_ptr(), _TYPES[dtype], t,
          slots.data_ptr(), _err(dev_err, dev))
    return dict(K=K, V=V)


def attend_cache(Q: torch.Tensor, cache: dict, block_table: torch.Tensor, ctx_len: torch.Tensor,
                 seq_len: torch.Tensor, q_start: torch.Tensor, max_q: int | None = None,
                 scale: float | None = None, want_lse: bool = False,
                 out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 dev_err: torch.Tensor | None = None) -> dict:
    """Attention over all visible keys of each request (alhr_attend_cache).

    Q bf16 or fp16 [tokens, q_heads, d] (rows contiguous, strides multiples of 8 numbers), q_heads
    a multiple of the cache's heads; block_table int32 [R, max_blocks]; ctx_len, seq_len int32
    [R]; q_start int32 [R + 1]. Row t of request r sees the keys
    [0, min(ctx_len[r] + t - q_start[r] + 1, seq_len[r])). max_q: no request has more rows (it
    chooses the kernels; unknown: None); scale: 1 / sqrt(d) unless given. Returns out, of Q's type
    (rows outside every request keep what they hold), and lse float32 [tokens, q_heads] if asked
    for. workspace: uint8, at least attend_cache_workspace(...) bytes; calls that may run at the
    same time need one each. dev_err: DEVERR_BLOCK for a block number outside the cache;
    DEVERR_TIMEOUT, not expected, where the outputs are not to be used."""
    dev = _cuda(Q, "Q")
    c = _struct(cache, dev)
    if Q.dim() != 3 or Q.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"Q: bf16 or fp16 [tokens, q_heads, d] expected, got {Q.dtype} "
                         f"{tuple(Q.shape)}")
    if block_table.dim() != 2:
        raise ValueError("block_table: [requests, max_blocks] expected")
    t, hq, _ = Q.shape
    r, width = block_table.shape
    qt, qh = _rows(Q, (t, hq, c.d), Q.dtype, "Q", dev)
    table = _need(block_table, torch.int32, (r, width), "block_table", dev)
    ctx = _need(ctx_len, torch.int32, (r,), "ctx_len", dev)
    seq = _need(seq_len, torch.int32, (r,), "seq_len", dev)
    start = _need(q_start, torch.int32, (r + 1,), "q_start", dev)
    if max_q is not None and max_q < 1 and t > 0:
        raise ValueError(f"max_q {max_q}: at least 1, or None")
    if out is None:
        out = Q.new_empty((t, hq, c.d))
    else:
        _need(out, Q.dtype, (t, hq, c.d), "out", dev)
    lse = Q.new_empty((t, hq), dtype=torch.float32) if want_lse else None
    q = QueriesStruct(r, t, hq, width, max_q or 0, _TYPES[Q.dtype], qt, qh,
                      1.0 / math.sqrt(c.d) if scale is None else scale)
    cp, qp = ctypes.byref(c), ctypes.byref(q)
    if workspace is None:
        workspace = Q.new_empty(_workspace(cp, qp, dev), dtype=torch.uint8)
    elif workspace.dtype != torch.uint8 or workspace.device != dev \
            or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected contiguous uint8 on {dev}")
    _call("alhr_attend_cache", dev, cp, qp, Q.data_ptr(), table, ctx, seq, start, out.data_ptr(),
          None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
          _err(dev_err, dev))
    return dict(out=out, lse=lse) if want_lse else dict(out=out)


def _workspace(cp, qp, dev) -> int:
    if _current_device() == dev.index:
        return alhr.lib().alhr_attend_cache_workspace(cp, qp)
    with torch.cuda.device(dev):
        return alhr.lib().alhr_attend_cache_workspace(cp, qp)


def attend_cache_workspace(Q: torch.Tensor, cache: dict, block_table: torch.Tensor) -> int:
    """Bytes of attend_cache's workspace for these tensors."""
    dev = _cuda(Q, "Q")
    c = _struct(cache, dev)
    q = QueriesStruct(block_table.shape[0], Q.shape[0], Q.shape[1], block_table.shape[1], 0,
                      _TYPES[Q.dtype], 0, 0, 1.0)
    return _workspace(ctypes.byref(c), ctypes.byref(q), dev)


def attend_cache_selected(Q: torch.Tensor, cache: dict, block_table: torch.Tensor,
                          ctx_len: torch.Tensor, seq_len: torch.Tensor, idx: torch.Tensor,
                          count: torch.Tensor, scale: float | None = None,
                          out: torch.Tensor | None = None,
                          dev_err: torch.Tensor | None = None) -> torch.Tensor:
    """alhr.attend over the cache: exact attention over selected positions, e.g. route's idx and
    count (alhr_attend_cache_selected). Q int8, bf16 or fp16 [B, H, nq, d], H a multiple of the
    cache's heads; block_table int32 [B, max_blocks]; ctx_len, seq_len int32 [B], row t at
    position ctx_len + t; idx int32 [B, H, nq, max_keys], count int32 [B, H, nq]; scale:
    1 / sqrt(d) unless given. Returns out float32 [B, H, nq, d]."""
    dev = _cuda(Q, "Q")
    c = _struct(cache, dev)
    if Q.dim() != 4 or Q.dtype not in (torch.int8, torch.bfloat16, torch.float16):
        raise ValueError(f"Q: int8, bf16 or fp16 [B, H, nq, d] expected, got {Q.dtype} "
                         f"{tuple(Q.shape)}")
    if block_table.dim() != 2 or idx.dim() != 4:
        raise ValueError("block_table [B, max_blocks] and idx [B, H, nq, max_keys] expected")
    B, H, nq, _ = Q.shape
    _need(Q, Q.dtype, (B, H, nq, c.d), "Q", dev)
    width, keys = block_table.shape[1], idx.shape[3]
    table = _need(block_table, torch.int32, (B, width), "block_table", dev)
    ctx = _need(ctx_len, torch.int32, (B,), "ctx_len", dev)
    seq = _need(seq_len, torch.int32, (B,), "seq_len", dev)
    ip = _need(idx, torch.int32, (B, H, nq, keys), "idx", dev)
    np_ = _need(count, torch.int32, (B, H, nq), "count", dev)
    if out is None:
        out = torch.empty((B, H, nq, c.d), dtype=torch.float32, device=dev)
    else:
        _need(out, torch.float32, (B, H, nq, c.d), "out", dev)
    s = SelectionStruct(B, H, nq, keys, width, _TYPES[Q.dtype],
                        1.0 / math.sqrt(c.d) if scale is None else scale)
    _call("alhr_attend_cache_selected", dev, ctypes.byref(c), ctypes.byref(s), Q.data_ptr(), table,
          ctx, seq, ip, np_, out.data_ptr(), _err(dev_err, dev))
    return out
