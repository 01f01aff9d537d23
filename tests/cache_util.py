"""The paged 8-bit cache by its definition, in 64 bits (plans in whole numbers), and its inputs."""
import math

import torch

FULL = {torch.int8: 127.0, torch.float8_e4m3fn: 256.0}
SAT = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
TINY = 2.0 ** -100


def ceil_div(a, b):
    return -(-a // b)


def plan_ref(ctx, new, table, free, first, tokens, bs, blocks):
    """alhr_plan_blocks over lists: (q_start, seq_len, slots, positions, free_next, table, flags)."""
    width = len(table[0]) if table else 1
    cap, flags = width * bs, 0
    table = [row[:] for row in table]
    first = min(max(first, 0), len(free))
    q_start, seq_len = [0], []
    slots, positions = [-1] * tokens, [-1] * tokens
    at = first
    for r in range(len(ctx)):
        n = max(new[r], 0)
        lo = q_start[-1]
        rows = min(lo + n, tokens) - lo
        flags |= 0x10 if rows < n else 0
        q_start.append(lo + rows)
        c = min(max(ctx[r], 0), cap)
        end = min(c + rows, cap)
        flags |= 0x10 if end - c < rows else 0
        held, total = ceil_div(c, bs), ceil_div(end, bs)
        have = held
        for j in range(held, total):
            if at < len(free):
                b = free[at]
                if not 0 <= b < blocks:
                    b, flags = -1, flags | 0x20
                table[r][j] = b
                have = j + 1
            else:
                table[r][j] = -1
                flags |= 0x10
            at += 1
        seq_len.append(min(end, have * bs))
        for t in range(rows):
            p = c + t
            positions[lo + t] = p
            if p < end:
                b = table[r][p // bs]
                if 0 <= b < blocks:
                    slots[lo + t] = b * bs + p % bs
                elif p // bs < held:
                    flags |= 0x20
    return q_start, seq_len, slots, positions, min(at, len(free)), table, flags


def encode(x, dtype):
    """fp32 numbers to codes: nearest, ties to even, saturated, NaN as 0."""
    x = torch.where(x.isnan(), torch.zeros_like(x), x).clamp(-SAT[dtype], SAT[dtype])
    return (x.round() if dtype == torch.int8 else x).to(dtype)


def store_ref(x, codes, scale, slots):
    """alhr_store_cache of one of K and V in its own fp32 steps (they are exact to the bit): x
    [T, H, d] fp32 on the CPU; codes [blocks, H, bs, d] and scale [blocks, H] are changed."""
    blocks, heads, bs, d = codes.shape
    dt = codes.dtype
    runs, slots = [], slots.tolist()
    for t, s in enumerate(slots):
        if not 0 <= s < blocks * bs:
            continue
        if runs and runs[-1][1] == t and s % bs and slots[t - 1] + 1 == s:
            runs[-1][1] = t + 1
        else:
            runs.append([t, t + 1])
    for a, b in runs:
        page, off = divmod(slots[a], bs)
        for h in range(heads):
            part = x[a:b, h]
            finite = part[part.isfinite()]
            amax = finite.abs().max() if finite.numel() else torch.tensor(0.0)
            old = scale[page, h].clone() if off else torch.tensor(0.0)
            s = torch.maximum(torch.maximum(old, amax / FULL[dt]), torch.tensor(TINY))
            if off and s > old:
                codes[page, h, :off] = encode(codes[page, h, :off].float() * (old / s), dt)
            codes[page, h, off:off + b - a] = encode(part / s, dt)
            scale[page, h] = s


def numbers(codes, scale):
    """What a cache's codes stand for, in 64 bits."""
    return codes.float().double() * scale.double()[:, :, None, None]


def score_error(d, most):
    """Relative error of exp(s) and absolute error of s, for |q| . |k| * scale <= most: the
    products of codes and queries are exact, the d additions and three multiplications (scales,
    log2 e) round at 2^-24 of at most `most` each, and the subtraction of the maximum and the
    power of two (2 ulp) add a few roundings of numbers that are no larger than 2 * most."""
    return (d + 16) * 2.0 ** -24 * (most + 1.0)


def attend_ref(q, k, v, kscale, vscale, table, ctx, seq, q_start, scale, k_all=None):
    """alhr_attend_cache in 64 bits. Returns out, lse, weight (sum p |v|: what a relative error of
    the weights can move), most (|q| . |k| * scale), which rows belong to a request and small:
    what an absolute error of 1 in every weight can move, for weights 2^(x_j - M),
    x_j = log2(exp(s_j) vscale_j), that multiply codes and of which the largest is at least 1:
    sum |code_j| / l with l = sum 2^(x_j - M) / vscale_j >= 1 / vscale_top, so that
    small = vscale_top sum |code_j|."""
    T, hq, d = q.shape
    blocks, hkv, bs, _ = k.shape
    width, g = table.shape[1], hq // hkv
    dev = q.device
    out = torch.zeros(T, hq, d, dtype=torch.float64, device=dev)
    weight, small = torch.zeros_like(out), torch.zeros_like(out)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device=dev)
    owned = torch.zeros(T, dtype=torch.bool)
    most = 0.0
    ctx, seq, q_start = ctx.tolist(), seq.tolist(), q_start.tolist()
    for r in range(len(ctx)):
        lo, hi = max(q_start[r], 0), min(q_start[r + 1], T)
        if hi <= lo:
            continue
        owned[lo:hi] = True
        n = max(0, min(seq[r], ctx[r] + hi - lo, width * bs))
        if n == 0:
            continue
        pages = table[r, :ceil_div(n, bs)].long()
        ok = ((pages >= 0) & (pages < blocks)).repeat_interleave(bs)[:n]
        pages = pages.clamp(0, blocks - 1)
        take = lambda x, s: numbers(x[pages], s[pages]).transpose(0, 1).reshape(hkv, -1, d)[:, :n]
        K, V = take(k, kscale), take(v, vscale)
        codes = torch.nan_to_num(take(v, torch.ones_like(vscale))).abs()
        vs = vscale[pages].double().T.repeat_interleave(bs, 1)[:, :n].clamp(min=TINY)
        pos = ctx[r] + torch.arange(hi - lo, device=dev)
        seen = (torch.arange(n, device=dev)[None] <= pos[:, None]) & ok[None]
        for h in range(hkv):
            Q = q[lo:hi, h * g:(h + 1) * g].double()
            s = torch.einsum("tgd,nd->tgn", Q, K[h]) * scale
            most = max(most, float(torch.einsum("tgd,nd->tgn", Q.abs(), K[h].abs()).max()) * abs(scale))
            s = s.masked_fill(~seen[:, None], -math.inf)
            l = torch.logsumexp(s, -1)
            p = torch.exp(s - torch.where(l.isinf(), torch.zeros_like(l), l)[..., None])
            # a masked key's weight is 0 whatever its value is
            out[lo:hi, h * g:(h + 1) * g] = p @ torch.nan_to_num(V[h])
            weight[lo:hi, h * g:(h + 1) * g] = p @ torch.nan_to_num(V[h]).abs()
            lse[lo:hi, h * g:(h + 1) * g] = l
            top = vs[h][(s + vs[h].log()).argmax(-1)]
            small[lo:hi, h * g:(h + 1) * g] = top[..., None] * (
                seen.double() @ codes[h])[:, None]
    return out, lse, weight, most, owned, small


def random_cache(blocks, hkv, bs, d, dtype, g, dev, spread=0.4):
    """Random codes over the whole range and scales that differ from block to block."""
    x = lambda: torch.randn(blocks, hkv, bs, d, generator=g, device=dev)
    c = (lambda: (x() * 40).round().clamp(-127, 127).to(dtype)) if dtype == torch.int8 else \
        (lambda: (x() * 100).clamp(-448, 448).to(dtype))
    base = 0.025 if dtype == torch.int8 else 0.01
    s = lambda: base * torch.exp(spread * torch.randn(blocks, hkv, generator=g, device=dev))
    return dict(k=c(), v=c(), k_scale=s(), v_scale=s())


def scattered_table(lens, bs, blocks, width, g, dev):
    """Pages of every request from a random order; -1 behind them."""
    order = torch.randperm(blocks, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=dev)
    at = 0
    for r, n in enumerate(lens):
        p = ceil_div(n, bs)
        table[r, :p] = order[at:at + p]
        at += p
    assert at <= blocks
    return table
