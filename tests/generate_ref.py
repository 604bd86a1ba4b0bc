"""Plain numpy reference of the generation step: the NVFP4 cache layout, its quantizer, the page and slot maps,
attention and the products with NVFP4 weights, in 64 bits (the quantizer in FP32, operation by operation, as its
definition has it).  Shares no code with the library."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=np.float64)
E2M1_16 = np.concatenate([E2M1, -E2M1])
E4M3 = np.array([np.nan if c & 127 == 127 else (-1.0 if c & 128 else 1.0) * (
    (c & 7) * 2.0 ** -9 if (c >> 3) & 15 == 0 else (1 + (c & 7) / 8) * 2.0 ** (((c >> 3) & 15) - 7)) for c in range(256)])


def bf16_bits(a):
    """FP32 array -> BF16 bit patterns (round to nearest even); NaN stays NaN."""
    u = np.ascontiguousarray(a, dtype=np.float32).view(np.uint32)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(np.asarray(a, dtype=np.float32)), np.uint16(0x7FC0), r)


def bf16_value(b):
    return (np.asarray(b, dtype=np.uint32) << 16).view(np.float32)


def _nearest(v, grid):
    """Index of the grid point nearest to v >= 0 (ties to the even index, saturating)."""
    v = np.asarray(v, dtype=np.float64)
    hi = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
    lo = hi - 1
    below, above = v - grid[lo], grid[hi] - v
    return np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)


def quantize_blocks(x, S):
    """x [..., 16] FP32, S [...] FP32 -> (codes [..., 16], block scale bytes [...])."""
    x, S = np.asarray(x, dtype=np.float32), np.broadcast_to(np.asarray(S, dtype=np.float32), x.shape[:-1])
    f = np.float32
    with np.errstate(all="ignore"):
        amax = np.abs(x).max(-1)                                     # NaN spreads
        t = (amax / f(6.0)) / np.where(S == 0, f(1), S)
        bs = np.where(np.isnan(t), 127, _nearest(np.where(np.isnan(t), 0, t), E4M3[:127]))
        bs = np.where(S == 0, 0, bs).astype(np.uint8)
        d = E4M3[bs].astype(f) * S
        r = np.minimum(np.where(d == 0, f(0), f(1) / np.where(d == 0, f(1), d)), np.finfo(f).max).astype(f)
        y = x * r[..., None]
        codes = _nearest(np.where(np.isnan(y), 0, np.abs(y)), E2M1).astype(np.uint8)
    return codes | (np.signbit(x).astype(np.uint8) << 3), bs


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(b):
    return np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1)


def v_scale_position(i):
    return i ^ ((i >> 1) & 1)


def cache_write(cache, slot, k, v, s_k, s_v, page):
    """Write one token's k, v [heads, D] (FP32 values) into cache [pages, heads, page / 16, 18 D]."""
    heads, D = k.shape
    p, off = slot // page, slot % page
    g, i = off // 16, off % 16
    for h in range(heads):
        rec = cache[p, h, g]
        for base, x, S in ((0, k[h], s_k[h]), (9 * D, v[h], s_v[h])):
            codes, bs = quantize_blocks(x.reshape(-1, 16), np.full(D // 16, S, np.float32))
            rec[base + i * (D // 2):base + (i + 1) * (D // 2)] = pack(codes.reshape(-1))
            if base == 0:
                rec[8 * D + i * (D // 16):8 * D + (i + 1) * (D // 16)] = bs
            else:
                rec[17 * D + np.arange(D // 16) * 16 + v_scale_position(i)] = bs


def cache_read(cache, slot, page):
    """(k, v) of one slot as val(code) * val(block scale), [heads, D] each (64 bits, without S)."""
    p, off = slot // page, slot % page
    g, i = off // 16, off % 16
    rec = cache[p, :, g]
    D = rec.shape[-1] // 18
    k = E2M1_16[unpack(rec[:, i * (D // 2):(i + 1) * (D // 2)])]
    v = E2M1_16[unpack(rec[:, 9 * D + i * (D // 2):9 * D + (i + 1) * (D // 2)])]
    ks = E4M3[rec[:, 8 * D + i * (D // 16):8 * D + (i + 1) * (D // 16)]]
    vs = E4M3[rec[:, 17 * D + np.arange(D // 16) * 16 + v_scale_position(i)]]
    return k * np.repeat(ks, 16, -1), v * np.repeat(vs, 16, -1)


def slots(seq, new, page, table, free, count, max_tokens):
    """The maps of a step, request by request: dict of outputs (the table as a new array)."""
    table, width = table.copy(), table.shape[1]
    seq, new = np.maximum(seq, 0), np.maximum(new, 0)
    left = max(0, min(int(count), len(free)))
    slot, pos = [], []
    for r in range(len(seq)):
        for c in range(-(-int(seq[r]) // page), min(-(-int(seq[r] + new[r]) // page), width)):
            table[r, c] = free[left - 1] if left > 0 else -1
            left -= left > 0
        for p in range(int(seq[r]), int(seq[r] + new[r])):
            at = table[r, p // page] if p // page < width else -1
            slot.append(at * page + p % page if at >= 0 else -1)
            pos.append(p)
    n = len(slot)
    fill = [-1] * max(0, max_tokens - n)
    slot = np.array((slot + fill)[:max_tokens], dtype=np.int64)
    return {"block_table": table, "q_start": np.concatenate([[0], np.cumsum(new)]), "total_lens": seq + new, "slots": slot,
            "positions": np.array((pos + fill)[:max_tokens]), "free_left": left, "unplaced": n - int((slot >= 0).sum())}


def attention(q, q_start, seq_lens, table, cache, s_k, s_v, scale, page, window=0):
    """64-bit attention.  q [T, heads, D] values.  Returns out, lse and, for error bounds, mix [T, heads, D] = sum p |v| / sum p
    and reach [T, heads] = the largest scale * sum |q| |k| over the attended positions."""
    T, heads, D = q.shape
    kv = cache.shape[1]
    out, mix = np.zeros(q.shape), np.zeros(q.shape)
    lse, reach = np.full((T, heads), -np.inf), np.zeros((T, heads))
    for r in range(len(seq_lens)):
        n = int(q_start[r + 1] - q_start[r])
        if n <= 0:
            continue
        L = max(0, int(seq_lens[r]))
        K, V, there = np.zeros((L, kv, D)), np.zeros((L, kv, D)), np.zeros(L, bool)
        for j in range(L):
            at = table[r, j // page] if j // page < table.shape[1] else -1
            if 0 <= at < cache.shape[0]:
                K[j], V[j] = cache_read(cache, int(at) * page + j % page, page)
                there[j] = True
        K, V = K * np.asarray(s_k, np.float64)[None, :, None], V * np.asarray(s_v, np.float64)[None, :, None]
        for i in range(n):
            t, pos = int(q_start[r]) + i, L - n + i
            lo = max(0, pos - window + 1) if window else 0
            js = np.arange(lo, max(lo, pos + 1))
            js = js[there[js]] if len(js) else js
            if not len(js):
                continue
            for h in range(heads):
                k, v = K[js, h // (heads // kv)], V[js, h // (heads // kv)]
                z = scale * (k @ q[t, h])
                m = z.max()
                p = np.exp(z - m)
                out[t, h] = p @ v / p.sum()
                mix[t, h] = p @ np.abs(v) / p.sum()
                lse[t, h] = m + np.log(p.sum())
                reach[t, h] = abs(scale) * (np.abs(k) @ np.abs(q[t, h])).max()
    return out, lse, mix, reach


def gemm_layout(compact):
    """Block scales [rows, cols] -> the GEMM scale layout."""
    rows, cols = compact.shape
    nct = -(-cols // 4)
    out = np.zeros(-(-rows // 128) * nct * 512, np.uint8)
    r, c = np.arange(rows)[:, None], np.arange(cols)[None, :]
    out[(r // 128 * nct + c // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + c % 4] = compact
    return out
