"""The operators of 4-bit decoding: what is measured, their plain forms and their definitions in 64 bits.

One generation step over NVFP4 weights and an NVFP4 key/value cache calls, in this order, the page and slot
maps of the new tokens (`slots`), the products with 4-bit weights (`matvec`), the write of the new keys and
values into the cache and their reading back (`cache`), and the attention over the cache (`attention`).

The cache is one byte tensor [pages, kv heads, page_size / 16, 18 * head_dim].  The last axis holds 16 tokens of
one head: 16 rows of K codes (head_dim / 2 bytes, the even element in the low nibble), 16 rows of K block scales
(head_dim / 16 E4M3 bytes), 16 rows of V codes, and the V block scales with the block index first, the 16
tokens of a block side by side with token i at position i ^ ((i >> 1) & 1).  A value is
val(code) * val(block scale) * S, with one FP32 S per kv head for K and one for V.  Slot number: page *
page_size + offset inside the page.
"""
import numpy as np
import torch

own = False

_BF16_STEP = 16                                       # elements that share a block scale
_WORKSPACE_BYTES = 64 << 20                           # one workspace for every attention call of a program


# --------------------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------------------

def listed():
    return [
        # page and slot maps of a decoding batch: one new token for most requests, none for idle ones
        {"name": "slots_decode_64", "op": "slots", "requests": 64, "longest": 8191, "most_new": 1, "page": 16},
        # the same for a batch with prompts in it: thousands of new tokens, ragged
        {"name": "slots_prompts_500", "op": "slots", "requests": 500, "longest": 4099, "most_new": 129, "page": 32},
        # new keys and values of a decoding batch into the cache, and back as BF16
        {"name": "cache_decode_64", "op": "cache", "tokens": 64, "kv_heads": 8, "head_dim": 128, "page": 16},
        # a long prompt's keys and values, odd in length
        {"name": "cache_prompt_16381", "op": "cache", "tokens": 16381, "kv_heads": 8, "head_dim": 128, "page": 64},
        # one request with a short context: latency counts
        {"name": "attention_one_short", "op": "attention", "requests": 1, "longest": 777, "most_new": 1, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 16, "window": 0},
        # one request with a very long context: the work has to be split along it
        {"name": "attention_one_long", "op": "attention", "requests": 1, "longest": 131071, "most_new": 1, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 64, "window": 0},
        # a full decoding batch, ragged, the largest case
        {"name": "attention_batch_64", "op": "attention", "requests": 64, "longest": 8192, "most_new": 1, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 16, "window": 0},
        # several drafted tokens a request are verified at once, fewer kv heads, small head dimension, a window
        {"name": "attention_drafts_24", "op": "attention", "requests": 24, "longest": 5003, "most_new": 6, "heads": 32,
         "kv_heads": 4, "head_dim": 64, "page": 32, "window": 4000},
        # square projection of one token: the smallest product
        {"name": "matvec_1x4096x4096", "op": "matvec", "tokens": 1, "outputs": 4096, "inputs": 4096, "per_row": False,
         "fp32_out": False},
        # feed-forward width, a few tokens
        {"name": "matvec_5x12288x4096", "op": "matvec", "tokens": 5, "outputs": 12288, "inputs": 4096, "per_row": True,
         "fp32_out": False},
        # output head of one token: FP32 logits over an odd number of entries
        {"name": "matvec_1x151937x2048", "op": "matvec", "tokens": 1, "outputs": 151937, "inputs": 2048,
         "per_row": True, "fp32_out": True},
        # a decoding batch through the long contraction
        {"name": "matvec_16x4096x14336", "op": "matvec", "tokens": 16, "outputs": 4096, "inputs": 14336,
         "per_row": False, "fp32_out": False},
    ]


def _log_between(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["slots", "cache", "attention", "attention", "matvec", "matvec"])
    if op == "slots":
        return {"op": op, "requests": _log_between(rng, 1, 600), "longest": _log_between(rng, 16, 9000),
                "most_new": rng.choice([1, 1, _log_between(rng, 2, 130)]), "page": rng.choice([16, 32, 64, 128])}
    if op == "cache":
        return {"op": op, "tokens": _log_between(rng, 1, 16381), "kv_heads": rng.choice([1, 2, 4, 8]),
                "head_dim": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 128])}
    if op == "attention":
        kv_heads, head_dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        requests = _log_between(rng, 1, 64)
        longest = _log_between(rng, 16, min(131071, 64 * 8192 // requests))
        return {"op": op, "requests": requests, "longest": longest,
                "most_new": min(longest, rng.choice([1, 1, rng.randint(2, 8)])),
                "heads": kv_heads * rng.choice([1, 2, 4, 5, 8]), "kv_heads": kv_heads, "head_dim": head_dim,
                "page": rng.choice([16, 32, 64, 128]), "window": rng.choice([0, 0, 0, _log_between(rng, 16, 4096)])}
    tokens, inputs = _log_between(rng, 1, 16), 16 * _log_between(rng, 16, 896)
    return {"op": op, "tokens": tokens, "outputs": _log_between(rng, 64, min(151937, 250_000_000 // inputs)),
            "inputs": inputs, "per_row": rng.random() < 0.5, "fp32_out": rng.random() < 0.3}


# --------------------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------------------

def _ceil_div(a, b):
    return (a + b - 1) // b


def _lengths(case):
    """Tokens of each request (new ones included) and how many of them are new: ragged, the longest at its full
    length, in larger batches one idle request and one that has just begun.  They go with the case."""
    rng = np.random.default_rng([case["requests"], case["longest"]])
    n, longest, most = case["requests"], case["longest"], case["most_new"]
    total = rng.integers(max(1, longest // 4), longest + 1, n)
    total[rng.integers(n)] = longest
    new = rng.integers(1, most + 1, n) if most > 1 else np.ones(n, np.int64)
    if n >= 8:
        total[2], new[2] = 0, 0
        total[5], new[5] = 1, 1
    return total, np.minimum(new, total)


def _page_table(case, total, seed):
    """A table of distinct pages in random order, -1 where a request has none, and the number of pages."""
    rng = np.random.default_rng([seed, 11])
    per = _ceil_div(total, case["page"])
    pages = int(per.sum()) + 3
    order = rng.permutation(pages)
    table = np.full((len(total), max(1, int(per.max())) + 1), -1, np.int64)
    table[np.arange(table.shape[1])[None, :] < per[:, None]] = order[:int(per.sum())]
    return table, pages, order[int(per.sum()):]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    def i32(a):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)

    s = {"case": case, "op": case["op"]}
    if case["op"] == "slots":
        total, new = _lengths(case)
        before = total - new
        table, pages, rest = _page_table(case, before, seed)
        table = np.pad(table, ((0, 0), (0, _ceil_div(case["longest"], case["page"]) + 1 - table.shape[1])),
                       constant_values=-1) if table.shape[1] <= _ceil_div(case["longest"], case["page"]) else table
        need = int((_ceil_div(total, case["page"]) - _ceil_div(before, case["page"])).sum())
        free = np.concatenate([rest, pages + np.arange(need + 5)])
        most = int(new.sum()) + 7                      # a buffer of fixed length, longer than what is needed
        s |= {"seq_lens": i32(before), "new_lens": i32(new), "page": case["page"], "block_table": i32(table),
              "free_pages": i32(np.random.default_rng([seed, 12]).permutation(free)), "free_count": i32([len(free) - 2]),
              "most": most, "q_start": i32(np.zeros(len(new) + 1)), "total_lens": i32(np.zeros(len(new))),
              "slots": i32(np.zeros(most)), "positions": i32(np.zeros(most)), "free_left": i32([0]),
              "unplaced": i32([0])}
        return s
    if case["op"] == "matvec":
        m, n, k = case["tokens"], case["outputs"], case["inputs"]
        x = normal(m, k)
        x[:, torch.randint(k, (max(1, k // 200),), generator=g, device=dev)] *= 20.0   # outlier channels
        s["x"] = x.to(torch.bfloat16)
        amax_row = 2688.0 * (0.02 * 5 / 2688.0) * (0.75 + 0.5 * torch.rand(n, generator=g, device=dev))
        s["s2"] = (amax_row / 2688.0) if case["per_row"] else amax_row[:1] / 2688.0
        scale_of = s["s2"].expand(n)
        code, bs = _quantize(0.02 * normal(n, k), scale_of[:, None])
        s["q"] = _pack_nibbles(code)
        rows, cols = _ceil_div(n, 128) * 128, _ceil_div(k // 16, 4) * 4
        s["s"] = torch.zeros(rows * cols, dtype=torch.uint8, device=dev)
        s["s"][_scale_places(n, k, dev).reshape(-1)] = bs.reshape(-1)
        s["y"] = torch.empty((m, n), dtype=torch.float32 if case["fp32_out"] else torch.bfloat16, device=dev)
        return s
    heads, dim, page = case["kv_heads"], case["head_dim"], case["page"]
    s["s_k"] = (4.0 + 4.0 * torch.rand(heads, generator=g, device=dev)) / 2688.0      # calibrated per head
    s["s_v"] = (4.0 + 4.0 * torch.rand(heads, generator=g, device=dev)) / 2688.0
    channel = 0.5 + torch.rand((1, heads, dim), generator=g, device=dev)              # keys have loud channels
    if case["op"] == "cache":
        t = case["tokens"]
        pages = _ceil_div(t, page) + 4
        qkv = normal(t, 3 * heads, dim)                # q, k and v of one projection side by side
        qkv[:, heads:2 * heads] *= channel
        s["qkv"] = qkv.to(torch.bfloat16)
        s["k"], s["v"] = s["qkv"][:, heads:2 * heads], s["qkv"][:, 2 * heads:]
        order = torch.randperm(pages, generator=g, device=dev)
        at = torch.arange(t, device=dev) + page // 3    # the first page is partly filled already
        s["slots"] = (order[at // page] * page + at % page).to(torch.int32)
        s["cache"] = torch.zeros((pages, heads, page // 16, 18 * dim), dtype=torch.uint8, device=dev)
        s["k_out"] = torch.empty((t, heads, dim), dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.empty((t, heads, dim), dtype=torch.bfloat16, device=dev)
        return s
    total, new = _lengths(case)
    table, pages, _ = _page_table(case, total, seed)
    tokens = int(new.sum())
    s |= {"q": normal(tokens, case["heads"], dim).to(torch.bfloat16), "q_start": i32(np.concatenate([[0], np.cumsum(new)])),
          "seq_lens": i32(total), "block_table": i32(table), "max_q": int(new.max()), "scale": dim ** -0.5,
          "window": case["window"], "longest": int(total.max()),
          "out": torch.empty((tokens, case["heads"], dim), dtype=torch.bfloat16, device=dev),
          "lse": torch.empty((tokens, case["heads"]), dtype=torch.float32, device=dev),
          "workspace": torch.empty(_WORKSPACE_BYTES, dtype=torch.uint8, device=dev)}
    code, bs = _quantize(normal(pages * page, heads, dim) * channel, s["s_k"][None, :, None])
    kc = _pack_nibbles(code).view(pages, page // 16, 16, heads, dim // 2).permute(0, 3, 1, 2, 4).reshape(pages, heads, page // 16, 8 * dim)
    ks = bs.view(pages, page // 16, 16, heads, dim // 16).permute(0, 3, 1, 2, 4).reshape(pages, heads, page // 16, dim)
    code, bs = _quantize(normal(pages * page, heads, dim), s["s_v"][None, :, None])
    vc = _pack_nibbles(code).view(pages, page // 16, 16, heads, dim // 2).permute(0, 3, 1, 2, 4).reshape(pages, heads, page // 16, 8 * dim)
    place = torch.arange(16, device=dev)
    vs = bs.view(pages, page // 16, 16, heads, dim // 16)[:, :, place ^ ((place >> 1) & 1)].permute(0, 3, 1, 4, 2).reshape(pages, heads, page // 16, dim)
    s["cache"] = torch.cat([kc, ks, vc, vs], -1)
    return s


# --------------------------------------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------------------------------------

def _quantize(x, S):
    """E2M1 codes [..., n] and E4M3 block scale bytes [..., n / 16] of x under the second-level scale S [..., 1]:
    bs = E4M3(amax / 6 / S), code = E2M1(x * (1 / (bs * S))), rounded to nearest even, saturating."""
    blocks = x.unflatten(-1, (-1, _BF16_STEP))
    amax = blocks.abs().amax(-1)
    S = S.expand(amax.shape)
    bs8 = torch.where(S == 0, torch.zeros_like(amax), amax / torch.full_like(amax, 6.0) / S).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = bs8.float() * S
    r = torch.where(d == 0, torch.zeros_like(d), torch.ones_like(d) / d).clamp(max=torch.finfo(torch.float32).max)
    y = (blocks * r[..., None]).flatten(-2)
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
            + 8 * torch.signbit(y).to(torch.uint8))
    return code, bs8.view(torch.uint8)


def _pack_nibbles(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _unpack_values(codes):
    """FP32 values of packed E2M1 codes, the even element from the low nibble."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=codes.device)
    byte = torch.arange(256, device=codes.device)
    return torch.stack([table[byte & 15], table[byte >> 4]], -1)[codes.int()].flatten(-2)


def _scale_places(rows, k, device):
    """Byte offsets [rows, k / 16] of the block scales in the GEMM scale layout (512-byte tiles of 128 rows x 4)."""
    r, c = torch.arange(rows, device=device)[:, None], torch.arange(k // 16, device=device)[None, :]
    return (r // 128 * _ceil_div(k // 16, 4) + c // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + c % 4


def _dequantize(codes, scales, S):
    return _unpack_values(codes) * scales.view(torch.float8_e4m3fn).float().repeat_interleave(_BF16_STEP, -1) * S


def _places(slots, cache, page):
    """Byte offsets in the cache of K codes, K scales, V codes and V scales for each slot and head."""
    _, heads, groups, record = cache.shape
    dim, dev = record // 18, cache.device
    slot = slots.long()[:, None]
    base = ((slot // page * heads + torch.arange(heads, device=dev)[None, :]) * groups + slot % page // 16) * record
    i = (slot % 16)[..., None]
    code, block = torch.arange(dim // 2, device=dev), torch.arange(dim // 16, device=dev)
    base = base[..., None]
    return (base + i * (dim // 2) + code, base + 8 * dim + i * (dim // 16) + block, base + 9 * dim + i * (dim // 2) + code,
            base + 17 * dim + block * 16 + (i ^ ((i >> 1) & 1)))


def _plain_slots(s):
    seq, new, page, table = s["seq_lens"].long(), s["new_lens"].long(), s["page"], s["block_table"].long()
    width = table.shape[1]
    total = seq + new
    q_start = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    had = (seq + page - 1) // page
    have = torch.maximum(((total + page - 1) // page).clamp(max=width), had)
    need = have - had
    base = need.cumsum(0) - need
    free = s["free_count"].long()
    column = torch.arange(width, device=seq.device)[None, :]
    k = base[:, None] + column - had[:, None]
    fresh = (column >= had[:, None]) & (column < have[:, None])
    given = s["free_pages"].long()[(free - 1 - k).clamp(0, s["free_pages"].numel() - 1)]
    table = torch.where(fresh, torch.where(k < free, given, -torch.ones_like(k)), table)
    t = torch.arange(s["most"], device=seq.device)
    r = torch.searchsorted(q_start[1:].contiguous(), t, right=True).clamp(max=seq.numel() - 1)
    real = t < q_start[-1]
    pos = seq[r] + t - q_start[r]
    at = table[r, (pos // page).clamp(max=width - 1)]
    placed = real & (pos // page < width) & (at >= 0)
    slots = torch.where(placed, at * page + pos % page, -torch.ones_like(pos))
    return {"block_table": table.int(), "q_start": q_start.int(), "total_lens": total.int(), "slots": slots.int(),
            "positions": torch.where(real, pos, -torch.ones_like(pos)).int(),
            "free_left": (free - need.sum()).clamp(min=0).int(), "unplaced": (q_start[-1] - placed.sum()).int().reshape(1)}


def _plain_cache(s):
    cache, page = s["cache"], s["case"]["page"]
    k_code, k_bs = _quantize(s["k"].float(), s["s_k"][None, :, None])
    v_code, v_bs = _quantize(s["v"].float(), s["s_v"][None, :, None])
    kc, ks, vc, vs = _places(s["slots"], cache, page)
    flat = cache.view(-1)
    flat[kc], flat[ks], flat[vc], flat[vs] = _pack_nibbles(k_code), k_bs, _pack_nibbles(v_code), v_bs
    return {"k": _dequantize(flat[kc], flat[ks], s["s_k"][None, :, None]).to(torch.bfloat16),
            "v": _dequantize(flat[vc], flat[vs], s["s_v"][None, :, None]).to(torch.bfloat16)}


def _plain_attention(s):
    case, cache = s["case"], s["cache"]
    page, heads, kv_heads, dim = case["page"], case["heads"], case["kv_heads"], case["head_dim"]
    n, most = s["seq_lens"].numel(), s["max_q"]
    length, dev = s["longest"], cache.device
    used = -(-length // page)
    got = cache[s["block_table"][:, :used].long().clamp(min=0)].transpose(1, 2).flatten(2, 3)     # [n, kv, groups, 18 dim]
    kc, ks, vc, vs = got.split([8 * dim, dim, 8 * dim, dim], -1)
    k = _dequantize(kc.unflatten(-1, (16, -1)).contiguous(), ks.unflatten(-1, (16, -1)).contiguous(), s["s_k"][None, :, None, None, None])
    i = torch.arange(16, device=dev)
    vs = vs.unflatten(-1, (-1, 16))[..., i ^ ((i >> 1) & 1)].transpose(-1, -2)
    v = _dequantize(vc.unflatten(-1, (16, -1)).contiguous(), vs.contiguous(), s["s_v"][None, :, None, None, None])
    k, v = k.flatten(2, 3), v.flatten(2, 3)                                                       # [n, kv, tokens, dim]
    start = s["q_start"].long()
    count = start[1:] - start[:-1]
    j = torch.arange(most, device=dev)
    row = (start[:-1, None] + j[None, :]).clamp(max=s["q"].shape[0] - 1)                          # [n, most]
    q = s["q"].float()[row].view(n, most, kv_heads, heads // kv_heads, dim).permute(0, 2, 1, 3, 4).flatten(2, 3)
    scores = (q @ k.transpose(-1, -2)) * s["scale"]
    pos = (s["seq_lens"].long()[:, None] - count[:, None] + j[None, :])[:, None, :, None]          # [n, 1, most, 1]
    at = torch.arange(k.shape[2], device=dev)[None, None, None, :]
    seen = (at <= pos) & (at > pos - s["window"] if s["window"] else at >= 0) & (at < s["seq_lens"].long()[:, None, None, None])
    seen = seen.repeat_interleave(heads // kv_heads, 2)
    scores = scores.masked_fill(~seen, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top.isinf(), torch.zeros_like(top), top))
    l = p.sum(-1, keepdim=True)
    out = torch.where(l > 0, (p @ v) / l, torch.zeros_like(l))
    lse = top + torch.log(l)
    out = out.unflatten(2, (most, -1)).permute(0, 2, 1, 3, 4).reshape(n * most, heads, dim)
    lse = lse.squeeze(-1).unflatten(2, (most, -1)).permute(0, 2, 1, 3).reshape(n * most, heads)
    t = torch.arange(s["q"].shape[0], device=dev)
    r = torch.searchsorted(start[1:].contiguous(), t, right=True)
    pick = r * most + t - start[r]
    return {"out": out[pick].to(torch.bfloat16), "lse": lse[pick]}


def _plain_matvec(s):
    n, k = s["q"].shape[0], s["x"].shape[1]
    w = _dequantize(s["q"], s["s"][_scale_places(n, k, s["q"].device)], 1.0)
    return {"y": ((s["x"].float() @ w.t()) * s["s2"][None, :]).to(s["y"].dtype)}


def run(state):
    s = state
    if not own:
        return {"slots": _plain_slots, "cache": _plain_cache, "attention": _plain_attention, "matvec": _plain_matvec}[s["op"]](s)
    import microscaled_precision_numerics_gb300 as mx
    if s["op"] == "slots":
        mx.mx_kv_slots(s["seq_lens"], s["new_lens"], s["page"], s["block_table"], s["free_pages"], s["free_count"], s["q_start"],
                       s["total_lens"], s["slots"], s["positions"], s["free_left"], s["unplaced"])
        return {name: s[name] for name in ("block_table", "q_start", "total_lens", "slots", "positions", "free_left", "unplaced")}
    if s["op"] == "cache":
        mx.mx_nvfp4_kv_append(s["k"], s["v"], s["slots"], s["s_k"], s["s_v"], s["cache"])
        mx.mx_nvfp4_kv_gather(s["cache"], s["slots"], s["s_k"], s["s_v"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if s["op"] == "attention":
        mx.mx_nvfp4_kv_attention(s["q"], s["q_start"], s["seq_lens"], s["block_table"], s["cache"], s["s_k"], s["s_v"], s["scale"],
                                 s["max_q"], s["out"], s["workspace"], lse=s["lse"], window=s["window"])
        return {"out": s["out"], "lse": s["lse"]}
    mx.mx_nvfp4_matvec(s["x"], s["q"], s["s"], s["s2"], mx.MX_SCOPE_ROW if s["case"]["per_row"] else mx.MX_SCOPE_TENSOR, s["y"])
    return {"y": s["y"]}


# --------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------------------------------------

def work(case):
    if case["op"] == "slots":
        total, new = _lengths(case)
        need = int((_ceil_div(total, case["page"]) - _ceil_div(total - new, case["page"])).sum())
        return {"bytes": 4 * (4 * len(new) + 1 + 2 * need + 2 * int(new.sum()) + 4), "flops": 0}
    if case["op"] == "cache":
        values = 2 * case["tokens"] * case["kv_heads"] * case["head_dim"]
        # each BF16 value is read, 9/16 byte is written, read again, and a BF16 value is written
        return {"bytes": values * (2 + 0.5625 + 0.5625 + 2) + 8 * case["tokens"], "flops": 4 * values}
    if case["op"] == "attention":
        total, new = _lengths(case)
        window = case["window"] or case["longest"]
        first = np.maximum(0, total - new + 1 - window)
        read = int(np.where(new > 0, total - first, 0).sum())
        pairs = sum(int(np.minimum(np.arange(t - m + 1, t + 1), window).sum()) for t, m in zip(total, new))
        rows = int(new.sum()) * case["heads"]
        return {"bytes": read * case["kv_heads"] * case["head_dim"] * 2 * 0.5625 + rows * (4 * case["head_dim"] + 4),
                "flops": 4 * pairs * case["heads"] * case["head_dim"]}
    m, n, k = case["tokens"], case["outputs"], case["inputs"]
    return {"bytes": n * k * 0.5625 + 2 * m * k + (4 if case["fp32_out"] else 2) * m * n + 4 * (n if case["per_row"] else 1),
            "flops": 2 * m * n * k}


# --------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------------------------

_E2M1 = np.array([(-1.0 if c & 8 else 1.0) * (0.5 * (c & 1) if not c & 6 else (1 + 0.5 * (c & 1)) * 2.0 ** (((c >> 1) & 3) - 1))
                  for c in range(16)])
_E4M3 = np.array([(-1.0 if c & 128 else 1.0) * (np.nan if c & 127 == 127 else (c & 7) * 2.0 ** -9 if not c & 120 else
                                                (1 + (c & 7) / 8) * 2.0 ** (((c >> 3) & 15) - 7)) for c in range(256)])


def _nearest_even(value, grid):
    """The non-negative grid points nearest to value (ties to the point of even index, beyond the last: the last)."""
    hi = np.clip(np.searchsorted(grid, value), 1, len(grid) - 1)
    lo = hi - 1
    below, above = value - grid[lo], grid[hi] - value
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return grid[np.where(up, hi, lo)]


def _fake_quantized(x, S):
    """x [..., heads, dim] in 64 bits as the values its codes and scales stand for."""
    b = x.reshape(*x.shape[:-1], -1, 16)
    S = S.reshape(1, -1, 1)
    bs = _nearest_even(np.abs(b).max(-1) / 6 / S, _E4M3[:127])
    step = np.where(bs * S > 0, bs * S, 1.0)[..., None]
    return (np.sign(b) * _nearest_even(np.abs(b) / step, _E2M1[:8]) * (bs * S)[..., None]).reshape(x.shape)


def exact(case, seed):
    if case["op"] == "slots":
        return None                                    # whole numbers
    s = prepare(case, seed)
    host = lambda t: t.cpu().numpy()                   # noqa: E731
    if case["op"] == "cache":
        return {"k": _fake_quantized(host(s["k"].double()), host(s["s_k"].double())),
                "v": _fake_quantized(host(s["v"].double()), host(s["s_v"].double()))}
    e2m1, e4m3 = torch.from_numpy(_E2M1).cuda(), torch.from_numpy(_E4M3).cuda()
    if case["op"] == "matvec":
        m, n, k = case["tokens"], case["outputs"], case["inputs"]
        x, y = s["x"].double(), torch.empty((m, n), dtype=torch.float64, device="cuda")
        tiles = s["s"].view(-1, _ceil_div(k // 16, 4), 32, 4, 4)      # [row bands, column tiles, row in 32, band of 32, column]
        for band in range(tiles.shape[0]):
            rows = min(128, n - 128 * band)
            bs = e4m3[tiles[band].permute(2, 1, 0, 3).reshape(128, -1)[:rows, :k // 16].long()]
            q = s["q"][128 * band:128 * band + rows].long()
            w = torch.stack([e2m1[q & 15], e2m1[q >> 4]], -1).view(rows, k // 16, 16) * bs[..., None]
            y[:, 128 * band:128 * band + rows] = x @ w.view(rows, k).t()
        return {"y": host(y * s["s2"].double()[None, :])}
    page, heads, kv, dim = case["page"], case["heads"], case["kv_heads"], case["head_dim"]
    out = torch.zeros((s["q"].shape[0], heads, dim), dtype=torch.float64, device="cuda")
    lse = torch.full((s["q"].shape[0], heads), -np.inf, dtype=torch.float64, device="cuda")
    start, total, table = host(s["q_start"]), host(s["seq_lens"]), host(s["block_table"])
    s_k, s_v = s["s_k"].double(), s["s_v"].double()
    order = torch.tensor([i ^ ((i >> 1) & 1) for i in range(16)], device="cuda")
    for r in range(len(total)):
        length, count = int(total[r]), int(start[r + 1] - start[r])
        if not length or not count:
            continue
        pages = torch.from_numpy(table[r, :_ceil_div(length, page)].astype(np.int64)).cuda()
        rec = s["cache"][pages].permute(1, 0, 2, 3).reshape(kv, -1, 18 * dim).long()

        def decoded(codes, scales, S):
            v = torch.stack([e2m1[codes & 15], e2m1[codes >> 4]], -1).view(kv, -1, 16, dim // 16, 16)
            return (v * e4m3[scales][..., None] * S[:, None, None, None, None]).reshape(kv, -1, dim)[:, :length]

        K = decoded(rec[..., :8 * dim].reshape(kv, -1, 16, dim // 2), rec[..., 8 * dim:9 * dim].reshape(kv, -1, 16, dim // 16), s_k)
        V = decoded(rec[..., 9 * dim:17 * dim].reshape(kv, -1, 16, dim // 2),
                    rec[..., 17 * dim:].reshape(kv, -1, dim // 16, 16)[..., order].transpose(-1, -2), s_v)
        for i in range(count):
            pos = length - count + i
            lo = max(0, pos - case["window"] + 1) if case["window"] else 0
            if pos < lo:
                continue
            q = s["q"][int(start[r]) + i].double().view(kv, heads // kv, dim)
            z = torch.einsum("hgd,htd->hgt", q, K[:, lo:pos + 1]) * s["scale"]
            lse[int(start[r]) + i] = torch.logsumexp(z, -1).reshape(heads)
            out[int(start[r]) + i] = torch.einsum("hgt,htd->hgd", torch.softmax(z, -1), V[:, lo:pos + 1]).reshape(heads, dim)
    return {"out": host(out), "lse": host(lse)}
