"""The operators between the products of a layer with routed experts: what is measured, their plain forms and
their definitions in 64 bits.

A layer of this kind calls, in this order, the root-mean-square norm with the residual's addition, whose output comes in
MXFP8 for the product that reads it (`norm`), the router's choice of experts for each token (`route`), the tokens sorted by
expert (`dispatch`) for the grouped products, and the experts' rows brought back to their tokens with the router's
weights (`combine`).  `norm_backward` and `combine_backward` are their gradients, a `route` with a step has its own too; the
gradient of `dispatch` is a `combine` without weights.

MXFP8: blocks of 32 E4M3 codes under one E8M0 byte, 2^(byte - 127), byte = max(exponent field of the block's largest magnitude
- 8, 0).  The scale bytes lie in the GEMM's layout: 512-byte tiles of 128 rows x 4 scale columns, in row-major tile order,
with (r, c) at (r % 32) * 16 + (r / 32 % 4) * 4 + c % 4 of its tile; padding is zero.  In the grouped layout every expert's rows
start on a tile.
"""
import numpy as np
import torch

own = False

_EPS = 1e-6


# --------------------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one token of a generating request, into the attention's or the experts' first product: latency counts
        {"name": "norm_token_1x2048", "op": "norm", "rows": 1, "cols": 2048, "residual": True, "y": True, "row": True,
         "col": False, "weight_fp32": False},
        # a prompt of odd length at the feed-forward width
        {"name": "norm_prompt_1003x14336", "op": "norm", "rows": 1003, "cols": 14336, "residual": False, "y": False, "row": True,
         "col": False, "weight_fp32": True},
        # a training step's tokens: both orientations, for the product and for its weight gradient
        {"name": "norm_train_8192x4096", "op": "norm", "rows": 8192, "cols": 4096, "residual": True, "y": False, "row": True,
         "col": True, "weight_fp32": False},
        # gradient of the norm for a short packed sequence of odd length
        {"name": "norm_backward_777x2048", "op": "norm_backward", "rows": 777, "cols": 2048, "dsum": True, "weight_fp32": True},
        # the same for a training step
        {"name": "norm_backward_8192x4096", "op": "norm_backward", "rows": 8192, "cols": 4096, "dsum": True,
         "weight_fp32": False},
        # experts of a decoding batch's tokens
        {"name": "route_decode_64", "op": "route", "tokens": 64, "experts": 128, "top_k": 8, "normalize": True, "fp32": True,
         "masked": 0, "step": False},
        # experts of a training step's tokens with the gradient of the logits, one expert out of service
        {"name": "route_step_8192", "op": "route", "tokens": 8192, "experts": 128, "top_k": 8, "normalize": True, "fp32": False,
         "masked": 1, "step": True},
        # a decoding batch sorted by expert, a few of its tokens idle: latency counts
        {"name": "dispatch_decode_61", "op": "dispatch", "tokens": 61, "experts": 128, "top_k": 8, "hidden": 2048, "idle": 3,
         "codes": True},
        # a training step's tokens sorted by expert, as MXFP8
        {"name": "dispatch_step_8192", "op": "dispatch", "tokens": 8192, "experts": 128, "top_k": 8, "hidden": 2048, "idle": 0,
         "codes": True},
        # the experts' rows of a decoding batch back to its tokens
        {"name": "combine_decode_61", "op": "combine", "tokens": 61, "experts": 128, "top_k": 8, "hidden": 2048, "idle": 3,
         "weights": True, "residual": True},
        # a training step's rows back to its tokens
        {"name": "combine_step_8192", "op": "combine", "tokens": 8192, "experts": 128, "top_k": 8, "hidden": 2048, "idle": 0,
         "weights": True, "residual": False},
        # and the gradients of the rows and of the weights
        {"name": "combine_backward_8192", "op": "combine_backward", "tokens": 8192, "experts": 128, "top_k": 8, "hidden": 2048,
         "idle": 0},
    ]


def _log_between(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "route", "dispatch", "combine", "combine_backward"])
    if op in ("norm", "norm_backward"):
        cols = 32 * _log_between(rng, 4, 512)
        rows = _log_between(rng, 1, min(8192, 8192 * 4096 // cols))
        weight_fp32 = rng.random() < 0.5
        if op == "norm_backward":
            return {"op": op, "rows": rows, "cols": cols, "dsum": rng.random() < 0.7, "weight_fp32": weight_fp32}
        col = rng.random() < 0.4
        return {"op": op, "rows": max(32, rows // 32 * 32) if col else rows, "cols": cols, "residual": rng.random() < 0.7,
                "y": rng.random() < 0.5, "row": not col or rng.random() < 0.8, "col": col, "weight_fp32": weight_fp32}
    experts = rng.choice([8, 16, 32, 60, 64, 128, 160, 256, 512])
    top_k = rng.randint(1, 8)
    tokens = _log_between(rng, 1, 8192)
    if op == "route":
        return {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "normalize": rng.random() < 0.6,
                "fp32": rng.random() < 0.5, "masked": rng.choice([0, 0, rng.randint(1, experts - top_k) if experts > top_k else 0]),
                "step": rng.random() < 0.5}
    hidden = 32 * _log_between(rng, 4, max(4, min(256, 8192 * 8 * 2048 // (tokens * top_k) // 32)))
    case = {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "hidden": hidden,
            "idle": rng.choice([0, 0, rng.randint(0, tokens - 1)])}
    if op == "dispatch":
        case["codes"] = rng.random() < 0.6
    if op == "combine":
        case |= {"weights": rng.random() < 0.7, "residual": rng.random() < 0.5}
    return case


# --------------------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------------------

def _ceil_div(a, b):
    return (a + b - 1) // b


def _scale_bytes(rows, cols):
    return _ceil_div(rows, 128) * _ceil_div(cols // 32, 4) * 512


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    def empty(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device=dev)

    s = {"case": case, "op": case["op"]}
    if case["op"] in ("norm", "norm_backward"):
        rows, cols = case["rows"], case["cols"]
        x = normal(rows, cols)
        x[:, torch.randint(cols, (max(1, cols // 200),), generator=g, device=dev)] *= 20.0   # outlier channels
        s["x"] = x.to(torch.bfloat16)
        s["weight"] = (1.0 + 0.1 * normal(cols)).to(torch.float32 if case["weight_fp32"] else torch.bfloat16)
        if case["op"] == "norm_backward":
            s["dy"] = (0.01 * normal(rows, cols)).to(torch.bfloat16)
            s["dsum"] = (0.01 * normal(rows, cols)).to(torch.bfloat16) if case["dsum"] else None
            s["dx"], s["dweight"] = empty(rows, cols), empty(cols, dtype=torch.float32)
            s["workspace"] = empty(64 << 20, dtype=torch.uint8)      # one for all such calls of a program
            return s
        s["residual"] = (3.0 * normal(rows, cols)).to(torch.bfloat16) if case["residual"] else None
        s["out"] = {"sum_out": empty(rows, cols) if case["residual"] else None, "y": empty(rows, cols) if case["y"] else None}
        for name, a, b in (("row", rows, cols), ("col", cols, rows)):
            s["out"]["q_" + name] = empty(a, b, dtype=torch.uint8) if case[name] else None
            s["out"]["s_" + name] = empty(_scale_bytes(a, b), dtype=torch.uint8) if case[name] else None
        return s
    t, experts, k = case["tokens"], case["experts"], case["top_k"]
    popular = normal(experts)                                         # some experts are asked for more than others
    logits = normal(t, experts) * 1.5 + 0.7 * popular
    if case["op"] == "route":
        logits[:, torch.randperm(experts, generator=g, device=dev)[:case["masked"]]] = float("-inf")
        s["logits"] = logits.to(torch.float32 if case["fp32"] else torch.bfloat16)
        s["ids"], s["weights"] = empty(t, k, dtype=torch.int32), empty(t, k, dtype=torch.float32)
        if case["step"]:
            s["dweights"], s["dlogits"] = 0.01 * normal(t, k), torch.zeros_like(s["logits"])
        return s
    value, ids = logits.topk(min(k, experts), -1)
    s["ids"] = ids.to(torch.int32)
    s["weights"] = torch.softmax(value, -1)
    s["ids"][torch.randperm(t, generator=g, device=dev)[:case["idle"]]] = -1
    s["ids"] = s["ids"].contiguous()
    n, hidden = t * k, case["hidden"]
    if case["op"] == "dispatch":
        s["group_offsets"] = empty(experts + 1, dtype=torch.int64)
        s["rows"], s["source"] = empty(t, k, dtype=torch.int32), empty(n, dtype=torch.int32)
        s["workspace"] = empty(16 << 20, dtype=torch.uint8)
        x = normal(t, hidden).to(torch.bfloat16)
        if case["codes"]:
            s["q"], s["s"] = _quantize_rows(x.float())
            s["q_out"] = empty(n, hidden, dtype=torch.uint8)
            s["s_out"] = empty(_scale_bytes(n + 127 * experts, hidden), dtype=torch.uint8)
        else:
            s["x"], s["y"] = x, empty(n, hidden)
        return s
    _, s["rows"], _ = _sorted_by_expert(s["ids"], experts)
    s["z"] = normal(n, hidden).to(torch.bfloat16)
    if case["op"] == "combine":
        s["weights"] = s["weights"] if case["weights"] else None
        s["residual"] = (3.0 * normal(t, hidden)).to(torch.bfloat16) if case["residual"] else None
        s["y"] = empty(t, hidden)
        return s
    s["dy"] = (0.01 * normal(t, hidden)).to(torch.bfloat16)
    s["dz"], s["dweights"] = empty(n, hidden), empty(t, k, dtype=torch.float32)
    return s


# --------------------------------------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------------------------------------

def _scale_places(rows, columns, device):
    """Byte offsets [rows, columns] of the scales in the GEMM layout; `rows` a count or the row numbers themselves."""
    r = rows.long()[:, None] if torch.is_tensor(rows) else torch.arange(rows, device=device)[:, None]
    c = torch.arange(columns, device=device)[None, :]
    return (r // 128 * _ceil_div(columns, 4) + c // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + c % 4


def _quantize_rows(x):
    """E4M3 codes [rows, cols] and E8M0 scales in the GEMM layout of x [rows, cols] (FP32 that holds BF16 values), as bytes."""
    rows, cols = x.shape
    blocks = x.unflatten(-1, (-1, 32))
    field = (blocks.abs().amax(-1).view(torch.int32) >> 23) & 255
    byte = (field - 8).clamp(min=0)
    inverse = ((254 - byte) << 23).view(torch.float32)
    codes = (blocks * inverse[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).flatten(-2)
    scales = torch.zeros(_scale_bytes(rows, cols), dtype=torch.uint8, device=x.device)
    scales[_scale_places(rows, cols // 32, x.device)] = byte.to(torch.uint8)
    return codes.view(torch.uint8), scales


def _as_values(out):
    """Codes and scale bytes as the numbers that they stand for."""
    kind = {"q": torch.float8_e4m3fn, "s": torch.float8_e8m0fnu}
    return {name: v.view(kind[name[0]]) if v.dtype == torch.uint8 else v for name, v in out.items() if v is not None}


def _plain_norm(s):
    case = s["case"]
    h = s["x"]
    out = {}
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(torch.bfloat16)
        out["sum_out"] = h
    f = h.float()
    y = (f * (1.0 / torch.sqrt(f.square().mean(-1, keepdim=True) + _EPS)) * s["weight"].float()).to(torch.bfloat16)
    if case["y"]:
        out["y"] = y
    if case["row"]:                                    # the codes are those of the BF16 output, as the products' other operands'
        out["q_row"], out["s_row"] = _quantize_rows(y.float())
    if case["col"]:
        out["q_col"], out["s_col"] = _quantize_rows(y.float().t().contiguous())
    return _as_values(out)


def _plain_norm_backward(s):
    h, dy, w = s["x"].float(), s["dy"].float(), s["weight"].float()
    r = 1.0 / torch.sqrt(h.square().mean(-1, keepdim=True) + _EPS)
    n = h * r
    dn = dy * w
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(torch.bfloat16), "dweight": (dy * n).sum(0)}


def _plain_route(s):
    case, z = s["case"], s["logits"].float()
    k = case["top_k"]
    order = torch.sort(z, dim=-1, descending=True, stable=True)       # of equal ones the lowest index first
    ids, chosen = order.indices[:, :k], order.values[:, :k]
    top = chosen[:, :1]
    e = torch.exp(chosen - top)
    every = torch.exp(z - top)
    total = (e if case["normalize"] else every).sum(-1, keepdim=True)
    w = e / total
    out = {"ids": ids.int(), "weights": w}
    if case["step"]:
        d = w * (s["dweights"] - (w * s["dweights"]).sum(-1, keepdim=True))
        if case["normalize"]:
            dz = torch.zeros_like(z).scatter(1, ids, d)
        else:
            g = torch.zeros_like(z).scatter(1, ids, s["dweights"])
            dz = every / total * (g - (w * s["dweights"]).sum(-1, keepdim=True))
        out["dlogits"] = dz.to(s["logits"].dtype)
    return out


def _sorted_by_expert(ids, experts):
    """First row of each expert [experts + 1], the row of each choice (-1: an idle one's), and each row's choice (-1 from the last on)."""
    flat = ids.reshape(-1).long()
    n, dev = flat.numel(), ids.device
    key = torch.where(flat < 0, torch.full_like(flat, experts), flat)
    order = torch.sort(key, stable=True).indices
    offsets = torch.searchsorted(key[order], torch.arange(experts + 1, device=dev))
    at = torch.arange(n, device=dev)
    rows = torch.empty_like(flat)
    rows[order] = torch.where(at < offsets[-1], at, torch.full_like(at, -1))
    source = torch.where(at < offsets[-1], order, torch.full_like(order, -1))
    return offsets, rows.view(ids.shape).int(), source.int()


def _plain_dispatch(s):
    case = s["case"]
    experts, hidden, k = case["experts"], case["hidden"], case["top_k"]
    offsets, rows, source = _sorted_by_expert(s["ids"], experts)
    out = {"group_offsets": offsets, "rows": rows, "source": source}
    have = (source >= 0)[:, None]
    token = source.long().clamp(min=0) // k
    if not case["codes"]:
        out["y"] = torch.where(have, s["x"][token], torch.zeros_like(s["x"][:1]))
        return out
    out["q_out"] = torch.where(have, s["q"][token], torch.zeros_like(s["q"][:1]))
    size = offsets[1:] - offsets[:-1]
    tiles = (size + 127) // 128
    start = (tiles.cumsum(0) - tiles) * 128                           # first padded row of each expert
    at = torch.arange(source.numel(), device=source.device)
    e = torch.searchsorted(offsets, at, right=True).clamp(max=experts) - 1
    padded = start[e] + at - offsets[e]
    mine = s["s"][_scale_places(token, hidden // 32, source.device)]
    place = _scale_places(padded, hidden // 32, source.device)
    last = _scale_bytes(source.numel() + 127 * experts, hidden)
    scales = torch.zeros(last + 1, dtype=torch.uint8, device=source.device)
    scales[torch.where(have, place, torch.full_like(place, last))] = mine
    out["s_out"] = scales[:last]
    return _as_values(out)


def _plain_combine(s):
    rows = s["rows"].long()
    z = s["z"].float()[rows.clamp(min=0)]                             # [tokens, top_k, hidden]
    w = s["weights"] if s["weights"] is not None else torch.ones_like(rows, dtype=torch.float32)
    y = torch.where(rows[..., None] >= 0, w[..., None] * z, torch.zeros_like(z)).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(torch.bfloat16)}


def _plain_combine_backward(s):
    rows, dy = s["rows"].long(), s["dy"].float()
    have = rows >= 0
    dw = torch.where(have, (s["z"].float()[rows.clamp(min=0)] * dy[:, None, :]).sum(-1), torch.zeros_like(s["weights"]))
    n = s["z"].shape[0]
    dz = torch.zeros((n + 1, dy.shape[1]), dtype=torch.bfloat16, device=dy.device)
    dz[torch.where(have, rows, torch.full_like(rows, n))] = (s["weights"][..., None] * dy[:, None, :]).to(torch.bfloat16)
    return {"dz": dz[:n], "dweights": dw}


def run(state):
    s = state
    if not own:
        return {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "route": _plain_route, "dispatch": _plain_dispatch,
                "combine": _plain_combine, "combine_backward": _plain_combine_backward}[s["op"]](s)
    import microscaled_precision_numerics_gb300 as mx
    case = s["case"]
    if s["op"] == "norm":
        mx.mx_rmsnorm_mxfp8(s["x"], s["weight"], _EPS, residual=s["residual"], **s["out"])
        return _as_values(s["out"])
    if s["op"] == "norm_backward":
        mx.mx_rmsnorm_backward(s["dy"], s["x"], s["weight"], _EPS, s["dx"], s["dweight"], s["workspace"], dsum=s["dsum"])
        return {"dx": s["dx"], "dweight": s["dweight"]}
    if s["op"] == "route":
        mx.mx_moe_route(s["logits"], s["ids"], s["weights"], normalize=case["normalize"])
        out = {"ids": s["ids"], "weights": s["weights"]}
        if case["step"]:
            mx.mx_moe_route_backward(s["logits"], s["ids"], s["dweights"], s["dlogits"], normalize=case["normalize"])
            out["dlogits"] = s["dlogits"]
        return out
    if s["op"] == "dispatch":
        mx.mx_moe_sort(s["ids"], s["group_offsets"], s["rows"], s["source"], s["workspace"])
        out = {name: s[name] for name in ("group_offsets", "rows", "source")}
        if not case["codes"]:
            mx.mx_moe_dispatch(s["x"], s["rows"], s["y"])
            return out | {"y": s["y"]}
        mx.mx_moe_dispatch_quantized(mx.MX_FMT_MXFP8, s["q"], s["s"], s["rows"], s["group_offsets"], s["q_out"], s["s_out"])
        return out | _as_values({"q_out": s["q_out"], "s_out": s["s_out"]})
    if s["op"] == "combine":
        mx.mx_moe_combine(s["z"], s["rows"], s["y"], weights=s["weights"], residual=s["residual"])
        return {"y": s["y"]}
    mx.mx_moe_combine_backward(s["dy"], s["z"], s["rows"], s["weights"], s["dz"], s["dweights"])
    return {"dz": s["dz"], "dweights": s["dweights"]}


# --------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------------------------------------

def work(case):
    if case["op"] in ("norm", "norm_backward"):
        values, weight = case["rows"] * case["cols"], case["cols"] * (4 if case["weight_fp32"] else 2)
        if case["op"] == "norm_backward":
            return {"bytes": values * (6 + 2 * case["dsum"]) + weight + 4 * case["cols"], "flops": 12 * values}
        per = 2 + 4 * case["residual"] + 2 * case["y"] + 1.03125 * (case["row"] + case["col"])
        return {"bytes": values * per + weight, "flops": 6 * values}
    t, n = case["tokens"], case["tokens"] * case["top_k"]
    if case["op"] == "route":
        logits = t * case["experts"] * (4 if case["fp32"] else 2)
        return {"bytes": logits * (2 if case["step"] else 1) + n * (12 if case["step"] else 8), "flops": 4 * t * case["experts"]}
    hidden, used = case["hidden"], (t - case["idle"]) * case["top_k"]
    if case["op"] == "dispatch":
        per = 1.03125 if case["codes"] else 2
        return {"bytes": 12 * n + 8 * (case["experts"] + 1) + (t - case["idle"] + used) * hidden * per, "flops": 0}
    if case["op"] == "combine":
        return {"bytes": n * (4 + 4 * case["weights"]) + 2 * hidden * (used + t * (1 + case["residual"])), "flops": 2 * used * hidden}
    return {"bytes": 12 * n + 2 * hidden * (t + 2 * used), "flops": 3 * used * hidden}


# --------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------------------------

def _e4m3(v):
    """The E4M3 value nearest to v (ties to the even mantissa), saturating, in 64 bits."""
    a = np.abs(v)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(a, 1e-300))), -6) - 3)
    return np.sign(v) * np.minimum(np.round(a / step) * step, 448.0)


def _mxfp8_values(x, band=1024):
    """(codes, scales in the GEMM layout) of x [rows, cols], 64 bits, as values."""
    rows, cols = x.shape
    columns = cols // 32
    scale = np.zeros((_ceil_div(rows, 128) * 128, _ceil_div(columns, 4) * 4))
    scale[:] = 2.0 ** -127                                            # what the padding's zero byte stands for
    codes = np.empty_like(x)
    for at in range(0, rows, band):
        b = x[at:at + band].reshape(-1, columns, 32)
        amax = np.abs(b).max(-1)
        two = np.exp2(np.maximum(np.where(amax > 0, np.floor(np.log2(np.where(amax > 0, amax, 1.0))), -127) - 8, -127))
        scale[at:at + band, :columns][:len(two)] = two
        codes[at:at + band] = _e4m3(b / two[..., None]).reshape(-1, cols)
    tiles = scale.reshape(-1, 4, 32, scale.shape[1] // 4, 4)          # [row tile, row / 32, row % 32, column tile, column % 4]
    return codes, np.ascontiguousarray(tiles.transpose(0, 3, 2, 1, 4)).reshape(-1)


def exact(case, seed):
    s = prepare(case, seed)
    host = lambda t: t.cpu().numpy()                                  # noqa: E731
    bf16 = lambda t: t.to(torch.bfloat16).double()                    # noqa: E731
    if case["op"] in ("norm", "norm_backward"):
        h, w = s["x"].double(), s["weight"].double()
        if case["op"] == "norm":
            out = {}
            if case["residual"]:
                h = bf16(h + s["residual"].double())
                out["sum_out"] = host(h)
            y = h / (h.pow(2).sum(-1, keepdim=True) / case["cols"] + _EPS).sqrt() * w
            if case["y"]:
                out["y"] = host(y)
            if case["row"]:
                out["q_row"], out["s_row"] = _mxfp8_values(host(bf16(y)))
            if case["col"]:
                out["q_col"], out["s_col"] = _mxfp8_values(host(bf16(y).t().contiguous()))
            return out
        dy = s["dy"].double()
        root = (h.pow(2).sum(-1, keepdim=True) / case["cols"] + _EPS).sqrt()
        inner = (dy * w * h).sum(-1, keepdim=True)
        dx = dy * w / root - h * inner / (case["cols"] * root.pow(3))
        if case["dsum"]:
            dx = dx + s["dsum"].double()
        return {"dx": host(dx), "dweight": host((dy * h / root).sum(0))}
    if case["op"] == "route":
        z = host(s["logits"].double())
        t, k = case["tokens"], case["top_k"]
        ids = np.argsort(-z, axis=-1, kind="stable")[:, :k]
        e = np.exp(z - z.max(-1, keepdims=True))
        picked = np.take_along_axis(e, ids, 1)
        total = picked.sum(-1, keepdims=True) if case["normalize"] else e.sum(-1, keepdims=True)
        out = {"ids": None, "weights": picked / total}
        if case["step"]:
            dw = host(s["dweights"].double())
            dz = np.zeros_like(z)
            inner = (dw * out["weights"]).sum(-1, keepdims=True)
            if not case["normalize"]:
                dz = -e / total * inner
            for j in range(k):
                part = out["weights"][:, j:j + 1] * (dw[:, j:j + 1] - (inner if case["normalize"] else 0.0))
                np.put_along_axis(dz, ids[:, j:j + 1], np.take_along_axis(dz, ids[:, j:j + 1], 1) + part, 1)
            out["dlogits"] = dz
        return out
    if case["op"] == "dispatch":
        return None                                                   # whole numbers, and values that are moved
    rows, z = s["rows"].long(), s["z"].double()
    have = rows >= 0
    if case["op"] == "combine":
        y = s["residual"].double() if case["residual"] else torch.zeros((rows.shape[0], z.shape[1]), dtype=torch.float64, device=z.device)
        for j in range(case["top_k"]):
            on = have[:, j]
            w = s["weights"][on, j, None].double() if case["weights"] else 1.0
            y[on] = y[on] + w * z[rows[on, j]]
        return {"y": host(y)}
    dy, dz, dw = s["dy"].double(), torch.zeros_like(z), torch.zeros_like(s["weights"], dtype=torch.float64)
    for j in range(case["top_k"]):
        on = have[:, j]
        dz[rows[on, j]] = s["weights"][on, j, None].double() * dy[on]
        dw[on, j] = (z[rows[on, j]] * dy[on]).sum(-1)
    return {"dz": host(dz), "dweights": host(dw)}
