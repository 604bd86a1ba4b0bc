"""The operators between a layer's products at sizes whose offsets pass 31 bits, and the sort's form for many choices: the last
rows against the same rows on their own, orders against their definition on the device."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.fixture(scope="module")
def mx():
    import microscaled_precision_numerics_gb300 as m
    m.lib()
    return m


def test_norm_and_gradient_past_31_bits(mx):
    rows, cols, tail = 140000, 16384, 32                   # 2.3e9 elements
    x = torch.randn((rows, cols), device=DEV, dtype=BF)
    res = x.roll(1, 1)
    w = torch.randn(cols, device=DEV)
    out = mx.alloc_mxfp8(rows, cols, DEV)
    y = torch.empty_like(x)
    mx.mx_rmsnorm_mxfp8(x, w, 1e-6, residual=res, sum_out=res, y=y, **out)
    few = {k: v for k, v in mx.alloc_mxfp8(tail, cols, DEV).items()}
    s, y2 = torch.empty((tail, cols), device=DEV, dtype=BF), torch.empty((tail, cols), device=DEV, dtype=BF)
    at = slice(rows - tail, rows)
    mx.mx_rmsnorm_mxfp8(x[at], w, 1e-6, residual=x[at].roll(1, 1), sum_out=s, y=y2, **few)
    assert torch.equal(res[at], s) and torch.equal(y[at], y2)
    assert torch.equal(out["q_row"][at], few["q_row"]) and torch.equal(out["q_col"][:, at], few["q_col"])
    del out, few
    dx, dx2, dw = torch.empty_like(x), torch.empty((tail, cols), device=DEV, dtype=BF), torch.empty(cols, device=DEV)
    ws = torch.empty(mx.rmsnorm_workspace_bytes(rows, cols), dtype=U8, device=DEV)
    mx.mx_rmsnorm_backward(y, res, w, 1e-6, dx, dw, ws, dsum=x)
    mx.mx_rmsnorm_backward(y[at], res[at], w, 1e-6, dx2, torch.empty_like(dw), ws, dsum=x[at])
    assert torch.equal(dx[at], dx2)
    # a column's sum over 140000 rows against one in FP64 of the rows' FP32 products (n within 24 roundings of FP32)
    c = slice(5, cols, 4099)
    r = torch.cat([part.double().square().mean(-1) for part in res.split(2000)]).add(1e-6).rsqrt()
    want = (y[:, c].double() * res[:, c].double() * r[:, None]).sum(0)
    size = (y[:, c].double() * res[:, c].double() * r[:, None]).abs().sum(0)
    assert ((dw[c].double() - want).abs() <= (rows / 152 + 300) * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("experts", [5, 128, 1024])
def test_sort_of_many_choices(mx, experts):
    """Twenty million choices: every one has its row, rows are in the order of experts, choices of one expert in theirs."""
    tokens, k = 2500001, 8
    n = tokens * k
    ids = torch.randint(-1, experts, (tokens, k), dtype=I32, device=DEV)
    offsets, rows, source = (torch.empty(experts + 1, dtype=torch.int64, device=DEV), torch.empty_like(ids),
                             torch.empty(n, dtype=I32, device=DEV))
    ws = torch.empty(mx.moe_sort_workspace_bytes(n, experts), dtype=U8, device=DEV)
    mx.mx_moe_sort(ids, offsets, rows, source, ws)
    flat, used = ids.view(-1), int(offsets[-1])
    counts = torch.bincount(flat[flat >= 0].long(), minlength=experts)
    assert torch.equal(offsets[1:], counts.cumsum(0)) and int(offsets[0]) == 0
    assert (source[used:] == -1).all() and (rows.view(-1)[flat < 0] == -1).all()
    src = source[:used].long()
    key = flat[src].long() * n + src
    assert (key[1:] > key[:-1]).all()
    assert torch.equal(rows.view(-1)[src], torch.arange(used, dtype=I32, device=DEV))


def test_dispatch_and_combine_past_31_bits(mx):
    tokens, k, experts, hidden = 131072, 4, 64, 4608       # 2.4e9 elements of the experts' rows
    n = tokens * k
    ids = torch.randint(0, experts, (tokens, k), dtype=I32, device=DEV)
    offsets, rows, source = (torch.empty(experts + 1, dtype=torch.int64, device=DEV), torch.empty_like(ids),
                             torch.empty(n, dtype=I32, device=DEV))
    mx.mx_moe_sort(ids, offsets, rows, source, torch.empty(mx.moe_sort_workspace_bytes(n, experts), dtype=U8, device=DEV))
    x = torch.randn((tokens, hidden), device=DEV, dtype=BF)
    z = torch.empty((n, hidden), device=DEV, dtype=BF)
    mx.mx_moe_dispatch(x, rows, z)
    pick = torch.cat([torch.arange(64, device=DEV), torch.randint(0, n, (4000,), device=DEV), torch.arange(n - 64, n, device=DEV)])
    assert torch.equal(z[pick], x[source[pick].long() // k])
    a = mx.alloc_mxfp8(tokens, hidden, DEV, colwise=False)
    mx.mx_quantize_mxfp8(x, **a)
    q, s = torch.empty((n, hidden), dtype=U8, device=DEV), torch.empty(mx.grouped_scale_bytes(n, experts, hidden, 32), dtype=U8, device=DEV)
    mx.mx_moe_dispatch_quantized(mx.MX_FMT_MXFP8, a["q_row"], a["s_row"], rows, offsets, q, s)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    mx.mx_quantize_mxfp8_grouped(z, offsets, q2, s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    y = torch.empty_like(x)
    quarter = torch.full((tokens, k), 0.25, device=DEV)
    mx.mx_moe_combine(z, rows, y, weights=quarter)         # four times a quarter, exactly
    assert torch.equal(y, x)
    dz, dw = torch.empty_like(z), torch.empty_like(quarter)
    mx.mx_moe_combine_backward(x, z, rows, quarter, dz, dw)
    assert torch.equal(dz[pick], (x[source[pick].long() // k].float() * 0.25).to(BF))
    want = x.double().square().sum(-1, keepdim=True).expand(tokens, k)
    assert ((dw.double() - want).abs() <= (hidden / 256 + 40) * 2.0 ** -24 * want).all()


def test_choice_of_many_tokens(mx):
    z = torch.randn((1 << 20, 2048 // 16), device=DEV, dtype=BF)
    ids, w = torch.empty((1 << 20, 8), dtype=I32, device=DEV), torch.empty((1 << 20, 8), device=DEV)
    mx.mx_moe_route(z, ids, w)
    order = torch.sort(z.float(), dim=-1, descending=True, stable=True)
    assert torch.equal(ids, order.indices[:, :8].int())
    want = torch.softmax(order.values[:, :8].double(), -1)
    assert ((w.double() - want).abs() <= want * 2.0 ** -24 * 80).all()


def test_norm_of_more_threads_than_32_bits(mx):
    """2^27 - 1 narrow rows, 32 threads each: the last rows, and the scale row that fills up the last tile, which is cleared."""
    rows, cols, tail = (1 << 27) - 1, 32, 127
    x = torch.randn((1 << 20, cols), device=DEV, dtype=BF).repeat(128, 1)[:rows]
    w = torch.randn(cols, device=DEV, dtype=BF)
    out, few = mx.alloc_mxfp8(rows, cols, DEV, colwise=False), mx.alloc_mxfp8(tail, cols, DEV, colwise=False)
    for o in (out, few):
        o["s_row"].fill_(255)
    mx.mx_rmsnorm_mxfp8(x, w, 1e-6, **out)
    mx.mx_rmsnorm_mxfp8(x[rows - tail:], w, 1e-6, **few)
    assert torch.equal(out["q_row"][rows - tail:], few["q_row"])
    assert torch.equal(out["s_row"].view(-1)[-512:], few["s_row"].view(-1))
    scales = few["s_row"].view(32, 4, 4)                   # row 32 q + r of the tile at [r, q], its columns 1 to 3 padding
    assert scales[31, 3].eq(0).all() and scales[:, :, 0].eq(0).sum() == 1 and scales[:, :, 1:].eq(0).all()
