"""The forms that the operators between a layer's products take by their sizes: every kind of width of the norm from 512 rows on,
wide rows that FP32 does not hold, rows of logits that are not finite, long runs of the norm gradient's rings with what each turn
adds, and the sort on both sides of its switches.  Against the 64-bit forms of layer_ref.py and against the same rows in another
form."""
import numpy as np
import pytest
import torch

import layer_ref as ref
from test_gpu_layer import codes_of, host, mx, rand, run_norm, run_sort, same, some_ids, within, y_bound      # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def norm_into_marked(mx, x, w, eps, res):
    """(sum, y) of a call without codes, into buffers that held a mark."""
    y, s = torch.full_like(x, 77.0), None if res is None else torch.full_like(x, 77.0)
    mx.mx_rmsnorm_mxfp8(x, w, eps, residual=res, sum_out=s, y=y)
    return s, y


# 8, 16 and 24 columns beyond each multiple of 1024
RAGGED = [1024 * k + r for k in range(1, 16) for r in (8, 16, 24)]


@pytest.mark.parametrize("cols", RAGGED + [264, 520, 1016, 1000, 2040, 4096, 5120, 8184, 12288, 16376, 16384])
def test_norm_of_512_rows_and_more_at_every_kind_of_width(mx, cols):
    """The same rows in a call of 512 and in calls of fewer, which take another form, and some of them against 64 bits."""
    x, res = rand(101, 512, cols), rand(102, 512, cols, scale=3.0)
    w = rand(103, cols, scale=0.2).float() + 1.0
    for r in (None, res):
        s, y = norm_into_marked(mx, x, w, 1e-6, r)
        for part in (slice(0, 300), slice(300, 512)):
            s2, y2 = norm_into_marked(mx, x[part], w, 1e-6, None if r is None else r[part])
            assert torch.equal(y[part], y2) and (r is None or torch.equal(s[part], s2))
        some = slice(0, 512, 73)
        h, _, want = ref.norm(host(x[some]), host(w), 1e-6, None if r is None else host(r[some]))
        within(y[some], want, y_bound(want))
        assert r is None or np.array_equal(host(s[some]), h)


@pytest.mark.parametrize("rows,cols", [(513, 288), (600, 1032), (777, 2056), (512, 3080), (1003, 14336), (520, 15384), (2000, 1056), (801, 4096),
                                       (515, 992)])
@pytest.mark.parametrize("weight", [BF, F32])
@pytest.mark.parametrize("with_residual", [False, True])
def test_norm_of_many_rows(mx, rows, cols, weight, with_residual):
    x, res = rand(104, rows, cols), rand(105, rows, cols, scale=3.0) if with_residual else None
    w = (1.0 + 0.2 * torch.randn(cols, generator=torch.Generator().manual_seed(106))).to(weight).to(DEV)
    codes = cols % 32 == 0
    y = torch.full_like(x, 77.0)
    s, y, out = run_norm(mx, x, w, 1e-6, res, row=codes, sum_out=None if res is None else torch.full_like(x, 77.0), y=y)
    h, _, want = ref.norm(host(x), host(w), 1e-6, None if res is None else host(res))
    if res is not None:
        assert np.array_equal(host(s), h)
    within(y, want, y_bound(want))
    if codes:
        same(out, codes_of(mx, y, True, False))


@pytest.mark.parametrize("rows,cols,col", [(7, 4096, False), (7, 8192, False), (5, 16384, False), (700, 1056, False), (601, 2048, False),
                                           (520, 1032, False), (64, 1536, True), (32, 5120, True), (64, 8224, True), (32, 16384, True)])
def test_norm_of_wide_rows_beyond_the_range_of_squares(mx, rows, cols, col):
    """Ordinary rows, rows whose squares pass FP32's range on either side and rows that are not finite, in one call."""
    x, w = rand(107, rows, cols), rand(108, cols, scale=0.2).float() + 1.0
    x[1::7] *= 2.0 ** 70                                   # (exact: powers of two)
    x[2::7] *= 2.0 ** -80
    x[3::14, cols - 1], x[4::14, 3] = float("inf"), float("nan")
    fine = torch.ones(rows, dtype=torch.bool, device=DEV)
    fine[3::14] = fine[4::14] = False
    codes = cols % 32 == 0
    _, y, out = run_norm(mx, x, w, 0.0, row=codes, col=col)
    _, _, want = ref.norm(host(x[fine]), host(w), 0.0)
    within(y[fine], want, y_bound(want))
    assert torch.isnan(y[4::14]).all() and torch.isnan(y[3::14, -1]).all() and not y[3::14, :-1].any()
    if codes or col:
        same(out, codes_of(mx, y, codes, col))


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("experts,k", [(12, 3), (100, 8), (300, 5), (1024, 32)])
def test_route_gradient_of_rows_that_are_not_finite(mx, normalize, dtype, experts, k):
    """Such a row's softmax is NaN everywhere, and so is what it passes on: all of the row, or (over the chosen) the chosen ones."""
    inf, nan = float("inf"), float("nan")
    z = torch.randn((6, experts), generator=torch.Generator().manual_seed(120)).to(dtype).to(DEV)
    z[0, 7] = inf
    z[1, 2], z[1, 9] = nan, -inf
    z[2, 4], z[2, 5] = inf, nan
    z[3, 6], z[3, 7:] = inf, -inf                          # fewer than k may be left
    z[4, 3] = -inf                                         # an ordinary row
    z[5] = -inf
    ids = torch.empty((6, k), dtype=torch.int32, device=DEV)
    w, dw = torch.empty((6, k), device=DEV), torch.randn((6, k), generator=torch.Generator().manual_seed(121)).to(DEV)
    mx.mx_moe_route(z, ids, w, normalize=normalize)
    dz = torch.full_like(z, 99.0)
    mx.mx_moe_route_backward(z, ids, dw, dz, normalize=normalize)
    got, chosen = host(dz), np.zeros((6, experts), bool)
    for t in range(6):
        chosen[t, host(ids)[t][host(ids)[t] >= 0]] = True
    for t in range(4):
        if normalize:
            assert np.isnan(got[t, chosen[t]]).all() and not got[t, ~chosen[t]].any()
        else:
            assert np.isnan(got[t]).all()
    assert np.isfinite(got[4:]).all() and got[4, 3] == 0 and not got[5].any()


# Sizes of which every CTA of the gradient has at least three turns on 152 SMs: (rows, cols, most turns of a CTA's row or lane's).
# Rows that share a warp: 304 CTAs of 8 warps with 4, 2 or 1 rows each.  A CTA a row: up to four CTAs an SM.
LONG = [(30000, 64), (15001, 128), (7600, 256), (7501, 512), (7400, 1000), (2000, 1032), (1501, 2048), (1400, 4096), (1001, 5120), (960, 8192),
        (520, 8200), (500, 16384)]


def longest_chain(rows, cols):
    """Additions that one summand of dweight may pass: the turns of a lane or thread, then at most 2 in the butterfly, 8 warps or 2 CTAs,
    10 loads of the second kernel and 5 levels of its butterfly."""
    side = 4 if cols <= 64 else 2 if cols <= 128 else 1
    turns = -(-rows // (304 * 8 * side)) if cols <= 1024 else -(-rows // 152)        # (a CTA an SM at least, whatever the form)
    return turns + 25


@pytest.mark.parametrize("rows,cols", LONG)
def test_norm_gradient_over_many_turns(mx, rows, cols):
    """Ordinary rows and ones that FP32 does not hold side by side.  n has 24 roundings beside the sums'."""
    h, dy, dsum = rand(109, rows, cols), rand(110, rows, cols, scale=0.01), rand(111, rows, cols, scale=0.01)
    w = rand(112, cols, scale=0.2).float() + 1.0
    h[1::7] *= 2.0 ** 70                                   # (exact: powers of two)
    h[2::7] *= 2.0 ** -80
    dy[3::5] *= 2.0 ** -40
    dx, dw = torch.empty_like(h), torch.full((cols,), 9.0, device=DEV)
    ws = torch.full((mx.rmsnorm_workspace_bytes(rows, cols),), 255, dtype=U8, device=DEV)
    mx.mx_rmsnorm_backward(dy, h, w, 0.0, dx, dw, ws, dsum=dsum)
    want, wdw, bound, size = ref.norm_backward(host(dy), host(h), host(w), 0.0, host(dsum))
    within(dx, want, bound)
    within(dw, wdw, (longest_chain(rows, cols) + 24) * ref.EPS32 * size)


@pytest.mark.parametrize("rows,cols", LONG)
def test_norm_gradient_takes_every_row_into_dweight(mx, rows, cols):
    """dy is zero but in a few rows, so that a row left out shows whole."""
    h, w = rand(113, rows, cols), torch.ones(cols, dtype=BF, device=DEV)
    ws = torch.full((mx.rmsnorm_workspace_bytes(rows, cols),), 255, dtype=U8, device=DEV)
    n = host(h)
    n = n / np.sqrt((n * n).mean(-1, keepdims=True) + 1e-6)
    for picked in ([0], [rows - 1], [rows - 2, rows // 2, 1], list(range(5, rows, 101))):
        dy = torch.zeros_like(h)
        dy[picked] = rand(114, len(picked), cols)
        dx, dw = torch.empty_like(h), torch.full((cols,), 9.0, device=DEV)
        mx.mx_rmsnorm_backward(dy, h, w, 1e-6, dx, dw, ws)
        each = host(dy[picked]) * n[picked]
        within(dw, each.sum(0), (len(picked) + 24 + 25) * ref.EPS32 * np.abs(each).sum(0))


# choices on both sides of 16384, 32768, 65536 and 131072
@pytest.mark.parametrize("tokens,k,experts", [(2048, 8, 128), (2731, 6, 33), (4096, 8, 1000), (10923, 3, 128), (65537, 1, 7), (8193, 8, 60),
                                              (16384, 8, 1024), (12000, 9, 513), (43691, 3, 1024)])
@pytest.mark.parametrize("idle", [0.0, 0.3])
def test_sort_on_both_sides_of_its_switches(mx, tokens, k, experts, idle):
    ids = some_ids(115, tokens, k, experts, idle, distinct=False)
    got = run_sort(mx, ids, experts)
    for a, b, name in zip(got, ref.sort(host(ids), experts), ("group_offsets", "rows", "source")):
        assert np.array_equal(host(a), b), name
    a, b, _ = run_sort(mx, ids, experts, source=False)
    assert torch.equal(a, got[0]) and torch.equal(b, got[1])
