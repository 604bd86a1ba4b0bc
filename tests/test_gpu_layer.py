"""The operators between a layer's products on the device against the 64-bit forms of layer_ref.py: the norm with residual and
MXFP8 output, the router's choice, the rows by expert and back, and the gradients.  Codes and scales are compared byte for byte
with the framework's quantizers."""
import numpy as np
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.fixture(scope="module")
def mx():
    import microscaled_precision_numerics_gb300 as m
    m.lib()
    return m


def host(t):
    return t.detach().double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def rand(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(BF).to(DEV)


def strided(t, extra=24, fill=7.0):
    """A copy of a 2-D tensor inside a wider one, so that its rows are not back to back."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=t.dtype, device=t.device)
    wide[:, 8:8 + t.shape[1]] = t
    return wide[:, 8:8 + t.shape[1]]


def within(got, want, bound):
    got, want, bound = host(got), np.asarray(want), np.broadcast_to(bound, np.shape(want))
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size} beyond the bound, first at {np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]} +- {bound[bad][0]}"


def y_bound(y):
    # sums: a chain of 8 and at most 12 levels; mean, eps, root, quotient and two products add 6, and r takes half of the sum's
    return np.abs(y) * (ref.HALF16 + 24 * ref.EPS32) + ref.TINY16


def run_norm(mx, x, w, eps, residual=None, row=True, col=False, sum_out=None, y=None):
    rows, cols = x.shape
    out = mx.alloc_mxfp8(rows, cols, DEV, rowwise=row, colwise=col)
    for t in out.values():
        t.fill_(0xA5)
    s = (sum_out if sum_out is not None else torch.empty_like(residual)) if residual is not None else None
    y = torch.empty((rows, cols), dtype=BF, device=DEV) if y is None else y
    mx.mx_rmsnorm_mxfp8(x, w, eps, residual=residual, sum_out=s, y=y, **out)
    return s, y, out


def codes_of(mx, y, row, col):
    out = mx.alloc_mxfp8(y.shape[0], y.shape[1], DEV, rowwise=row, colwise=col)
    for t in out.values():
        t.fill_(0x5A)
    mx.mx_quantize_mxfp8(y, **out)
    return out


def same(a, b):
    for name in a:
        assert torch.equal(a[name], b[name]), name


NORM_SIZES = [(1, 32), (1, 2048), (3, 96), (33, 160), (130, 256), (5, 288), (7, 1056), (2, 8192), (3, 8224), (2, 16384), (257, 992)]


@pytest.mark.parametrize("rows,cols", NORM_SIZES)
@pytest.mark.parametrize("weight", [BF, F32])
@pytest.mark.parametrize("with_residual", [False, True])
def test_norm_rows(mx, rows, cols, weight, with_residual):
    x, res = rand(1, rows, cols), rand(2, rows, cols, scale=3.0) if with_residual else None
    w = (1.0 + 0.2 * torch.randn(cols, generator=torch.Generator().manual_seed(3))).to(weight).to(DEV)
    s, y, out = run_norm(mx, x, w, 1e-6, res)
    h, _, want = ref.norm(host(x), host(w), 1e-6, None if res is None else host(res))
    if res is not None:
        assert np.array_equal(host(s), h)
    within(y, want, y_bound(want))
    same(out, codes_of(mx, y, True, False))


BOTH = [(rows, cols, row) for rows, cols in ((32, 32), (32, 136), (64, 256), (96, 288), (160, 1056), (32, 8224), (64, 16384), (416, 512),
                                             (128, 4096), (32, 8)) for row in (False, True) if not row or cols % 32 == 0]


@pytest.mark.parametrize("rows,cols,row", BOTH)
@pytest.mark.parametrize("with_residual", [False, True])
def test_norm_both_orientations(mx, rows, cols, row, with_residual):
    x, res = rand(4, rows, cols), rand(5, rows, cols, scale=2.0) if with_residual else None
    w = (1.0 + 0.2 * torch.randn(cols, generator=torch.Generator().manual_seed(6))).to(BF).to(DEV)
    s, y, out = run_norm(mx, x, w, 1e-5, res, row=row, col=True)
    h, _, want = ref.norm(host(x), host(w), 1e-5, None if res is None else host(res))
    if res is not None:
        assert np.array_equal(host(s), h)
    within(y, want, y_bound(want))
    same(out, codes_of(mx, y, row, True))
    # the codes alone are the same, and so with the sum in the residual's or x's own place
    alone = {k: torch.zeros_like(v) for k, v in out.items()}
    mx.mx_rmsnorm_mxfp8(x, w, 1e-5, residual=res, **alone)
    same(out, alone)
    if res is not None:
        for which in (0, 1):
            a, b = x.clone(), res.clone()
            again = {k: torch.zeros_like(v) for k, v in out.items()}
            mx.mx_rmsnorm_mxfp8(a, w, 1e-5, residual=b, sum_out=(a, b)[which], **again)
            same(out, again)
            assert torch.equal((a, b)[which], s)


def test_norm_rows_do_not_depend_on_the_batch_or_the_outputs(mx):
    x, w = rand(7, 192, 1312), rand(8, 1312, scale=0.1).float() + 1.0
    _, y, _ = run_norm(mx, x, w, 1e-6, row=True, col=True)
    for first, count in ((0, 1), (17, 5), (64, 128)):
        _, part, _ = run_norm(mx, x[first:first + count], w, 1e-6)
        assert torch.equal(part, y[first:first + count])


def test_norm_strided_views(mx):
    x, res, w = rand(9, 37, 320), rand(10, 37, 320), torch.ones(320, dtype=BF, device=DEV)
    s, y, out = run_norm(mx, x, w, 1e-6, res)
    ys, ss = strided(torch.zeros_like(x)), strided(torch.zeros_like(x))
    s2, y2, out2 = run_norm(mx, strided(x), w, 1e-6, strided(res), sum_out=ss, y=ys)
    assert torch.equal(s, s2) and torch.equal(y, y2)
    same(out, out2)
    for wide in (ys, ss):
        around = wide.as_strided((37, 344), (344, 1), wide.storage_offset() - 8)
        assert (around[:, :8] == 7.0).all() and (around[:, 328:] == 7.0).all()


@pytest.mark.parametrize("col", [False, True])
@pytest.mark.parametrize("value,eps", [(3.0e38, 1e-6), (2.0e20, 1e-6), (1e-25, 0.0), (1e-38, 0.0), (1e-20, 1e-30), (1e-30, 1e-6)])
def test_norm_beyond_the_range_of_squares(mx, value, eps, col):
    x = (torch.rand((32, 544), generator=torch.Generator().manual_seed(11)).to(DEV) * 0.9 + 0.1).mul(value).to(BF)
    w = torch.full((544,), 1.5, dtype=F32, device=DEV)
    _, y, out = run_norm(mx, x, w, eps, col=col)
    _, _, want = ref.norm(host(x), host(w), eps)
    within(y, want, y_bound(want))
    same(out, codes_of(mx, y, True, col))


def test_norm_zero_rows_and_rows_that_are_not_finite(mx):
    x, w = rand(12, 64, 512), torch.ones(512, dtype=BF, device=DEV)
    x[3] = 0
    x[5, 100], x[40, 7], x[41, 7], x[41, 9] = float("nan"), float("inf"), float("-inf"), float("nan")
    _, y, out = run_norm(mx, x, w, 1e-6, row=True, col=True)
    got = host(y)
    assert not got[3].any() and np.isnan(got[5]).all() and np.isnan(got[41]).all()
    assert np.isnan(got[40, 7]) and not np.delete(got[40], 7).any()
    rest = [r for r in range(64) if r not in (5, 40, 41)]
    _, _, want = ref.norm(host(x)[rest], 1.0, 1e-6)
    within(y[rest], want, y_bound(want))
    same(out, codes_of(mx, y, True, True))
    zero = torch.zeros((2, 512), dtype=BF, device=DEV)
    _, y, _ = run_norm(mx, zero, w, 0.0)                   # 0 / 0
    assert torch.isnan(y).all()


@pytest.mark.parametrize("rows,cols", [(61, 8), (100, 64), (1001, 136), (77901, 40), (78001, 64), (39000, 96), (39001, 128), (19501, 224), (19499, 256)])
def test_norm_of_narrow_rows(mx, rows, cols):
    """Rows that share a warp: ordinary ones, ones that FP32 does not hold and ones that are not finite side by side."""
    x, w = rand(13, rows, cols), rand(14, cols, scale=0.2).float() + 1.0
    x[1::7] *= 2.0 ** 70                                   # (exact: a power of two)
    x[2::7] *= 2.0 ** -80
    x[3::7, cols - 1], x[5::14, 3] = float("inf"), float("nan")
    fine = torch.ones(rows, dtype=torch.bool, device=DEV)
    fine[3::7] = fine[5::14] = False
    codes = cols % 32 == 0
    _, y, out = run_norm(mx, x, w, 0.0, row=codes)
    _, _, want = ref.norm(host(x[fine]), host(w), 0.0)
    within(y[fine], want, y_bound(want))
    assert torch.isnan(y[5::14]).all() and torch.isnan(y[3::7, -1]).all() and not y[3::7, :-1].any()
    if codes:
        same(out, codes_of(mx, y, True, False))
    # with a residual, in views with other strides, and column-wise codes too: the same rows
    half = x * 0.5
    ys, ss = strided(torch.zeros_like(x)), strided(torch.zeros_like(x))
    mx.mx_rmsnorm_mxfp8(strided(half), w, 0.0, residual=strided(half, extra=40), sum_out=ss, y=ys)
    assert torch.equal(ss.nan_to_num(7.0), x.nan_to_num(7.0)) and torch.equal(ys.nan_to_num(7.0), y.nan_to_num(7.0))
    around = ys.as_strided((rows, cols + 24), (cols + 24, 1), ys.storage_offset() - 8)
    assert (around[:, :8] == 7.0).all() and (around[:, cols + 8:] == 7.0).all()
    some = rows // 32 * 32
    _, both, _ = run_norm(mx, x[:some], w, 0.0, row=codes, col=True)
    assert torch.equal(both.nan_to_num(7.0), y[:some].nan_to_num(7.0))


BACKWARD_SIZES = [(1, 8), (1, 2048), (5, 96), (33, 1000), (700, 256), (3, 8200), (2, 16384), (311, 2048), (2000, 512), (4001, 128), (5, 5120),
                  (470, 4104), (9, 8192), (1900, 1024), (3700, 72)]


@pytest.mark.parametrize("rows,cols", BACKWARD_SIZES)
@pytest.mark.parametrize("weight", [BF, F32])
@pytest.mark.parametrize("with_dsum", [False, True])
def test_norm_backward(mx, rows, cols, weight, with_dsum):
    h, dy = rand(21, rows, cols, scale=2.0), rand(22, rows, cols, scale=0.01)
    dsum = rand(23, rows, cols, scale=0.01) if with_dsum else None
    w = (1.0 + 0.2 * torch.randn(cols, generator=torch.Generator().manual_seed(24))).to(weight).to(DEV)
    dx, dw = torch.empty_like(h), torch.full((cols,), 9.0, device=DEV)
    ws = torch.full((mx.rmsnorm_workspace_bytes(rows, cols),), 255, dtype=U8, device=DEV)
    mx.mx_rmsnorm_backward(dy, h, w, 1e-6, dx, dw, ws, dsum=dsum)
    want, wdw, bound, size = ref.norm_backward(host(dy), host(h), host(w), 1e-6, None if dsum is None else host(dsum))
    within(dx, want, bound)
    # a column's sum is at most rows additions in any order, and n has 24 roundings
    within(dw, wdw, (rows + 32) * ref.EPS32 * size + 1e-30)
    for alias in ("dy", "dsum") if with_dsum else ("dy",):
        a = {"dy": dy.clone(), "dsum": None if dsum is None else dsum.clone()}
        dw2 = torch.empty_like(dw)
        mx.mx_rmsnorm_backward(a["dy"], h, w, 1e-6, a[alias], dw2, ws, dsum=a["dsum"])
        assert torch.equal(a[alias], dx) and torch.equal(dw, dw2)


@pytest.mark.parametrize("rows,cols", [(9001, 64), (77901, 40), (39001, 128), (40000, 72), (19501, 224), (40011, 256),
                                       (20001, 384), (9001, 512), (9003, 776), (5000, 1000), (4999, 1024)])
def test_norm_backward_of_narrow_rows(mx, rows, cols):
    """Many rows to a warp, ordinary ones and ones that FP32 does not hold side by side, in views with other strides."""
    h, dy, dsum = rand(30, rows, cols), rand(31, rows, cols, scale=0.01), rand(32, rows, cols, scale=0.01)
    w = rand(33, cols, scale=0.2).float() + 1.0
    h[1::7] *= 2.0 ** 70                                   # (exact: powers of two)
    h[2::7] *= 2.0 ** -80
    dy[3::5] *= 2.0 ** -40
    dx, dw = torch.empty_like(h), torch.full((cols,), 9.0, device=DEV)
    ws = torch.full((mx.rmsnorm_workspace_bytes(rows, cols),), 255, dtype=U8, device=DEV)
    mx.mx_rmsnorm_backward(dy, h, w, 0.0, dx, dw, ws, dsum=dsum)
    want, wdw, bound, size = ref.norm_backward(host(dy), host(h), host(w), 0.0, host(dsum))
    within(dx, want, bound)
    within(dw, wdw, (rows + 32) * ref.EPS32 * size + 1e-30)
    views, dw2 = [strided(t, extra) for t, extra in ((dy, 24), (h, 40), (dsum, 32), (torch.zeros_like(h), 24))], torch.empty_like(dw)
    mx.mx_rmsnorm_backward(views[0], views[1], w, 0.0, views[3], dw2, ws, dsum=views[2])
    assert torch.equal(views[3], dx) and torch.equal(dw, dw2)
    around = views[3].as_strided((rows, cols + 24), (cols + 24, 1), views[3].storage_offset() - 8)
    assert (around[:, :8] == 7.0).all() and (around[:, cols + 8:] == 7.0).all()
    few = torch.empty((37, cols), dtype=BF, device=DEV)
    mx.mx_rmsnorm_backward(dy[-37:], h[-37:], w, 0.0, few, dw2, ws, dsum=dsum[-37:])
    assert torch.equal(few, dx[-37:])


def test_norm_backward_against_differences(mx):
    """The directional derivative of sum(dy * y) by central differences in 64 bits.  The step leaves an error of its square."""
    h, dy, w = rand(25, 9, 352), rand(26, 9, 352), rand(27, 352).float() + 1.0
    dx, dw = torch.empty_like(h), torch.empty(352, device=DEV)
    mx.mx_rmsnorm_backward(dy, h, w, 1e-6, dx, dw, torch.empty(1 << 20, dtype=U8, device=DEV))
    rng = np.random.default_rng(1)
    vh, vw = rng.standard_normal((9, 352)), rng.standard_normal(352)

    def loss(step):
        return (host(dy) * ref.norm(host(h) + step * vh, host(w) + step * vw, 1e-6)[2]).sum()

    slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
    got = (host(dx) * vh).sum() + (host(dw) * vw).sum()
    room = (np.abs(host(dx) * vh)).sum() * ref.HALF16 + 1e-4 * np.abs(slope) + 1e-6
    assert abs(got - slope) <= room


@pytest.mark.parametrize("value,grad,eps", [(2.0e20, 1.0, 1e-6), (1e-25, 1.0, 0.0), (1.0, 1e36, 1e-6), (1e-10, 1e-33, 0.0), (1e15, 1e-25, 1e-6),
                                            (1e-12, 1e25, 1e-30)])
def test_norm_backward_beyond_the_range_of_products(mx, value, grad, eps):
    h = (rand(28, 6, 640) * value).to(BF)
    dy = (rand(29, 6, 640) * grad).to(BF)
    w = torch.ones(640, dtype=F32, device=DEV)
    dx, dw = torch.empty_like(h), torch.empty(640, device=DEV)
    mx.mx_rmsnorm_backward(dy, h, w, eps, dx, dw, torch.empty(1 << 20, dtype=U8, device=DEV))
    want, wdw, bound, size = ref.norm_backward(host(dy), host(h), host(w), eps)
    within(dx, want, bound)
    within(dw, wdw, 64 * ref.EPS32 * size + 2.0 ** -140)


# ------------------------------------------------------------------------------------------------
# the router's choice
# ------------------------------------------------------------------------------------------------

def run_route(mx, z, k, normalize):
    ids = torch.full((z.shape[0], k), 99, dtype=I32, device=DEV)
    w = torch.full((z.shape[0], k), 99.0, device=DEV)
    mx.mx_moe_route(z, ids, w, normalize=normalize)
    return ids, w


def weight_bound(z, w):
    # exp within 2 steps, its argument's rounding, the total of at most 1024 terms (32 a lane and 5 levels), the quotient
    with np.errstate(invalid="ignore"):
        return w * ref.EPS32 * (64 + 2 * np.nan_to_num(np.ptp(np.where(np.isfinite(z), z, 0.0), axis=-1, keepdims=True))) + 2.0 ** -140


ROUTE_SIZES = [(1, 1, 1), (5, 3, 3), (64, 128, 8), (33, 60, 4), (7, 64, 6), (130, 200, 10), (9, 256, 32), (6, 511, 2), (3, 1024, 16), (1001, 16, 1)]


@pytest.mark.parametrize("tokens,experts,k", ROUTE_SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("normalize", [False, True])
def test_route_and_gradient(mx, tokens, experts, k, dtype, normalize):
    z = (torch.randn((tokens, experts), generator=torch.Generator().manual_seed(31)) * 3).to(dtype).to(DEV)
    if experts > 8:
        z[:, 3] = z[:, 5]                                  # ties
        z[tokens // 2, 1] = float("-inf")
    ids, w = run_route(mx, z, k, normalize)
    want_ids, want_w = ref.route(host(z), k, normalize)
    assert np.array_equal(host(ids), want_ids)
    within(w, want_w, weight_bound(host(z), want_w))
    dw = torch.randn((tokens, k), generator=torch.Generator().manual_seed(32)).to(DEV)
    dz = torch.full_like(z, 99.0)
    mx.mx_moe_route_backward(z, ids, dw, dz, normalize=normalize)
    want, mag = ref.route_backward(host(z), want_ids, host(dw), normalize)
    near = mag * ref.EPS32 * (160 + 4 * np.ptp(np.where(np.isfinite(host(z)), host(z), 0.0), axis=-1, keepdims=True)) + 2.0 ** -130
    within(dz, want, near if dtype == F32 else near * 1.01 + ref.HALF16 * np.abs(want))


def test_route_gradient_against_differences(mx):
    rng = np.random.default_rng(2)
    z = torch.from_numpy(rng.standard_normal((11, 40))).float().to(DEV)
    dw = torch.from_numpy(rng.standard_normal((11, 6))).float().to(DEV)
    v = rng.standard_normal((11, 40))
    for normalize in (False, True):
        ids, _ = run_route(mx, z, 6, normalize)
        dz = torch.empty_like(z)
        mx.mx_moe_route_backward(z, ids, dw, dz, normalize=normalize)

        def loss(step):
            x = host(z) + step * v
            e = np.exp(x)
            picked = np.take_along_axis(e, host(ids), 1)
            return (host(dw) * picked / (picked if normalize else e).sum(-1, keepdims=True)).sum()

        slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
        assert abs((host(dz) * v).sum() - slope) <= 1e-5 * np.abs(host(dz) * v).sum() + 1e-7


@pytest.mark.parametrize("normalize", [False, True])
def test_route_rows_that_leave_little_or_are_not_finite(mx, normalize):
    inf, nan = float("inf"), float("nan")
    z = torch.randn((8, 37), generator=torch.Generator().manual_seed(33)).to(DEV)
    z[0] = -inf                                            # nothing left
    z[1] = -inf
    z[1, 20], z[1, 4] = 1.0, -3.0                          # two left
    z[2, 9] = nan
    z[3, 11] = inf
    z[4] = torch.finfo(F32).min                            # the lowest value is a value
    z[5] = 0.0
    z[5, ::2] = -0.0                                       # zeros of both signs are equal
    z[6] = z[6] * 1e30
    ids, w = run_route(mx, z, 5, normalize)
    want_ids, want_w = ref.route(host(z), 5, normalize)
    assert np.array_equal(host(ids), want_ids)
    assert (host(ids)[0] == -1).all() and host(ids)[1].tolist() == [20, 4, -1, -1, -1]
    assert not host(w)[0].any() and np.isnan(host(w)[2]).all() and np.isnan(host(w)[3]).all()
    fine = [0, 1, 4, 5, 6, 7]
    within(w[fine], want_w[fine], np.maximum(weight_bound(host(z)[fine], want_w[fine]).clip(max=1e-5), 0) + 1e-6 * want_w[fine])
    dz = torch.full_like(z, 99.0)
    mx.mx_moe_route_backward(z, ids, torch.ones_like(w), dz, normalize=normalize)
    assert not host(dz)[0].any()
    masked = host(dz)[1][np.isneginf(host(z)[1])]
    assert not masked.any() and np.isnan(host(dz)[2, 9])


@pytest.mark.parametrize("experts,k", [(256, 8), (300, 32), (512, 1), (1024, 20)])
def test_route_many_experts_with_equal_and_masked_logits(mx, experts, k):
    """Rows that leave many equal candidates, few or none, or whose largest all lie in one lane's experts."""
    z = torch.randn((12, experts), generator=torch.Generator().manual_seed(37)).to(DEV)
    z[0] = 1.0                                             # all equal
    z[1] = torch.randint(0, 3, (experts,), generator=torch.Generator().manual_seed(38)).float().to(DEV)
    z[2] = -float("inf")
    z[3] = -float("inf")
    z[3, experts // 2] = -1e30
    z[4, 5::32] += 100.0                                   # the largest in lane 5
    z[5, ::2] = -float("inf")
    z[6] = torch.arange(experts, device=DEV).float()
    z[7] = -torch.arange(experts, device=DEV).float()
    z[8, 70:90] = float("nan")
    z[9] = torch.finfo(F32).min
    for normalize in (False, True):
        ids, w = run_route(mx, z, k, normalize)
        want_ids, want_w = ref.route(host(z), k, normalize)
        assert np.array_equal(host(ids), want_ids)
        fine = [r for r in range(12) if r != 8]
        within(w[fine], want_w[fine], np.minimum(weight_bound(host(z)[fine], want_w[fine]), 2e-5) + 2e-6 * want_w[fine])
        assert np.isnan(host(w)[8]).all()


def test_route_gradient_of_ids_given_twice_or_outside(mx):
    z = torch.randn((4, 12), generator=torch.Generator().manual_seed(34)).to(DEV)
    ids = torch.tensor([[3, 3, 1], [-1, 12, 5], [-1, -1, -1], [0, 11, 0]], dtype=I32, device=DEV)
    dw = torch.randn((4, 3), generator=torch.Generator().manual_seed(35)).to(DEV)
    for normalize in (False, True):
        dz = torch.full_like(z, 99.0)
        mx.mx_moe_route_backward(z, ids, dw, dz, normalize=normalize)
        want, mag = ref.route_backward(host(z), host(ids), host(dw), normalize)
        within(dz, want, 200 * ref.EPS32 * mag)


def test_route_strided_logits(mx):
    z = rand(36, 50, 72)
    a, b = run_route(mx, z, 4, True), run_route(mx, strided(z), 4, True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    wide = strided(torch.zeros_like(z))
    dz = torch.empty_like(z)
    mx.mx_moe_route_backward(strided(z), a[0], a[1], wide)
    mx.mx_moe_route_backward(z, a[0], a[1], dz)
    assert torch.equal(wide, dz)


# ------------------------------------------------------------------------------------------------
# rows by expert and back
# ------------------------------------------------------------------------------------------------

def some_ids(seed, tokens, k, experts, idle=0.0, distinct=True):
    rng = np.random.default_rng(seed)
    if distinct and k <= experts:
        ids = np.argsort(rng.random((tokens, experts)), axis=1)[:, :k]
    else:
        ids = rng.integers(0, experts, (tokens, k))
    ids[rng.random((tokens, k)) < idle] = -1
    return torch.from_numpy(ids.astype(np.int32)).to(DEV)


def run_sort(mx, ids, experts, source=True):
    n = ids.numel()
    offsets = torch.full((experts + 1,), 77, dtype=torch.int64, device=DEV)
    rows, src = torch.full_like(ids, 77), torch.full((n,), 77, dtype=I32, device=DEV)
    ws = torch.full((mx.moe_sort_workspace_bytes(n, experts),), 255, dtype=U8, device=DEV)
    mx.mx_moe_sort(ids, offsets, rows, src if source else None, ws)
    return offsets, rows, src


SORT_SIZES = [(1, 1, 1), (1, 8, 128), (3, 2, 5), (61, 8, 128), (513, 8, 16), (4096, 1, 7), (4097, 1, 1024), (700, 6, 60), (8192, 8, 128),
              (5000, 32, 1024), (2049, 2, 33), (16385, 8, 40), (150000, 8, 64), (40000, 4, 1024)]


@pytest.mark.parametrize("tokens,k,experts", SORT_SIZES)
@pytest.mark.parametrize("idle", [0.0, 0.3])
def test_sort(mx, tokens, k, experts, idle):
    ids = some_ids(41, tokens, k, experts, idle, distinct=tokens < 10000)
    got = run_sort(mx, ids, experts)
    for a, b, name in zip(got, ref.sort(host(ids), experts), ("group_offsets", "rows", "source")):
        assert np.array_equal(host(a), b), name
    a, b, _ = run_sort(mx, ids, experts, source=False)
    assert torch.equal(a, got[0]) and torch.equal(b, got[1])


@pytest.mark.parametrize("experts", [1, 40, 600])
def test_sort_one_expert_for_all_none_for_all_and_ids_outside(mx, experts):
    for fill in (experts - 1, -1, experts, 2 ** 31 - 1, -2 ** 31):
        for tokens in (9, 9001):
            ids = torch.full((tokens, 3), fill, dtype=I32, device=DEV)
            for a, b in zip(run_sort(mx, ids, experts), ref.sort(host(ids), experts)):
                assert np.array_equal(host(a), b)


MOVES = [(1, 1, 4, 8), (1, 8, 128, 2048), (61, 8, 128, 512), (37, 6, 60, 1000), (300, 4, 9, 136), (40, 32, 64, 264), (5, 3, 8, 16384), (2000, 2, 16, 32)]


@pytest.mark.parametrize("tokens,k,experts,hidden", MOVES)
@pytest.mark.parametrize("view", [False, True])
def test_dispatch(mx, tokens, k, experts, hidden, view):
    ids = some_ids(42, tokens, k, experts, 0.2)
    _, rows, source = run_sort(mx, ids, experts)
    x = rand(43, tokens, hidden)
    y = torch.full((tokens * k, hidden), 5.0, dtype=BF, device=DEV)
    y = strided(y) if view else y
    mx.mx_moe_dispatch(strided(x) if view else x, rows, y)
    src = host(source)
    want = np.where((src >= 0)[:, None], host(x)[np.maximum(src, 0) // k], 5.0)
    assert np.array_equal(host(y), want)


@pytest.mark.parametrize("tokens,k,experts,hidden", [(1, 1, 4, 32), (1, 8, 128, 2048), (61, 8, 128, 256), (37, 6, 60, 992), (300, 4, 9, 160),
                                                     (40, 32, 64, 288), (5, 3, 8, 16384), (1000, 2, 3, 512), (900, 8, 1024, 64),
                                                     (30, 3, 5, 8480), (2500, 1, 9, 96), (5000, 3, 40, 160), (20000, 5, 300, 32), (2600, 20, 64, 96),
                                                     (2433, 32, 40, 64), (4867, 2, 7, 2112)])
@pytest.mark.parametrize("idle", [0.0, 0.4])
def test_dispatch_quantized_is_the_grouped_quantizer_of_the_dispatched_rows(mx, tokens, k, experts, hidden, idle):
    ids = some_ids(44, tokens, k, experts, idle)
    offsets, rows, _ = run_sort(mx, ids, experts)
    used, n = int(offsets[-1]), tokens * k
    x = rand(45, tokens, hidden)
    y = torch.zeros((n, hidden), dtype=BF, device=DEV)
    mx.mx_moe_dispatch(x, rows, y)
    # MXFP8
    a = mx.alloc_mxfp8(tokens, hidden, DEV, colwise=False)
    mx.mx_quantize_mxfp8(x, **a)
    q = torch.full((n, hidden), 0x33, dtype=U8, device=DEV)
    s = torch.full((mx.grouped_scale_bytes(n, experts, hidden, 32),), 0x33, dtype=U8, device=DEV)
    mx.mx_moe_dispatch_quantized(mx.MX_FMT_MXFP8, a["q_row"], a["s_row"], rows, offsets, q, s)
    assert (q[used:] == 0x33).all()
    if used:
        want_q = torch.empty((used, hidden), dtype=U8, device=DEV)
        want_s = torch.empty(mx.grouped_scale_bytes(used, experts, hidden, 32), dtype=U8, device=DEV)
        mx.mx_quantize_mxfp8_grouped(y[:used], offsets, want_q, want_s)
        assert torch.equal(q[:used], want_q) and torch.equal(s[:want_s.numel()], want_s)
        assert not s[want_s.numel():].any()
    else:
        assert not s.any()
    # NVFP4
    a = mx.alloc_nvfp4_rows(tokens, hidden, DEV)
    mx.mx_nvfp4_quantize_per_token(x, a["q"], a["s"], a["s2"])
    out = mx.alloc_nvfp4_rows_grouped(n, experts, hidden, DEV)
    for t in out.values():
        t.fill_(0x33)
    mx.mx_moe_dispatch_quantized(mx.MX_FMT_NVFP4, a["q"], a["s"], rows, offsets, out["q"], out["s"], s2=a["s2"], s2_out=out["s2"])
    assert (out["q"][used:] == 0x33).all() and (out["s2"][used:] == 0x33).all()
    if used:
        want = mx.alloc_nvfp4_rows_grouped(used, experts, hidden, DEV)
        mx.mx_nvfp4_quantize_per_token_grouped(y[:used], offsets, want["q"], want["s"], want["s2"])
        assert torch.equal(out["q"][:used], want["q"]) and torch.equal(out["s2"][:used], want["s2"])
        assert torch.equal(out["s"][:want["s"].numel()], want["s"]) and not out["s"][want["s"].numel():].any()


@pytest.mark.parametrize("tokens,k,experts,hidden", MOVES)
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("with_residual", [False, True])
def test_combine(mx, tokens, k, experts, hidden, weighted, with_residual):
    ids = some_ids(46, tokens, k, experts, 0.2)
    ids[tokens // 2] = -1                                  # a token without an expert
    _, rows, source = run_sort(mx, ids, experts)
    z = rand(47, tokens * k, hidden)
    z[int((host(source) >= 0).sum()):] = float("nan")      # rows that none names
    w = torch.rand((tokens, k), generator=torch.Generator().manual_seed(48)).to(DEV) if weighted else None
    if weighted:
        w[rows < 0] = float("nan")                   # weights of choices that are left out
    res = rand(49, tokens, hidden, scale=3.0) if with_residual else None
    y = torch.full((tokens, hidden), 5.0, dtype=BF, device=DEV)
    mx.mx_moe_combine(z, rows, y, weights=w, residual=res)
    want, mag = ref.combine(host(z), host(rows), None if w is None else host(w), None if res is None else host(res))
    within(y, want, ref.HALF16 * np.abs(want) + (k + 2) * 1.01 * ref.EPS32 * mag + ref.TINY16)
    wide = strided(res) if with_residual else strided(torch.zeros_like(y))
    mx.mx_moe_combine(strided(z), rows, wide, weights=w, residual=wide if with_residual else None)   # in the residual's place
    assert torch.equal(wide, y)


@pytest.mark.parametrize("tokens,k,experts,hidden", MOVES)
def test_combine_backward(mx, tokens, k, experts, hidden):
    ids = some_ids(50, tokens, k, experts, 0.2)
    _, rows, source = run_sort(mx, ids, experts)
    z, dy = rand(51, tokens * k, hidden), rand(52, tokens, hidden)
    z[int((host(source) >= 0).sum()):] = float("nan")
    w = torch.rand((tokens, k), generator=torch.Generator().manual_seed(53)).to(DEV)
    dz, dw = torch.full_like(z, 5.0), torch.full((tokens, k), 5.0, device=DEV)
    mx.mx_moe_combine_backward(dy, z, rows, w, dz, dw)
    want, want_dw, mag = ref.combine_backward(host(dy), host(z), host(rows), host(w), np.full(z.shape, 5.0))
    within(dz, want, (ref.HALF16 + 1.01 * ref.EPS32) * np.abs(want))
    within(dw, want_dw, (hidden / 256 + 40) * ref.EPS32 * mag)
    zs, dw2 = strided(z), torch.empty_like(dw)
    mx.mx_moe_combine_backward(strided(dy), zs, rows, w, zs, dw2)                    # the gradient in the rows' own place
    used = source >= 0
    assert torch.equal(zs[used], dz[used]) and torch.equal(dw, dw2)


def test_combine_gradients_against_differences(mx):
    """combine is linear in z and in the weights: the gradients along a direction are differences of whole steps."""
    ids = some_ids(54, 20, 4, 8)
    _, rows, _ = run_sort(mx, ids, 8)
    z, dy, dx = rand(55, 80, 96), rand(56, 20, 96), torch.empty((20, 96), dtype=BF, device=DEV)
    w = torch.rand((20, 4), generator=torch.Generator().manual_seed(57)).to(DEV)
    dz, dw = torch.empty_like(z), torch.empty_like(w)
    mx.mx_moe_combine_backward(dy, z, rows, w, dz, dw)
    rng = np.random.default_rng(3)
    vz, vw = rng.standard_normal(z.shape), rng.standard_normal(w.shape)
    f = lambda a, b: (host(dy) * ref.combine(a, host(rows), b)[0]).sum()             # noqa: E731
    for got, v, slope in ((dz, vz, f(host(z) + vz, host(w)) - f(host(z), host(w))), (dw, vw, f(host(z), host(w) + vw) - f(host(z), host(w)))):
        assert abs((host(got) * v).sum() - slope) <= ref.HALF16 * np.abs(host(got) * v).sum() + 1e-9 * abs(slope) + 1e-9
    # and dispatch's gradient is the plain combine: <dispatch(x), u> = <x, combine(u)>
    x, u = rand(58, 20, 96), rand(59, 80, 96)
    y = torch.empty_like(u)
    mx.mx_moe_dispatch(x, rows, y)
    mx.mx_moe_combine(u, rows, dx)
    want, _ = ref.combine(host(u), host(rows))
    assert abs((host(y) * host(u)).sum() - (host(x) * want).sum()) <= 1e-9 * np.abs(host(y) * host(u)).sum()
    within(dx, want, ref.HALF16 * np.abs(want) + 8 * ref.EPS32 * np.abs(host(u)).max())


def test_rows_outside_the_buffers_are_skipped(mx):
    rows = torch.tensor([[0, 9], [-5, 2], [2 ** 31 - 1, 1]], dtype=I32, device=DEV)
    x, y = rand(60, 3, 64), torch.full((4, 64), 5.0, dtype=BF, device=DEV)
    mx.mx_moe_dispatch(x, rows, y)
    assert torch.equal(y[0], x[0]) and torch.equal(y[2], x[1]) and torch.equal(y[1], x[2]) and (y[3] == 5.0).all()
    z, out = rand(61, 4, 64), torch.empty((3, 64), dtype=BF, device=DEV)
    mx.mx_moe_combine(z, rows, out)
    assert torch.equal(out, z[torch.tensor([0, 2, 1], device=DEV)])
    a = mx.alloc_mxfp8(3, 64, DEV, colwise=False)
    mx.mx_quantize_mxfp8(x, **a)
    q, s = torch.full((4, 64), 0x33, dtype=U8, device=DEV), torch.empty(mx.grouped_scale_bytes(4, 2, 64, 32), dtype=U8, device=DEV)
    mx.mx_moe_dispatch_quantized(mx.MX_FMT_MXFP8, a["q_row"], a["s_row"], rows, torch.tensor([0, 2, 3], device=DEV), q, s)
    assert torch.equal(q[0], a["q_row"][0]) and torch.equal(q[2], a["q_row"][1]) and (q[3] == 0x33).all()


# ------------------------------------------------------------------------------------------------
# streams, graphs, devices
# ------------------------------------------------------------------------------------------------

def a_layer(mx, x, res, w, experts, state):
    """Norm, choice, sort, dispatch and combine of rows doubled by plain torch, and the gradients, into the buffers of `state`."""
    s = state
    mx.mx_rmsnorm_mxfp8(x, w, 1e-6, residual=res, sum_out=s["sum"], y=s["y"], q_row=s["q"], s_row=s["s"])
    s["logits"].copy_(s["y"][:, :experts])
    mx.mx_moe_route(s["logits"], s["ids"], s["weights"])
    mx.mx_moe_sort(s["ids"], s["offsets"], s["rows"], s["source"], s["ws"])
    mx.mx_moe_dispatch(s["y"], s["rows"], s["z"])
    mx.mx_moe_dispatch_quantized(mx.MX_FMT_MXFP8, s["q"], s["s"], s["rows"], s["offsets"], s["zq"], s["zs"])
    s["z"].mul_(2.0)
    mx.mx_moe_combine(s["z"], s["rows"], s["out"], weights=s["weights"], residual=s["sum"])
    mx.mx_moe_combine_backward(s["out"], s["z"], s["rows"], s["weights"], s["dz"], s["dweights"])
    mx.mx_moe_combine(s["dz"], s["rows"], s["dy"])
    mx.mx_moe_route_backward(s["logits"], s["ids"], s["dweights"], s["dlogits"])
    mx.mx_rmsnorm_backward(s["dy"], s["sum"], w, 1e-6, s["dx"], s["dw"], s["ws"], dsum=s["out"])
    return ("sum", "y", "q", "s", "ids", "weights", "offsets", "rows", "source", "z", "zq", "zs", "out", "dz", "dweights", "dy", "dlogits", "dx", "dw")


def layer_state(mx, t, hidden, k, experts):
    e = lambda *shape, dtype=BF: torch.zeros(shape, dtype=dtype, device=DEV)         # noqa: E731
    n = t * k
    return {"sum": e(t, hidden), "y": e(t, hidden), "q": e(t, hidden, dtype=U8), "s": e(mx.scale_bytes(t, hidden, 32), dtype=U8),
            "logits": e(t, experts), "ids": e(t, k, dtype=I32), "weights": e(t, k, dtype=F32), "offsets": e(experts + 1, dtype=torch.int64),
            "rows": e(t, k, dtype=I32), "source": e(n, dtype=I32), "ws": e(max(mx.moe_sort_workspace_bytes(n, experts),
                                                                                mx.rmsnorm_workspace_bytes(t, hidden)), dtype=U8),
            "z": e(n, hidden), "zq": e(n, hidden, dtype=U8), "zs": e(mx.grouped_scale_bytes(n, experts, hidden, 32), dtype=U8),
            "out": e(t, hidden), "dz": e(n, hidden), "dweights": e(t, k, dtype=F32), "dy": e(t, hidden), "dlogits": e(t, experts),
            "dx": e(t, hidden), "dw": e(hidden, dtype=F32)}


@pytest.mark.parametrize("tokens", [1, 50, 900])
def test_run_of_all_eager_captured_replayed_and_on_two_streams(mx, tokens):
    hidden, k, experts = 256, 8, 128
    w = torch.ones(hidden, dtype=BF, device=DEV)
    inputs = [(rand(71 + i, tokens, hidden), rand(81 + i, tokens, hidden)) for i in range(3)]
    want = []
    for x, res in inputs:
        s = layer_state(mx, tokens, hidden, k, experts)
        names = a_layer(mx, x, res, w, experts, s)
        torch.cuda.synchronize()
        want.append({n: s[n].clone() for n in names})
    # one graph, replayed on changing inputs
    x, res, s = inputs[0][0].clone(), inputs[0][1].clone(), layer_state(mx, tokens, hidden, k, experts)
    a_layer(mx, x, res, w, experts, s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a_layer(mx, x, res, w, experts, s)
    for i in (1, 2, 0):
        x.copy_(inputs[i][0])
        res.copy_(inputs[i][1])
        g.replay()
        torch.cuda.synchronize()
        for n in want[i]:
            assert torch.equal(s[n], want[i][n]), n
    # two streams at once, each with its own buffers
    streams, states = [torch.cuda.Stream(), torch.cuda.Stream()], [layer_state(mx, tokens, hidden, k, experts) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                a_layer(mx, inputs[i][0], inputs[i][1], w, experts, states[i])
    torch.cuda.synchronize()
    for i in range(2):
        for n in want[i]:
            assert torch.equal(states[i][n], want[i][n]), n
    mx.check_device_status()


def test_large_sizes_pass_32_bits(mx):
    """Rows whose byte offsets pass 2^32: combine and dispatch at the end of a large buffer."""
    hidden, total = 8192, 300000                           # 4.9 GB
    z = torch.zeros((total, hidden), dtype=BF, device=DEV)
    rows = torch.tensor([[total - 1, 0], [5, total - 2]], dtype=I32, device=DEV)
    x = rand(90, 2, hidden)
    mx.mx_moe_dispatch(x, rows, z)
    assert torch.equal(z[total - 1], x[0]) and torch.equal(z[total - 2], x[1]) and torch.equal(z[0], x[0])
    y = torch.empty((2, hidden), dtype=BF, device=DEV)
    mx.mx_moe_combine(z, rows, y, weights=torch.full((2, 2), 0.5, device=DEV))
    assert torch.equal(y, x)
