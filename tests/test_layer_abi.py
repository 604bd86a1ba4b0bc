"""Host-side validation of the entry points of include/mxnum_layer.h: each refusal returns its status before anything touches a
GPU, every declared symbol is exported and bound, the binding refuses tensors of another kind, and the 64-bit forms that
the GPU tests compare with agree with differences of themselves."""
import ctypes
import os
import re

import numpy as np
import pytest

import layer_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mxnum_layer.h")

# fake, never dereferenced device addresses
A = ctypes.c_void_p(0x10000)
A8 = ctypes.c_void_p(0x10008)
A2 = ctypes.c_void_p(0x10002)
NUL = None
OK, INVALID, ALIGNMENT, UNSUPPORTED = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from microscaled_precision_numerics_gb300 import _build
    import microscaled_precision_numerics_gb300 as mx
    _build.build()
    return mx.lib()


def test_every_declared_symbol_is_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mx_[a-z0-9_]+)\s*\(", text)))
    assert names == ["mx_moe_combine", "mx_moe_combine_backward", "mx_moe_dispatch", "mx_moe_dispatch_quantized", "mx_moe_route",
                     "mx_moe_route_backward", "mx_moe_sort", "mx_moe_sort_workspace_bytes", "mx_rmsnorm_backward", "mx_rmsnorm_mxfp8",
                     "mx_rmsnorm_workspace_bytes"]
    for name in names:
        assert getattr(lib, name).argtypes is not None, name


NORM = dict(x=A, ldx=64, residual=A, ldr=64, weight=A, weight_type=0, eps=1e-6, rows=32, cols=64, sum=A, lds=64, y=A, ldy=64, q_row=A, s_row=A,
            q_col=A, s_col=A, stream=NUL)
NORM_BACKWARD = dict(dy=A, lddy=64, h=A, ldh=64, weight=A, weight_type=1, eps=1e-6, rows=3, cols=64, dsum=A, ldds=64, dx=A, lddx=64, dweight=A,
                     workspace=A, workspace_bytes=1 << 30, stream=NUL)
ROUTE = dict(logits=A, logits_type=0, ldl=16, tokens=4, experts=16, top_k=2, normalize=1, ids=A, weights=A, stream=NUL)
ROUTE_BACKWARD = dict(logits=A, logits_type=1, ldl=16, tokens=4, experts=16, top_k=2, normalize=0, ids=A, dweights=A, dlogits=A, ldd=16, stream=NUL)
SORT = dict(ids=A, tokens=4, top_k=2, experts=16, group_offsets=A, rows=A, source=A, workspace=A, workspace_bytes=1 << 20, stream=NUL)
DISPATCH = dict(x=A, ldx=64, tokens=4, hidden=64, rows=A, top_k=2, y=A, ldy=64, total_rows=8, stream=NUL)
QUANTIZED = dict(fmt=1, q=A, s=A, s2=A, tokens=4, hidden=64, rows=A, top_k=2, G=16, group_offsets=A, q_out=A, s_out=A, s2_out=A, total_rows=8,
                 stream=NUL)
COMBINE = dict(z=A, ldz=64, total_rows=8, hidden=64, rows=A, weights=A, tokens=4, top_k=2, residual=A, ldr=64, y=A, ldy=64, stream=NUL)
COMBINE_BACKWARD = dict(dy=A, lddy=64, z=A, ldz=64, total_rows=8, hidden=64, rows=A, weights=A, tokens=4, top_k=2, dz=A, lddz=64, dweights=A,
                        stream=NUL)


def check(f, base, want, **changed):
    assert set(changed) <= set(base)
    assert f(*{**base, **changed}.values()) == want, changed


def check_common(f, base, must, sixteen, four, sizes, strides):
    for p in must:
        check(f, base, INVALID, **{p: NUL})
    for p in sixteen:
        check(f, base, ALIGNMENT, **{p: A8})
    for p in four:
        check(f, base, ALIGNMENT, **{p: A2})
    for p in sizes:
        check(f, base, INVALID, **{p: 0})
        check(f, base, INVALID, **{p: -1})
    for p, odd in strides:
        check(f, base, INVALID, **{p: base[p] - 8})
        if odd:
            check(f, base, ALIGNMENT, **{p: base[p] + 4})


def test_norm_refusals(lib):
    f = lib.mx_rmsnorm_mxfp8
    check_common(f, NORM, ("x", "weight", "s_row", "s_col"), ("x", "residual", "weight", "sum", "y", "q_row", "s_row", "q_col", "s_col"), (),
                 ("rows", "cols"), [(p, True) for p in ("ldx", "ldr", "lds", "ldy")])
    check(f, NORM, INVALID, residual=NUL)                  # a sum of nothing
    check(f, NORM, INVALID, y=NUL, q_row=NUL, q_col=NUL)
    check(f, NORM, INVALID, weight_type=2)
    for eps in (-1e-6, float("nan"), float("inf")):
        check(f, NORM, INVALID, eps=eps)
    wide = {k: 1 << 15 for k in ("ldx", "ldr", "lds", "ldy")}
    check(f, NORM, UNSUPPORTED, rows=40)                   # column-wise blocks
    check(f, NORM, UNSUPPORTED, cols=48)                   # row-wise blocks
    check(f, NORM, ALIGNMENT, cols=44)
    check(f, NORM, UNSUPPORTED, cols=16384 + 32, **wide)
    check(f, NORM, UNSUPPORTED, rows=1 << 31)


def test_norm_backward_refusals(lib):
    f = lib.mx_rmsnorm_backward
    check_common(f, NORM_BACKWARD, ("dy", "h", "weight", "dx", "dweight", "workspace"), ("dy", "h", "weight", "dsum", "dx", "workspace"),
                 ("dweight",), ("rows", "cols"), [(p, True) for p in ("lddy", "ldh", "ldds", "lddx")])
    check(f, NORM_BACKWARD, INVALID, workspace_bytes=lib.mx_rmsnorm_workspace_bytes(3, 64) - 1)
    check(f, NORM_BACKWARD, INVALID, eps=-1.0)
    check(f, NORM_BACKWARD, UNSUPPORTED, cols=16392, **{k: 1 << 15 for k in ("lddy", "ldh", "ldds", "lddx")})
    for bad in ((0, 64), (3, 0), (-1, 64), (3, 16385)):
        assert lib.mx_rmsnorm_workspace_bytes(*bad) == 0
    assert 0 < lib.mx_rmsnorm_workspace_bytes(1 << 20, 16384) <= 64 << 20


def test_route_refusals(lib):
    f = lib.mx_moe_route
    check_common(f, ROUTE, ("logits", "ids", "weights"), (), ("logits", "ids", "weights"), ("tokens", "experts", "top_k"), [("ldl", False)])
    f2 = lib.mx_moe_route_backward
    check_common(f2, ROUTE_BACKWARD, ("logits", "ids", "dweights", "dlogits"), (), ("logits", "ids", "dweights", "dlogits"),
                 ("tokens", "experts", "top_k"), [("ldl", False), ("ldd", False)])
    for g, base in ((f, ROUTE), (f2, ROUTE_BACKWARD)):
        check(g, base, INVALID, logits_type=2)
        check(g, base, INVALID, normalize=2)
        check(g, base, INVALID, top_k=17)
        strides = {k: 2000 for k in ("ldl", "ldd") if k in base}
        check(g, base, UNSUPPORTED, experts=1025, **strides)
        check(g, base, UNSUPPORTED, experts=64, top_k=33, **strides)
        check(g, base, UNSUPPORTED, tokens=1 << 30)


def test_sort_refusals(lib):
    f = lib.mx_moe_sort
    check_common(f, SORT, ("ids", "group_offsets", "rows", "workspace"), ("group_offsets", "workspace"), ("ids", "rows", "source"),
                 ("tokens", "top_k", "experts"), [])
    check(f, SORT, UNSUPPORTED, experts=1025)
    check(f, SORT, UNSUPPORTED, top_k=33)
    check(f, SORT, UNSUPPORTED, tokens=1 << 30)
    check(f, SORT, INVALID, workspace_bytes=lib.mx_moe_sort_workspace_bytes(8, 16) - 1)
    for bad in ((0, 8), (8, 0), (8, 1025), (1 << 31, 8), (-8, 8)):
        assert lib.mx_moe_sort_workspace_bytes(*bad) == 0
    assert 0 < lib.mx_moe_sort_workspace_bytes((1 << 31) - 1, 1024) <= 16 << 20


def test_rows_refusals(lib):
    check_common(lib.mx_moe_dispatch, DISPATCH, ("x", "rows", "y"), ("x", "y"), ("rows",), ("tokens", "hidden", "top_k", "total_rows"),
                 [("ldx", True), ("ldy", True)])
    check_common(lib.mx_moe_combine, COMBINE, ("z", "rows", "y"), ("z", "residual", "y"), ("rows", "weights"),
                 ("tokens", "hidden", "top_k", "total_rows"), [("ldz", True), ("ldr", True), ("ldy", True)])
    check_common(lib.mx_moe_combine_backward, COMBINE_BACKWARD, ("dy", "z", "rows", "weights", "dz", "dweights"), ("dy", "z", "dz"),
                 ("rows", "weights", "dweights"), ("tokens", "hidden", "top_k", "total_rows"), [("lddy", True), ("ldz", True), ("lddz", True)])
    check_common(lib.mx_moe_dispatch_quantized, QUANTIZED, ("q", "s", "s2", "rows", "group_offsets", "q_out", "s_out", "s2_out"),
                 ("q", "s", "group_offsets", "q_out", "s_out"), ("s2", "rows", "s2_out"), ("tokens", "hidden", "top_k", "total_rows", "G"), [])
    check(lib.mx_moe_dispatch_quantized, QUANTIZED, INVALID, fmt=0)                   # MXFP8 has no second scales
    check(lib.mx_moe_dispatch_quantized, QUANTIZED, INVALID, fmt=2)
    check(lib.mx_moe_dispatch_quantized, QUANTIZED, INVALID, G=1025)
    check(lib.mx_moe_dispatch_quantized, QUANTIZED, UNSUPPORTED, hidden=48)
    for f, base, ld in ((lib.mx_moe_dispatch, DISPATCH, ("ldx", "ldy")), (lib.mx_moe_combine, COMBINE, ("ldz", "ldr", "ldy")),
                        (lib.mx_moe_combine_backward, COMBINE_BACKWARD, ("lddy", "ldz", "lddz"))):
        check(f, base, ALIGNMENT, hidden=60)
        check(f, base, UNSUPPORTED, top_k=33)
        check(f, base, UNSUPPORTED, tokens=1 << 30)
        check(f, base, UNSUPPORTED, total_rows=1 << 31)
        check(f, base, UNSUPPORTED, hidden=(1 << 23) + 8, **{k: 1 << 24 for k in ld})


def test_binding_refuses_tensors_of_another_kind(lib):
    import torch
    import microscaled_precision_numerics_gb300 as mx
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.ones(64)
    ids, f32 = torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2))
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    off = torch.zeros(9, dtype=torch.int64)
    with pytest.raises(TypeError):
        mx.mx_rmsnorm_mxfp8(x.float(), w, 1e-6, y=x)
    with pytest.raises(TypeError):
        mx.mx_rmsnorm_mxfp8(x, w.half(), 1e-6, y=x)
    with pytest.raises(ValueError):
        mx.mx_rmsnorm_mxfp8(x.t(), w, 1e-6, y=x)
    with pytest.raises(TypeError):
        mx.mx_moe_route(x.half(), ids, f32)
    with pytest.raises(ValueError):
        mx.mx_moe_route(x, ids[0], f32)
    with pytest.raises(ValueError):
        mx.mx_moe_dispatch(x[:3], ids, x)
    # everything in order, but on the CPU
    for call in (lambda: mx.mx_rmsnorm_mxfp8(x, w, 1e-6, y=x), lambda: mx.mx_rmsnorm_backward(x, x, w, 1e-6, x, w, ws),
                 lambda: mx.mx_moe_route(x, ids, f32), lambda: mx.mx_moe_route_backward(x, ids, f32, x), lambda: mx.mx_moe_sort(ids, off, ids, None, ws),
                 lambda: mx.mx_moe_dispatch(x, ids, x), lambda: mx.mx_moe_combine(x, ids, x), lambda: mx.mx_moe_combine_backward(x, x, ids, f32, x, f32)):
        with pytest.raises(ValueError):
            call()


def test_rounding_to_bf16_is_to_the_nearest_even():
    import torch
    a = np.random.default_rng(1).standard_normal(10000).astype(np.float32)
    a = np.concatenate([a, (a.view(np.uint32) & 0xFFFF0000 | 0x8000).view(np.float32)])
    assert np.array_equal(ref.bf16(a), torch.from_numpy(a).to(torch.bfloat16).double().numpy())


def test_gradients_of_the_plain_forms_against_differences():
    """Central differences of the forward forms; the step's square is 1e-10 and the values are of order one."""
    rng = np.random.default_rng(5)
    h, w, dy = rng.standard_normal((6, 40)), rng.standard_normal(40), rng.standard_normal((6, 40))
    dx, dw, _, _ = ref.norm_backward(dy, h, w, 1e-3)
    z, dwt = rng.standard_normal((6, 12)), rng.standard_normal((6, 3))
    for value, grads in (((h, w), (dx, dw)),):
        for which in range(2):
            v = rng.standard_normal(value[which].shape)
            f = lambda s: (dy * ref.norm(*[a + s * v if i == which else a for i, a in enumerate(value)], 1e-3)[2]).sum()  # noqa: B023, E731
            assert abs((f(1e-5) - f(-1e-5)) / 2e-5 - (grads[which] * v).sum()) < 1e-6
    for normalize in (False, True):
        ids, _ = ref.route(z, 3, normalize)
        dz, _ = ref.route_backward(z, ids, dwt, normalize)
        v = rng.standard_normal(z.shape)
        f = lambda s: (dwt * ref.route(z + s * v, 3, normalize)[1]).sum()           # noqa: B023, E731
        assert abs((f(1e-6) - f(-1e-6)) / 2e-6 - (dz * v).sum()) < 1e-6


def test_plain_sort_and_combine():
    ids = np.array([[2, 0], [-1, 2], [0, 5]], np.int32)
    offsets, rows, source = ref.sort(ids, 4)
    assert offsets.tolist() == [0, 2, 2, 4, 4] and rows.tolist() == [[2, 0], [-1, 3], [1, -1]] and source.tolist() == [1, 4, 0, 3, -1, -1]
    z = np.arange(12.0).reshape(6, 2)
    y, _ = ref.combine(z, rows, np.full((3, 2), 2.0), np.ones((3, 2)))
    assert y.tolist() == [[1 + 2 * 4 + 0, 1 + 2 * 5 + 2 * 1], [1 + 2 * 6, 1 + 2 * 7], [1 + 2 * 2, 1 + 2 * 3]]
