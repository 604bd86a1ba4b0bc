"""The binding refuses tensors of the layer's entry points that hold enough elements in another shape: a choice's values by
[top_k, tokens], a norm's weights of another width.  On CPU tensors, which are refused last of all: the message tells."""
import pytest
import torch

import layer_ref as ref                                    # noqa: F401  (the tests' folder is on the path)
import microscaled_precision_numerics_gb300 as mx

I32, F32, BF = torch.int32, torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    from microscaled_precision_numerics_gb300 import _build
    _build.build()
    return mx.lib()


T, K, E, H = 6, 2, 16, 64


def calls():
    x, z, logits = torch.zeros((T, H), dtype=BF), torch.zeros((T * K, H), dtype=BF), torch.zeros((T, E))
    ids = torch.zeros((T, K), dtype=I32)
    off, ws = torch.zeros(E + 1, dtype=torch.int64), torch.zeros(1 << 16, dtype=torch.uint8)
    f = lambda: torch.zeros((T, K))                                                   # noqa: E731
    return {
        "route weights": lambda t: mx.mx_moe_route(logits, ids, t, True),
        "route_backward dweights": lambda t: mx.mx_moe_route_backward(logits, ids, t, logits),
        "combine weights": lambda t: mx.mx_moe_combine(z, ids, x, weights=t),
        "combine_backward weights": lambda t: mx.mx_moe_combine_backward(x, z, ids, t, z, f()),
        "combine_backward dweights": lambda t: mx.mx_moe_combine_backward(x, z, ids, f(), z, t),
        "sort rows": lambda t: mx.mx_moe_sort(ids, off, t.to(I32), None, ws),
    }


@pytest.mark.parametrize("name", sorted(calls()))
def test_values_of_choices_in_another_order_are_refused(name):
    call, what = calls()[name], name.split()[1]
    for shape in ((K, T), (T * K, 1), (1, T * K), (K, T, 1)):
        with pytest.raises(ValueError, match=rf"{what} must be \[{T}, {K}\], got"):
            call(torch.zeros(shape))
    # [tokens, top_k], a longer one's first rows and the same values in one row of memory go on to the refusal of the CPU
    for shape in ((T, K), (T + 3, K), (T * K,)):
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call(torch.zeros(shape))
    with pytest.raises(ValueError, match="holds .* bytes"):
        call(torch.zeros((T - 1, K)))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_weights_of_another_width_are_refused(dtype):
    x, dw, ws = torch.zeros((T, H), dtype=BF), torch.zeros(H), torch.zeros(1 << 16, dtype=torch.uint8)
    forward = lambda w: mx.mx_rmsnorm_mxfp8(x, w, 1e-6, y=x)                          # noqa: E731
    backward = lambda w: mx.mx_rmsnorm_backward(x, x, w, 1e-6, x, dw, ws)             # noqa: E731
    for call in (forward, backward):
        for n in (H - 8, H + 8, 2 * H):
            with pytest.raises(ValueError, match=rf"weight must be \[{H}\], got"):
                call(torch.ones(n, dtype=dtype))
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call(torch.ones(H, dtype=dtype))
