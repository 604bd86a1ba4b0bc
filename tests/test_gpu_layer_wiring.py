"""What meets before the norm's gradient in examples/experts_layer.py: the experts' rows brought back to their tokens and the router's
path, against 64 bits of both, with a bound far below either, so that a path left out or taken twice shows."""
import numpy as np
import pytest
import torch

import layer_ref as ref
from test_gpu_layer_example import example, host           # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,hidden,experts,top_k", [(1, 256, 8, 2), (77, 512, 8, 2), (300, 256, 16, 4)])
def test_gradient_of_the_norms_output_is_the_experts_and_the_routers(example, tokens, hidden, experts, top_k):        # noqa: F811
    torch.manual_seed(13)
    layer = example.Layer(hidden, 256, experts, top_k, seed=15)
    x, res, dout = (torch.randn((tokens, hidden), device="cuda").to(torch.bfloat16) for _ in range(3))
    layer.forward(x, res)
    g, t = layer.backward(dout), layer.trace
    logits, router = host(g["logits"]), host(layer.router)
    by_router, size = logits @ router, np.abs(logits) @ np.abs(router)
    want, mag = ref.combine(host(g["rows"]), host(t["rows"]), None, by_router)
    # the router's product: experts + 2 roundings of FP32 and one to BF16; then combine's
    bound = (experts + 2) * ref.EPS32 * size + ref.HALF16 * np.abs(by_router)
    bound = 1.01 * bound + ref.HALF16 * (np.abs(want) + bound) + (top_k + 2) * 1.01 * ref.EPS32 * mag + ref.TINY16
    assert (np.abs(host(g["y"]) - want) <= bound).all()
    by_experts = want - by_router
    for path in (by_router, by_experts):
        assert np.linalg.norm(path) > 5 * np.linalg.norm(bound)
