"""The layer with routed experts of examples/experts_layer.py: every link of its forward and backward against 64-bit forms of
the link on the tensors that went into it, and the whole gradient against differences of a 64-bit layer over the values that the
codes stand for."""
import os
import sys

import numpy as np
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import experts_layer
    return experts_layer


def host(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def dequantized(mx, q, s, rows, cols):
    y = torch.empty((rows, cols), dtype=torch.bfloat16, device=q.device)
    mx.mx_dequantize_bf16(mx.MX_FMT_MXFP8, q, s, None, mx.MX_SCOPE_NONE, rows, cols, y)
    return host(y)


def fake(mx, x):
    """The values that the row-wise MXFP8 codes of x stand for."""
    o = mx.alloc_mxfp8(x.shape[0], x.shape[1], x.device, colwise=False)
    mx.mx_quantize_mxfp8(x.contiguous(), **o)
    return dequantized(mx, o["q_row"], o["s_row"], *x.shape)


def product_near(got, a, b, what):
    """The bar of the products' own tests: a relative Frobenius error of at most 1e-2."""
    want = a @ b.T
    err = np.linalg.norm(host(got) - want) / np.linalg.norm(want)
    assert err <= 1e-2, (what, err)


@pytest.mark.parametrize("tokens,hidden,experts,top_k", [(1, 256, 8, 2), (77, 512, 8, 2), (300, 256, 16, 4)])
def test_layer_link_by_link(example, tokens, hidden, experts, top_k):
    mx = example.mx
    torch.manual_seed(3)
    layer = example.Layer(hidden, 256, experts, top_k, seed=5)
    x, res, dout = (torch.randn((tokens, hidden), device="cuda").to(torch.bfloat16) for _ in range(3))
    layer.forward(x, res)
    g, t = layer.backward(dout), layer.trace
    mx.check_device_status()
    h, _, y = ref.norm(host(x), 1.0, example.EPS, host(res))
    assert np.array_equal(host(t["sum"]), h)
    assert (np.abs(host(t["y"]) - y) <= np.abs(y) * (ref.HALF16 + 24 * ref.EPS32) + ref.TINY16).all()
    ids, w = ref.route(host(t["logits"]), top_k, True)
    assert np.array_equal(host(t["ids"]), ids) and (np.abs(host(t["weights"]) - w) <= 1e-5 * w).all()
    offsets, rows, source = ref.sort(ids, experts)
    assert np.array_equal(host(t["offsets"]), offsets) and np.array_equal(host(t["rows"]), rows)
    token = source // top_k
    y_fake = fake(mx, t["y"])
    for e in range(experts):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        part = slice(int(a), int(b))
        wu, wd = (fake(mx, m.w[e]) for m in (layer.gate_up, layer.down))
        # the data gradients read the weights by columns, quantized along the other axis
        wut, wdt = (fake(mx, m.w[e].t()) for m in (layer.gate_up, layer.down))
        product_near(t["gate_up"][part], y_fake[token[part]], wu, "gate_up")
        product_near(t["z"][part], fake(mx, t["act"][part]), wd, "down")
        product_near(g["act"][part], fake(mx, g["z"][part]), wdt, "down's gradient")
        product_near(g["rows"][part], fake(mx, g["gate_up"][part]), wut, "gate_up's gradient")
    out, mag = ref.combine(host(t["z"]), rows, host(t["weights"]), host(t["sum"]))
    assert (np.abs(host(t["out"]) - out) <= ref.HALF16 * np.abs(out) + (top_k + 2) * 1.01 * ref.EPS32 * mag + ref.TINY16).all()
    dz, dw, mag = ref.combine_backward(host(dout), host(t["z"]), rows, host(t["weights"]), np.zeros(t["z"].shape))
    assert (np.abs(host(g["z"]) - dz) <= (ref.HALF16 + 1.01 * ref.EPS32) * np.abs(dz)).all()
    assert (np.abs(host(g["weights"]) - dw) <= 60 * ref.EPS32 * mag).all()
    dlogits, mag = ref.route_backward(host(t["logits"]), ids, host(g["weights"]), True)
    assert (np.abs(host(g["logits"]) - dlogits) <= 300 * ref.EPS32 * mag + 1e-30).all()
    dx, dnorm, bound, size = ref.norm_backward(host(g["y"]), host(t["sum"]), 1.0, example.EPS, host(dout))
    assert (np.abs(host(g["dx"]) - dx) <= bound).all()
    assert (np.abs(host(g["norm"]) - dnorm) <= (tokens + 32) * ref.EPS32 * size + 1e-30).all()


def test_whole_gradient_against_differences(example):
    """The layer in 64 bits without any rounding: its directional derivatives by differences, against the example's gradients.  Each of
    the backward's five tensors on the way carries an MXFP8 rounding of at most 2^-4 of a value; over thousands of values their
    errors are independent, so the directional derivative is off by less than 2^-4 of the gradient's norm along a random
    direction, five times over."""
    torch.manual_seed(7)
    layer = example.Layer(256, 256, 8, 2, seed=9)
    x, res, dout = (torch.randn((64, 256), device="cuda").to(torch.bfloat16) for _ in range(3))
    layer.forward(x, res)
    g, t = layer.backward(dout), layer.trace
    ids = torch.from_numpy(host(t["ids"])).long()
    up, down, router = (torch.from_numpy(host(v)) for v in (layer.gate_up.w, layer.down.w, layer.router))

    def loss(h, w):
        y = h / (h.pow(2).mean(-1, keepdim=True) + example.EPS).sqrt() * w
        weights = torch.softmax((y @ router.t()).gather(1, ids), -1)
        out = h.clone()
        for j in range(2):
            gu = torch.einsum("toh,th->to", up[ids[:, j]], y)
            gate, u = gu.chunk(2, -1)
            out = out + weights[:, j, None] * torch.einsum("tho,to->th", down[ids[:, j]], torch.nn.functional.silu(gate) * u)
        return float((out * torch.from_numpy(host(dout))).sum())

    h, w = torch.from_numpy(host(t["sum"])), torch.from_numpy(host(layer.norm))
    gen = torch.Generator().manual_seed(11)
    for which, grad in ((0, g["dx"]), (1, g["norm"])):
        for _ in range(3):
            v = torch.randn((h, w)[which].shape, generator=gen, dtype=torch.float64)
            at = lambda s: loss(h + s * v, w) if which == 0 else loss(h, w + s * v)                # noqa: B023, E731
            slope, got = (at(1e-4) - at(-1e-4)) / 2e-4, float((torch.from_numpy(host(grad)) * v).sum())
            norm = float(grad.double().norm())
            assert abs(got - slope) <= 5 * 2.0 ** -4 * norm, (which, got, slope, norm)


def test_example_runs(example, monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["experts_layer.py", "--tokens", "33", "--hidden", "256"])
    example.main()
    assert "tokens of each expert" in capsys.readouterr().out
