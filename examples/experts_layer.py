"""A feed-forward layer with routed experts in MXFP8, forward and backward, by the library's calls for everything between and
in the experts' products: random weights, a batch of tokens.

    python examples/experts_layer.py [--tokens 200] [--hidden 512] [--experts 8] [--top-k 2]

Forward: norm of the residual stream with its MXFP8 output (mx_rmsnorm_mxfp8), the router's choice (mx_moe_route), the tokens
sorted by expert (mx_moe_sort, mx_moe_dispatch_quantized), gate and up in one grouped product, the activation, down, and the
experts' rows back to their tokens with the router's weights and the residual (mx_moe_combine).  Backward: the same way back
(mx_moe_combine_backward, grouped products with the weights' column-wise copies, mx_moe_combine without weights,
mx_moe_route_backward, mx_rmsnorm_backward).  The roundings to MXFP8 count as the identity.  The router's product, the activation and
the experts' weight gradients are plain torch.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import microscaled_precision_numerics_gb300 as mx

EPS = 1e-6


class Experts:
    """Weights [experts, out, in] as MXFP8 for a grouped product (rows) and for its data gradient (columns)."""

    def __init__(self, w):
        self.w, (self.n, self.out, self.inp) = w, w.shape
        each = [mx.alloc_mxfp8(self.out, self.inp, w.device) for _ in range(self.n)]
        for one, o in zip(w, each):
            mx.mx_quantize_mxfp8(one, **o)
        self.q, self.s, self.qt, self.st = (torch.stack([o[k] for o in each]) for k in ("q_row", "s_row", "q_col", "s_col"))

    def __call__(self, offsets, q, s):
        return grouped(offsets, q, s, self.q, self.s, self.out, self.inp)

    def gradient(self, offsets, dy):
        return grouped(offsets, *quantize(offsets, dy), self.qt, self.st, self.inp, self.out)


def grouped(offsets, q, s, b, sb, n, k):
    d = torch.zeros((q.shape[0], n), dtype=torch.bfloat16, device=q.device)
    mx.mx_grouped_scaled_gemm(mx.MX_FMT_MXFP8, offsets, q, s, None, b, sb, None, n, k, d)
    return d


def quantize(offsets, x):
    """Expert-sorted rows as MXFP8 (codes, scales)."""
    rows, cols = x.shape
    q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    s = torch.empty(mx.grouped_scale_bytes(rows, offsets.numel() - 1, cols, 32), dtype=torch.uint8, device=x.device)
    mx.mx_quantize_mxfp8_grouped(x, offsets, q, s)
    return q, s


def activation(gate_up):
    gate, up = gate_up.float().chunk(2, -1)
    return (torch.nn.functional.silu(gate) * up).to(torch.bfloat16)


def activation_backward(gate_up, da):
    gate, up = gate_up.float().chunk(2, -1)
    s, da = torch.sigmoid(gate), da.float()
    return torch.cat([da * up * s * (1 + gate * (1 - s)), da * gate * s], -1).to(torch.bfloat16)


class Layer:
    def __init__(self, hidden=512, ffn=256, experts=8, top_k=2, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def weight(*shape):
            return (torch.randn(shape, generator=g, device=device) * shape[-1] ** -0.5).to(torch.bfloat16)

        self.hidden, self.experts, self.top_k = hidden, experts, top_k
        self.norm = torch.ones(hidden, device=device)
        self.router = weight(experts, hidden)
        self.gate_up, self.down = Experts(weight(experts, 2 * ffn, hidden)), Experts(weight(experts, hidden, ffn))

    def forward(self, x, residual):
        """The residual stream behind the layer (BF16 [tokens, hidden]): x + residual + what the experts add."""
        T, H, G, k, dev = x.shape[0], self.hidden, self.experts, self.top_k, x.device
        t = self.trace = {"x": x, "residual": residual}
        e = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device=dev)      # noqa: E731
        codes = mx.alloc_mxfp8(T, H, dev, colwise=False)
        t["sum"], t["y"] = e(T, H), e(T, H)
        mx.mx_rmsnorm_mxfp8(x, self.norm, EPS, residual=residual, sum_out=t["sum"], y=t["y"], **codes)
        t["logits"] = t["y"].float() @ self.router.float().t()
        t["ids"], t["weights"] = e(T, k, dtype=torch.int32), e(T, k, dtype=torch.float32)
        mx.mx_moe_route(t["logits"], t["ids"], t["weights"])
        t["offsets"], t["rows"], t["source"] = e(G + 1, dtype=torch.int64), e(T, k, dtype=torch.int32), e(T * k, dtype=torch.int32)
        mx.mx_moe_sort(t["ids"], t["offsets"], t["rows"], t["source"], e(mx.moe_sort_workspace_bytes(T * k, G), dtype=torch.uint8))
        t["q"], t["s"] = e(T * k, H, dtype=torch.uint8), e(mx.grouped_scale_bytes(T * k, G, H, 32), dtype=torch.uint8)
        mx.mx_moe_dispatch_quantized(mx.MX_FMT_MXFP8, codes["q_row"], codes["s_row"], t["rows"], t["offsets"], t["q"], t["s"])
        t["gate_up"] = self.gate_up(t["offsets"], t["q"], t["s"])
        t["act"] = activation(t["gate_up"])
        t["z"] = self.down(t["offsets"], *quantize(t["offsets"], t["act"]))
        t["out"] = e(T, H)
        mx.mx_moe_combine(t["z"], t["rows"], t["out"], weights=t["weights"], residual=t["sum"])
        return t["out"]

    def backward(self, dout):
        """Gradients {name: tensor}; dx is that of x and of the residual alike."""
        t, T, k, dev = self.trace, dout.shape[0], self.top_k, dout.device
        g = {}
        g["z"], g["weights"] = torch.zeros_like(t["z"]), torch.empty_like(t["weights"])
        mx.mx_moe_combine_backward(dout, t["z"], t["rows"], t["weights"], g["z"], g["weights"])
        g["act"] = self.down.gradient(t["offsets"], g["z"])
        g["gate_up"] = activation_backward(t["gate_up"], g["act"])
        g["rows"] = self.gate_up.gradient(t["offsets"], g["gate_up"])
        g["logits"] = torch.empty_like(t["logits"])
        mx.mx_moe_route_backward(t["logits"], t["ids"], g["weights"], g["logits"])
        by_router = (g["logits"] @ self.router.float()).to(torch.bfloat16)
        g["y"] = torch.empty_like(dout)
        mx.mx_moe_combine(g["rows"], t["rows"], g["y"], residual=by_router)
        g["dx"], g["norm"] = torch.empty_like(dout), torch.empty_like(self.norm)
        ws = torch.empty(mx.rmsnorm_workspace_bytes(T, self.hidden), dtype=torch.uint8, device=dev)
        mx.mx_rmsnorm_backward(g["y"], t["sum"], self.norm, EPS, g["dx"], g["norm"], ws, dsum=dout)
        g["router"] = g["logits"].t() @ t["y"].float()
        token = t["source"].long().clamp(min=0) // k
        ends = t["offsets"].tolist()
        g["down"] = torch.stack([g["z"][a:b].float().t() @ t["act"][a:b].float() for a, b in zip(ends, ends[1:])])
        g["up"] = torch.stack([g["gate_up"][a:b].float().t() @ t["y"][token[a:b]].float() for a, b in zip(ends, ends[1:])])
        return g


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=200)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--top-k", type=int, default=2)
    args = ap.parse_args()
    torch.manual_seed(1)
    layer = Layer(args.hidden, experts=args.experts, top_k=args.top_k)
    x, residual = (torch.randn((args.tokens, args.hidden), device="cuda").to(torch.bfloat16) for _ in range(2))
    out = layer.forward(x, residual)
    grads = layer.backward(torch.ones_like(out))
    mx.check_device_status()
    size = (layer.trace["offsets"][1:] - layer.trace["offsets"][:-1]).tolist()
    print(f"{args.tokens} tokens, {args.top_k} of {args.experts} experts each; tokens of each expert: {size}")
    for name, v in grads.items():
        print(f"  d{name:8s} {tuple(v.shape)}, norm {float(v.float().norm()):.4f}")


if __name__ == "__main__":
    main()
