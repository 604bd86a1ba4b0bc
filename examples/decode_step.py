"""Generation with NVFP4 weights and an NVFP4 key/value cache, by the library's calls alone for everything that
reads weights or cache: one decoder layer and an output head, random weights, a batch of requests of different lengths.

    python examples/decode_step.py [--steps 8] [--requests 4] [--hidden 512]

Each step makes the page and slot maps of the new tokens (mx_kv_slots, updating lengths and free pages in place),
projects them with NVFP4 weights (mx_nvfp4_matvec), writes keys and values into the cache (mx_nvfp4_kv_append), attends over it
(mx_nvfp4_kv_attention) and goes on through the output projection, the gated feed-forward and the head.  The first step
is the prompts', in slices of at most MX_MATVEC_MAX_TOKENS tokens.  Norms, activation and the choice of the next
token are plain torch.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import microscaled_precision_numerics_gb300 as mx


class Linear:
    """A weight [out, in] as NVFP4 rows: codes, GEMM-layout block scales, one FP32 scale per row."""

    def __init__(self, w):
        self.out, self.inp = w.shape
        self.w = mx.alloc_nvfp4_rows(self.out, self.inp, w.device)
        mx.mx_nvfp4_quantize_per_token(w, self.w["q"], self.w["s"], self.w["s2"])

    def __call__(self, x, dtype=torch.bfloat16):
        y = torch.empty((x.shape[0], self.out), dtype=dtype, device=x.device)
        for i in range(0, x.shape[0], mx.MX_MATVEC_MAX_TOKENS):
            part = slice(i, i + mx.MX_MATVEC_MAX_TOKENS)
            mx.mx_nvfp4_matvec(x[part], self.w["q"], self.w["s"], self.w["s2"], mx.MX_SCOPE_ROW, y[part])
        return y

    def dequantized(self):
        y = torch.empty((self.out, self.inp), dtype=torch.bfloat16, device=self.w["q"].device)
        mx.mx_dequantize_bf16(mx.MX_FMT_NVFP4, self.w["q"], self.w["s"], self.w["s2"], mx.MX_SCOPE_ROW, self.out, self.inp, y)
        return y


def norm(x):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Decoder:
    """One decoder layer over `requests` requests with a paged NVFP4 cache, and an output head."""

    def __init__(self, requests, hidden=512, heads=8, kv_heads=2, head_dim=64, ffn=1024, vocab=1000, longest=256, page=16, seed=0,
                 device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def weight(out, inp):
            return (torch.randn((out, inp), generator=g, device=device) * inp ** -0.5).to(torch.bfloat16)

        self.heads, self.kv_heads, self.dim, self.page = heads, kv_heads, head_dim, page
        self.embedding = weight(vocab, hidden)
        self.qkv = Linear(weight((heads + 2 * kv_heads) * head_dim, hidden))
        self.o = Linear(weight(hidden, heads * head_dim))
        self.gate_up = Linear(weight(2 * ffn, hidden))
        self.down = Linear(weight(hidden, ffn))
        self.head = Linear(weight(vocab, hidden))
        per = -(-longest // page)
        i32 = {"dtype": torch.int32, "device": device}
        self.cache = mx.alloc_nvfp4_kv_cache(requests * per, page, kv_heads, head_dim, device)
        self.s_k = torch.full((kv_heads,), 8.0 / 2688, device=device)     # covers |k|, |v| up to 8
        self.s_v = torch.full((kv_heads,), 8.0 / 2688, device=device)
        self.lens = torch.zeros(requests, **i32)
        self.table = torch.full((requests, per), -1, **i32)
        self.free = torch.arange(requests * per, **i32)
        self.free_count = torch.full((1,), requests * per, **i32)
        self.q_start = torch.zeros(requests + 1, **i32)
        self.unplaced = torch.zeros(1, **i32)
        self.workspace = torch.empty(mx.kv_attention_workspace_bytes(head_dim), dtype=torch.uint8, device=device)

    def step(self, tokens, new_lens, most_new=None):
        """Logits (FP32) of the new tokens: tokens [T] of all requests in order, new_lens [requests] how many each has (on the
        device), most_new the largest of them, which attention lays its work out for (T where it is not known)."""
        T, H, KV, D = tokens.numel(), self.heads, self.kv_heads, self.dim
        x = self.embedding[tokens]
        slots = torch.empty(T, dtype=torch.int32, device=x.device)
        positions = torch.empty_like(slots)
        mx.mx_kv_slots(self.lens, new_lens, self.page, self.table, self.free, self.free_count, self.q_start, self.lens, slots, positions,
                       self.free_count, self.unplaced)
        qkv = self.qkv(norm(x)).view(T, H + 2 * KV, D)
        mx.mx_nvfp4_kv_append(qkv[:, H:H + KV], qkv[:, H + KV:], slots, self.s_k, self.s_v, self.cache)
        attended = torch.empty((T, H, D), dtype=torch.bfloat16, device=x.device)
        mx.mx_nvfp4_kv_attention(qkv[:, :H], self.q_start, self.lens, self.table, self.cache, self.s_k, self.s_v, D ** -0.5,
                                 most_new or T, attended, self.workspace)
        x = x + self.o(attended.view(T, H * D))
        gate, up = self.gate_up(norm(x)).float().chunk(2, -1)
        x = x + self.down((torch.nn.functional.silu(gate) * up).to(torch.bfloat16))
        self.trace = {"qkv": qkv, "attended": attended, "slots": slots, "positions": positions, "x": x}
        return self.head(norm(x), torch.float32)


def generate(decoder, prompts, steps):
    """Greedy tokens [requests, steps] after the prompts (lists of token numbers)."""
    dev = decoder.lens.device
    new = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device=dev)
    logits = decoder.step(torch.tensor([t for p in prompts for t in p], device=dev), new, max(len(p) for p in prompts))
    last = logits[decoder.q_start[1:].long() - 1].argmax(-1)
    ones, out = torch.ones_like(new), []
    for _ in range(steps):
        out.append(last)
        last = decoder.step(last, ones, 1).argmax(-1)
    return torch.stack(out, 1)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--hidden", type=int, default=512)
    args = ap.parse_args()
    torch.manual_seed(1)
    decoder = Decoder(args.requests, hidden=args.hidden, longest=64 + args.steps)
    prompts = [torch.randint(1000, (int(n),)).tolist() for n in torch.randint(1, 60, (args.requests,))]
    tokens = generate(decoder, prompts, args.steps)
    mx.check_device_status()
    print(f"lengths {decoder.lens.tolist()}, {int(decoder.free_count)} pages free, {int(decoder.unplaced)} tokens without a page")
    for prompt, row in zip(prompts, tokens.tolist()):
        print(f"{len(prompt):3d} prompt tokens -> {row}")


if __name__ == "__main__":
    main()
