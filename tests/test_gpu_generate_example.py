"""GPU: the generation example runs the operators together; every step against dense torch on the dequantized weights
and the cached values read back (relative Frobenius error <= 1e-2, the bar of the GEMM tests)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOL = 1e-2


def load():
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def err(got, want):
    return float((got.double() - want.double()).norm() / want.double().norm())


def dense_check(ex, d, tokens, logits, lens, new):
    """The step's intermediate results recomputed in FP32 from its own inputs."""
    import microscaled_precision_numerics_gb300 as mx
    H, KV, D = d.heads, d.kv_heads, d.dim
    x = d.embedding[tokens]
    qkv = ex.norm(x).float() @ d.qkv.dequantized().float().t()
    assert err(d.trace["qkv"].flatten(1), qkv) <= TOL
    start, want = 0, torch.zeros_like(d.trace["attended"], dtype=torch.float32)
    for r, (total, n) in enumerate(zip(lens, new)):
        at = torch.arange(total, device=x.device)
        slots = (d.table[r, at // d.page] * d.page + at % d.page).to(torch.int32)
        k, v = (torch.empty((total, KV, D), dtype=torch.bfloat16, device=x.device) for _ in range(2))
        mx.mx_nvfp4_kv_gather(d.cache, slots, d.s_k, d.s_v, k, v)
        assert torch.equal(slots[total - n:], d.trace["slots"][start:start + n])
        # the cache holds the step's keys and values to 4 bits: within half of the widest code gap (2 of 6) and
        # the scale's rounding (1/16) of the block's largest element
        fresh = d.trace["qkv"][start:start + n, H:H + KV].float()
        gap = fresh.view(n, KV, D // 16, 16).abs().amax(-1, keepdim=True).expand(n, KV, D // 16, 16).reshape(n, KV, D)
        assert ((k[total - n:].float() - fresh).abs() <= gap * (1 / 6 + 1 / 16 + 1 / 128)).all()
        q = d.trace["qkv"][start:start + n, :H].float()
        k, v = (t.float().repeat_interleave(H // KV, 1) for t in (k, v))
        s = torch.einsum("nhd,thd->hnt", q, k) * D ** -0.5
        s = s.masked_fill(at[None, :] > (total - n + torch.arange(n, device=x.device))[:, None], float("-inf"))
        want[start:start + n] = torch.einsum("hnt,thd->nhd", s.softmax(-1), v)
        start += n
    assert err(d.trace["attended"], want) <= TOL
    y = x.float() + (d.trace["attended"].flatten(1).float() @ d.o.dequantized().float().t()).to(torch.bfloat16).float()
    gate, up = (ex.norm(y.to(torch.bfloat16)).float() @ d.gate_up.dequantized().float().t()).chunk(2, -1)
    y = y.to(torch.bfloat16).float() + (torch.nn.functional.silu(gate) * up).to(torch.bfloat16).float() @ d.down.dequantized().float().t()
    assert err(d.trace["x"], y) <= TOL
    assert err(logits, ex.norm(d.trace["x"]).float() @ d.head.dequantized().float().t()) <= TOL


def test_generation_step_by_step():
    ex = load()
    prompts = [[5, 7, 11], list(range(40)), [1], list(range(100, 117))]
    d = ex.Decoder(4, longest=64)
    dev = d.lens.device
    new = [len(p) for p in prompts]
    tokens = torch.tensor([t for p in prompts for t in p], device=dev)
    lens = list(new)
    logits = d.step(tokens, torch.tensor(new, dtype=torch.int32, device=dev))
    dense_check(ex, d, tokens, logits, lens, new)
    for _ in range(3):                                                   # the third request idles: no tokens in these steps
        tokens = logits[d.q_start[1:].long() - 1].argmax(-1)[[0, 1, 3]] if len(new) == 4 and new[2] else logits.argmax(-1)
        new = [1, 1, 0, 1]
        lens = [a + b for a, b in zip(lens, new)]
        logits = d.step(tokens, torch.tensor(new, dtype=torch.int32, device=dev))
        assert d.lens.tolist() == lens and int(d.unplaced) == 0
        dense_check(ex, d, tokens, logits, lens, new)
    assert int(d.free_count) == 16 - sum(-(-n // d.page) for n in lens)


def test_example_main(capsys, monkeypatch):
    ex = load()
    monkeypatch.setattr("sys.argv", ["decode_step.py", "--steps", "3", "--requests", "3", "--hidden", "256"])
    ex.main()
    out = capsys.readouterr().out
    assert " 0 tokens without a page" in out and out.count("prompt tokens ->") == 3
