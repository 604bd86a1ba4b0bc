"""GPU: attention over the NVFP4 cache at the edges of its arithmetic and arguments.  Against the 64-bit reference; bounds as in
test_gpu_generate.py, with the term of small probabilities derived anew where it is used."""
import numpy as np
import pytest
import torch

import generate_ref as ref
from gpu_util import DEV, bf16_dev, to_np_u16
from test_gpu_generate import attention_case, check_attention, done, f32, i32, mx, wide    # noqa: F401  (mx is the fixture)
from test_gpu_generate_example import load

pytestmark = pytest.mark.gpu


def sink_case(D, L, new, group, kv, page, nats, *sinks, zero=True):
    """One request: keys are zero but for the positions `sinks`, which score `nats` (a little more from head to head); their values
    are zero and all others are positive, so the output is made of small probabilities alone."""
    rng = np.random.default_rng(L + D)
    width = -(-L // page)
    codes_v, one = rng.integers(1, 8, (width * page, kv, D)).astype(np.uint8), 0x38           # 0x38: E4M3 1.0
    if zero:
        codes_v[list(sinks)] = 0
    codes_k = np.zeros_like(codes_v)
    codes_k[list(sinks)] = 6                                                                  # 4.0
    cache = np.zeros((width, kv, page // 16, 18 * D), np.uint8)
    order = rng.permutation(width)
    for j in range(width * page):
        r, i = cache[order[j // page], :, j % page // 16], j % 16
        r[:, i * (D // 2):(i + 1) * (D // 2)] = ref.pack(codes_k[j])
        r[:, 8 * D + i * (D // 16):8 * D + (i + 1) * (D // 16)] = one
        r[:, 9 * D + i * (D // 2):9 * D + (i + 1) * (D // 2)] = ref.pack(codes_v[j])
        r[:, 17 * D + np.arange(D // 16) * 16 + ref.v_scale_position(i)] = one
    scale = D ** -0.5
    s_k, s_v = np.full(kv, nats / (scale * D * 4), np.float32), np.full(kv, 1 / 6, np.float32)
    q = np.ones((new, kv * group, D)) * (1 + np.arange(kv * group) / 64)[None, :, None]
    return bf16_dev(ref.bf16_bits(q)), [0, new], [L], order[None, :], torch.from_numpy(cache).to(DEV), s_k, s_v, scale


SINKS = [(64, 384, 1, 4, 1, 16, 0), (64, 384, 5, 4, 1, 32, 0), (128, 383, 1, 8, 2, 16, 0), (128, 380, 3, 4, 2, 16, 0), (256, 384, 1, 2, 1, 16, 0),
         (256, 384, 5, 2, 1, 16, 0),
         (128, 1000, 1, 4, 1, 16, 0),                                       # divided inside a cluster
         (64, 2000, 2, 4, 2, 16, 20000)]                                    # split over the GPU


@pytest.mark.parametrize("nats", [3e4, 2e7, 1e10, 1e20])
@pytest.mark.parametrize("D,L,new,group,kv,page,more", SINKS)
def test_large_scores(mx, D, L, new, group, kv, page, more, nats):       # noqa: F811
    """Two equal keys whose scores are so large that their products with scale and log2 e differ by rounding alone: each
    has half of the weight all the same, so the output is the mean of two values, off by 2^-11 of it (P) and BF16's rounding."""
    q, q_start, lens, table, cache, s_k, s_v, scale = sink_case(D, L, new, group, kv, page, nats, 5, L // 2, zero=False)
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float32, device=DEV)
    ws = torch.empty(mx.kv_attention_workspace_bytes(D), dtype=torch.uint8, device=DEV)
    mx.mx_nvfp4_kv_attention(q, i32(q_start), i32(lens), i32(wide(table, more // page)), cache, f32(s_k), f32(s_v), scale, new, out, ws, lse=lse)
    done(mx)
    o, l, _, _ = ref.attention(ref.bf16_value(to_np_u16(q)).astype(np.float64), q_start, lens, table, cache.cpu().numpy(), s_k, s_v, scale, page)
    assert (np.abs(out.float().cpu().numpy() - o) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(o)).all()
    # FP32: the sum of D products, three scalings, the product with ln 2
    assert (np.abs(lse.cpu().numpy() - l) <= (D + 6) * 2.0 ** -24 * np.abs(l)).all()


@pytest.mark.parametrize("nats", [16.6, 17.0, 17.7, 18.5])
@pytest.mark.parametrize("D,L,new,group,kv,page,more", SINKS)
def test_small_probabilities_beside_a_large_one(mx, D, L, new, group, kv, page, more, nats):       # noqa: F811
    """The probabilities of all but one position are 2^-24 to 2^-27 of the largest.  Each enters the second product as FP16
    of 2^7 times itself relative to the running maximum: off by 2^-11 relatively or 2^-25 absolutely, which is 2^-32 of the
    largest, so |error of o| <= (4 eps + 2^-10 + n 2^-24) mix + n 2^-32 max|v| + 2^-8 |o|."""
    for sink in (0, L // 2):
        q, q_start, lens, table, cache, s_k, s_v, scale = sink_case(D, L, new, group, kv, page, nats, sink)
        out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
        lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float32, device=DEV)
        ws = torch.empty(mx.kv_attention_workspace_bytes(D), dtype=torch.uint8, device=DEV)
        mx.mx_nvfp4_kv_attention(q, i32(q_start), i32(lens), i32(wide(table, more // page)), cache, f32(s_k), f32(s_v), scale, new, out, ws, lse=lse)
        done(mx)
        o, l, mix, reach = ref.attention(ref.bf16_value(to_np_u16(q)).astype(np.float64), q_start, lens, table, cache.cpu().numpy(), s_k, s_v,
                                         scale, page)
        eps = (D + 4) * 2.0 ** -24 * reach + 2.0 ** -23 * (np.abs(l) + np.log(L) + reach)
        vmax = 6 * float(np.max(s_v))
        bound = (4 * eps[..., None] + 2.0 ** -10 + L * 2.0 ** -24) * mix + L * 2.0 ** -32 * vmax + 2.0 ** -8 * 1.01 * np.abs(o)
        got = out.float().cpu().numpy().astype(np.float64)
        bad = ~(np.abs(got - o) <= bound)
        assert not bad.any(), f"sink {sink}: {int(bad.sum())} of {bad.size} off, {got[bad][0]} want {o[bad][0]} within {bound[bad][0]}"
        bad = ~(np.abs(lse.cpu().numpy() - l) <= eps + 2.0 ** -20 + L * 2.0 ** -24 + 2.0 ** -22 * np.abs(l))
        assert not bad.any()


@pytest.mark.parametrize("window", [0, 30])
@pytest.mark.parametrize("heads,kv,D", [(4, 4, 64), (8, 2, 128), (4, 1, 256)])
def test_max_q_below_the_new_tokens(mx, heads, kv, D, window):       # noqa: F811
    """A max_q below a request's new tokens: its first max_q rows are as with all of them, later ones are not written."""
    page, new = 16, [5, 1, 7, 3]
    q, q_start, lens, table, cache, s_k, s_v = attention_case(31, [90, 33, 40, 3], new, heads, kv, D, page)
    o, l, mix, reach = ref.attention(ref.bf16_value(to_np_u16(q)).astype(np.float64), q_start, lens, table, cache.cpu().numpy(), s_k, s_v,
                                     D ** -0.5, page, window)
    ws = torch.empty(mx.kv_attention_workspace_bytes(D), dtype=torch.uint8, device=DEV)
    for max_q in (1, 2, 4):
        out = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full(q.shape[:2], 9.0, dtype=torch.float32, device=DEV)
        for tab in (table, wide(table, 200)):
            mx.mx_nvfp4_kv_attention(q, i32(q_start), i32(lens), i32(tab), cache, f32(s_k), f32(s_v), D ** -0.5, max_q, out, ws, lse=lse,
                                     window=window)
            done(mx)
            kept = np.concatenate([s + np.arange(min(n, max_q)) for s, n in zip(q_start, new)])
            rest = np.setdiff1d(np.arange(len(o)), kept)
            got, got_l = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
            assert (got[rest] == 9).all() and (got_l[rest] == 9).all()
            eps = ((D + 4) * 2.0 ** -24 * reach + 2.0 ** -23 * (np.abs(l) + np.log(90) + reach))[kept]
            bound = (4 * eps[..., None] + 2.0 ** -10 + 90 * 2.0 ** -24) * mix[kept] + 90 * 2.0 ** -32 * 6 * 448 * s_v.max() + 2.0 ** -8 * 1.01 * np.abs(o[kept])
            assert (np.abs(got - o)[kept] <= bound + 1e-30).all()
            assert (np.abs(got_l - l)[kept] <= eps + 2.0 ** -20 + 90 * 2.0 ** -24 + 2.0 ** -22 * np.abs(l[kept])).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 3])
def test_nan_value_of_small_probability(mx, D, new):       # noqa: F811
    """A NaN among the values reaches every row that attends to its position, whatever its probability and wherever the position lies:
    in the last tile, part of which is masked, as in one that is not."""
    L, group, kv, page = 148, 4, 2, 16
    q, q_start, lens, table, cache, s_k, s_v, scale = sink_case(D, L, new, group, kv, page, 40.0, 3)      # the rest at 2^-57
    args = (i32(q_start), i32(lens), i32(table))
    ws = torch.empty(mx.kv_attention_workspace_bytes(D), dtype=torch.uint8, device=DEV)

    def attend(c, window):
        out = torch.zeros_like(q)
        mx.mx_nvfp4_kv_attention(q, *args, c, f32(s_k), f32(s_v), scale, new, out, ws, window=window)
        done(mx)
        return out

    for window in (0, 146):                                                 # 146: the first tile is masked in part
        base = attend(cache, window)
        assert base.isfinite().all()
        for tok in (2, 4, 20, 100, 127, 128, 140, L - 2, L - 1):
            hurt = cache.clone()
            hurt[int(table[0, tok // page]), 1, 0, 17 * D + ref.v_scale_position(tok % 16)] = 0x7F        # block 0 of kv head 1
            out = attend(hurt, window)
            for t in range(new):
                pos = L - new + t
                sees = tok <= pos and (window == 0 or tok > pos - window)
                assert out[t, group:, :16].isnan().all() == sees and out[t, group:, :16].isnan().any() == sees, (tok, t)
                assert torch.equal(out[t, group:, 16:], base[t, group:, 16:]) and torch.equal(out[t, :group], base[t, :group])


@pytest.mark.parametrize("scale", [0.0, 0.1])
@pytest.mark.parametrize("scale_v", [1e-34, 1e-36, 1e33])
@pytest.mark.parametrize("lens,new,heads,kv,D,page,more", [([300, 40], [1, 1], 8, 2, 64, 16, 0), ([300, 40], [3, 2], 8, 2, 128, 16, 0),
                                                           ([900], [1], 8, 2, 128, 16, 0), ([1500, 700], [2, 1], 8, 2, 256, 16, 20000)])
def test_value_scales_near_the_ends_of_fp32(mx, lens, new, heads, kv, D, page, more, scale_v, scale):       # noqa: F811
    """S_v so small that divided by the sum of the probabilities, most of all of equal ones, it would have few bits left or none."""
    q, q_start, lens, table, cache, s_k, s_v = attention_case(41, lens, new, heads, kv, D, page, scale_v=scale_v)
    out, _ = check_attention(mx, q, q_start, lens, wide(table, more // page), cache, s_k, s_v, scale, page, host_cache=cache.cpu().numpy())
    want, l, mix, reach = ref.attention(ref.bf16_value(to_np_u16(q)).astype(np.float64), q_start, lens, table, cache.cpu().numpy(), s_k, s_v, scale, page)
    # check_attention's bound has a floor of 1e-30 for zeros, which is above these outputs; BF16's smallest step here instead
    n = int(max(lens))
    eps = (D + 4) * 2.0 ** -24 * reach + 2.0 ** -23 * (np.abs(l) + np.log(n) + reach)
    bound = (4 * eps[..., None] + 2.0 ** -10 + n * 2.0 ** -24) * mix + n * 2.0 ** -32 * 6 * 448 * s_v.max() + 2.0 ** -8 * 1.01 * np.abs(want) + 2.0 ** -133
    assert (np.abs(out.float().cpu().numpy() - want) <= bound).all()


def test_example_passes_the_largest_number_of_new_tokens(mx, monkeypatch):       # noqa: F811
    """max_q of the example's attention calls: the longest prompt, then one token a request, not the whole batch's tokens."""
    ex, seen = load(), []
    real = ex.mx.mx_nvfp4_kv_attention
    monkeypatch.setattr(ex.mx, "mx_nvfp4_kv_attention", lambda *a, **k: (seen.append(a[8]), real(*a, **k))[1])
    prompts = [[5, 7, 11], [1], list(range(17))]
    tokens = ex.generate(ex.Decoder(3, longest=32), prompts, 3)
    done(mx)
    assert seen == [17, 1, 1, 1]
    # a step that is not told takes the batch's number of tokens, which is never too small, and gives the same tokens
    d = ex.Decoder(3, longest=32)
    new = torch.tensor([3, 1, 17], dtype=torch.int32, device=DEV)
    logits = d.step(torch.tensor([t for p in prompts for t in p], device=DEV), new)
    assert seen[-1] == 21 and torch.equal(logits[d.q_start[1:].long() - 1].argmax(-1), tokens[:, 0])
