"""GPU: the generation operators on runs as long as those that they are made for -- contexts whose page look-ups are
refilled many times, pieces joined in several passes, weights whose rows a CTA takes in several turns, activations staged in
stretches -- against 64-bit references computed on the device.

Bounds as in test_gpu_generate.py, where they are derived, but for two terms that grow with the length there.
Sums: no FP32 sum here is one chain over the n positions.  A warp sums what it has of its CTA's run and the joins add four
warps and the pieces, so with c = positions of a warp + 4 + pieces (chain() below) c 2^-24 takes the place of n 2^-24.
Small probabilities: each enters the second product as FP16 of 2^7 times itself relative to the running maximum, off by
2^-25 absolutely at most, so n 2^-32 max|v| takes the place of n 2^-24 max|v|."""
import numpy as np
import pytest
import torch

import generate_ref as ref
from gpu_util import DEV
from test_gpu_generate import done, f32, i32, mx, ref_places    # noqa: F401  (mx is the fixture)

pytestmark = pytest.mark.gpu


def table_of(values):
    return torch.from_numpy(np.asarray(values)).to(DEV)


def make_cache(g, pages, page, kv, D):
    """A random cache, with value magnitudes that differ by token, and its values [pages * page tokens, kv, D] left in bytes:
    decode() reads them back by the layout's definition."""
    cache = torch.randint(0, 256, (pages, kv, page // 16, 18 * D), generator=g, dtype=torch.uint8, device=DEV)
    scales = torch.randint(0x30, 0x40, (2, pages, kv, page // 16, D), generator=g, dtype=torch.uint8, device=DEV)     # 0.5 .. 1.875
    cache[..., 8 * D:9 * D], cache[..., 17 * D:] = scales[0], scales[1]
    return cache


def decode(cache, pages, page):
    """K and V of the pages in this order, [kv, tokens, D] in 64 bits; a negative page gives zeros."""
    _, kv, groups, record = cache.shape
    D = record // 18
    rec = cache[pages.clamp(min=0)].permute(1, 0, 2, 3).reshape(kv, -1, record)                  # [kv, groups, record]
    e2m1, e4m3 = table_of(ref.E2M1_16), table_of(ref.E4M3)
    place = torch.tensor([ref.v_scale_position(i) for i in range(16)], device=DEV)

    def values(codes, scales):                                                                    # [kv, groups, 16, D / 2], [.., D / 16]
        v = e2m1[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
        return (v.unflatten(-1, (-1, 16)) * e4m3[scales.int()][..., None]).flatten(-2).flatten(1, 2)

    K = values(rec[..., :8 * D].unflatten(-1, (16, -1)), rec[..., 8 * D:9 * D].unflatten(-1, (16, -1)))
    V = values(rec[..., 9 * D:17 * D].unflatten(-1, (16, -1)), rec[..., 17 * D:].unflatten(-1, (-1, 16))[..., place].transpose(-1, -2))
    return K, V


def attend(q, q_start, lens, table, cache, s_k, s_v, scale, page, window):
    """out, lse, mix and reach (as ref.attention's) in 64 bits, request by request; a table of device integers."""
    T, heads, D = q.shape
    kv = cache.shape[1]
    f = dict(dtype=torch.float64, device=DEV)
    out, mix = torch.zeros((T, heads, D), **f), torch.zeros((T, heads, D), **f)
    lse, reach = torch.full((T, heads), -np.inf, **f), torch.zeros((T, heads), **f)
    for r, L in enumerate(lens):
        lo, hi = int(q_start[r]), int(q_start[r + 1])
        L, n = int(L), hi - lo
        if n == 0 or L == 0:
            continue
        pages = table[r, :-(-L // page)].long()
        K, V = decode(cache, pages, page)
        K, V = K[:, :L] * s_k.double()[:, None, None], V[:, :L] * s_v.double()[:, None, None]
        there = (pages >= 0).repeat_interleave(page)[:L]
        at, pos = torch.arange(L, device=DEV), L - n + torch.arange(n, device=DEV)
        seen = there[None, :] & (at[None, :] <= pos[:, None]) & (at[None, :] > pos[:, None] - (window or L + n))
        x = q[lo:hi].double().view(n, kv, heads // kv, D).permute(1, 0, 2, 3)                    # [kv, n, group, D]
        z = torch.einsum("kngd,ktd->kngt", x, K) * scale
        z = z.masked_fill(~seen[None, :, None, :], float("-inf"))
        top = z.amax(-1, keepdim=True).clamp(min=-1e300)
        p = torch.exp(z - top)
        l = p.sum(-1, keepdim=True)
        put = lambda to, v: to[lo:hi].copy_(v.permute(1, 0, 2, 3).reshape(n, heads, -1).reshape(to[lo:hi].shape))    # noqa: E731
        put(out, torch.einsum("kngt,ktd->kngd", p, V) / l.clamp(min=1e-300))
        put(mix, torch.einsum("kngt,ktd->kngd", p, V.abs()) / l.clamp(min=1e-300))
        put(lse, top + torch.log(l))
        a = torch.einsum("kngd,ktd->kngt", x.abs(), K.abs()) * abs(scale)
        put(reach, a.masked_fill(~seen[None, :, None, :], 0.0).amax(-1, keepdim=True))
        del K, V, z, p, a
    return out, lse, mix, reach


def chain(lens, kv, col_tiles):
    """Positions of a warp, four warps and all pieces: at least two CTAs an SM share the tiles, of which an item has at most 16
    more than its context has; a warp takes a quarter of a CTA's, one more for the remainder, 32 positions each."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = sum((-(-int(n) // 32) + 16) * kv * col_tiles for n in lens)
    run = max(-(-tiles // (2 * sms - 4)), 8)
    return 32 * (run // 4 + 2) + 4 + 4 * sms


def check_long(mx, seed, lens, new, heads, kv, D, page, window=0, missing=(), late=False):       # noqa: F811
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    lens, new = np.asarray(lens), np.asarray(new)
    per = -(-lens // page)
    pages = int(per.sum()) + 2
    order = torch.randperm(pages, generator=g, device=DEV)
    table = torch.full((len(lens), int(per.max()) + 1), -1, dtype=torch.int32, device=DEV)
    first = np.concatenate([[0], np.cumsum(per)])
    for r in range(len(lens)):
        table[r, :per[r]] = order[first[r]:first[r + 1]].int()
    cache = make_cache(g, pages, page, kv, D)
    if late:                                                              # block scales of the keys grow along each context from 0.5 to 3.75
        for r in range(len(lens)):
            step = torch.arange(int(per[r]), device=DEV) * 24 // max(1, int(per[r]))
            cache[table[r, :per[r]].long(), :, :, 8 * D:9 * D] = (0x30 + step).to(torch.uint8)[:, None, None, None]
    for r, column in missing:
        table[r, column] = -1
    q_start = np.concatenate([[0], np.cumsum(new)])
    q = torch.randn((int(q_start[-1]), heads, D), generator=g, device=DEV).to(torch.bfloat16)
    s_k = (1 + torch.rand(kv, generator=g, device=DEV)) / 3
    s_v = (1 + torch.rand(kv, generator=g, device=DEV)) / 3
    out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), dtype=torch.float32, device=DEV)
    ws = torch.full((mx.kv_attention_workspace_bytes(D),), 255, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    mx.mx_nvfp4_kv_attention(q, i32(q_start), i32(lens), table, cache, s_k, s_v, D ** -0.5, int(new.max()), out, ws, lse=lse, window=window)
    done(mx)
    o, l, mix, reach = attend(q, q_start, lens, table, cache, s_k, s_v, D ** -0.5, page, window)
    group = heads // kv
    n, c = int(lens.max()), chain(lens, kv, -(-int(new.max()) * group // 8))
    empty = l == -np.inf
    assert torch.equal(lse == -np.inf, empty) and not out[empty].any()
    lf = torch.where(empty, torch.zeros_like(l), l)
    eps = (D + 4) * 2.0 ** -24 * reach + 2.0 ** -23 * (lf.abs() + np.log(n) + reach)
    bound = (4 * eps[..., None] + 2.0 ** -10 + c * 2.0 ** -24) * mix + n * 2.0 ** -32 * 6 * 1.875 * float(s_v.max()) + 2.0 ** -8 * 1.01 * o.abs() + 1e-30
    bad = ~((out.double() - o).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off: {out[bad][:3].tolist()} want {o[bad][:3].tolist()} within {bound[bad][:3].tolist()}"
    bad = ~(torch.where(empty, torch.zeros_like(l), lse.double() - l).abs() <= eps + 2.0 ** -20 + c * 2.0 ** -24 + 2.0 ** -22 * lf.abs())
    assert not bad.any(), f"lse: {int(bad.sum())} of {bad.numel()} off: {lse[bad][:3].tolist()} want {l[bad][:3].tolist()}"


def ragged(seed, n, lo, hi):
    lens = np.random.default_rng(seed).integers(lo, hi + 1, n)
    lens[-1] = hi
    return lens


@pytest.mark.parametrize("D,heads,kv,page,drafts,window", [(128, 32, 8, 16, 1, 0), (64, 32, 8, 64, 1, 0), (256, 8, 4, 32, 1, 0),       # one fragment
                                                           (128, 32, 4, 32, 2, 0), (64, 32, 8, 16, 4, 0), (256, 8, 4, 16, 5, 0),  # two
                                                           (128, 32, 8, 128, 1, 5000), (64, 32, 4, 32, 6, 4000)])
@pytest.mark.parametrize("late", [False, True])
def test_batch_of_long_contexts(mx, D, heads, kv, page, drafts, window, late):       # noqa: F811
    """Hundreds of tiles a CTA: each warp refills its look-ups several times.  Pages are missing on both sides of such a
    refill.  With late maxima the running one is raised all along the contexts."""
    lens = ragged(D, 48, 2000, 8192)
    new = np.random.default_rng(drafts).integers(1, drafts + 1, 48)
    missing = [(3, int(lens[3]) // page // 2), (7, 0), (9, int(lens[9] - 1) // page), (47, 8192 // page - 3)]
    check_long(mx, 1, lens, new, heads, kv, D, page, window, missing, late)


@pytest.mark.parametrize("D,heads,kv,drafts", [(128, 4, 1, 1), (128, 8, 1, 3), (64, 8, 2, 1), (256, 2, 1, 1), (256, 8, 1, 3)])
@pytest.mark.parametrize("late", [False, True])
def test_one_very_long_context(mx, D, heads, kv, drafts, late):       # noqa: F811
    """Hundreds of pieces an item, joined by all warps of a CTA in several passes."""
    check_long(mx, 2, [131071], [drafts], heads, kv, D, 64, 0, [(0, 700), (0, 1000), (0, 2047)], late)


@pytest.mark.parametrize("requests", [120, 700])
@pytest.mark.parametrize("D,group", [(128, 4), (64, 16), (256, 2)])
def test_long_contexts_among_short_ones(mx, D, group, requests):       # noqa: F811
    """Dozens of pieces an item where there are many items (a warp joins a column in several passes), no more and more than CTAs."""
    lens = ragged(requests, requests, 0, 40)
    lens[[2, requests // 2, requests - 1]] = 70001, 30011, 65537
    new = np.minimum(lens, 1)
    check_long(mx, 3, lens, new, group, 1, D, 16, 0, [(2, 2000), (requests - 1, 4095)], True)


# ------------------------------------------------------------------------------------------------
# products
# ------------------------------------------------------------------------------------------------

def check_product(mx, M, N, K, per_row, fp32):       # noqa: F811
    g = torch.Generator(device=DEV)
    g.manual_seed(M + N + K)
    q = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device=DEV)
    bs = torch.randint(0, 120, (N, K // 16), generator=g, dtype=torch.uint8, device=DEV)
    s = torch.full((mx.scale_bytes(N, K, 16),), 0x7F, dtype=torch.uint8, device=DEV)          # padding: not read into any result
    s[torch.from_numpy(ref_places(N, K)).to(DEV)] = bs
    s2 = (0.5 + torch.rand(N if per_row else 1, generator=g, device=DEV)) * 1e-3
    x = torch.randn((M, K), generator=g, device=DEV).to(torch.bfloat16)
    y = torch.full((M, N), float("nan"), dtype=torch.float32 if fp32 else torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    mx.mx_nvfp4_matvec(x, q, s, s2, mx.MX_SCOPE_ROW if per_row else mx.MX_SCOPE_TENSOR, y)
    done(mx)
    e2m1, e4m3, xd = table_of(ref.E2M1_16), table_of(ref.E4M3), x.double()
    for r in range(0, N, 20000):
        part = slice(r, min(N, r + 20000))
        w = e2m1[torch.stack([q[part] & 15, q[part] >> 4], -1).flatten(1).int()]
        w = (w.unflatten(1, (-1, 16)) * e4m3[bs[part].int()][..., None]).flatten(1)
        sc = (s2[part] if per_row else s2).double()[None, :]
        want, absprod = (xd @ w.t()) * sc, (xd.abs() @ w.abs().t()) * sc
        lost = 2.0 ** -40 * xd.abs().amax(1, keepdim=True) * w.abs().sum(1)[None, :] * sc
        # a sum of K terms whose chains are at most (K of a warp) + 16 warps * 8 CTAs long; K bounds them from K = 256 on
        bound = K * 2.0 ** -24 * (1 + 2.0 ** -10) * absprod + lost + 2.0 ** -23 * want.abs() + (0 if fp32 else 2.0 ** -8 * 1.01 * want.abs()) + 1e-37
        got = y[:, part].double()
        bad = ~((got - want).abs() <= bound)
        assert not bad.any(), f"rows {r}..: {int(bad.sum())} off, {got[bad][:3].tolist()} want {want[bad][:3].tolist()}"
        # In the mean: every matrix instruction (16 products) and every scaling of a step (128) errs by at most 2^-23 of the largest
        # of what it adds, which for these random signs is within four times the size of the whole sum; a block of 16 products that
        # is missing, or another's, is off by sqrt(16 / K) of it.
        mean = 4 * 2.0 ** -23 * (K / 16 + K / 128 + 128) + (0 if fp32 else 2.0 ** -8)
        assert float((got - want).norm() / want.norm()) <= mean


@pytest.mark.parametrize("M,N,K", [(1, 151937, 2048), (4, 57611, 3152), (16, 40001, 2064), (9, 30000, 4096),                 # several turns of rows
                                   (2, 20000, 8208), (8, 18060, 5104), (3, 40000, 4096), (13, 9001, 14352), (16, 25000, 8192),
                                   (16, 33000, 14336)])
def test_product_in_several_turns(mx, M, N, K):       # noqa: F811
    check_product(mx, M, N, K, True, True)
    check_product(mx, M, N, K, False, False)


@pytest.mark.parametrize("M,N,K", [(16, 300, 40016), (16, 64, 65536), (12, 5000, 53248), (16, 20000, 30736), (8, 700, 61456), (8, 20001, 57344)])
def test_product_with_activations_in_stretches(mx, M, N, K):       # noqa: F811
    check_product(mx, M, N, K, True, True)
