"""GPU: the generation step over NVFP4 weights and an NVFP4 key/value cache (page and slot maps, cache write and
read, attention over the cache, products of a few tokens) against a plain 64-bit reference.

Integers, codes, block scales and BF16 values read back must be equal.  The error bounds of the two computed operators
are derived from their roundings:

products   y is a sum of K exact products in FP32, in any order: |error| <= K 2^-24 sum |x w| (1 + 2^-10), then the
           multiplication by s2 (2^-24 |y|) and the rounding to BF16 (2^-8 |y|, its unit
           roundoff with 8 significant bits; for FP32 outputs none).  Elements of
           x below 2^-29 of their row's largest may lose bits of their own: at most 2^-40 max |x| each.
attention  a score errs by eps = (D + 4) 2^-24 reach (FP32 sum of D exact products and its scalings; reach = largest
           scale * sum |q||k|) + 2^-23 (|m| + reach) (the maximum and the exponent's argument); a probability by
           2 eps + 2^-21 relatively (exp) and, entering the second product as FP16, by 2^-11 relatively and 2^-24 of
           the largest absolutely; so |error of o| <= (4 eps + 2^-10) mix + n 2^-24 max|v|, mix = sum p|v| / sum p, the
           FP32 sums over n positions adding n 2^-24 mix, and BF16 rounding 2^-8 |o|.
           |error of lse| <= eps + 2^-20 + n 2^-24 + 2^-22 |lse|."""
import numpy as np
import pytest
import torch

import generate_ref as ref
from gpu_util import DEV, bf16_dev, to_np_u16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import microscaled_precision_numerics_gb300 as m
    m.lib()
    return m


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.atleast_1d(a), dtype=np.int32)).to(DEV)


def f32(a):
    return torch.from_numpy(np.ascontiguousarray(np.atleast_1d(a), dtype=np.float32)).to(DEV)


def done(mx):
    torch.cuda.synchronize()
    mx.check_device_status()


# ------------------------------------------------------------------------------------------------
# page and slot maps
# ------------------------------------------------------------------------------------------------

def run_slots(mx, seq, new, page, table, free, count, most, in_place=False):
    R = len(seq)
    s, n, c = i32(seq), i32(new), i32(count)
    tab = i32(table)
    tot, left = (s, c) if in_place else (i32(np.zeros(R)), i32(0))
    start, slots, pos, un = i32(np.full(R + 1, 99)), i32(np.full(most, 99)), i32(np.full(most, 99)), i32(99)
    mx.mx_kv_slots(s, n, page, tab, i32(free), c, start, tot, slots, pos, left, un)
    done(mx)
    want = ref.slots(np.asarray(seq), np.asarray(new), page, np.asarray(table), np.asarray(free), count, most)
    for name, got in (("block_table", tab), ("q_start", start), ("total_lens", tot), ("slots", slots), ("positions", pos),
                      ("free_left", left), ("unplaced", un)):
        w = np.atleast_1d(want[name])
        assert np.array_equal(got.cpu().numpy(), w), name
    return want


def slots_case(R, longest, most_new, page, seed, spare=4, width_less=0):
    rng = np.random.default_rng(seed)
    seq = rng.integers(0, longest + 1, R)
    new = rng.integers(0, most_new + 1, R)
    width = max(1, -(-(longest + most_new) // page) - width_less)
    table = np.full((R, width), -1)
    had = np.minimum(-(-seq // page), width)
    ids = rng.permutation(int(had.sum()) + R * (most_new // page + 2) + spare)
    table[np.arange(width)[None, :] < had[:, None]] = ids[:int(had.sum())]
    return seq, new, table, ids[int(had.sum()):]


@pytest.mark.parametrize("R,longest,most_new,page", [(1, 0, 1, 16), (1, 40, 300, 16), (5, 100, 1, 64), (64, 500, 1, 16),
                                                     (63, 50, 90, 48), (1000, 20, 9, 16), (1025, 3, 3, 16), (4096, 5, 2, 32)])
@pytest.mark.parametrize("in_place", [False, True])
def test_slots(mx, R, longest, most_new, page, in_place):
    seq, new, table, free = slots_case(R, longest, most_new, page, R + longest)
    most = int(new.sum()) + 5
    run_slots(mx, seq, new, page, table, free, len(free) - 1, most, in_place)


def test_slots_no_new_tokens(mx):
    seq, new, table, free = slots_case(7, 40, 3, 16, 0)
    want = run_slots(mx, seq, np.zeros(7, int), 16, table, free, len(free), 4)
    assert want["unplaced"] == 0 and (want["slots"] == -1).all()


def test_slots_stack_runs_out(mx):
    seq, new, table, free = slots_case(40, 60, 50, 16, 3)
    want = run_slots(mx, seq, new, 16, table, free, 11, int(new.sum()), True)
    assert want["free_left"] == 0 and want["unplaced"] > 0
    run_slots(mx, seq, new, 16, table, free, 0, int(new.sum()))
    run_slots(mx, seq, new, 16, table, free, -3, int(new.sum()))
    run_slots(mx, seq, new, 16, table, free, len(free) + 100, int(new.sum()))     # clamped to the stack's capacity


def test_slots_narrow_table_and_short_outputs(mx):
    seq, new, table, free = slots_case(40, 200, 50, 16, 4, width_less=6)
    run_slots(mx, seq, new, 16, table, free, len(free), int(new.sum()) - 30)
    run_slots(mx, seq, new, 16, table, free, len(free), 3000 + int(new.sum()))


def test_slots_negative_lengths_count_as_zero(mx):
    seq, new, table, free = slots_case(9, 60, 20, 16, 5)
    seq[2], new[4], seq[7], new[7] = -5, -1, -2, 6
    table[[2, 7]] = -1
    run_slots(mx, seq, new, 16, table, free, len(free), int(np.maximum(new, 0).sum()) + 2)


def test_slots_strided_table(mx):
    seq, new, table, free = slots_case(6, 60, 20, 16, 6)
    wide = torch.full((6, table.shape[1] + 9), 77, dtype=torch.int32, device=DEV)
    view = wide[:, :table.shape[1]]
    view.copy_(i32(table))
    most = int(new.sum())
    outs = [i32(np.zeros(7)), i32(np.zeros(6)), i32(np.zeros(most)), i32(np.zeros(most)), i32(0), i32(0)]
    mx.mx_kv_slots(i32(seq), i32(new), 16, view, i32(free), i32(len(free)), *outs)
    done(mx)
    want = ref.slots(seq, new, 16, table, free, len(free), most)
    assert np.array_equal(view.cpu().numpy(), want["block_table"]) and (wide[:, table.shape[1]:] == 77).all()
    assert np.array_equal(outs[2].cpu().numpy(), want["slots"])


# ------------------------------------------------------------------------------------------------
# cache write and read
# ------------------------------------------------------------------------------------------------

def kv_inputs(rng, T, heads, D, spread=1.0):
    return [ref.bf16_bits(rng.standard_normal((T, heads, D)) * spread * np.exp2(rng.integers(-3, 4, (T, heads, 1)))) for _ in range(2)]


@pytest.mark.parametrize("T,heads,D,page", [(1, 1, 64, 16), (3, 2, 128, 32), (17, 8, 128, 16), (50, 3, 64, 48), (33, 1, 256, 16),
                                            (130, 4, 128, 64)])
def test_append_and_gather(mx, T, heads, D, page):
    rng = np.random.default_rng(T + D)
    pages = T // page + 3
    k, v = kv_inputs(rng, T, heads, D)
    s_k, s_v = rng.uniform(0.5, 2, heads).astype(np.float32) / 448, rng.uniform(0.5, 2, heads).astype(np.float32) / 448
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    if T > 2:
        slots[1], slots[T - 1] = -1, pages * page                 # skipped: below and beyond the cache
    start = rng.integers(0, 256, (pages, heads, page // 16, 18 * D)).astype(np.uint8)
    want = start.copy()
    for t in range(T):
        if 0 <= slots[t] < pages * page:
            ref.cache_write(want, int(slots[t]), ref.bf16_value(k[t]), ref.bf16_value(v[t]), s_k, s_v, page)
    # k and v as views of a fused projection
    fused = torch.zeros((T, 3 * heads + 1, D), dtype=torch.bfloat16, device=DEV)
    kd, vd = fused[:, heads:2 * heads], fused[:, 2 * heads:3 * heads]
    kd.copy_(bf16_dev(k))
    vd.copy_(bf16_dev(v))
    cache = torch.from_numpy(start).to(DEV)
    mx.mx_nvfp4_kv_append(kd, vd, i32(slots), f32(s_k), f32(s_v), cache)
    done(mx)
    assert np.array_equal(cache.cpu().numpy(), want)

    back = torch.full((T, 2 * heads + 1, D), 7.0, dtype=torch.bfloat16, device=DEV)
    ko, vo = back[:, :heads], back[:, heads:2 * heads]
    mx.mx_nvfp4_kv_gather(cache, i32(slots), f32(s_k), f32(s_v), ko, vo)
    done(mx)
    for t in range(T):
        if 0 <= slots[t] < pages * page:
            a, b = ref.cache_read(want, int(slots[t]), page)
            assert np.array_equal(to_np_u16(ko[t]), ref.bf16_bits(a.astype(np.float32) * s_k[:, None])), t
            assert np.array_equal(to_np_u16(vo[t]), ref.bf16_bits(b.astype(np.float32) * s_v[:, None])), t
        else:
            assert not ko[t].any() and not vo[t].any()
    assert (back[:, 2 * heads:] == 7.0).all()


def test_append_extreme_values(mx):
    """Clipped blocks, subnormals, zeros, a zero and a tiny S, infinities and NaN, against the same rules."""
    D, heads, page = 64, 5, 16
    rng = np.random.default_rng(0)
    x = rng.standard_normal((8, heads, D)).astype(np.float32)
    x[0] *= 1e5
    x[1] *= 1e-6
    x[2] = 0
    x[3, :, :16] = 2.0 ** -133
    x[4, :, 3] = np.inf
    x[5, :, 20] = np.nan
    x[6] *= 1e30
    bits = ref.bf16_bits(x)
    s = np.array([1 / 448, 0.0, 1e-38, 3.0, 2.0 ** -10], np.float32)
    want = np.zeros((1, heads, 1, 18 * D), np.uint8)
    for t in range(8):
        ref.cache_write(want, t, ref.bf16_value(bits[t]), ref.bf16_value(bits[t]), s, s, page)
    cache = mx.alloc_nvfp4_kv_cache(1, page, heads, D, DEV)
    d = bf16_dev(bits)
    mx.mx_nvfp4_kv_append(d, d, i32(np.arange(8)), f32(s), f32(s), cache)
    done(mx)
    got = cache.cpu().numpy()
    # the codes of a block that holds a NaN are not specified (its scale is NaN)
    for a in (got, want):
        for base in (0, 9 * D):
            a[0, :, 0, base + 5 * D // 2 + 8:base + 5 * D // 2 + 16] = 0
    assert np.array_equal(got, want)


def test_cache_beyond_32_bit_offsets(mx):
    D, heads, page = 128, 8, 64
    pages = (5 << 30) // (page * heads * 18 * D // 16)
    cache = torch.zeros((pages, heads, page // 16, 18 * D), dtype=torch.uint8, device=DEV)
    rng = np.random.default_rng(1)
    k, v = kv_inputs(rng, 9, heads, D)
    s = np.full(heads, 1 / 448, np.float32)
    slots = np.arange(9) + (pages - 1) * page + 3
    mx.mx_nvfp4_kv_append(bf16_dev(k), bf16_dev(v), i32(slots), f32(s), f32(s), cache)
    small = np.zeros((1, heads, page // 16, 18 * D), np.uint8)
    for t in range(9):
        ref.cache_write(small, t + 3, ref.bf16_value(k[t]), ref.bf16_value(v[t]), s, s, page)
    assert np.array_equal(cache[-1:].cpu().numpy(), small) and not cache[:-1].any()
    ko, vo = (torch.empty((9, heads, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    mx.mx_nvfp4_kv_gather(cache, i32(slots), f32(s), f32(s), ko, vo)
    want = np.stack([ref.cache_read(small, t + 3, page)[0] for t in range(9)])
    assert np.array_equal(to_np_u16(ko), ref.bf16_bits(want.astype(np.float32) * s[:, None]))
    # attention reads the last page too
    q = bf16_dev(ref.bf16_bits(rng.standard_normal((1, 16, D))))
    check_attention(mx, q, [0, 1], [12], np.array([[pages - 1]]), cache, s, s, D ** -0.5, page, host_cache=small, host_table=np.array([[0]]))


# ------------------------------------------------------------------------------------------------
# attention
# ------------------------------------------------------------------------------------------------

def check_attention(mx, q, q_start, lens, table, cache, s_k, s_v, scale, page, window=0, host_cache=None, host_table=None,
                    max_q=None, out=None):
    T, heads, D = q.shape
    host = host_cache if host_cache is not None else cache.cpu().numpy()
    out = torch.full((T, heads, D), float("nan"), dtype=torch.bfloat16, device=DEV) if out is None else out
    lse = torch.full((T, heads), float("nan"), dtype=torch.float32, device=DEV)
    ws = torch.full((mx.kv_attention_workspace_bytes(D),), 255, dtype=torch.uint8, device=DEV)
    n = int(np.max(np.diff(q_start))) if max_q is None else max_q
    args = (q, i32(q_start), i32(lens), i32(table), cache, f32(s_k), f32(s_v), scale, n)
    mx.mx_nvfp4_kv_attention(*args, out, ws, lse=lse, window=window)
    done(mx)
    qv = ref.bf16_value(to_np_u16(q)).astype(np.float64)
    o, l, mix, reach = ref.attention(qv, q_start, lens, table if host_table is None else host_table, host, s_k, s_v, scale, page, window)
    got, got_l = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    empty = np.isneginf(l)
    assert np.array_equal(np.isneginf(got_l), empty) and not got[empty].any()
    count = max(1, int(np.max(lens)))
    lf = np.where(empty, 0.0, l)
    eps = (D + 4) * 2.0 ** -24 * reach + 2.0 ** -23 * (np.abs(lf) + np.log(count) + reach)
    big = np.abs(o).max() if o.size else 0.0
    vmax = max(6 * 448 * float(np.max(s_v)), big)
    bound = (4 * eps[..., None] + 2.0 ** -10 + count * 2.0 ** -24) * mix + count * 2.0 ** -24 * vmax + 2.0 ** -8 * 1.01 * np.abs(o) + 1e-30
    assert np.isfinite(got).all()
    bad = np.abs(got - o) > bound
    assert not bad.any(), f"{int(bad.sum())} elements off, first {np.argwhere(bad)[0]}: {got[bad][0]} want {o[bad][0]}"
    bad = np.abs(np.where(empty, 0.0, got_l) - lf) > eps + 2.0 ** -20 + count * 2.0 ** -24 + 2.0 ** -22 * np.abs(lf)
    assert not bad.any(), f"lse off: {got_l[bad][:3]} want {l[bad][:3]}"
    return out, lse


def attention_case(seed, lens, new, heads, kv, D, page, junk=255, scale_v=1.0):
    """A cache holding the requests' tokens in pages in random order; everything else in it is `junk` (255: NaN scales)."""
    rng = np.random.default_rng(seed)
    lens, new = np.asarray(lens), np.asarray(new)
    per = -(-lens // page)
    pages = int(per.sum()) + 2
    order = rng.permutation(pages)
    table = np.full((len(lens), int(per.max()) + 1), -1)
    table[np.arange(table.shape[1])[None, :] < per[:, None]] = order[:int(per.sum())]
    D16 = D // 16
    cache = np.full((pages, kv, page // 16, 18 * D), junk, np.uint8)
    s_k, s_v = (rng.uniform(4, 8, kv).astype(np.float32) / 2688 for _ in range(2))
    s_v = s_v * np.float32(scale_v)
    for r in range(len(lens)):
        L = int(lens[r])
        if not L:
            continue
        kc, ks = ref.quantize_blocks(rng.standard_normal((L, kv, D16, 16)), s_k[None, :, None] * np.ones((L, 1, D16), np.float32))
        vc, vs = ref.quantize_blocks(rng.standard_normal((L, kv, D16, 16)) * scale_v, s_v[None, :, None] * np.ones((L, 1, D16), np.float32))
        kc, vc = ref.pack(kc.reshape(L, kv, D)), ref.pack(vc.reshape(L, kv, D))
        for j in range(L):
            p, g, i = table[r, j // page], j % page // 16, j % 16
            rec = cache[p, :, g]
            rec[:, i * (D // 2):(i + 1) * (D // 2)] = kc[j]
            rec[:, 8 * D + i * D16:8 * D + (i + 1) * D16] = ks[j]
            rec[:, 9 * D + i * (D // 2):9 * D + (i + 1) * (D // 2)] = vc[j]
            rec[:, 17 * D + np.arange(D16) * 16 + ref.v_scale_position(i)] = vs[j]
    q_start = np.concatenate([[0], np.cumsum(new)])
    q = bf16_dev(ref.bf16_bits(rng.standard_normal((int(q_start[-1]), heads, D)) * 1.5))
    return q, q_start, lens, table, torch.from_numpy(cache).to(DEV), s_k, s_v


ATTENTION_CASES = [
    ([1], [1], 4, 4, 64, 16, 0),                                   # one token of context
    ([15, 16, 17, 31, 32, 33], [1] * 6, 8, 2, 128, 16, 0),         # around the record and tile lengths
    ([63, 64, 65, 127, 129], [1] * 5, 8, 1, 128, 64, 0),
    ([200, 0, 1, 77], [1, 0, 1, 1], 8, 2, 128, 32, 0),             # an idle request in the batch
    ([130, 95], [4, 3], 4, 1, 64, 16, 0),                          # drafts: 12 and 16 rows
    ([100, 300, 5], [9, 20, 5], 6, 2, 128, 16, 0),                 # longer runs of new tokens, odd group
    ([90], [90], 2, 1, 64, 16, 0),                                 # a whole prompt
    ([700], [1], 32, 8, 128, 16, 0),
    ([1500, 3], [1, 1], 5, 1, 128, 48, 0),                         # group of five, pages of 48
    ([400, 33], [1, 2], 8, 2, 256, 16, 0),
    ([2100], [1], 16, 1, 64, 128, 0),                              # group of sixteen
    ([300, 50, 20], [3, 1, 2], 4, 2, 128, 16, 17),                 # windows: inside a tile,
    ([300, 50, 20], [3, 1, 2], 4, 2, 64, 16, 1),                   # of one position,
    ([500], [40], 4, 2, 128, 32, 64),                              # shorter than the run of new tokens,
    ([300, 50], [1, 1], 4, 2, 128, 16, 100000),                    # longer than the context
    ([260, 260, 260], [1, 1, 1], 40, 1, 128, 16, 0),               # group of forty: several row tiles
]


@pytest.mark.parametrize("lens,new,heads,kv,D,page,window", ATTENTION_CASES)
def test_attention(mx, lens, new, heads, kv, D, page, window):
    q, q_start, lens, table, cache, s_k, s_v = attention_case(1, lens, new, heads, kv, D, page)
    check_attention(mx, q, q_start, lens, table, cache, s_k, s_v, D ** -0.5, page, window)


def wide(table, columns):
    """The table with columns of -1 behind: contexts of wide tables are split among CTAs, those of narrow ones are not."""
    return np.pad(table, ((0, 0), (0, columns)), constant_values=-1)


@pytest.mark.parametrize("lens,new,heads,kv,D,page,window", ATTENTION_CASES)
def test_attention_wide_table(mx, lens, new, heads, kv, D, page, window):
    q, q_start, lens, table, cache, s_k, s_v = attention_case(1, lens, new, heads, kv, D, page)
    check_attention(mx, q, q_start, lens, wide(table, 5000 // page), cache, s_k, s_v, D ** -0.5, page, window)


@pytest.mark.parametrize("group,drafts", [(2, 1), (6, 3)])
def test_attention_more_items_than_ctas(mx, group, drafts):
    """Hundreds of short contexts and a few long ones, split and not."""
    rng = np.random.default_rng(12)
    lens = rng.integers(0, 24, 260)
    lens[[3, 77, 200]] = 1300, 641, 33
    new = np.minimum(lens, rng.integers(1, drafts + 1, 260))
    q, q_start, lens, table, cache, s_k, s_v = attention_case(13, lens, new, 4 * group, 4, 64, 16)
    check_attention(mx, q, q_start, lens, table, cache, s_k, s_v, 0.125, 16)
    short = lens < 700
    keep = np.flatnonzero(short)
    rows = np.concatenate([np.arange(q_start[r], q_start[r + 1]) for r in keep]).astype(int)
    starts = np.concatenate([[0], np.cumsum(np.diff(q_start)[keep])])
    check_attention(mx, q[torch.from_numpy(rows).to(DEV)].contiguous(), starts, lens[keep], np.ascontiguousarray(table[keep][:, :50]), cache,
                    s_k, s_v, 0.125, 16)


@pytest.mark.parametrize("positions", [500, 1200, 40000])
@pytest.mark.parametrize("lens,new,heads,kv,D,page,window", ATTENTION_CASES)
def test_attention_table_widths(mx, lens, new, heads, kv, D, page, window, positions):
    """Contexts divided inside a cluster, where short ones leave some of its CTAs nothing, and split over the GPU."""
    q, q_start, lens, table, cache, s_k, s_v = attention_case(1, lens, new, heads, kv, D, page)
    check_attention(mx, q, q_start, lens, wide(table, positions // page), cache, s_k, s_v, D ** -0.5, page, window)


@pytest.mark.parametrize("requests", [5, 9, 18, 27])
def test_attention_clusters_of_every_size(mx, requests):
    """Ragged batches of 8 kv heads, an idle request and a short one in each, with one and with several new tokens."""
    rng = np.random.default_rng(requests)
    lens = rng.integers(1, 420, requests)
    lens[[1, 3, 4]] = 0, 415, 1
    for most in (1, 3):
        new = np.minimum(lens, rng.integers(1, most + 1, requests))
        q, q_start, lens_, table, cache, s_k, s_v = attention_case(21, lens, new, 32, 8, 64, 16)
        for window in (0, 40):
            check_attention(mx, q, q_start, lens_, table, cache, s_k, s_v, 0.125, 16, window)


def test_attention_cluster_nan_key_and_value(mx):
    """One bad scale in one CTA's part of a context: a key's reaches all of its head, a value's its block of 16 only."""
    L, D, kv, group = 900, 128, 2, 4
    q, q_start, lens, table, cache, s_k, s_v = attention_case(22, [L], [1], kv * group, kv, D, 16)
    good, _ = check_attention(mx, q, q_start, lens, table, cache, s_k, s_v, 0.09, 16)
    ws = torch.empty(mx.kv_attention_workspace_bytes(D), dtype=torch.uint8, device=DEV)
    for tok in (0, 450, L - 1):
        rec = int(table[0, tok // 16])
        for at, sees in ((8 * D + (tok % 16) * (D // 16), slice(None)), (17 * D + 3 * 16 + ref.v_scale_position(tok % 16), slice(48, 64))):
            hurt = cache.clone()
            hurt[rec, 1, 0, at] = 0x7F
            out = torch.zeros_like(good)
            mx.mx_nvfp4_kv_attention(q, i32(q_start), i32(lens), i32(table), hurt, f32(s_k), f32(s_v), 0.09, 1, out, ws)
            done(mx)
            want = torch.zeros(D, dtype=torch.bool, device=DEV)
            want[sees] = True
            assert torch.equal(out[0, :group], good[0, :group])
            assert torch.equal(out[0, group:].isnan(), want.expand(group, D))
            assert torch.equal(out[0, group:][:, ~want], good[0, group:][:, ~want])


def test_attention_many_ragged_requests(mx):
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 120, 150)
    new = np.minimum(lens, rng.integers(0, 3, 150))
    q, q_start, lens, table, cache, s_k, s_v = attention_case(3, lens, new, 4, 2, 64, 16)
    check_attention(mx, q, q_start, lens, table, cache, s_k, s_v, 0.125, 16, max_q=7)


def test_attention_rows_with_nothing_to_attend(mx):
    """More new tokens than cached ones (positions below zero), and requests of length zero with tokens."""
    q, q_start, lens, table, cache, s_k, s_v = attention_case(4, [3, 40, 0], [3, 2, 0], 4, 2, 64, 16)
    q = torch.cat([q, q])[:8]
    check_attention(mx, q, np.array([0, 5, 7, 8]), lens, table, cache, s_k, s_v, 0.125, 16)


def test_attention_leaves_padding_rows_alone(mx):
    """More rows than the requests have tokens (a buffer of fixed length): the rest keeps what it holds."""
    q, q_start, lens, table, cache, s_k, s_v = attention_case(14, [50, 1000], [2, 1], 4, 2, 64, 16)
    for tab in (table, wide(table, 10)):
        q6 = torch.cat([q, q])[:6]
        out = torch.full((6, 4, 64), 9.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((6, 4), 9.0, dtype=torch.float32, device=DEV)
        ws = torch.empty(mx.kv_attention_workspace_bytes(64), dtype=torch.uint8, device=DEV)
        mx.mx_nvfp4_kv_attention(q6, i32(q_start), i32(lens), i32(tab), cache, f32(s_k), f32(s_v), 0.125, 2, out, ws, lse=lse)
        done(mx)
        want, want_lse = check_attention(mx, q, q_start, lens, tab, cache, s_k, s_v, 0.125, 16)
        assert torch.equal(out[:3], want) and torch.equal(lse[:3], want_lse)
        assert (out[3:] == 9).all() and (lse[3:] == 9).all()


def test_attention_skips_missing_pages(mx):
    q, q_start, lens, table, cache, s_k, s_v = attention_case(5, [200, 64, 40], [2, 1, 1], 4, 2, 128, 16)
    table[0, 3], table[0, 12], table[1, :4], table[2, 1] = -1, 10 ** 6, -1, -7
    check_attention(mx, q, q_start, lens, table, cache, s_k, s_v, 0.09, 16)
    # a table too narrow for the length
    check_attention(mx, q, q_start, lens, np.ascontiguousarray(table[:, :6]), cache, s_k, s_v, 0.09, 16)


@pytest.mark.parametrize("scale", [4.0, -1.0, 0.0, 1e-6])
def test_attention_sharp_and_flat(mx, scale):
    """Scores far apart (one position takes all), negative and zero scales."""
    q, q_start, lens, table, cache, s_k, s_v = attention_case(6, [333, 70], [1, 2], 8, 2, 64, 16)
    check_attention(mx, q, q_start, lens, table, cache, s_k, s_v, scale, 16)


@pytest.mark.parametrize("scale_v", [1e-20, 1e20])
def test_attention_value_scales(mx, scale_v):
    q, q_start, lens, table, cache, s_k, s_v = attention_case(7, [150], [1], 8, 2, 128, 16, scale_v=scale_v)
    check_attention(mx, q, q_start, lens, table, cache, s_k, s_v, 0.09, 16)


def test_attention_wide_range_queries(mx):
    """Queries with elements far apart in size, very large, very small and zero ones."""
    q, q_start, lens, table, cache, s_k, s_v = attention_case(8, [150, 40, 60], [1, 1, 1], 4, 1, 64, 16)
    v = q.float()
    v[0] *= torch.exp2(torch.randint(-30, 1, v[0].shape, device=DEV).float())
    v[1] *= 1e-30
    v[2, 0] = 0
    v[2, 1] *= 1e20
    q = v.to(torch.bfloat16)
    host = cache.cpu().numpy()
    check_attention(mx, q[:2], [0, 1, 2], lens[:2], table[:2], cache, s_k, s_v, 0.125, 16, host_cache=host)
    check_attention(mx, q[2:], [0, 1], lens[2:], table[2:], cache, s_k, s_v, 1e-21, 16, host_cache=host)


def test_attention_nan_key_spreads_inside_its_head_only(mx):
    q, q_start, lens, table, cache, s_k, s_v = attention_case(9, [70, 70], [1, 1], 4, 2, 64, 16)
    good, _ = check_attention(mx, q, q_start, lens, table, cache, s_k, s_v, 0.125, 16)
    cache[int(table[0, 1]), 1, 0, 8 * 64 + 5 * 4] = 0x7F                 # K scale of token 21, request 0, kv head 1
    out = torch.empty_like(good)
    ws = torch.empty(mx.kv_attention_workspace_bytes(64), dtype=torch.uint8, device=DEV)
    mx.mx_nvfp4_kv_attention(q, i32(q_start), i32(lens), i32(table), cache, f32(s_k), f32(s_v), 0.125, 1, out, ws)
    done(mx)
    assert out[0, 2:].isnan().all() and torch.equal(out[0, :2], good[0, :2]) and torch.equal(out[1], good[1])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_nan_value_reaches_only_rows_that_attend_to_it(mx, D):
    """A NaN block scale of V at a position that some rows of a run of new tokens mask (a later token, or one before the
    window): those rows are as without it, the others have NaN in that block of 16 dimensions and nowhere else."""
    kv, group, n, L = 2, 3, 6, 75
    q, q_start, lens, table, cache, s_k, s_v = attention_case(11, [L], [n], kv * group, kv, D, 16)
    window = 20
    base, _ = check_attention(mx, q, q_start, lens, table, cache, s_k, s_v, 0.1, 16, window)
    blk = D // 16 - 1
    for tok in (L - 3, L - n - window + 3):                             # masked by the first rows; by the last rows
        hurt = cache.clone()
        i = tok % 16
        hurt[int(table[0, tok // 16]), 1, 0, 17 * D + blk * 16 + ref.v_scale_position(i)] = 0xFF
        out = torch.zeros_like(base)
        ws = torch.empty(mx.kv_attention_workspace_bytes(D), dtype=torch.uint8, device=DEV)
        mx.mx_nvfp4_kv_attention(q, i32(q_start), i32(lens), i32(table), hurt, f32(s_k), f32(s_v), 0.1, n, out, ws, window=window)
        done(mx)
        for t in range(n):
            pos = L - n + t
            sees = pos - window < tok <= pos
            assert torch.equal(out[t, :group], base[t, :group])
            assert out[t, group:, blk * 16:].isnan().all() == sees and out[t, group:, blk * 16:].isnan().any() == sees
            assert torch.equal(out[t, group:, :blk * 16], base[t, group:, :blk * 16])
            if not sees:
                assert torch.equal(out[t], base[t])


def test_attention_strided_stream_graph_and_repeatable(mx):
    """q and out as views of larger tensors, on a side stream, captured in a graph and replayed: the same bits."""
    q, q_start, lens, table, cache, s_k, s_v = attention_case(10, [900, 35, 410], [1, 2, 1], 8, 2, 128, 16)
    out, lse = check_attention(mx, q, q_start, lens, table, cache, s_k, s_v, 0.09, 16)
    big_q = torch.full((4, 11, 160), 3.0, dtype=torch.bfloat16, device=DEV)
    big_q[:, 2:10, 16:144] = q
    big_o = torch.full((4, 10, 136), 5.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(mx.kv_attention_workspace_bytes(128), dtype=torch.uint8, device=DEV)
    lse2 = torch.empty_like(lse)
    args = (big_q[:, 2:10, 16:144], i32(q_start), i32(lens), i32(table), cache, f32(s_k), f32(s_v), 0.09, 2,
            big_o[:, 1:9, :128], ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    mx.mx_nvfp4_kv_attention(*args, lse=lse2, stream=side)
    side.synchronize()
    assert torch.equal(big_o[:, 1:9, :128], out) and torch.equal(lse2, lse)
    assert (big_o[:, 0] == 5).all() and (big_o[:, 9] == 5).all() and (big_o[:, :, 128:] == 5).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.mx_nvfp4_kv_attention(*args, lse=lse2)
    big_o.fill_(0)
    lse2.fill_(0)
    for _ in range(2):
        graph.replay()
    done(mx)
    assert torch.equal(big_o[:, 1:9, :128], out) and torch.equal(lse2, lse)


# ------------------------------------------------------------------------------------------------
# products of a few tokens
# ------------------------------------------------------------------------------------------------

def check_matvec(mx, x_bits, N, per_row, fp32, seed=0, x=None, y=None):
    M, K = x_bits.shape
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (N, K)).astype(np.uint8)
    bs = rng.integers(0, 120, (N, K // 16)).astype(np.uint8)
    s2 = rng.uniform(0.5, 2, N if per_row else 1).astype(np.float32) * 1e-3
    layout = ref.gemm_layout(bs)
    pad = np.ones_like(layout, bool)
    pad[ref_places(N, K)] = False
    layout[pad] = 0x7F                                                   # the padding is not read into any result
    xd = bf16_dev(x_bits) if x is None else x
    yd = torch.full((M, N), float("nan"), dtype=torch.float32 if fp32 else torch.bfloat16, device=DEV) if y is None else y
    mx.mx_nvfp4_matvec(xd, torch.from_numpy(ref.pack(codes)).to(DEV), torch.from_numpy(layout).to(DEV), f32(s2),
                       mx.MX_SCOPE_ROW if per_row else mx.MX_SCOPE_TENSOR, yd)
    done(mx)
    w = ref.E2M1_16[codes] * np.repeat(ref.E4M3[bs], 16, -1)
    xv = ref.bf16_value(x_bits).astype(np.float64)
    got = yd.double().cpu().numpy()
    return got, xv, w, s2.astype(np.float64)


def ref_places(N, K):
    nct = -(-(K // 16) // 4)
    r, c = np.arange(N)[:, None], np.arange(K // 16)[None, :]
    return (r // 128 * nct + c // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + c % 4


def assert_matvec(got, xv, w, s2, fp32):
    want = (xv @ w.T) * s2[None, :]
    K = xv.shape[1]
    absprod = (np.abs(xv) @ np.abs(w).T) * s2[None, :]
    lost = 2.0 ** -40 * np.abs(xv).max(1, keepdims=True) * np.abs(w).sum(1)[None, :] * s2[None, :]
    bound = K * 2.0 ** -24 * (1 + 2.0 ** -10) * absprod + lost + 2.0 ** -23 * np.abs(want) + (0 if fp32 else 2.0 ** -8 * 1.01 * np.abs(want)) + 1e-37
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{int(bad.sum())} elements off, first {np.argwhere(bad)[0]}: {got[bad][0]} want {want[bad][0]}"


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 25, 33, 64])
@pytest.mark.parametrize("N,K,per_row,fp32", [(300, 1024, True, False), (1, 16, False, True), (129, 272, True, True)])
def test_matvec(mx, M, N, K, per_row, fp32):
    x = ref.bf16_bits(np.random.default_rng(M).standard_normal((M, K)))
    assert_matvec(*check_matvec(mx, x, N, per_row, fp32, seed=N), fp32)


@pytest.mark.parametrize("M,N,K", [(1, 64, 4096), (1, 5, 16384), (3, 128, 14336), (16, 200, 8208), (64, 96, 14336), (1, 2, 48), (2, 1000, 32),
                                   (1, 20001, 144), (11, 4097, 528)])
def test_matvec_shapes(mx, M, N, K):
    x = ref.bf16_bits(np.random.default_rng(K).standard_normal((M, K)))
    for per_row, fp32 in ((False, False), (True, True)):
        assert_matvec(*check_matvec(mx, x, N, per_row, fp32, seed=M), fp32)


def test_matvec_wide_range_inputs(mx):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((6, 512))
    x[0] *= 1e30
    x[1] *= 1e-33
    x[2] = 0
    x[3] *= np.exp2(rng.integers(-40, 1, 512))
    x[4, :256] *= 1e-25
    x[5, 256:] *= 1e12
    assert_matvec(*check_matvec(mx, ref.bf16_bits(x), 200, True, True), True)


def test_matvec_not_finite_inputs_stay_in_their_token(mx):
    x = np.random.default_rng(0).standard_normal((3, 256))
    x[1, 77], x[2, 5] = np.nan, np.inf
    bits = ref.bf16_bits(x)
    got, xv, w, s2 = check_matvec(mx, bits, 140, False, True)
    assert_matvec(got[:1], xv[:1], w, s2, True)
    assert np.isnan(got[1]).all()
    infinite = w[:, 5] != 0
    assert np.isnan(got[2][~infinite]).all() and np.array_equal(got[2][infinite], np.sign(w[infinite, 5]) * np.inf)


def test_matvec_strided_views(mx):
    x = ref.bf16_bits(np.random.default_rng(5).standard_normal((5, 512)))
    wide = torch.full((5, 1024), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 256:768] = bf16_dev(x)
    for fp32 in (False, True):
        y = torch.full((5, 301), 7.0, dtype=torch.float32 if fp32 else torch.bfloat16, device=DEV)
        got = check_matvec(mx, x, 150, True, fp32, x=wide[:, 256:768], y=y[:, 8:158])
        assert_matvec(*got, fp32)
        assert (y[:, :8] == 7).all() and (y[:, 158:] == 7).all()


def test_matvec_takes_the_quantizers_weights(mx):
    """A weight quantized by the 2D quantizer (per-tensor scale) and by the per-token one (per-row scales)."""
    rng = np.random.default_rng(6)
    wb = ref.bf16_bits(rng.standard_normal((256, 512)) * 0.02)
    x = ref.bf16_bits(rng.standard_normal((4, 512)))
    w2 = mx.alloc_nvfp4_weight_2d(1, 256, 512, DEV)
    mx.mx_nvfp4_quantize_weight_2d(bf16_dev(wb).unsqueeze(0), w2["q_row"], w2["s_row"], w2["q_col"], w2["s_col"], w2["s_w"], w2["ws"])
    rows = mx.alloc_nvfp4_rows(256, 512, DEV)
    mx.mx_nvfp4_quantize_per_token(bf16_dev(wb), rows["q"], rows["s"], rows["s2"])
    for q, s, s2, scope in ((w2["q_row"][0], w2["s_row"], w2["s_w"], mx.MX_SCOPE_TENSOR), (rows["q"], rows["s"], rows["s2"], mx.MX_SCOPE_ROW)):
        y = torch.empty((4, 256), dtype=torch.float32, device=DEV)
        mx.mx_nvfp4_matvec(bf16_dev(x), q, s, s2, scope, y)
        done(mx)
        codes = ref.unpack(q.cpu().numpy())
        bs = s.cpu().numpy()[ref_places(256, 512)]
        w = ref.E2M1_16[codes] * np.repeat(ref.E4M3[bs], 16, -1)
        assert_matvec(y.double().cpu().numpy(), ref.bf16_value(x).astype(np.float64), w,
                      np.broadcast_to(s2.double().cpu().numpy(), (256,)), True)


def test_matvec_graph_and_repeatable(mx):
    x = bf16_dev(ref.bf16_bits(np.random.default_rng(7).standard_normal((3, 4096))))
    q = torch.randint(0, 256, (500, 2048), dtype=torch.uint8, device=DEV)
    s = torch.randint(0, 120, (mx.scale_bytes(500, 4096, 16),), dtype=torch.uint8, device=DEV)
    y = [torch.zeros((3, 500), dtype=torch.float32, device=DEV) for _ in range(3)]
    one = f32(1.0)
    mx.mx_nvfp4_matvec(x, q, s, one, mx.MX_SCOPE_TENSOR, y[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    mx.mx_nvfp4_matvec(x, q, s, one, mx.MX_SCOPE_TENSOR, y[1], stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.mx_nvfp4_matvec(x, q, s, one, mx.MX_SCOPE_TENSOR, y[2])
    graph.replay()
    done(mx)
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])
