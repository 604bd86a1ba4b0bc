"""Host-side validation of the generation entry points (include/mxnum_generate.h): each refusal returns its status before
anything touches a GPU, every declared symbol is exported, and the reference's quantizer agrees with the C oracle."""
import ctypes
import os
import re

import numpy as np
import pytest

import generate_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mxnum_generate.h")

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
    assert names == ["mx_kv_attention_workspace_bytes", "mx_kv_page_bytes", "mx_kv_slots", "mx_nvfp4_kv_append",
                     "mx_nvfp4_kv_attention", "mx_nvfp4_kv_gather", "mx_nvfp4_matvec"]
    for name in names:
        assert getattr(lib, name).argtypes is not None, name


def test_sizes(lib):
    assert lib.mx_kv_page_bytes(16, 8, 128) == 8 * 2304
    assert lib.mx_kv_page_bytes(48, 1, 64) == 3 * 1152
    for bad in ((0, 8, 128), (24, 8, 128), (16, 0, 128), (16, 8, 96), (-16, 8, 128)):
        assert lib.mx_kv_page_bytes(*bad) == 0
    for dim in (64, 128, 256):
        assert 0 < lib.mx_kv_attention_workspace_bytes(dim) <= 64 << 20
    assert lib.mx_kv_attention_workspace_bytes(96) == 0


@pytest.mark.parametrize("page_size,kv_heads,head_dim", [((1 << 20) + 16, 8, 128), (16, 65536, 128), (1 << 40, 1, 64), (16, 1 << 40, 64),
                                                         (1 << 20, 65535, 256), (48, 65535, 64)])
def test_page_bytes_are_of_sizes_that_the_cache_takes(lib, page_size, kv_heads, head_dim):
    """0 exactly where an append to such a cache is refused for its sizes (checked before anything is launched: no slots)."""
    import microscaled_precision_numerics_gb300 as mx
    taken = page_size <= 1 << 20 and kv_heads <= 65535
    assert lib.mx_kv_page_bytes(page_size, kv_heads, head_dim) == (page_size * kv_heads * 18 * head_dim // 16 if taken else 0)
    bad = {**APPEND, "pages": 1, "page_size": page_size, "kv_heads": kv_heads, "head_dim": head_dim, "k_token": 1 << 20, "v_token": 1 << 20,
           "k_head": 256, "v_head": 256, "T": 1, "slots": A if not taken else NUL}
    assert lib.mx_nvfp4_kv_append(*bad.values()) == (INVALID if taken else UNSUPPORTED)
    if not taken:
        with pytest.raises(ValueError):
            mx.alloc_nvfp4_kv_cache(0, page_size, kv_heads, head_dim, "cpu")


SLOTS = dict(seq_lens=A, new_lens=A, requests=4, page_size=16, block_table=A, table_width=8, table_stride=8, free_pages=A,
             free_capacity=10, free_count=A, q_start=A, total_lens=A, slots=A, positions=A, max_tokens=5, free_left=A,
             unplaced=A, stream=NUL)
APPEND = dict(k=A, k_token=512, k_head=128, v=A, v_token=512, v_head=128, slots=A, T=3, s_k=A, s_v=A, cache=A, pages=4,
              page_size=16, kv_heads=4, head_dim=128, stream=NUL)
GATHER = dict(cache=A, pages=4, page_size=16, kv_heads=4, head_dim=128, slots=A, T=3, s_k=A, s_v=A, k=A, k_token=512,
              k_head=128, v=A, v_token=512, v_head=128, stream=NUL)
ATTENTION = dict(q=A, q_token=1024, q_head=128, T=3, heads=8, q_start=A, seq_lens=A, requests=2, max_q=2, block_table=A,
                 table_width=8, table_stride=8, cache=A, pages=4, page_size=16, kv_heads=4, head_dim=128, s_k=A, s_v=A,
                 scale=0.1, window=0, out=A, o_token=1024, o_head=128, lse=A, workspace=A, workspace_bytes=64 << 20,
                 stream=NUL)
MATVEC = dict(x=A, ldx=64, q=A, s=A, s2=A, scope=1, M=1, N=8, K=64, y=A, ldy=8, y_fp32=0, stream=NUL)


def check(f, base, want, **changed):
    assert set(changed) <= set(base)
    assert f(*{**base, **changed}.values()) == want, changed


def test_slots_refusals(lib):
    f = lib.mx_kv_slots
    for name in ("seq_lens", "new_lens", "block_table", "free_pages", "free_count", "q_start", "total_lens", "slots",
                 "positions", "free_left", "unplaced"):
        check(f, SLOTS, INVALID, **{name: NUL})
        check(f, SLOTS, ALIGNMENT, **{name: A2})
    for name in ("requests", "page_size", "table_width", "max_tokens"):
        check(f, SLOTS, INVALID, **{name: 0})
        check(f, SLOTS, INVALID, **{name: -1})
    check(f, SLOTS, INVALID, free_capacity=-1)
    check(f, SLOTS, INVALID, table_stride=7)
    check(f, SLOTS, UNSUPPORTED, page_size=24)
    check(f, SLOTS, UNSUPPORTED, page_size=(1 << 20) + 16)
    check(f, SLOTS, UNSUPPORTED, requests=4097)
    check(f, SLOTS, UNSUPPORTED, max_tokens=1 << 31)
    check(f, SLOTS, UNSUPPORTED, table_width=1 << 30, table_stride=1 << 30)


@pytest.mark.parametrize("name", ["append", "gather"])
def test_cache_refusals(lib, name):
    f, base = (lib.mx_nvfp4_kv_append, APPEND) if name == "append" else (lib.mx_nvfp4_kv_gather, GATHER)
    for p in ("k", "v", "slots", "s_k", "s_v", "cache"):
        check(f, base, INVALID, **{p: NUL})
    for p in ("k", "v", "cache"):
        check(f, base, ALIGNMENT, **{p: A8})
    for p in ("slots", "s_k", "s_v"):
        check(f, base, ALIGNMENT, **{p: A2})
    for p in ("T", "pages", "page_size", "kv_heads", "head_dim"):
        check(f, base, INVALID, **{p: 0})
        check(f, base, INVALID, **{p: -1})
    for p in ("k_token", "v_token", "k_head", "v_head"):
        check(f, base, INVALID, **{p: 120})
        check(f, base, ALIGNMENT, **{p: 516})
    check(f, base, UNSUPPORTED, page_size=40)
    check(f, base, UNSUPPORTED, head_dim=96)
    check(f, base, UNSUPPORTED, pages=1 << 28)
    check(f, base, UNSUPPORTED, T=1 << 27)
    check(f, base, UNSUPPORTED, kv_heads=65536)


def test_attention_refusals(lib):
    f = lib.mx_nvfp4_kv_attention
    for p in ("q", "q_start", "seq_lens", "block_table", "cache", "s_k", "s_v", "out", "workspace"):
        check(f, ATTENTION, INVALID, **{p: NUL})
    for p in ("q", "cache", "out", "workspace"):
        check(f, ATTENTION, ALIGNMENT, **{p: A8})
    for p in ("q_start", "seq_lens", "block_table", "s_k", "s_v", "lse"):
        check(f, ATTENTION, ALIGNMENT, **{p: A2})
    for p in ("T", "heads", "requests", "max_q", "table_width", "pages", "page_size", "kv_heads", "head_dim"):
        check(f, ATTENTION, INVALID, **{p: 0})
        check(f, ATTENTION, INVALID, **{p: -1})
    check(f, ATTENTION, INVALID, heads=6)
    check(f, ATTENTION, INVALID, window=-1)
    check(f, ATTENTION, INVALID, scale=float("nan"))
    check(f, ATTENTION, INVALID, table_stride=7)
    check(f, ATTENTION, INVALID, workspace_bytes=lib.mx_kv_attention_workspace_bytes(128) - 1)
    check(f, ATTENTION, ALIGNMENT, q_head=132)
    check(f, ATTENTION, ALIGNMENT, o_token=1028)
    check(f, ATTENTION, UNSUPPORTED, head_dim=96)
    check(f, ATTENTION, UNSUPPORTED, requests=4097)
    check(f, ATTENTION, UNSUPPORTED, window=1 << 31)
    check(f, ATTENTION, UNSUPPORTED, max_q=1 << 30)
    check(f, ATTENTION, UNSUPPORTED, table_width=1 << 28, table_stride=1 << 28)


def test_matvec_refusals(lib):
    f = lib.mx_nvfp4_matvec
    for p in ("x", "q", "s", "s2", "y"):
        check(f, MATVEC, INVALID, **{p: NUL})
    for p in ("x", "q", "s", "y"):
        check(f, MATVEC, ALIGNMENT, **{p: A8})
    check(f, MATVEC, ALIGNMENT, s2=A2)
    for p in ("M", "N", "K"):
        check(f, MATVEC, INVALID, **{p: 0})
        check(f, MATVEC, INVALID, **{p: -1})
    check(f, MATVEC, INVALID, ldx=56)
    check(f, MATVEC, INVALID, ldy=7)
    check(f, MATVEC, INVALID, scope=0)
    check(f, MATVEC, INVALID, scope=3)
    check(f, MATVEC, INVALID, y_fp32=2)
    check(f, MATVEC, ALIGNMENT, ldx=68)
    check(f, MATVEC, UNSUPPORTED, M=65)
    check(f, MATVEC, UNSUPPORTED, K=40, ldx=40)
    check(f, MATVEC, UNSUPPORTED, N=1 << 31, ldy=1 << 31)


def test_binding_refuses_what_the_pointers_cannot_show():
    """The binding checks types, shapes and sizes on the tensors themselves (CPU tensors here: a correct set of arguments
    gets as far as the device check)."""
    import torch
    import microscaled_precision_numerics_gb300 as mx
    bf, i, f = torch.bfloat16, torch.int32, torch.float32
    z = lambda *s, dtype=bf: torch.zeros(s, dtype=dtype)                # noqa: E731
    cache, s, slots = z(2, 4, 1, 18 * 64, dtype=torch.uint8), z(4, dtype=f), z(3, dtype=i)
    good = (z(3, 4, 64), z(3, 4, 64), slots, s, s, cache)
    for call, args in ((mx.mx_nvfp4_kv_append, good), (mx.mx_nvfp4_kv_gather, (cache, slots, s, s, good[0], good[1]))):
        with pytest.raises(ValueError, match="CUDA"):
            call(*args)
    for bad in ((z(3, 4, 32),) + good[1:], (z(3, 4, 64, dtype=f),) + good[1:], (good[0], z(2, 4, 64)) + good[2:],
                (z(3, 64, 4).transpose(1, 2),) + good[1:], good[:2] + (z(2, dtype=i),) + good[3:],
                good[:3] + (z(3, dtype=f),) + good[4:], good[:5] + (z(2, 4, 1, 100, dtype=torch.uint8),)):
        with pytest.raises((ValueError, TypeError)) as e:
            mx.mx_nvfp4_kv_append(*bad)
        assert "CUDA" not in str(e.value)
    with pytest.raises(TypeError):
        mx.mx_nvfp4_kv_append(*good[:2], z(3, dtype=torch.int64), *good[3:])
    with pytest.raises(ValueError):
        mx.mx_nvfp4_matvec(z(1, 64), z(8, 16, dtype=torch.uint8), z(512, dtype=torch.uint8), z(1, dtype=f), 1, z(1, 8))
    with pytest.raises(TypeError):
        mx.mx_nvfp4_matvec(z(1, 64), z(8, 32, dtype=torch.uint8), z(512, dtype=torch.uint8), z(1, dtype=f), 1,
                           z(1, 8, dtype=torch.float16))
    with pytest.raises(ValueError):
        mx.mx_nvfp4_matvec(z(1, 64), z(8, 32, dtype=torch.uint8), z(100, dtype=torch.uint8), z(1, dtype=f), 1, z(1, 8))
    with pytest.raises(ValueError):
        mx.alloc_nvfp4_kv_cache(4, 24, 8, 128, "cpu")
    assert mx.alloc_nvfp4_kv_cache(4, 32, 8, 128, "cpu").shape == (4, 8, 2, 2304)


def test_reference_quantizer_agrees_with_the_oracle(orc):
    """Codes and block scales under a given S: the oracle's per-token quantizer fixes S = amax / 2688."""
    rng = np.random.default_rng(0)
    bits = ref.bf16_bits(rng.standard_normal((40, 128)) * np.exp2(rng.integers(-6, 6, (40, 1))))
    q, s, s_tok = orc.nvfp4_quantize_per_token(bits)
    codes, bs = ref.quantize_blocks(ref.bf16_value(bits).reshape(40, 8, 16), s_tok[:, None])
    assert np.array_equal(ref.pack(codes.reshape(40, 128)), q) and np.array_equal(bs, s)
    assert np.array_equal(ref.gemm_layout(bs), orc.scales_to_gemm_layout(s))
