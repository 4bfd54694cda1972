"""The 4-bit key/value cache without a GPU: pins of its oracle, and what the
entry points refuse before anything is launched."""

import numpy as np
import pytest
import torch

import exact_io_aware_84_b200 as fa
from oracle import attn_fwd_ref, kv4_attn_ref, kv4_quantise_ref, kv4_values_ref, round16_ref
from test_binding_host import _FakeCuda

P = 0x10000  # any 256-byte aligned address: no call here gets as far as using it


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_rounding_is_the_16_bit_type_s(dtype):
    t = torch.bfloat16 if dtype == "bf16" else torch.float16
    g = torch.Generator().manual_seed(1)
    x = torch.randn(4000, generator=g, dtype=torch.float64) * 10.0 ** torch.randint(-6, 4, (4000,), generator=g)
    # via float32 the rounding would be double: compare on float32 inputs
    x = x.float()
    assert np.array_equal(round16_ref(x.double().numpy(), dtype), x.to(t).double().numpy())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_quantiser_takes_the_nearest_of_its_sixteen_levels(dtype):
    t = torch.bfloat16 if dtype == "bf16" else torch.float16
    g = torch.Generator().manual_seed(2)
    x = torch.randn(300, 64, generator=g).to(t).double().numpy()
    n, s = kv4_quantise_ref(x, dtype)
    s32 = np.repeat(s, 32, -1)
    assert n.min() == -8 and n.max() <= 7
    assert np.array_equal(round16_ref(s, dtype), s)
    levels = np.arange(-8, 8)[:, None, None] * s32
    best = np.abs(levels - x).min(0)
    assert np.array_equal(np.abs(n * s32 - x), best)                       # nothing nearer
    ext = np.abs(x).reshape(300, 2, 32).max(-1)
    got = np.abs(n * s32).reshape(300, 2, 32).max(-1)
    assert np.array_equal(got, ext)                                        # the largest comes back exactly


def test_quantiser_ties_signs_and_zeros():
    x = np.zeros((4, 32))
    x[0, :3] = [8.0, -8.0, 0.5]                 # +-ext alike: the negative one decides, s = 1
    x[1, :4] = [16.0, 3.0, -3.0, -16.5]         # s = 2.0625
    x[2, :3] = [np.inf, np.nan, -1.0]
    n, s = kv4_quantise_ref(x, "bf16")
    assert s[0, 0] == 1.0 and list(n[0, :3]) == [7, -8, 1]                  # a tie goes up in x/s
    assert s[1, 0] == 2.0625 and n[1, 3] == -8 and n[1, 0] == 7
    assert s[2, 0] == -float.fromhex("0x1.fep124") and list(n[2, :3]) == [-8, 0, 0]
    assert s[3, 0] == 0 and not n[3].any() and not kv4_values_ref(x, "bf16")[3].any()


@pytest.mark.parametrize("causal", [False, True])
def test_attention_oracle_is_plain_attention_when_nothing_was_cached_before(causal):
    rng = np.random.default_rng(3)
    q, k, v = (rng.standard_normal((2, 3, 9, 64)) for _ in range(3))
    o, lse, _ = kv4_attn_ref(q, k, v, [0, 0], [9, 9], 0.125, causal)
    o_ref, lse_ref = attn_fwd_ref(q, k, v, 0.125, causal)
    assert np.allclose(o, o_ref, atol=1e-12) and np.allclose(lse, lse_ref, atol=1e-12)


def _write(lib, k=P, v=P, pool=P, table=P, start=P, count=None, B=1, Hkv=2, T=1, d=64, n_pages=4, page=16, max_pages=2,
           dtype=0):
    return lib.fa_kv4_write(k, v, pool, table, start, count, B, Hkv, T, d, n_pages, page, max_pages, dtype, None)


def _read(lib, k=P, v=P, pool=P, table=P, start=P, count=None, B=1, Hkv=2, T=1, d=64, n_pages=4, page=16, max_pages=2,
          dtype=0):
    return lib.fa_kv4_read(pool, table, start, count, k, v, B, Hkv, T, d, n_pages, page, max_pages, dtype, None)


def _fwd(lib, q=P, pool=P, table=P, start=P, count=None, o=P, lse=P, ws=P, ws_bytes=1 << 40, B=1, H=4, Hkv=2, T=1, d=64,
         n_pages=4, page=16, max_pages=2, scale=0.125, causal=1, dtype=0):
    return lib.fa_fwd_kv4(q, pool, table, start, count, o, lse, ws, ws_bytes, B, H, Hkv, T, d, n_pages, page,
                          max_pages, scale, causal, dtype, None)


SIZES = [dict(B=0), dict(Hkv=0), dict(T=0), dict(T=-3), dict(n_pages=0), dict(max_pages=0), dict(page=0), dict(page=8),
         dict(page=48), dict(page=512), dict(page=256, max_pages=1 << 23), dict(B=1 << 20, Hkv=1 << 10, T=4),
         dict(B=1 << 20, Hkv=1 << 12)]


@pytest.mark.parametrize("call", [_write, _read, _fwd])
def test_sizes_are_refused(call):
    lib = fa.load_library()
    for kw in SIZES:
        if call is _fwd and "Hkv" in kw:
            kw = dict(kw, H=kw["Hkv"])
        assert call(lib, **kw) == fa.FA_ERR_INVALID_ARG, kw
    assert call(lib, d=96) == fa.FA_ERR_UNSUPPORTED
    assert call(lib, dtype=4) == fa.FA_ERR_UNSUPPORTED
    for name in ("pool", "table", "start"):
        assert call(lib, **{name: None}) == fa.FA_ERR_INVALID_ARG
    assert call(lib, pool=P + 8) == fa.FA_ERR_MISALIGNED
    for name in ("table", "start", "count"):
        assert call(lib, **{name: P + 2}) == fa.FA_ERR_MISALIGNED


def test_row_arguments_are_refused():
    lib = fa.load_library()
    for call in (_write, _read):
        assert call(lib, k=None) == fa.FA_ERR_INVALID_ARG
        assert call(lib, v=None) == fa.FA_ERR_INVALID_ARG
        assert call(lib, v=P + 8) == fa.FA_ERR_MISALIGNED
        assert call(lib, dtype=2) == fa.FA_ERR_UNSUPPORTED       # rows have no float32 form
    assert _fwd(lib, q=None) == fa.FA_ERR_INVALID_ARG
    assert _fwd(lib, lse=None) == fa.FA_ERR_INVALID_ARG
    assert _fwd(lib, H=5) == fa.FA_ERR_INVALID_ARG
    assert _fwd(lib, scale=0.0) == fa.FA_ERR_INVALID_ARG
    assert _fwd(lib, scale=float("nan")) == fa.FA_ERR_INVALID_ARG
    assert _fwd(lib, o=P + 4) == fa.FA_ERR_MISALIGNED
    assert _fwd(lib, ws=None) == fa.FA_ERR_WORKSPACE
    assert _fwd(lib, ws_bytes=0) == fa.FA_ERR_WORKSPACE
    assert _fwd(lib, ws=P + 16) == fa.FA_ERR_MISALIGNED


def test_sizes_of_pool_and_workspace():
    assert fa.fa_kv4_pool_bytes(5, 3, 32, 128) == 5 * 3 * 32 * 128 * 2 * 9 // 16
    assert fa.fa_kv4_pool_bytes(5, 3, 24, 128) == 0
    assert fa.fa_kv4_pool_bytes(1 << 20, 8, 256, 128) == (1 << 20) * 8 * 16 * 18 * 128   # past 32 bits
    assert fa.fa_fwd_kv4_workspace_size(2, 8, 2, 1, 128) > 0
    assert fa.fa_fwd_kv4_workspace_size(2, 8, 3, 1, 128) == 0
    assert fa.fa_status_string(fa.FA_ERR_PAGE) == "FA_ERR_PAGE"
    with pytest.raises(ValueError):
        fa.fa_kv4_pool(4, 2, 20, 64, device="cpu")


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_valid_calls_without_a_device_report_it():
    lib = fa.load_library()
    for call in (_write, _read, _fwd):
        assert call(lib) == fa.FA_ERR_NO_DEVICE


class _Ints(_FakeCuda):
    def __init__(self, shape, dtype=torch.int32, **kw):
        super().__init__(shape, dtype=dtype, **kw)


class _Strided(_FakeCuda):
    def is_contiguous(self):
        return False


def _good():
    return dict(rows=_FakeCuda((3, 4, 5, 64)), pool=_FakeCuda((7, 4, 2, 18 * 64), dtype=torch.uint8),
                page_table=_Ints((3, 6)), start=_Ints((3,)), count=_Ints((3,)))


BAD = [("rows", torch.zeros(3, 4, 5, 64, dtype=torch.bfloat16), "CUDA"),
       ("rows", _Strided((3, 4, 5, 64)), "contiguous"),
       ("pool", torch.zeros(7, 4, 2, 18 * 64, dtype=torch.uint8), "pool"),
       ("pool", _FakeCuda((7, 4, 2, 18 * 64)), "pool"),
       ("pool", _FakeCuda((7, 4, 2, 18 * 128), dtype=torch.uint8), "pool holds"),
       ("pool", _FakeCuda((7, 4, 2, 18 * 64), dtype=torch.uint8, device="cuda:1"), "device"),
       ("page_table", _Ints((2, 6)), "page_table"),
       ("page_table", _Ints((3, 6), dtype=torch.int64), "int32"),
       ("page_table", torch.zeros(3, 6, dtype=torch.int32), "CUDA"),
       ("start", _Ints((3, 1)), "start"),
       ("start", _Ints((4,)), "start"),
       ("start", torch.zeros(3, dtype=torch.int32), "CUDA"),
       ("start", _Ints((3,), device="cuda:1"), "device"),
       ("count", _Ints((2,)), "count"),
       ("count", _Ints((3,), dtype=torch.int64), "int32")]


@pytest.mark.parametrize("name,value,word", BAD)
def test_binding_refuses_before_the_library_is_reached(name, value, word, monkeypatch):
    monkeypatch.setattr(fa, "load_library", lambda: pytest.fail("the library must not be reached"))
    a = dict(_good(), **{name: value})
    cache = (a["pool"], a["page_table"], a["start"], a["count"])
    with pytest.raises(ValueError, match=word):
        fa.fa_kv4_write(a["rows"], a["rows"], *cache)
    with pytest.raises(ValueError, match=word):
        fa.fa_fwd_kv4(a["rows"], *cache)
    with pytest.raises(ValueError, match=word):
        fa.fa_kv4_read(*cache, k=a["rows"], v=a["rows"])


def test_binding_refuses_what_does_not_fit_together(monkeypatch):
    monkeypatch.setattr(fa, "load_library", lambda: pytest.fail("the library must not be reached"))
    a = _good()
    cache = (a["pool"], a["page_table"], a["start"], a["count"])
    with pytest.raises(ValueError, match="match"):
        fa.fa_kv4_write(a["rows"], _FakeCuda((3, 4, 5, 64), dtype=torch.float16), *cache)
    with pytest.raises(ValueError, match="multiple"):
        fa.fa_fwd_kv4(_FakeCuda((3, 6, 5, 64)), *cache)
    with pytest.raises(ValueError, match="N and dtype"):
        fa.fa_kv4_read(*cache, N=4)
    with pytest.raises(ValueError, match="N and dtype"):
        fa.fa_kv4_read(*cache, N=4, k=a["rows"], v=a["rows"])
    with pytest.raises(ValueError, match="both"):
        fa.fa_kv4_read(*cache, k=a["rows"])
