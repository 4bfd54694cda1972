"""The 4-bit key/value cache on the GPU (fa_kv4_write, fa_kv4_read, fa_fwd_kv4)
against the float64 oracle.

Tolerances.  What is read back is one rounding of n s to the 16-bit type:
equal.  For attention let A = sum_j P_j |v_j| of an output element, u the half
step of O's type (eps/2; 0 for float32) and delta a bound on the error of a
score S in natural-log units:
  * a score's group sums add products of at most (256 + 15) |q| and start at
    264 |q| in float32, at most 3 roundings or truncations of 2^-23 relative:
    delta1 = 3 * 2^-23 * 535 * scale * sum_g |s_g| sum_{i in g} |q_i|, and
    joining groups, scaling and the exponent's argument add
    delta2 = 8 * 2^-24 * |S|max;
  * LSE: delta plus 2^-14 for exp, log and the float32 sums (625 additions of
    2^-24 each at the longest here);
  * O: A (2^-11 + 2 delta + 2^-13) for P s rounded to fp16 (half a step, 2^-11),
    the scores' errors in numerator and denominator, and exp and sums; plus
    2^-24 max|v| per key for P s below fp16's normal range; plus u |O|.
"""

import numpy as np
import pytest
import torch

import exact_io_aware_84_b200 as fa
from oracle import kv4_attn_ref, kv4_quantise_ref, kv4_values_ref, round16_ref
from parity import to64

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _rows(g, dtype, *shape):
    return torch.randn(*shape, generator=g).to(TYPES[dtype])


def _table(g, B, per, n_pages):
    return torch.randperm(n_pages, generator=g)[: B * per].reshape(B, per).to(torch.int32)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Cache:
    """A pool with random pages, filled with 0xff bytes (NaN scales) first, and what it should hold."""

    def __init__(self, B, Hkv, d, dtype, page, longest, seed=0, spare=3):
        self.g = torch.Generator().manual_seed(seed)
        self.B, self.Hkv, self.d, self.dtype, self.page = B, Hkv, d, dtype, page
        self.per = -(-longest // page)
        n_pages = B * self.per + spare
        self.pool = fa.fa_kv4_pool(n_pages, Hkv, page, d)
        self.pool.fill_(255)
        self.table = _table(self.g, B, self.per, n_pages).cuda()
        self.k = np.zeros((B, Hkv, self.per * page, d))
        self.v = np.zeros_like(self.k)
        self.ks = np.zeros((B, Hkv, self.per * page, d // 32))

    def write(self, start, T, count=None, k=None, v=None):
        k = _rows(self.g, self.dtype, self.B, self.Hkv, T, self.d) if k is None else k
        v = _rows(self.g, self.dtype, self.B, self.Hkv, T, self.d) if v is None else v
        fa.fa_kv4_write(k.cuda(), v.cuda(), self.pool, self.table, _ints(start), None if count is None else _ints(count))
        for b in range(self.B):
            n = T if count is None else max(0, min(T, count[b]))
            at = slice(start[b], start[b] + n)
            self.k[b, :, at] = kv4_values_ref(to64(k)[b, :, :n], self.dtype)
            self.v[b, :, at] = kv4_values_ref(to64(v)[b, :, :n], self.dtype)
            self.ks[b, :, at] = kv4_quantise_ref(to64(k)[b, :, :n], self.dtype)[1]

    def check_read(self, start, N, count=None):
        k, v = fa.fa_kv4_read(self.pool, self.table, _ints(start), None if count is None else _ints(count), N=N,
                              dtype=TYPES[self.dtype])
        for got, ref in ((k, self.k), (v, self.v)):
            want = np.zeros((self.B, self.Hkv, N, self.d))
            for b in range(self.B):
                n = N if count is None else max(0, min(N, count[b]))
                want[b, :, :n] = round16_ref(ref[b, :, start[b] : start[b] + n], self.dtype)
            assert np.array_equal(to64(got), want)

    def check_attention(self, q, start, count=None, causal=True, scale=None, o_fp32=False, missing=None, **kw):
        T = q.shape[2]
        n = [T] * self.B if count is None else [max(0, min(T, c)) for c in count]
        scale = self.d**-0.5 if scale is None else scale
        o, lse = fa.fa_fwd_kv4(q.cuda(), self.pool, self.table, _ints(start), None if count is None else _ints(count),
                               causal=causal, scale=scale, o_fp32=o_fp32, **kw)
        check(self, q, o, lse, start, n, causal, scale, missing)
        return o, lse


def check(c, q, o, lse, start, n, causal, scale, missing=None):
    torch.cuda.synchronize()
    q64 = to64(q)
    o_ref, lse_ref, a = kv4_attn_ref(q64, c.k, c.v, start, n, scale, causal, missing)
    group = q.shape[1] // c.Hkv
    qa = np.abs(q64).reshape(*q64.shape[:-1], -1, 32).sum(-1)                      # [B,H,T,W]
    s = np.repeat(np.abs(c.ks).max(2), group, 1)                                   # [B,H,W]: largest over the keys
    kk = np.repeat(np.abs(c.k).max(2), group, 1)
    bound = scale * (qa * s[:, :, None]).sum(-1)
    most = scale * (np.abs(q64) * kk[:, :, None]).sum(-1)                          # >= |S|
    delta = 3 * 2.0**-23 * 535 * bound + 8 * 2.0**-24 * most
    got_o, got_l = to64(o), to64(lse)
    empty = np.isinf(lse_ref)
    assert np.array_equal(np.isinf(got_l) & (got_l < 0), empty)
    assert not got_o[empty].any()
    off_l = np.abs(np.where(empty, 0, got_l) - np.where(empty, 0, lse_ref))
    assert (off_l <= delta + 2.0**-14).all(), f"LSE off by {off_l.max():.3e}, delta {delta.max():.3e}"
    u = 0.0 if o.dtype == torch.float32 else torch.finfo(o.dtype).eps / 2
    keys = c.k.shape[2]
    tol = a * (2.0**-11 + 2 * delta[..., None] + 2.0**-13) + u * np.abs(o_ref) + keys * 2.0**-24 * np.abs(c.v).max() / 64
    off = np.abs(got_o - o_ref)
    assert (off <= tol).all(), f"O off by {off.max():.3e} where {tol.reshape(-1)[(off - tol).argmax()]:.3e} is allowed"


def _ok():
    assert fa.fa_last_device_status() == fa.FA_OK


# ---------------------------------------------------------------- writing and reading back


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("start,T", [(0, 1), (1, 1), (15, 1), (0, 16), (3, 2), (7, 50), (30, 3), (0, 300)])
def test_written_rows_read_back(start, T, page, d, dtype):
    c = Cache(2, 3, d, dtype, page, start + 16 + T, seed=start + T + d)
    first = [start, start + 16]
    c.write(first, T)
    c.check_read(first, T)
    _ok()


def test_counts_cut_rows_and_clamp():
    c = Cache(5, 2, 64, "bf16", 32, 80, seed=4)
    c.write([0] * 5, 70)
    before = c.pool.clone()
    c.write([11, 12, 13, 14, 15], 9, count=[0, 1, 8, 99, -3])
    c.check_read([0] * 5, 70, count=[70, 0, 69, 200, -1])
    c.check_read([0] * 5, 70)
    # nothing but the pages of sequences 1, 2 and 3 has changed
    same = [int(p) for b in (0, 4) for p in c.table[b]] + [p for p in range(c.pool.shape[0]) if p not in c.table]
    assert torch.equal(c.pool[same], before[same])
    _ok()


@pytest.mark.parametrize("d", [64, 128])
def test_a_token_touches_no_other_token_s_bytes(d):
    c = Cache(1, 2, d, "fp16", 16, 64, seed=5)
    c.write([0], 64)
    for at in (0, 1, 17, 30, 63):
        c.write([at], 1)
        c.check_read([0], 64)
    _ok()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_values_that_quantisers_trip_over(dtype):
    t = TYPES[dtype]
    top, tiny = torch.finfo(t).max, torch.finfo(t).smallest_normal
    g = torch.Generator().manual_seed(6)
    k = torch.randn(1, 2, 24, 64, generator=g).to(t)
    k[0, 0, 0] = 0
    k[0, 0, 1, 3], k[0, 0, 1, 40] = float("inf"), float("-inf")
    k[0, 0, 2, 5] = float("nan")
    k[0, 0, 3] = float("nan")
    k[0, 0, 4, 0::2], k[0, 0, 4, 1::2] = top, -top
    k[0, 0, 5] = tiny
    k[0, 0, 6] = tiny / 64                                     # subnormal
    k[0, 0, 7, 7] = tiny / 8
    k[0, 0, 8] = -0.0
    k[0, 0, 9, :32] = torch.arange(32) / 2                     # ties
    k[0, 0, 9, 32:] = -torch.arange(32) / 2
    k[0, 0, 10] = 1000 + torch.arange(64) * 4                  # far from zero
    k[0, 0, 11, 0], k[0, 0, 11, 1] = 3.0, -3.0                 # both signs at the maximum
    k[0, 1] = (torch.randint(-64, 65, (24, 64), generator=g) / 16).to(t)   # many exact ties
    c = Cache(1, 2, 64, dtype, 32, 24, seed=7)
    c.write([0], 24, k=k, v=k.flip(2).contiguous())
    c.check_read([0], 24)
    _ok()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_every_ratio_of_mantissas_rounds_as_defined(dtype):
    """Every mantissa of the largest element against every other mantissa, at the exponents where codes differ, both
    signs: a group holds its largest element and 31 others."""
    t = TYPES[dtype]
    m = 128 if dtype == "bf16" else 1024
    mant = 1 + torch.arange(m, dtype=torch.float64, device="cuda") / m
    others = (mant[None, :] * 2.0 ** -torch.arange(6, dtype=torch.float64, device="cuda")[:, None]).flatten()
    others = torch.cat([others, -others])
    others = torch.cat([others, others.new_zeros(-len(others) % 31)]).reshape(-1, 31)          # [g, 31]
    for sign in (1.0, -1.0):
        x = torch.empty(m, len(others), 32, dtype=torch.float64, device="cuda")
        x[:, :, 0] = sign * mant[:, None]
        x[:, :, 1:] = torch.where(others.abs()[None] <= mant[:, None, None], others[None], 0.0)
        rows = x.reshape(-1)
        rows = torch.cat([rows, rows.new_zeros(-len(rows) % 128)]).reshape(1, 1, -1, 128).to(t)  # exact
        n = rows.shape[2]
        page = 256
        pool = fa.fa_kv4_pool(-(-n // page), 1, page, 128)
        table = torch.arange(pool.shape[0], dtype=torch.int32, device="cuda").flip(0).reshape(1, -1).contiguous()
        fa.fa_kv4_write(rows, rows.flip(2).contiguous(), pool, table, _ints([0]))
        k, v = fa.fa_kv4_read(pool, table, _ints([0]), N=n, dtype=t)
        g = rows.double().reshape(-1, 32)
        hi, lo = g.amax(1), g.amin(1)
        s = (torch.where(hi > -lo, hi, lo) / -8).to(t).double()[:, None]
        code = torch.where(s == 0, 0.0, torch.floor((2 * g / torch.where(s == 0, 1.0, s) + 1) / 2).clamp(-8, 7))
        # 2 g / s + 1 in float64 is within 2^-49 of a ratio that is a whole number or 2^-12 away from one
        want = (code * s).to(t).reshape(rows.shape)
        assert torch.equal(k, want) and torch.equal(v, want.flip(2))
    _ok()


def test_reading_leaves_the_cache_and_its_neighbours_alone():
    c = Cache(2, 2, 128, "bf16", 16, 50, seed=8)
    c.write([0, 0], 50)
    before = c.pool.clone()
    out = torch.full((2, 2, 2, 9, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    fa.fa_kv4_read(c.pool, c.table, _ints([20, 33]), k=out[0], v=out[1])
    assert torch.equal(c.pool, before)
    assert np.array_equal(to64(out[0, 0]), round16_ref(c.k[0, :, 20:29], "bf16"))
    _ok()


def test_positions_without_a_page_are_left_out_and_reported():
    c = Cache(3, 2, 64, "bf16", 16, 64, seed=9)
    c.write([0, 0, 0], 64)
    c.table[0, 1] = c.pool.shape[0]          # a page past the pool
    c.table[1, 2] = -1
    before = c.pool.clone()
    k = _rows(c.g, "bf16", 3, 2, 1, 64).cuda()
    fa.fa_kv4_write(k, k, c.pool, c.table, _ints([20, 40, 64]))      # all three missing (64: past the table)
    assert fa.fa_last_device_status() == fa.FA_ERR_PAGE
    _ok()                                    # the record is cleared
    fa.fa_kv4_write(k, k, c.pool, c.table, _ints([-1, -5, -2147483648]))
    assert fa.fa_last_device_status() == fa.FA_ERR_PAGE
    fa.fa_kv4_write(k, k, c.pool, c.table, _ints([2147483647] * 3))
    assert fa.fa_last_device_status() == fa.FA_ERR_PAGE
    assert torch.equal(c.pool, before)
    missing = np.zeros((3, 64), bool)
    missing[0, 16:32] = missing[1, 32:48] = True
    for x in (c.k, c.v):
        x[np.broadcast_to(missing[:, None, :, None], x.shape)] = 0
    c.check_read([0, 0, 0], 64)
    assert fa.fa_last_device_status() == fa.FA_ERR_PAGE
    for causal in (False, True):
        c.check_attention(_rows(c.g, "bf16", 3, 4, 2, 64), [62, 62, 62], causal=causal, missing=missing)
        assert fa.fa_last_device_status() == fa.FA_ERR_PAGE
    # a table that ends before the tokens do
    c.check_attention(_rows(c.g, "bf16", 3, 4, 2, 64), [63, 62, 100], count=[2, 2, 2], causal=False, missing=missing)
    assert fa.fa_last_device_status() == fa.FA_ERR_PAGE
    # entries past a sequence's end are not looked at
    c.table[:, 1:] = -7
    c.check_attention(_rows(c.g, "bf16", 3, 4, 1, 64), [15, 15, 3])
    _ok()


# ---------------------------------------------------------------- attention


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 1), (12, 4), (5, 1), (20, 2), (33, 1)])
@pytest.mark.parametrize("T,causal", [(1, True), (3, True), (3, False)])
def test_attention(T, causal, H, Hkv, d, dtype):
    start = [0, 14, 300]
    c = Cache(3, Hkv, d, dtype, 32, 310, seed=H + Hkv + d + T)
    c.write([0] * 3, 310)
    c.check_attention(_rows(c.g, dtype, 3, H, T, d), start, causal=causal)
    _ok()


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 500, 1023, 2049, 5000])
@pytest.mark.parametrize("page", [16, 128])
def test_lengths(length, page):
    c = Cache(2, 2, 128, "bf16", page, length, seed=length)
    c.write([0, 0], length)
    c.check_attention(_rows(c.g, "bf16", 2, 8, 1, 128), [length - 1, length // 2])
    _ok()


@pytest.mark.parametrize("T", [2, 7, 16, 40, 100])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_several_new_tokens_on_top_of_a_prefix_or_of_nothing(T, causal, d):
    c = Cache(3, 2, d, "fp16", 16, T + 130, seed=T)
    start, count = [0, 129, 57], [T, T, (T + 1) // 2]
    c.write([0] * 3, T + 130)
    c.check_attention(_rows(c.g, "fp16", 3, 6, T, d), start, count=count, causal=causal)
    _ok()


def test_rows_that_see_no_key():
    c = Cache(5, 1, 64, "bf16", 16, 40, seed=11)
    c.write([0] * 5, 40)
    q = _rows(c.g, "bf16", 5, 3, 4, 64)
    c.check_attention(q, [10, 10, 0, 36, 0], count=[0, -4, 1, 4, 99])
    _ok()
    for causal in (True, False):                                     # tokens before the sequence's start see nothing
        c.check_attention(q, [-2, -4, -50, 5, -3], causal=causal)


def test_more_sequences_than_threads_many_of_them_empty():
    B = 700
    c = Cache(B, 1, 64, "bf16", 16, 16, seed=12)
    c.write([0] * B, 16)
    count = [1 if b % 7 in (1, 5) else 0 for b in range(B)]
    start = [b % 16 for b in range(B)]
    c.check_attention(_rows(c.g, "bf16", B, 2, 1, 64), start, count=count)
    c.check_attention(_rows(c.g, "bf16", B, 2, 1, 64), start, count=[0] * B)
    c.check_attention(_rows(c.g, "bf16", B, 2, 1, 64), start, count=[0] * (B - 1) + [1])
    _ok()


def test_uneven_lengths():
    start = [0, 4000, 17, 1, 900, 63, 64, 2222, 3, 130]
    c = Cache(10, 2, 128, "fp16", 64, 4002, seed=13)
    c.write([0] * 10, 4002)
    c.check_attention(_rows(c.g, "fp16", 10, 8, 2, 128), start)
    _ok()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_peaked_scores_late_maxima_and_large_scale(dtype):
    c = Cache(1, 1, 128, dtype, 16, 1500, seed=14)
    ramp = torch.linspace(0.1, 6.0, 1500)[None, None, :, None]        # the maximum keeps growing
    c.write([0], 1500, k=(_rows(c.g, "bf16", 1, 1, 1500, 128).float() * ramp).to(TYPES[dtype]))
    c.check_attention(_rows(c.g, dtype, 1, 8, 1, 128), [1499])
    c.check_attention(_rows(c.g, dtype, 1, 8, 1, 128), [1499], scale=1.0)
    c.check_attention(_rows(c.g, dtype, 1, 8, 1, 128) * 30, [1499])
    _ok()


@pytest.mark.parametrize("dtype,low,high", [("bf16", -60, 60), ("fp16", -9, 10)])
def test_values_of_any_magnitude(dtype, low, high):
    """V's scales grow and shrink along the sequence by powers of two; so do K's and q's."""
    t = TYPES[dtype]
    for k_exp in (low // 3, 0, high // 3):
        c = Cache(1, 1, 64, dtype, 16, 800, seed=15)
        v = torch.randn(1, 1, 800, 64, generator=c.g) * torch.exp2(torch.linspace(low, high, 800))[None, None, :, None]
        k = torch.randn(1, 1, 800, 64, generator=c.g) * 2.0**k_exp
        c.write([0], 800, k=k.to(t), v=v.to(t))
        q = (torch.randn(1, 8, 1, 64, generator=c.g) * 2.0**-k_exp).to(t)
        c.check_attention(q, [799], o_fp32=True)
        c.check_attention(q, [399], o_fp32=True)
    _ok()


def test_zero_values_and_zero_queries():
    c = Cache(1, 1, 64, "bf16", 16, 200, seed=16)
    zero = torch.zeros(1, 1, 200, 64, dtype=torch.bfloat16)
    c.write([0], 200, v=zero)
    c.check_attention(_rows(c.g, "bf16", 1, 4, 1, 64), [199])
    c.write([0], 100, k=zero[:, :, :100])
    c.write([100], 100, v=zero[:, :, :100] + 2.0**-70)
    c.check_attention(torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16), [199])
    _ok()


def test_what_lies_behind_the_last_key_does_not_matter():
    c = Cache(1, 2, 128, "bf16", 64, 128, seed=17)      # Cache fills the pool with NaN scales
    c.write([0], 70)
    a = c.check_attention(_rows(c.g, "bf16", 1, 8, 1, 128), [69])
    # tokens of the future, also within the block, and at the type's largest values
    big = torch.full((1, 2, 58, 128), torch.finfo(torch.bfloat16).max, dtype=torch.bfloat16)
    c.write([70], 58, k=big, v=-big)
    c.g.manual_seed(17)
    q = _rows(c.g, "bf16", 1, 8, 1, 128)
    o1, l1 = fa.fa_fwd_kv4(q.cuda(), c.pool, c.table, _ints([69]), causal=True)
    o2, l2 = fa.fa_fwd_kv4(q.cuda(), c.pool, c.table, _ints([68]), causal=True)
    assert torch.isfinite(o1).all() and torch.isfinite(l1).all() and torch.isfinite(o2).all()
    # a causal row next to one that does see them
    q2 = _rows(c.g, "bf16", 1, 8, 2, 128) * 1e-30
    o3, l3 = fa.fa_fwd_kv4(q2.cuda(), c.pool, c.table, _ints([69]), causal=True)
    assert torch.isfinite(o3[:, :, 0]).all() and torch.isfinite(l3).all()
    _ok()


def test_a_nan_query_spoils_its_own_row_only():
    c = Cache(1, 1, 64, "bf16", 16, 100, seed=18)
    c.write([0], 100)
    q = _rows(c.g, "bf16", 1, 12, 1, 64)
    o, _ = fa.fa_fwd_kv4(q.cuda(), c.pool, c.table, _ints([99]))
    bad = q.clone()
    bad[0, 5, 0, 9] = float("nan")
    p, l = fa.fa_fwd_kv4(bad.cuda(), c.pool, c.table, _ints([99]))
    keep = [h for h in range(12) if h != 5]
    assert torch.equal(o[:, keep], p[:, keep]) and torch.isnan(p[0, 5]).all() and torch.isnan(l[0, 5]).all()
    _ok()


def test_the_same_call_twice_gives_the_same_bits():
    c = Cache(4, 2, 128, "bf16", 32, 3000, seed=19)
    c.write([0] * 4, 3000)
    q = _rows(c.g, "bf16", 4, 8, 1, 128).cuda()
    start = _ints([2999, 1500, 77, 2000])
    o1, l1 = fa.fa_fwd_kv4(q, c.pool, c.table, start)
    for _ in range(5):
        o2, l2 = fa.fa_fwd_kv4(q, c.pool, c.table, start)
        assert torch.equal(o1, o2) and torch.equal(l1, l2)
    _ok()


def test_partial_results_of_two_caches_merge():
    """The prefix in one cache, the rest in another: fa_merge joins the two."""
    a = Cache(2, 2, 64, "fp16", 16, 96, seed=20)
    b = Cache(2, 2, 64, "fp16", 16, 40, seed=21)
    a.write([0, 0], 96)
    b.write([0, 0], 40)
    q = _rows(a.g, "fp16", 2, 6, 1, 64)
    o1, l1 = a.check_attention(q, [95, 95], o_fp32=True)
    o2, l2 = b.check_attention(q, [39, 39], o_fp32=True)
    fa.fa_merge(o1, l1, o2, l2)
    joined = Cache(2, 2, 64, "fp16", 16, 136, seed=22)
    for x in ("k", "v", "ks"):
        setattr(joined, x, np.concatenate([getattr(a, x)[:, :, :96], getattr(b, x)[:, :, :40]], 2))
    check(joined, q, o1, l1, [135, 135], [1, 1], True, 64**-0.5)
    _ok()


def test_a_cache_past_four_gigabytes():
    page, Hkv, d = 256, 8, 128
    n_pages = 15000
    need = fa.fa_kv4_pool_bytes(n_pages, Hkv, page, d)
    assert need > 1 << 32
    pool = fa.fa_kv4_pool(n_pages, Hkv, page, d)
    c = Cache(2, Hkv, d, "bf16", page, 600, seed=23)
    c.pool, c.table = pool, _ints([[14999, 0, 14001], [7500, 14998, 1]])
    c.write([0, 0], 600)
    c.check_read([0, 0], 600)
    c.check_attention(_rows(c.g, "bf16", 2, 8, 1, 128), [599, 300])
    _ok()


# A table with room for 2^17 positions: the attention then cannot count on short sequences, and divides
# all of them over the whole grid; with a tight one, few and short sequences get a cluster of CTAs each.


def _room(c, positions=1 << 17):
    wide = torch.full((c.B, positions // c.page), -7, dtype=torch.int32, device="cuda")
    wide[:, : c.table.shape[1]] = c.table
    c.table = wide.contiguous()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 1), (12, 4), (4, 2), (5, 1), (33, 1)])
@pytest.mark.parametrize("T,causal", [(1, True), (3, True), (3, False)])
def test_room_for_long_sequences(T, causal, H, Hkv, d, dtype):
    start = [0, 14, 900]
    c = Cache(3, Hkv, d, dtype, 32, 910, seed=H + Hkv + d + T)
    c.write([0] * 3, 910)
    _room(c)
    c.check_attention(_rows(c.g, dtype, 3, H, T, d), start, causal=causal)
    _ok()


@pytest.mark.parametrize("length", [1, 16, 63, 64, 65, 127, 129, 1023, 2049, 5000])
def test_room_and_lengths(length):
    c = Cache(2, 2, 128, "bf16", 16, length, seed=length)
    c.write([0, 0], length)
    _room(c)
    c.check_attention(_rows(c.g, "bf16", 2, 8, 1, 128), [length - 1, length // 2])
    _ok()


@pytest.mark.parametrize("T", [2, 16, 40, 100])
@pytest.mark.parametrize("d", [64, 128])
def test_room_and_several_new_tokens(T, d):
    c = Cache(3, 2, d, "fp16", 16, T + 130, seed=T)
    start, count = [0, 129, 57], [T, T, (T + 1) // 2]
    c.write([0] * 3, T + 130)
    _room(c)
    for causal in (False, True):
        c.check_attention(_rows(c.g, "fp16", 3, 6, T, d), start, count=count, causal=causal)
    _ok()


@pytest.mark.parametrize("wide", [False, True])
def test_more_units_than_warps(wide):
    """2400 key heads of short sequences, some of them empty."""
    B = 300
    c = Cache(B, 8, 64, "bf16", 64, 64, seed=27)
    c.write([0] * B, 64)
    if wide:
        _room(c, 1 << 12)
    count = [0 if b % 11 == 3 else 1 for b in range(B)]
    c.check_attention(_rows(c.g, "bf16", B, 8, 1, 64), [(b * 7) % 64 for b in range(B)], count=count)
    _ok()


def test_room_and_rows_that_see_no_key():
    c = Cache(5, 1, 64, "bf16", 16, 40, seed=11)
    c.write([0] * 5, 40)
    _room(c)
    q = _rows(c.g, "bf16", 5, 3, 4, 64)
    c.check_attention(q, [10, 10, 0, 36, 0], count=[0, -4, 1, 4, 99])
    for causal in (True, False):
        c.check_attention(q, [-2, -4, -50, 5, -3], causal=causal)
    _ok()


def test_room_and_missing_pages():
    c = Cache(2, 2, 64, "bf16", 16, 640, seed=28)
    c.write([0, 0], 640)
    _room(c)
    c.table[0, 3], c.table[1, 20] = c.pool.shape[0], -1
    missing = np.zeros((2, 640), bool)
    missing[0, 48:64] = missing[1, 320:336] = True
    for x in (c.k, c.v):
        x[np.broadcast_to(missing[:, None, :, None], x.shape)] = 0
    c.check_attention(_rows(c.g, "bf16", 2, 4, 2, 64), [638, 600], missing=missing)
    assert fa.fa_last_device_status() == fa.FA_ERR_PAGE


@pytest.mark.parametrize("wide", [False, True])
def test_one_channel_far_above_the_others(wide):
    """q enters relative to its row's largest element, and P s_V relative to the largest scale."""
    c = Cache(2, 1, 128, "bf16", 16, 700, seed=29)
    k, v = _rows(c.g, "bf16", 2, 1, 700, 128), _rows(c.g, "bf16", 2, 1, 700, 128)
    k[..., 5] *= 2.0**-12
    v[..., 70] *= 2.0**12
    c.write([0, 0], 700, k=k, v=v)
    if wide:
        _room(c)
    q = _rows(c.g, "bf16", 2, 8, 1, 128)
    q[..., 5] *= 2.0**12
    c.check_attention(q, [699, 350])
    _ok()


# ---------------------------------------------------------------- streams, graphs, use


def test_two_streams_with_a_workspace_each():
    c = Cache(3, 2, 128, "bf16", 16, 2000, seed=24)
    c.write([0] * 3, 2000)
    q = [_rows(c.g, "bf16", 3, 8, 1, 128).cuda() for _ in range(2)]
    start = _ints([1999, 1000, 1700])
    want = [fa.fa_fwd_kv4(x, c.pool, c.table, start) for x in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    need = fa.fa_fwd_kv4_workspace_size(3, 8, 2, 1, 128)
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            o, l = torch.empty_like(want[i][0]), torch.empty_like(want[i][1])
            fa.fa_fwd_kv4(q[i], c.pool, c.table, start, o=o, lse=l, workspace=ws[i], stream=s)
            got[i].append((o, l))
    torch.cuda.synchronize()
    for i in range(2):
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])
    _ok()


def test_decoding_after_a_prefill_eager_and_in_a_graph():
    """A prompt through fa_fwd_gqa and into the cache, then token by token:
    each step writes its key and value and attends, with positions advanced on
    the device; the same steps replayed from one captured graph."""
    B, H, Hkv, d, P, steps = 2, 8, 2, 64, 37, 20
    c = Cache(B, Hkv, d, "bf16", 16, P + steps, seed=25)
    g = c.g
    k, v = (_rows(g, "bf16", B, Hkv, P, d) for _ in range(2))
    prompt_o, prompt_lse = fa.fa_fwd_gqa(_rows(g, "bf16", B, H, P, d).cuda(), k.cuda(), v.cuda(), causal=True)
    assert torch.isfinite(prompt_o.float()).all() and torch.isfinite(prompt_lse).all()
    c.write([0] * B, P, k=k, v=v)
    qs, ks, vs = ([_rows(g, "bf16", B, h, 1, d) for _ in range(steps)] for h in (H, Hkv, Hkv))
    q, kk, vv = (torch.empty_like(x[0], device="cuda") for x in (qs, ks, vs))
    start = _ints([P] * B)
    ws = torch.empty(fa.fa_fwd_kv4_workspace_size(B, H, Hkv, 1, d), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((B, H, 1), device="cuda")

    def step():
        fa.fa_kv4_write(kk, vv, c.pool, c.table, start)
        fa.fa_fwd_kv4(q, c.pool, c.table, start, o=o, lse=lse, workspace=ws, causal=True)
        start.add_(1)

    def decode(go):
        start.fill_(P)
        out = []
        for i in range(steps):
            q.copy_(qs[i]), kk.copy_(ks[i]), vv.copy_(vs[i])
            go()
            out.append((o.clone(), lse.clone()))
        return out

    eager = decode(step)
    for i in range(steps):
        c.k[:, :, P + i] = kv4_values_ref(to64(ks[i])[:, :, 0], "bf16")
        c.v[:, :, P + i] = kv4_values_ref(to64(vs[i])[:, :, 0], "bf16")
        c.ks[:, :, P + i] = kv4_quantise_ref(to64(ks[i])[:, :, 0], "bf16")[1]
    for i in (0, 1, 10, 11, steps - 1):
        check(c, qs[i], *eager[i], [P + i] * B, [1] * B, True, d**-0.5)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for a, b in zip(eager, decode(graph.replay)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.check_read([0] * B, P + steps)
    _ok()


def test_a_binding_made_workspace_and_outputs_on_a_side_stream():
    c = Cache(1, 1, 128, "fp16", 16, 900, seed=26)
    c.write([0], 900)
    q = _rows(c.g, "fp16", 1, 4, 1, 128).cuda()
    want = fa.fa_fwd_kv4(q, c.pool, c.table, _ints([899]))
    start = _ints([899])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = fa.fa_fwd_kv4(q, c.pool, c.table, start)
        k, v = fa.fa_kv4_read(c.pool, c.table, start, N=1, dtype=torch.float16)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert np.array_equal(to64(k)[0, 0, 0], round16_ref(c.k[0, 0, 899], "fp16"))
    _ok()


def test_what_a_call_allocates_belongs_to_its_stream():
    """A block that the current stream has freed but not finished reading is not
    what a call on another stream writes to."""
    c = Cache(1, 2, 128, "bf16", 16, 4096, seed=30)
    c.write([0], 4096)
    start, q = _ints([4095]), _rows(c.g, "bf16", 1, 8, 1, 128).cuda()
    want = fa.fa_fwd_kv4(q, c.pool, c.table, start)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    need = fa.fa_fwd_kv4_workspace_size(1, 8, 2, 1, 128)
    for go in (lambda s: fa.fa_kv4_read(c.pool, c.table, _ints([0]), N=4096, dtype=torch.bfloat16, stream=s),
               lambda s: fa.fa_fwd_kv4(q, c.pool, c.table, start, stream=s)):
        for stream in (side, side.cuda_stream):
            torch.cuda.empty_cache()
            a = torch.full((2 * 4096 * 128,), 3.0, dtype=torch.bfloat16, device="cuda")
            b = torch.full((need,), 5, dtype=torch.uint8, device="cuda")
            torch.cuda.synchronize()
            torch.cuda._sleep(20_000_000)            # the current stream is busy, then reads a and b
            a2, b2 = a + 0, b + 0
            del a, b
            got = go(stream)
            torch.cuda.synchronize()
            assert (a2 == 3).all() and (b2 == 5).all()
            if got[0].shape == want[0].shape:
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    _ok()


@pytest.mark.parametrize("wide", [False, True])
def test_a_withheld_arrival_ends_with_a_status(wide):
    c = Cache(2, 2, 128, "bf16", 16, 2100, seed=31)
    c.write([0, 0], 2100)
    if wide:
        _room(c)
    q = _rows(c.g, "bf16", 2, 8, 1, 128)
    _ok()
    assert fa.fa_debug_set_wait_limit_ms(100) == fa.FA_OK
    assert fa.fa_debug_set_flags(4) == fa.FA_OK
    try:
        fa.fa_fwd_kv4(q.cuda(), c.pool, c.table, _ints([2099, 900]))
        assert fa.fa_last_device_status() == fa.FA_ERR_TIMEOUT
        assert fa.fa_last_device_status() == fa.FA_OK
    finally:
        fa.fa_debug_set_flags(0)
        fa.fa_debug_set_wait_limit_ms(1000)
    c.check_attention(q, [2099, 900])
    _ok()


@pytest.mark.parametrize("compiled", [True, False])
def test_both_bindings_do_the_same(compiled, monkeypatch):
    """The compiled binding and the package's own path: results, what is allocated, what is handed back."""
    if not compiled:
        monkeypatch.setattr(fa, "_compiled", lambda t: None)
    else:
        assert fa._compiled(torch.empty(1, device="cuda")) is not None
    c = Cache(3, 2, 64, "fp16", 16, 200, seed=32)
    c.write([0, 0, 0], 100)
    c.write([100, 0, 7], 20, count=[20, 3, 0])
    c.check_read([0, 0, 0], 120, count=[120, 100, 100])
    c.check_read([0, 1, 2], 90)
    q = _rows(c.g, "fp16", 3, 4, 2, 64)
    o, lse = c.check_attention(q, [60, 50, 98])
    assert o.dtype == torch.float16 and o.shape == q.shape and lse.shape == (3, 4, 2)
    o, _ = c.check_attention(q, [60, 50, 98], o_fp32=True, causal=False, count=[2, 1, 0], scale=0.25)
    assert o.dtype == torch.float32
    mine = torch.full((3, 4, 2, 64), 7.0, device="cuda"), torch.empty((3, 4, 2), device="cuda")
    ws = torch.empty(fa.fa_fwd_kv4_workspace_size(3, 4, 2, 2, 64), dtype=torch.uint8, device="cuda")
    got = fa.fa_fwd_kv4(q.cuda(), c.pool, c.table, _ints([60, 50, 98]), o=mine[0], lse=mine[1], workspace=ws, scale=1)
    assert got[0] is mine[0] and got[1] is mine[1]
    check(c, q, *got, [60, 50, 98], [2, 2, 2], False, 1.0)
    k, v = fa.fa_kv4_read(c.pool, c.table, _ints([5, 5, 5]), N=1, dtype=torch.float16)
    assert k.shape == v.shape == (3, 2, 1, 64) and k.data_ptr() != v.data_ptr()
    _ok()


@pytest.mark.parametrize("compiled", [True, False])
def test_both_bindings_refuse_the_same(compiled, monkeypatch):
    if not compiled:
        monkeypatch.setattr(fa, "_compiled", lambda t: None)
    c = Cache(2, 2, 64, "bf16", 16, 32, seed=33)
    k = _rows(c.g, "bf16", 2, 2, 3, 64).cuda()
    s = _ints([0, 0])
    bad = [(k, k.transpose(2, 3), c.pool, c.table, s), (k.float(), k.float(), c.pool, c.table, s), (k, k.half(), c.pool, c.table, s),
           (k, k[:1], c.pool, c.table, s), (k.cpu(), k, c.pool, c.table, s), (k, k, c.pool[:, :1], c.table, s),
           (k, k, c.pool.float(), c.table, s), (k, k, c.pool, c.table.long(), s), (k, k, c.pool, c.table[:1], s),
           (k, k, c.pool, c.table, s.long()), (k, k, c.pool, c.table, _ints([0])), (k, k, c.pool, c.table, s.cpu()),
           (k, k, c.pool, c.table.t(), s)]
    for args in bad:
        with pytest.raises((ValueError, TypeError)):
            fa.fa_kv4_write(*args)
        with pytest.raises((ValueError, TypeError, fa.FAError)):
            if args[1] is k or args[0].dtype == torch.float32:
                fa.fa_fwd_kv4(args[0], *args[2:])
            else:
                raise ValueError
    for kw in (dict(o=torch.empty(2, 2, 3, 64, device="cuda", dtype=torch.float64)), dict(lse=torch.empty(2, 2, 4, device="cuda")),
               dict(workspace=torch.empty(1 << 25, dtype=torch.uint8)), dict(o=torch.empty(2, 2, 3, 64))):
        with pytest.raises(ValueError):
            fa.fa_fwd_kv4(k, c.pool, c.table, s, **kw)
    with pytest.raises(fa.FAError, match="WORKSPACE"):
        fa.fa_fwd_kv4(k, c.pool, c.table, s, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fa.FAError, match="INVALID"):
        fa.fa_fwd_kv4(k, c.pool, c.table, s, scale=-1.0)
    with pytest.raises(fa.FAError, match="INVALID"):
        fa.fa_fwd_kv4(torch.cat([k, k[:, :1]], 1)[:, :0].contiguous(), c.pool, c.table, s)
    for n, t in ((None, torch.bfloat16), (4, torch.float32), (4, None)):
        with pytest.raises(ValueError):
            fa.fa_kv4_read(c.pool, c.table, s, N=n, dtype=t)
    with pytest.raises((RuntimeError, fa.FAError)):
        fa.fa_kv4_read(c.pool, c.table, s, N=0, dtype=torch.bfloat16)
    _ok()
