"""The 4-bit cache where calls touch its borders, against the float64 oracle
with a bound for each row of its own.

Tolerance of a row of O.  Only the keys j that the row sees enter it, with
P_j, A = sum_j P_j |v_j|, u and delta (from these keys' scales) as in
test_kv4_gpu: A (2^-11 + 2 delta + 2^-13) + u |O|.  P s_V is rounded to fp16
after a power of two has brought the row's largest product so far to 2^6 or
above, so that products below fp16's normal range are off by 2^-25 there: at
most 2^-31 of the largest, times |n| <= 8 a key, where the largest |v| of a
key is 8 s: keys * 2^-31 * max_j(P_j max|v_j|).  16-bit results add half a
step of their subnormals.
"""

import numpy as np
import pytest
import torch

import exact_io_aware_84_b200 as fa
from oracle import kv4_attn_ref, round16_ref
from parity import to64
from test_kv4_gpu import TYPES, Cache, _ints, _ok, _room, _rows

pytestmark = pytest.mark.gpu


def _seen(c, b, t, start, n, causal, missing):
    keys = start[b] + t + 1 if causal else start[b] + n[b]
    j = np.arange(max(0, min(keys, c.k.shape[2])))
    return j if missing is None else j[~missing[b, j]]


def strict(c, q, o, lse, start, n=None, causal=True, scale=None, missing=None):
    """O and LSE of every row against the oracle; each row's bound is made from the keys that it sees."""
    torch.cuda.synchronize()
    B, H, T, d = q.shape
    n = [T] * B if n is None else n
    scale = d**-0.5 if scale is None else scale
    q64, got_o, got_l = to64(q), to64(o), to64(lse)
    o_ref, lse_ref, a = kv4_attn_ref(q64, c.k, c.v, start, n, scale, causal, missing)
    u = 0.0 if o.dtype == torch.float32 else torch.finfo(o.dtype).eps / 2
    least = {torch.float32: 0.0, torch.bfloat16: 2.0**-134, torch.float16: 2.0**-25}[o.dtype]
    group = H // c.Hkv
    for b in range(B):
        for t in range(T):
            j = _seen(c, b, t, start, n, causal, missing) if t < n[b] else []
            for h in range(H):
                where = f"row {b, h, t}"
                if not len(j):
                    assert not got_o[b, h, t].any() and got_l[b, h, t] == -np.inf, where
                    continue
                k, v, ks = c.k[b, h // group, j], c.v[b, h // group, j], np.abs(c.ks[b, h // group, j]).max(0)
                qa = np.abs(q64[b, h, t])
                delta = (3 * 2.0**-23 * 535 * scale * (qa.reshape(-1, 32).sum(-1) * ks).sum()
                         + 8 * 2.0**-24 * scale * (qa * np.abs(k).max(0)).sum())
                assert abs(got_l[b, h, t] - lse_ref[b, h, t]) <= delta + 2.0**-14, f"LSE of {where}: {got_l[b, h, t]}, {lse_ref[b, h, t]}"
                s = scale * (k @ q64[b, h, t])
                p = np.exp(s - lse_ref[b, h, t])
                tol = (a[b, h, t] * (2.0**-11 + 2 * delta + 2.0**-13) + u * np.abs(o_ref[b, h, t]) + least
                       + len(j) * 2.0**-31 * (p * np.abs(v).max(-1)).max())
                off = np.abs(got_o[b, h, t] - o_ref[b, h, t])
                at = (off - tol).argmax() if not np.isnan(off).any() else np.isnan(off).argmax()
                assert (off <= tol).all(), (f"O of {where}, element {at}: {got_o[b, h, t, at]:.6e} for {o_ref[b, h, t, at]:.6e}, "
                                            f"{tol[at]:.3e} is allowed")


def attend(c, q, start, count=None, causal=True, scale=None, missing=None, **kw):
    """One call, checked row by row."""
    n = None if count is None else [max(0, min(q.shape[2], x)) for x in count]
    o, lse = fa.fa_fwd_kv4(q.cuda(), c.pool, c.table, _ints(start), None if count is None else _ints(count), causal=causal,
                           scale=scale, **kw)
    strict(c, q, o, lse, start, n, causal, scale, missing)
    return o, lse


# ---------------------------------------------------------------- the division over the whole grid


@pytest.mark.parametrize("B", [3, 127, 128, 129, 300])
def test_first_copies_after_the_plan(B):
    """The plan's sums lie where each CTA's first copies go (one sequence a thread, and several): call after call the
    same bits, and the right ones."""
    c = Cache(B, 1, 64, "bf16", 16, 96, seed=B)
    c.write([0] * B, 96)
    _room(c, 1 << 14)
    start = [(b * 37) % 96 for b in range(B)]
    q = _rows(c.g, "bf16", B, 2, 1, 64)
    o, lse = attend(c, q, start)
    q, s = q.cuda(), _ints(start)
    for _ in range(50):
        o2, lse2 = fa.fa_fwd_kv4(q, c.pool, c.table, s, causal=True)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    _ok()


# ---------------------------------------------------------------- writing and reading parts of a block


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
def test_every_part_of_a_block_is_written_and_read(d, dtype):
    """Some lanes of a warp have rows to write or read, others none: every first position and length within two blocks,
    a sequence each."""
    part = [(at, n) for at in range(16) for n in range(1, 18)]
    B = len(part)
    c = Cache(B, 1, d, dtype, 16, 33, seed=d)
    c.write([0] * B, 33)
    c.check_read([0] * B, 33)
    start, count = [at for at, _ in part], [n for _, n in part]
    c.write(start, 17, count=count)
    c.check_read([0] * B, 33)
    c.check_read(start, 17, count=count)
    _ok()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17])
def test_rows_end_anywhere_in_a_block(n, d, dtype):
    c = Cache(16, 2, d, dtype, 16, 33, seed=n + d)
    c.write([0] * 16, 33)
    c.check_read(list(range(16)), n)
    c.write(list(range(16)), n)
    c.check_read(list(range(16)), n)
    c.check_read([0] * 16, 33)
    _ok()


# ---------------------------------------------------------------- values far apart

SHARED = [(1, 1), (2, 1), (4, 2), (4, 1), (8, 1), (24, 2)]   # rows a key head: one column a row, two, four; two tiles; ...
FAR = [("bf16", 2.0**100), ("bf16", 2.0**30), ("fp16", 60000.0)]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype,far", FAR)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", SHARED)
def test_a_row_does_not_feel_keys_that_only_later_rows_see(H, Hkv, d, dtype, far, wide):
    """The last two of three tokens bring values far above all others; small ones all around (fp16: far below 1)."""
    c = Cache(2, Hkv, d, dtype, 16, 420, seed=H + d)
    small = 1.0 if dtype == "bf16" else 2.0**-10
    v = _rows(c.g, dtype, 2, Hkv, 420, d) * small
    start = [400, 61]
    for b, at in enumerate(start):
        v[b, :, at + 1] = far
        v[b, :, at + 2] = -far
    c.write([0, 0], 420, v=v)
    if wide:
        _room(c)
    attend(c, _rows(c.g, dtype, 2, H, 3, d), start, o_fp32=True)
    attend(c, _rows(c.g, dtype, 2, H, 3, d), start, count=[2, 1])
    _ok()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,T", [(1, 1), (4, 1), (8, 1), (5, 4)])
def test_a_key_of_no_weight_does_not_matter_whatever_its_value(H, T, d, wide):
    """One key's value is near the type's largest and its weight e^-200 or less: before, between and behind the others,
    with the maximum reached before it and after it."""
    for length, at in ((40, 0), (40, 17), (700, 0), (700, 333), (700, 690), (3000, 5), (3000, 64)):
        c = Cache(1, 1, d, "bf16", 16, length, seed=length + at)
        k, v = (_rows(c.g, "bf16", 1, 1, length, d) for _ in range(2))
        k += 3.0 * 8 / d**0.5
        k[:, :, at] = -30.0
        v[:, :, at] = 2.0**126
        c.write([0], length, k=k, v=v)
        if wide:
            _room(c)
        q = (_rows(c.g, "bf16", 1, H, T, d).float().abs() + 1).bfloat16()
        attend(c, q, [length - T], o_fp32=True)
    _ok()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("H,d", [(1, 64), (8, 128), (12, 128)])
def test_a_key_of_all_the_weight_and_no_value_leaves_the_others_exact(H, d, dtype, wide):
    for at in (0, 250):
        c = Cache(1, 1, d, dtype, 16, 500, seed=at + H)
        k, v = (_rows(c.g, dtype, 1, 1, 500, d) for _ in range(2))
        k *= 0.1
        k[:, :, at] = 24.0 * 8 / d / d**0.5 * 8          # scores of 1.5 * 24 or so above the others'
        v[:, :, at] = 0
        c.write([0], 500, k=k, v=v)
        if wide:
            _room(c)
        q = (_rows(c.g, dtype, 1, H, 1, d).float().abs() * 0.1 + 1).to(TYPES[dtype])
        attend(c, q, [499], o_fp32=True)
    _ok()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype,low,high", [("bf16", -60, 60), ("bf16", -125, 0), ("fp16", -14, 12)])
def test_magnitudes_along_the_sequence_row_by_row(dtype, low, high, wide):
    for up in (True, False):
        c = Cache(1, 1, 64, dtype, 16, 800, seed=int(up))
        ramp = torch.linspace(low, high, 800) if up else torch.linspace(high, low, 800)
        v = (torch.randn(1, 1, 800, 64, generator=c.g) * torch.exp2(ramp)[None, None, :, None]).to(TYPES[dtype])
        c.write([0], 800, v=v)
        if wide:
            _room(c)
        for H, T, at in ((8, 1, 799), (8, 1, 399), (1, 1, 90), (4, 3, 500), (4, 40, 700)):
            attend(c, _rows(c.g, dtype, 1, H, T, 64), [at], o_fp32=True)
    _ok()


@pytest.mark.parametrize("wide", [False, True])
def test_results_keep_their_bits_when_the_future_is_written(wide):
    c = Cache(1, 2, 128, "bf16", 64, 128, seed=17)      # Cache fills the pool with NaN scales
    if wide:
        _room(c)
    c.write([0], 70)
    q = _rows(c.g, "bf16", 1, 8, 1, 128)
    before = [attend(c, q, [at]) for at in (69, 68, 40)]
    big = torch.full((1, 2, 58, 128), torch.finfo(torch.bfloat16).max, dtype=torch.bfloat16)
    c.write([70], 58, k=big, v=-big)
    for at, (o, lse) in zip((69, 68, 40), before):
        o2, lse2 = fa.fa_fwd_kv4(q.cuda(), c.pool, c.table, _ints([at]), causal=True)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # the first of two causal rows, the second of which sees one of them
    q2 = torch.cat([q, q * 2.0**-110], 2)
    o3, lse3 = fa.fa_fwd_kv4(q2.cuda(), c.pool, c.table, _ints([69]), causal=True)
    c.k, c.v, c.ks = c.k[:, :, :70], c.v[:, :, :70], c.ks[:, :, :70]
    strict(c, q, o3[:, :, :1], lse3[:, :, :1], [69])
    _ok()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("apart", [12, 20, 24])
@pytest.mark.parametrize("H,d", [(1, 64), (2, 128), (4, 128), (8, 64), (16, 128)])
def test_groups_of_one_row_far_apart(H, d, apart, wide):
    """The first 32 elements of V lie far above the others, which are held to their own size as far as it is promised."""
    c = Cache(1, 1, d, "bf16", 16, 2000, seed=apart + H)
    v = _rows(c.g, "bf16", 1, 1, 2000, d)
    v[..., :32] *= 2.0**apart
    c.write([0], 2000, v=v)
    if wide:
        _room(c)
    attend(c, _rows(c.g, "bf16", 1, H, 1, d), [1999], o_fp32=True)
    _ok()


# ---------------------------------------------------------------- idle sequences of a padded batch


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("idle", [0, -5])
def test_an_idle_sequence_s_pages_are_not_looked_at(idle, d):
    """Sequences without tokens, whose pages do not exist and whose starts lie inside a block, past the table or before it."""
    c = Cache(6, 2, d, "bf16", 16, 48, seed=40)
    c.write([0] * 6, 48)
    before = c.pool.clone()
    c.table[1:] = -7
    start, count = [5, 7, 40, 48 + 9, -3, 2147483647], [3, idle, idle, idle, idle, idle]
    c.write(start, 3, count=count)
    _ok()
    rows = fa.fa_kv4_read(c.pool, c.table, _ints(start), _ints(count), N=20, dtype=torch.bfloat16)
    _ok()
    for x, held in zip(rows, (c.k, c.v)):
        assert not x[1:].any() and not x[0, :, 3:].any()
        assert np.array_equal(to64(x[0, :, :3]), round16_ref(held[0, :, 5:8], "bf16"))
    attend(c, _rows(c.g, "bf16", 6, 4, 3, d), start, count=count)
    _ok()
    used = (c.pool != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert used in ([], [int(c.table[0, 0])])


# ---------------------------------------------------------------- statuses


@pytest.mark.parametrize("page_first", [True, False])
def test_a_missing_page_does_not_hide_a_timeout(page_first):
    c = Cache(1, 2, 128, "bf16", 16, 200, seed=41)
    c.write([0], 200)
    q = _rows(c.g, "bf16", 1, 8, 1, 128).cuda()
    k = _rows(c.g, "bf16", 1, 2, 1, 128).cuda()
    _ok()

    def no_page():
        fa.fa_kv4_write(k, k, c.pool, c.table, _ints([c.per * 16]))

    if page_first:
        no_page()
    assert fa.fa_debug_set_wait_limit_ms(100) == fa.FA_OK
    assert fa.fa_debug_set_flags(4) == fa.FA_OK
    try:
        fa.fa_fwd_kv4(q, c.pool, c.table, _ints([199]))
        torch.cuda.synchronize()
    finally:
        fa.fa_debug_set_flags(0)
        fa.fa_debug_set_wait_limit_ms(1000)
    if not page_first:
        no_page()
    assert fa.fa_last_device_status() == fa.FA_ERR_TIMEOUT
    assert fa.fa_last_device_status() == fa.FA_ERR_PAGE
    _ok()


# ---------------------------------------------------------------- queries and scales at the ends


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("scale", [1e-20, 1e-25, 1e-38, 1e-45])
def test_rows_of_zeros_under_a_tiny_scale(scale, dtype, wide):
    """Every key that a row sees has the same weight, and those that it does not see have none."""
    c = Cache(2, 1, 64, dtype, 16, 150, seed=42)
    c.write([0, 0], 150)
    if wide:
        _room(c)
    q = torch.zeros(2, 4, 3, 64, dtype=TYPES[dtype])
    q[:, 1] = _rows(c.g, dtype, 2, 3, 64)
    attend(c, q, [100, 3], scale=scale)
    _ok()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("o_fp32", [True, False])
@pytest.mark.parametrize("H,d", [(1, 64), (4, 128), (8, 128), (12, 64)])
def test_values_at_the_end_of_bf16_s_range(H, d, o_fp32, wide):
    """Infinities are held as the largest finite values, and O, an average of them, is finite."""
    inf = float("inf")
    c = Cache(1, 1, d, "bf16", 16, 1500, seed=43)
    k = _rows(c.g, "bf16", 1, 1, 1500, d)
    k[:, :, 700:] *= 2
    c.write([0], 1500, k=k, v=torch.full((1, 1, 1500, d), inf, dtype=torch.bfloat16))
    if wide:
        _room(c)
    q = _rows(c.g, "bf16", 1, H, 1, d)
    for at in (0, 40, 1499):
        attend(c, q, [at], o_fp32=o_fp32)
    v = _rows(c.g, "bf16", 1, 1, 1500, d)
    v[:, :, 3::7, :40], v[:, :, 5::11, 40:] = inf, -inf
    c.write([0], 1500, v=v)
    for at in (40, 1499):
        attend(c, q, [at], o_fp32=o_fp32)
    _ok()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("o_fp32", [True, False])
@pytest.mark.parametrize("H,T,d", [(1, 1, 64), (4, 1, 128), (8, 1, 128), (12, 1, 64), (40, 10, 128)])
def test_values_at_the_end_of_fp16_s_range(H, T, d, o_fp32, wide):
    inf = float("inf")
    c = Cache(1, 1, d, "fp16", 16, 1500, seed=44)
    v = torch.full((1, 1, 1500, d), inf, dtype=torch.float16)
    v[..., 1::2] = -inf
    c.write([0], 1500, v=v)
    if wide:
        _room(c)
    q = _rows(c.g, "fp16", 1, H, T, d)
    for at in (0, 3, 40, 1499 - T):
        o, _ = attend(c, q, [at], o_fp32=o_fp32)
        assert torch.isfinite(o).all()
    _ok()


@pytest.mark.parametrize("T", [1, 12])
def test_one_key_s_rounding_does_not_take_fp16_past_its_range(T):
    """A key below the running maximum's move has nearly all the weight, which rounds: up by more than 2^-12 in some
    rows.  Every O is 65504; P s_V and the weights round by 2^-11, O's sums by 2^-13, O itself by 2^-11."""
    B, d, page = 600, 128, 64
    g = torch.Generator().manual_seed(45)
    pool = fa.fa_kv4_pool(B * 4, 2, page, d)
    table = torch.randperm(B * 4, generator=g).reshape(B, 4).to(torch.int32).cuda()
    k = torch.full((B, 2, 256, d), -2.0, dtype=torch.float16, device="cuda")
    k[:, :, 0], k[:, :, 80] = 0.0, 0.35
    fa.fa_kv4_write(k, torch.full_like(k, float("inf")), pool, table, _ints([0] * B))
    q = (_rows(g, "fp16", B, 2, T, d).float() * 0.2 + 0.5).half()
    o, _ = fa.fa_fwd_kv4(q.cuda(), pool, table, _ints([255 - T] * B), causal=True)
    assert ((o.float() - 65504).abs() <= 65504 * (2.0**-10 + 2.0**-13)).all()
    _ok()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("H,d", [(1, 64), (8, 128), (16, 128)])
@pytest.mark.parametrize("e", [-124, -116, -90, 60, 100])
def test_queries_of_any_magnitude_and_keys_that_make_up_for_it(e, H, d, wide):
    c = Cache(1, 1, d, "bf16", 16, 300, seed=46)
    k = (torch.randn(1, 1, 300, d, generator=c.g) * 2.0**-e).bfloat16()
    c.write([0], 300, k=k)
    if wide:
        _room(c)
    q = (torch.randn(1, H, 1, d, generator=c.g) * 2.0**e).bfloat16()
    attend(c, q, [299], o_fp32=True)
    _ok()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("H,d", [(1, 64), (4, 128), (8, 64), (12, 128)])
def test_a_key_of_hardly_any_weight_and_the_largest_value_counts(H, d, wide):
    """Weights of e^-88 to e^-102 times 3.4e38: below float32's smallest, and yet what O is made of; in the first step and
    later, before and behind the key of the largest score, all that a warp has."""
    for length, at, n in ((3, 0, 1), (3, 1, 1), (65, 64, 1), (300, 17, 1), (300, 250, 1), (300, 0, 64), (300, 64, 150), (1500, 700, 1)):
        c = Cache(1, 1, d, "bf16", 16, length, seed=47)
        k, v = _rows(c.g, "bf16", 1, 1, length, d) * 0.01, _rows(c.g, "bf16", 1, 1, length, d) * 2.0**-8
        k[:, :, at : at + n], v[:, :, at : at + n] = -96 / d**0.5, float("inf")
        c.write([0], length, k=k, v=v)
        if wide:
            _room(c)
        for weak in (0.92, 0.96, 1.0, 1.06):
            q = (weak * (1 + 0.01 * torch.rand(1, H, 1, d, generator=c.g))).bfloat16()
            attend(c, q, [length - 1], o_fp32=True)
    _ok()
