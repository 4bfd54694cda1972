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
from oracle import kv4_attn_ref
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
