"""CPU oracle for the 4-bit key/value cache: what it holds, and attention over it.

TEST INFRASTRUCTURE ONLY, like ``oracle.attention``.  Everything is float64;
the cache is represented by the rows that it stands for, position by position.
"""

from __future__ import annotations

import numpy as np

__all__ = ["round16_ref", "kv4_quantise_ref", "kv4_values_ref", "kv4_attn_ref"]

GROUP = 32
_FINITE = {"bf16": float.fromhex("0x1.fep127"), "fp16": 65504.0}


def round16_ref(x, dtype):
    """Round float64 values to bf16 or fp16 (nearest, ties to even), as float64."""
    x = np.asarray(x, np.float64)
    bits, low = (8, -133) if dtype == "bf16" else (11, -24)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.abs(x)))
    e = np.where(np.isfinite(e), e, 0.0)
    step = np.exp2(np.maximum(e - (bits - 1), low))
    return np.rint(x / step) * step


def kv4_quantise_ref(x, dtype):
    """(n, s) of rows x [..., d]: n int64 [..., d], s float64 [..., d/32]."""
    top = _FINITE[dtype]
    x = np.nan_to_num(np.asarray(x, np.float64), nan=0.0, posinf=top, neginf=-top)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    hi, lo = g.max(-1), g.min(-1)
    s = round16_ref(np.where(hi > -lo, hi, lo) / -8.0, dtype)
    s = np.where(np.abs(s) < 2.0**-126, 0.0, s)
    r = g / np.where(s == 0, 1.0, s)[..., None]
    n = np.clip(np.floor(r + 0.5), -8, 7)
    return np.where(s[..., None] == 0, 0, n).astype(np.int64).reshape(x.shape), s


def kv4_values_ref(x, dtype):
    """The values n s that rows x stand for in the cache, unrounded."""
    n, s = kv4_quantise_ref(x, dtype)
    return (n.reshape(*s.shape, GROUP) * s[..., None]).reshape(n.shape)


def kv4_attn_ref(q, k, v, start, count, scale, causal, missing=None):
    """O, LSE and sum_j P_j |v_j| of q [B,H,T,d] over k, v [B,Hkv,L,d] (position
    by position).  missing [B, L]: keys that do not exist."""
    B, H, T, d = q.shape
    group = H // k.shape[1]
    o, a = np.zeros_like(q), np.zeros_like(q)
    lse = np.full((B, H, T), -np.inf)
    for b in range(B):
        for t in range(count[b]):
            keys = start[b] + t + 1 if causal else start[b] + count[b]
            j = np.arange(max(0, min(keys, k.shape[2])))
            if missing is not None:
                j = j[~missing[b, j]]
            if not len(j):
                continue
            for h in range(H):
                s = scale * (k[b, h // group, j] @ q[b, h, t])
                m = s.max()
                p = np.exp(s - m)
                lse[b, h, t] = m + np.log(p.sum())
                p = p / p.sum()
                o[b, h, t] = p @ v[b, h // group, j]
                a[b, h, t] = p @ np.abs(v[b, h // group, j])
    return o, lse, a
