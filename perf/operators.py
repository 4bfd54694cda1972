"""The operators of serving from a key/value cache held in 4 bits, as cases that can be run and timed.

Two operators, three kinds of case ("op"):
  "store"  new tokens' keys and values are quantised into the paged cache and read back in 16 bits,
  "read"   a stretch of the cache is read back in 16 bits,
  "attend" a few new tokens' queries attend to everything that their sequence has in the cache.

The definition. A row of a key or value head is cut into groups of 32 elements. Of a group, ext is its largest
element if that exceeds the negative of its smallest one, else its smallest; the group's scale s is -ext/8 rounded to
the row's 16-bit type (below 2^-126 it is 0), and each element x is held as the whole number
n = min(max(floor(x/s + 1/2), -8), 7), 0 where s is 0; it stands for n*s.  A cache row read back is n*s rounded to
the 16-bit type; attention takes n*s unrounded.  Token t of sequence b sits at position start[b] + t, in slot
position % page of page page_table[b][position / page].  Query t attends the keys 0 .. start[b] + t when causal, else
the keys 0 .. start[b] + count[b] - 1; rows t >= count[b] are padding (O = 0, LSE = -inf).
"""

import math

import torch

#: Set by whoever runs the cases: the framework's operators (True), or their plain form (False).
own = False

GROUP = 32
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # One decoding step of 64 sequences: one new token each. All latency.
        dict(name="store-append", op="store", B=64, Hkv=8, T=1, d=128, start=4095, page=16, type="bf16", ragged=True),
        # Five proposed tokens for seven sequences, an odd shape.
        dict(name="store-draft", op="store", B=7, Hkv=12, T=5, d=64, start=611, page=32, type="fp16", ragged=True),
        # The prompts of a batch of two, 16 heads, 8192 tokens at once (the benchmark's d=128 shape).
        dict(name="store-prompt", op="store", B=2, Hkv=16, T=8192, d=128, start=0, page=64, type="bf16", ragged=False),
        # One sequence of 23400 steps with 12 heads of 64 (one trading day of seconds), written after a short prefix.
        dict(name="store-day", op="store", B=1, Hkv=12, T=23400, d=64, start=37, page=16, type="bf16", ragged=False),
        # Shared prefixes fetched for attention in 16 bits.
        dict(name="read-prefix", op="read", B=16, Hkv=8, T=6001, d=128, start=0, page=32, type="fp16", ragged=True),
        # One sequence, one token: the smallest decoding call.
        dict(name="attend-one", op="attend", B=1, H=32, Hkv=8, T=1, d=128, start=999, page=16, type="bf16", ragged=False, causal=True),
        # A batch of eight with 12 heads of 64 around 1024 tokens, every head its own keys.
        dict(name="attend-mha", op="attend", B=8, H=12, Hkv=12, T=1, d=64, start=1023, page=16, type="fp16", ragged=False, causal=True),
        # An ordinary serving batch: 64 sequences of uneven length, four query heads to a key head.
        dict(name="attend-batch", op="attend", B=64, H=32, Hkv=8, T=1, d=128, start=8191, page=64, type="bf16", ragged=True, causal=True),
        # The largest: eight sequences of 64 Ki tokens, eight query heads to a key head.
        dict(name="attend-long", op="attend", B=8, H=64, Hkv=8, T=1, d=128, start=65535, page=128, type="bf16", ragged=False, causal=True),
        # Four sequences of a trading day, 12 heads of 64.
        dict(name="attend-day", op="attend", B=4, H=12, Hkv=12, T=1, d=64, start=23399, page=16, type="bf16", ragged=False, causal=True),
        # Four proposed tokens a sequence are checked at once: 16 query rows to a key head.
        dict(name="attend-draft", op="attend", B=24, H=32, Hkv=8, T=4, d=128, start=5003, page=32, type="fp16", ragged=True, causal=True),
        # The next 96 tokens of two prompts on top of what is cached: many rows to a key head.
        dict(name="attend-chunk", op="attend", B=2, H=16, Hkv=4, T=96, d=64, start=3001, page=16, type="bf16", ragged=True, causal=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "store", "read", "attend", "attend", "attend", "attend"])
    c = dict(op=op, d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]), type=rng.choice(["bf16", "fp16"]), ragged=rng.random() < 0.6)
    if op == "attend":
        most = 8 * 8 * 65536  # sequences x key heads x keys; four times that for the scores
        while True:
            c.update(B=_log(rng, 1, 96), Hkv=rng.choice([1, 2, 4, 5, 8, 12]), T=rng.choice([1, 1, 1, 1, 2, 3, 5, 8, _log(rng, 8, 96)]),
                     start=_log(rng, 1, 40000) - 1, causal=rng.random() < 0.7)
            c["H"] = c["Hkv"] * rng.choice([1, 1, 2, 3, 4, 6, 8, 16])
            keys = c["B"] * (c["start"] + c["T"])
            if keys * c["Hkv"] <= most and keys * c["H"] * c["T"] <= 4 * most:
                return c
    while True:
        c.update(B=_log(rng, 1, 96), Hkv=rng.choice([1, 2, 4, 5, 8, 12, 16]), T=rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 8, 20000)]), start=_log(rng, 1, 10000) - 1)
        if op == "read":
            c["start"] = rng.choice([0, c["start"] % 777])
        rows = c["B"] * c["Hkv"] * (c["T"] + (c["start"] if op == "read" else 0))
        if rows <= (16 * 8 * 6001 if op == "read" else 2 * 16 * 8192):
            return c


def _starts(case):
    """Each sequence's start: all alike, or spread between a tenth and the whole of what the case names."""
    B, s = case["B"], case["start"]
    return [s if not case["ragged"] else s * (100 + (b * 611 + 357) % 901) // 1000 for b in range(B)]


def _counts(case):
    """How many of its T tokens each sequence has."""
    B, T = case["B"], case["T"]
    return [T if not case["ragged"] or T < 3 else T - (b * 5 + 2) % ((T + 2) // 3) for b in range(B)]


def work(case):
    d, T, type_bytes = case["d"], case["T"], 2
    row = d / 2 + d / GROUP * type_bytes  # one cached key or value row
    if case["op"] == "attend":
        keys = [s + n for s, n in zip(_starts(case), _counts(case))]
        pairs = sum(sum(min(s + (t + 1 if case["causal"] else n), k) for t in range(n)) for s, n, k in zip(_starts(case), _counts(case), keys))
        rows = case["B"] * case["H"] * T
        return {"bytes": 2 * sum(keys) * case["Hkv"] * row + rows * (2 * d * type_bytes + 4), "flops": 4 * pairs * case["H"] * d}
    rows = 2 * sum(_counts(case)) * case["Hkv"]
    out = 2 * case["B"] * case["Hkv"] * T
    if case["op"] == "read":
        return {"bytes": rows * row + out * d * type_bytes, "flops": rows * d}
    return {"bytes": rows * (d * type_bytes + row) + out * d * type_bytes, "flops": 4 * rows * d}


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _inputs(case, seed):
    """The inputs alone, from the seed. Keys have a few strong channels, and queries of real scores' spread."""
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    t, B, Hkv, d, page = TYPES[case["type"]], case["B"], case["Hkv"], case["d"], case["page"]
    starts, counts = _starts(case), _counts(case)
    per = -(-(max(starts) + case["T"]) // page)
    x = {"start": torch.tensor(starts, dtype=torch.int32, device="cuda"), "count": torch.tensor(counts, dtype=torch.int32, device="cuda"), "per": per, "pages": B * per + 3}
    x["table"] = torch.randperm(B * per + 3, generator=g, device="cuda")[: B * per].reshape(B, per).to(torch.int32)
    x["len"] = case["T"] if case["op"] == "store" else max(s + n for s, n in zip(starts, counts))
    strong = torch.exp(0.5 * _normal(g, 1, Hkv, 1, d))
    x["k"] = (_normal(g, B, Hkv, x["len"], d) * strong).to(t)
    x["v"] = _normal(g, B, Hkv, x["len"], d).to(t)
    if case["op"] == "attend":
        x["q"] = _normal(g, B, case["H"], case["T"], d).to(t)
    return x


def _quantise(x):
    """The whole numbers (int8) and scales of rows, by the definition above."""
    top = torch.finfo(x.dtype).max
    f = torch.nan_to_num(x.float(), nan=0.0, posinf=top, neginf=-top).unflatten(-1, (-1, GROUP))
    high, low = f.amax(-1, keepdim=True), f.amin(-1, keepdim=True)
    s = (torch.where(high > -low, high, low) * -0.125).to(x.dtype).float()
    none = s.abs() < 2.0**-126
    n = torch.floor(f / torch.where(none, 1.0, s) + 0.5).clamp(-8, 7)
    return torch.where(none, 0.0, n).to(torch.int8).flatten(-2), torch.where(none, 0.0, s).squeeze(-1).to(x.dtype)


def _values(n, s):
    return (n.float().unflatten(-1, (-1, GROUP)) * s.float().unsqueeze(-1)).flatten(-2)


def _slots(state, first, length):
    """Page and slot of positions first[b] .. first[b] + length - 1."""
    i = torch.arange(length, device="cuda")
    at = first.long()[:, None] + i[None, :]
    page = state["page"]
    return state["table"].long().gather(1, (at // page).clamp(max=state["table"].shape[1] - 1)), at % page


def _write_plain(state, k, v, first, count):
    pages, slots = _slots(state, first, k.shape[2])
    live = torch.arange(k.shape[2], device="cuda")[None, :] < count.long()[:, None]
    pages = torch.where(live, pages, state["k_n"].shape[0] - 1)  # padding goes to a page that nobody reads
    for name, x in (("k", k), ("v", v)):
        n, s = _quantise(x)
        state[name + "_n"][pages, :, slots] = n.transpose(1, 2)
        state[name + "_s"][pages, :, slots] = s.transpose(1, 2)


def _read_plain(state, first, count, length):
    pages, slots = _slots(state, first, length)
    live = (torch.arange(length, device="cuda")[None, :] < count.long()[:, None])[:, None, :, None]
    out = []
    for name in ("k", "v"):
        x = _values(state[name + "_n"][pages, :, slots], state[name + "_s"][pages, :, slots]).transpose(1, 2)
        out.append(torch.where(live, x, 0.0))
    return out


def prepare(case, seed):
    x = _inputs(case, seed)
    state = dict(case, keys=x["len"], table=x["table"], start=x["start"], count=x["count"], k=x["k"], v=x["v"], q=x.get("q"))
    t, Hkv, d, page = TYPES[case["type"]], case["Hkv"], case["d"], case["page"]
    if own:
        import exact_io_aware_84_b200 as fa

        state["fa"] = fa
        state["pool"] = fa.fa_kv4_pool(x["pages"], Hkv, page, d, device="cuda")
    else:
        for name in ("k", "v"):
            state[name + "_n"] = torch.zeros(x["pages"] + 1, Hkv, page, d, dtype=torch.int8, device="cuda")
            state[name + "_s"] = torch.zeros(x["pages"] + 1, Hkv, page, d // GROUP, dtype=t, device="cuda")
    if case["op"] == "store":
        return state
    zero, all_of = torch.zeros_like(x["start"]), x["start"] + x["count"]
    if own:
        fa.fa_kv4_write(state["k"], state["v"], state["pool"], state["table"], zero, all_of)
        if case["op"] == "attend":
            need = fa.fa_fwd_kv4_workspace_size(case["B"], case["H"], Hkv, case["T"], d)
            state["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    else:
        _write_plain(state, state["k"], state["v"], zero, all_of)
    state["k"] = state["v"] = None  # they are in the cache now
    return state


def _attend_plain(state):
    q, start, count = state["q"], state["start"].long(), state["count"].long()
    B, H, T, d = q.shape
    Hkv, length = state["Hkv"], state["keys"]
    k, v = _read_plain(state, torch.zeros_like(start), start + count, length)
    rows = q.float().reshape(B, Hkv, H // Hkv * T, d)
    scores = torch.matmul(rows, k.transpose(-1, -2)).reshape(B, H, T, length) * d**-0.5
    t, j = torch.arange(T, device="cuda"), torch.arange(length, device="cuda")
    limit = start[:, None] + t[None, :] + 1 if state["causal"] else (start + count)[:, None].expand(B, T)
    limit = torch.where(t[None, :] < count[:, None], limit, 0)
    scores = scores.masked_fill(j >= limit[:, None, :, None], -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, Hkv, H // Hkv * T, length), v).reshape(B, H, T, d) / torch.where(total == 0, 1.0, total)
    return o.to(q.dtype), (m + torch.log(total)).squeeze(-1)


def run(state):
    start, count, T = state["start"], state["count"], state["T"]
    if own:
        fa, pool, table = state["fa"], state["pool"], state["table"]
        if state["op"] == "attend":
            return fa.fa_fwd_kv4(state["q"], pool, table, start, count, workspace=state["workspace"], causal=state["causal"])
        if state["op"] == "store":
            fa.fa_kv4_write(state["k"], state["v"], pool, table, start, count)
        return fa.fa_kv4_read(pool, table, start, count, N=T, dtype=TYPES[state["type"]])
    if state["op"] == "attend":
        return _attend_plain(state)
    if state["op"] == "store":
        _write_plain(state, state["k"], state["v"], start, count)
    k, v = _read_plain(state, start, count, T)
    return k.to(TYPES[state["type"]]), v.to(TYPES[state["type"]])


def _held(rows):
    """What the cache stands for, in 64 bits: rows [..., d] of a 16-bit type."""
    x = rows.double().reshape(*rows.shape[:-1], -1, GROUP)
    up, down = x.max(-1).values, (-x).max(-1).values
    s = torch.where(up > down, -up, down).div(8).to(rows.dtype).double()[..., None]
    whole = torch.where(s == 0, torch.zeros_like(x), (2 * x / s + 1).div(2, rounding_mode="floor"))
    return (torch.minimum(torch.maximum(whole, torch.full_like(whole, -8)), torch.full_like(whole, 7)) * s).reshape(rows.shape)


def exact(case, seed):
    x = _inputs(case, seed)
    starts, counts, T, d = _starts(case), _counts(case), case["T"], case["d"]
    if case["op"] != "attend":
        first = [0] * case["B"] if case["op"] == "store" else starts
        out = []
        for rows in (x["k"], x["v"]):
            full = torch.zeros(case["B"], case["Hkv"], T, d, dtype=torch.float64, device="cuda")
            for b, n in enumerate(counts):
                have = rows[b, :, first[b] : first[b] + n]
                full[b, :, : have.shape[1]] = _held(have)
            out.append(full)
        return tuple(out)
    o = torch.zeros(case["B"], case["H"], T, d, dtype=torch.float64, device="cuda")
    lse = torch.full((case["B"], case["H"], T), -math.inf, dtype=torch.float64, device="cuda")
    each = case["H"] // case["Hkv"]
    for b, (s, n) in enumerate(zip(starts, counts)):
        for h in range(case["Hkv"]):
            k, v = _held(x["k"][b, h, : s + n]), _held(x["v"][b, h, : s + n])
            q = x["q"][b, h * each : (h + 1) * each, :n].double()
            a = torch.einsum("gtd,jd->gtj", q, k) / math.sqrt(d)
            if case["causal"]:
                seen = torch.ones(n, s + n, dtype=torch.bool, device="cuda").tril(diagonal=s)
                a = torch.where(seen, a, torch.full_like(a, -math.inf))
            lse[b, h * each : (h + 1) * each, :n] = torch.logsumexp(a, -1)
            o[b, h * each : (h + 1) * each, :n] = torch.einsum("gtj,jd->gtd", torch.softmax(a, -1), v)
    return o, lse
