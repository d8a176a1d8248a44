"""Operators of a serving step on the paged caches, in plain torch and as the library's calls.

Three operators: appending keys and values to the paged cache with their rotary positions
applied on the way (queries turned in the same call), attention of one or many new tokens of
each request within a sliding window and over the first tokens (sinks), and a cache held in 4
bits: its append, its rows read back, and decode attention over it.  run() takes the plain
form (own = False) or the library's calls (own = True) on the same inputs.
"""
from __future__ import annotations

import math
import random

import torch

own = False

D = 128  # head dimension of the cache
PAGE = 64  # tokens per page


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one chat's next token, far behind the tokens that its cache still holds: latency
        dict(name="append_step", op="append", requests=1, hq=32, hkv=8, held_lo=1000, held_hi=1000, new_lo=1, new_hi=1,
             rotary=128, interleaved=False, base=1000000.0, scaling="none", factor=1.0, offset=32768, mix=1),
        # a serving step: one token of each of 64 requests of odd lengths, GQA 8
        dict(name="append_batch", op="append", requests=64, hq=64, hkv=8, held_lo=0, held_hi=2000, new_lo=1, new_hi=1,
             rotary=128, interleaved=False, base=1000000.0, scaling="yarn", factor=4.0, offset=0, mix=2),
        # the serving loop's prefill chunk: the ends of two prompts and the most of a third
        dict(name="append_prefill", op="append", requests=3, hq=32, hkv=8, held_lo=77, held_hi=2500, new_lo=1303,
             new_hi=11000, rotary=128, interleaved=False, base=1000000.0, scaling="none", factor=1.0, offset=0, mix=3),
        # the next token of one long chat: latency
        dict(name="window_step", op="window", requests=1, hq=32, hkv=8, len_lo=32768, len_hi=32768, new_lo=1, new_hi=1,
             sink=4, window=1024, mix=4),
        # a serving step of 64 requests, many of them shorter than their window
        dict(name="window_batch", op="window", requests=64, hq=32, hkv=8, len_lo=1, len_hi=32768, new_lo=1, new_hi=1,
             sink=4, window=4096, mix=5),
        # a few drafted tokens of each request looked at in one step, GQA 8
        dict(name="window_drafts", op="window", requests=16, hq=64, hkv=8, len_lo=64, len_hi=16384, new_lo=3, new_hi=7,
             sink=4, window=2048, mix=6),
        # prompts of two requests, the second behind a history
        dict(name="window_prefill", op="window", requests=2, hq=32, hkv=8, len_lo=8192, len_hi=11011, new_lo=8192,
             new_hi=8192, sink=4, window=4096, mix=7),
        # a prompt's chunk behind a long history, everything before it visible
        dict(name="window_chunk", op="window", requests=1, hq=32, hkv=8, len_lo=32768, len_hi=32768, new_lo=2048,
             new_hi=2048, sink=0, window=0, mix=8),
        # short and one-token requests at odd lengths: latency
        dict(name="int4_short", op="int4", requests=5, hq=8, hkv=2, group=32, len_lo=1, len_hi=1000, mix=9),
        # the 8B-shaped layer's single request
        dict(name="int4_8b", op="int4", requests=1, hq=32, hkv=8, group=128, len_lo=32768, len_hi=32768, mix=10),
        # the long batch: 8 requests of 100000 tokens
        dict(name="int4_batch", op="int4", requests=8, hq=32, hkv=8, group=32, len_lo=100000, len_hi=100000, mix=11),
        # a prompt's chunk into the 4-bit cache, and the history read back for the chunk's own attention
        dict(name="int4_fill", op="fill", hkv=8, group=32, held=12345, new=8192, mix=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["append", "window", "window", "int4", "int4", "fill"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([4, 8])
    mix = rng.randrange(1 << 30)
    if op == "append":
        hi = _log_int(rng, 1, 9000)
        n = _log_int(rng, 1, max(1, min(64, 9000 // hi)))
        return dict(op=op, requests=n, hq=hq, hkv=hkv, held_lo=0, held_hi=_log_int(rng, 1, 4000), new_lo=rng.choice([1, hi]),
                    new_hi=hi, rotary=rng.choice([128, 128, 96, 64, 18, 2]), interleaved=rng.random() < 0.5,
                    base=rng.choice([10000.0, 500000.0, 1000000.0]), scaling=rng.choice(["none", "linear", "bands", "yarn"]),
                    factor=rng.choice([2.0, 4.0, 8.0]), offset=rng.choice([0, 0, _log_int(rng, 1, 1000000)]), mix=mix)
    if op == "window":
        new = rng.choice([1, 1, _log_int(rng, 2, 16), _log_int(rng, 17, 4096)])
        hi = max(new, _log_int(rng, 1, 40000))
        window = rng.choice([_log_int(rng, 1, 8192), 128 * rng.randrange(1, 33), 0])
        pairs = new * min(hi, window or hi) * hq  # of a request, at most
        n = _log_int(rng, 1, max(1, min(64, 600000 // hi, 2000000000 // pairs)))
        new = max(1, min(new, 2000000000 // (hi * hq)) if pairs > 2000000000 else new)
        return dict(op=op, requests=n, hq=hq, hkv=hkv, len_lo=rng.choice([1, hi, max(1, hi // 3)]), len_hi=hi,
                    new_lo=rng.choice([1, new]), new_hi=new, sink=rng.choice([0, 1, 4, 64, 130]), window=window, mix=mix)
    if op == "int4":
        hi = _log_int(rng, 1, 65536)
        n = _log_int(rng, 1, max(1, min(28, 600000 // hi)))
        return dict(op=op, requests=n, hq=hq, hkv=hkv, group=rng.choice([32, 128]), len_lo=rng.choice([1, hi, max(1, hi // 3)]),
                    len_hi=hi, mix=mix)
    return dict(op=op, hkv=hkv, group=rng.choice([32, 128]), held=_log_int(rng, 1, 12000) - 1, new=_log_int(rng, 1, 8192), mix=mix)


def _spread(case, n, lo, hi, salt):
    """n seeded lengths in [lo, hi], over their logarithm; the first two are the ends."""
    r = random.Random(case["mix"] * 31 + salt)
    out = [hi, lo] + [lo + _log_int(r, 1, hi - lo + 1) - 1 for _ in range(n)]
    return out[:n]


def _held(case):
    return _spread(case, case["requests"], case["held_lo"], case["held_hi"], 1)


def _context(case):
    return _spread(case, case["requests"], case["len_lo"], case["len_hi"], 2)


def _new(case):
    """New tokens of each request; in a window case they are the last of its tokens."""
    new = _spread(case, case["requests"], case["new_lo"], case["new_hi"], 3)
    return [min(n, L) for n, L in zip(new, _context(case))] if case["op"] == "window" else new


def _visible(pos, sink, window):
    """Tokens that the query at pos attends."""
    start = max(0, pos - window + 1) if window else 0
    return pos + 1 - start + min(sink, start)


def work(case):
    op = case["op"]
    if op == "append":
        rows = sum(_new(case))
        heads = case["hq"] + case["hkv"]
        return {"bytes": 2 * rows * (heads + case["hkv"]) * D * 2, "flops": 3 * rows * heads * case["rotary"]}
    if op == "window":
        pairs = read = 0
        for L, n in zip(_context(case), _new(case)):
            pairs += sum(_visible(p, case["sink"], case["window"]) for p in range(L - n, L))
            start = max(0, L - n - case["window"] + 1) if case["window"] else 0
            read += L - start + min(case["sink"], start)
        return {"bytes": read * case["hkv"] * 2 * D * 2 + 2 * sum(_new(case)) * case["hq"] * D * 2,
                "flops": 4 * pairs * case["hq"] * D}
    row = D // 2 + 4 * (D // case["group"])  # bytes of a token's row: codes, scales and zero points
    if op == "int4":
        total = sum(_context(case))
        return {"bytes": total * case["hkv"] * 2 * row + 2 * case["requests"] * case["hq"] * D * 2,
                "flops": 4 * total * case["hq"] * D}
    total = case["held"] + case["new"]
    return {"bytes": 2 * case["hkv"] * (case["new"] * (2 * D + row) + total * (row + 2 * D)),
            "flops": 2 * case["hkv"] * D * (4 * case["new"] + 2 * total)}


# ------------------------------------------------------------------ inputs
def _gen(*parts):
    s = 0
    for p in parts:
        s = (s * 1000003 + int(p) + 12345) & ((1 << 62) - 1)
    return torch.Generator(device="cuda").manual_seed(s)


def _tokens(n, hkv, seed, stream):
    """K and V rows bf16 [n, hkv, D]: N(0, 1) with outlier channels (four of K x20, two of V x8) and a log-normal
    factor per token vector, the distribution of the benchmark's workloads."""
    pick = random.Random(seed)
    scale = torch.ones(2, D, device="cuda")
    scale[0, pick.sample(range(D), 4)] = 20.0
    scale[1, pick.sample(range(D), 2)] = 8.0
    out = torch.empty(2, n, hkv, D, dtype=torch.bfloat16, device="cuda")
    for a in range(0, n, 16384):
        b = min(n, a + 16384)
        g = _gen(seed, stream, a)
        x = torch.randn(2, b - a, hkv, D, generator=g, device="cuda")
        norm = torch.exp(0.5 * torch.randn(2, b - a, hkv, 1, generator=g, device="cuda"))
        out[:, a:b] = x * norm * scale[:, None, None, :]
    return out[0], out[1]


def _frequencies(case):
    """fp64 frequencies (radians a position) of the rotary pairs, and the factor on the rotated channels."""
    R, base, factor = case["rotary"], case["base"], case["factor"]
    f = torch.tensor([base ** (-2.0 * i / R) for i in range(R // 2)], dtype=torch.float64)
    original = 32768
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "bands":
        turns = original * f / (2 * math.pi)  # turns within the original context
        mix = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return f / factor * (1 - mix) + f * mix, 1.0
    if case["scaling"] == "yarn":
        where = [R * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        low, high = max(math.floor(where[0]), 0), min(math.ceil(where[1]), R - 1)
        ramp = ((torch.arange(R // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _make_cache(case, lengths):
    """A cache of one layer with room for requests of these lengths."""
    import int2_rotated_kv_rotate_gb300 as pkg

    fmt = pkg.OSCAR_FORMAT_INT4 if "group" in case else pkg.OSCAR_FORMAT_BF16
    return pkg.KVCache(fmt=fmt, n_q_heads=case.get("hq", 4 * case["hkv"]), n_kv_heads=case["hkv"], group=case.get("group", 128),
                       n_layers=1, max_requests=len(lengths), max_pages=max(1, sum(_pages(L) for L in lengths)),
                       max_pages_per_request=max(1, max(_pages(L) for L in lengths)))


def _filled_cache(case, lengths, kv):
    """The cache with the requests' tokens in it, and their slots."""
    cache = _make_cache(case, lengths)
    slots = [cache.alloc() for _ in lengths]
    for slot, L, (K, V) in zip(slots, lengths, kv):
        if L:
            cache.reserve([slot], [L])
            cache.append(0, K, V)
            cache.commit()
    return cache, slots


def _prepare_append(case, seed):
    hq, hkv, held, new = case["hq"], case["hkv"], _held(case), _new(case)
    rows, total = sum(new), [h + n for h, n in zip(held, new)]
    # queries, keys and values are slices of one fused projection's rows
    qkv = torch.randn(rows, (hq + 2 * hkv) * D, generator=_gen(seed, 1, rows), device="cuda").to(torch.bfloat16)
    q, k, v = (x.view(rows, -1, D) for x in qkv.split([hq * D, hkv * D, hkv * D], dim=1))
    at = torch.cat([torch.arange(h, t) for h, t in zip(held, total)])  # places of the new tokens in their requests
    positions = (at + case["offset"]).to(torch.int32).cuda()
    st = dict(case=case, q=q, k=k, v=v, positions=positions)
    if own:
        from int2_rotated_kv_rotate_gb300 import RotaryEmbedding

        scaling = None if case["scaling"] == "none" else dict(type=case["scaling"], factor=case["factor"], original_context=32768)
        cache = _make_cache(case, total)
        cache.bf16_pages(0).zero_()
        slots = [cache.alloc() for _ in total]
        some = [i for i in range(len(held)) if held[i]]
        if some:  # the tokens held before (the append does not look at them)
            cache.reserve([slots[i] for i in some], [held[i] for i in some])
            cache.commit()
        cache.reserve(slots, new)
        page_of = [cache.pages(s) for s in slots]
        st.update(cache=cache, pool=cache.bf16_pages(0), q_out=torch.empty(rows, hq, D, dtype=torch.bfloat16, device="cuda"),
                  rotary=RotaryEmbedding(head_dim=D, rotary_dim=case["rotary"], base=case["base"],
                                         interleaved=case["interleaved"], scaling=scaling))
        # (a fresh pool hands its pages out in order: those of the tokens held, then those of the new ones)
        assert page_of == _page_ids(held, total)
    else:
        f, magnitude = _frequencies(case)
        ids = _page_ids(held, total)
        page = torch.cat([torch.tensor(p)[torch.arange(h, t) // PAGE] for p, h, t in zip(ids, held, total)])
        st.update(freq=f.cuda(), magnitude=magnitude, page=page.cuda(), place=(at % PAGE).cuda(),
                  pool=torch.zeros(max(1, sum(_pages(t) for t in total)), hkv, 2, PAGE, D, dtype=torch.bfloat16, device="cuda"))
    return st


def _page_ids(held, total):
    """Physical pages of requests that first held some tokens and then grew to their totals."""
    ids, next_page = [], 0
    for h in held:
        ids.append(list(range(next_page, next_page + _pages(h))))
        next_page += _pages(h)
    for p, t in zip(ids, total):
        more = _pages(t) - len(p)
        p += range(next_page, next_page + more)
        next_page += more
    return ids


def _prepare_window(case, seed):
    lengths, new = _context(case), _new(case)
    kv = [_tokens(L, case["hkv"], seed, i) for i, L in enumerate(lengths)]
    q = torch.randn(sum(new), case["hq"], D, generator=_gen(seed, 2), device="cuda").to(torch.bfloat16)
    st = dict(case=case, q=q)
    if own:
        cache, slots = _filled_cache(case, lengths, kv)
        cache.plan_window(slots, n_queries=new, n_sink=case["sink"], window=case["window"])
        st.update(cache=cache, out=torch.empty_like(q))
    else:
        st["kv"] = kv
    return st


def _quantize(x, group):
    """Codes (two to a byte), scales and zero points of rows [n, hkv, D] in bf16."""
    y = x.float().unflatten(-1, (D // group, group))
    low, high = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    # (a quotient of tensors: by a number, torch multiplies with its reciprocal)
    scale, zero = ((high - low) / torch.full_like(low, 15.0)).to(torch.bfloat16), low.to(torch.bfloat16)
    s = scale.float()
    codes = torch.where(s == 0, torch.zeros_like(y), ((y - zero.float()) / torch.where(s == 0, torch.ones_like(s), s)).round().clamp(0, 15))
    codes = codes.to(torch.uint8).flatten(-2)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), scale, zero


def _values(packed, scale, zero):
    """fp32 values [n, hkv, D] of codes, scales and zero points."""
    codes = torch.stack((packed & 15, packed >> 4), dim=-1).flatten(-2).float()
    return (codes.unflatten(-1, (scale.shape[-2], -1)) * scale.float() + zero.float()).flatten(-2)


def _prepare_int4(case, seed):
    lengths = _context(case)
    kv = [_tokens(L, case["hkv"], seed, i) for i, L in enumerate(lengths)]
    q = torch.randn(len(lengths), case["hq"], D, generator=_gen(seed, 3), device="cuda").to(torch.bfloat16)
    st = dict(case=case, q=q)
    if own:
        cache, slots = _filled_cache(case, lengths, kv)
        cache.plan(slots)
        st.update(cache=cache, out=torch.empty_like(q))
    else:
        st["kv"] = [[_quantize(x, case["group"]) for x in pair] for pair in kv]
    return st


def _prepare_fill(case, seed):
    held, new, hkv = case["held"], case["new"], case["hkv"]
    old, (k, v) = _tokens(held, hkv, seed, 0), _tokens(new, hkv, seed, 1)
    st = dict(case=case, k=k, v=v)
    shape = (held + new, hkv, D)
    if own:
        cache = _make_cache(case, [held + new])
        slot = cache.alloc()
        if held:
            cache.reserve([slot], [held])
            cache.append(0, *old)
            cache.commit()
        cache.reserve([slot], [new])
        st.update(cache=cache, slot=slot, k_out=torch.empty(shape, dtype=torch.bfloat16, device="cuda"),
                  v_out=torch.empty(shape, dtype=torch.bfloat16, device="cuda"))
    else:
        st["store"] = []
        for x in old:
            parts = _quantize(x, case["group"])
            room = [torch.empty((held + new,) + p.shape[1:], dtype=p.dtype, device="cuda") for p in parts]
            for r, p in zip(room, parts):
                r[:held] = p
            st["store"].append(room)
    return st


def prepare(case, seed):
    return {"append": _prepare_append, "window": _prepare_window, "int4": _prepare_int4,
            "fill": _prepare_fill}[case["op"]](case, seed)


# ------------------------------------------------------------------ one pass
def _run_append(st):
    case, R = st["case"], st["case"]["rotary"]
    if own:
        st["cache"].append_rotated(0, st["rotary"], st["k"], st["v"], q=st["q"], q_out=st["q_out"],
                                   positions=st["positions"] if case["offset"] else None)
        return st["q_out"], st["pool"]
    angle = st["positions"].double()[:, None] * st["freq"][None, :]  # in 64 bits: far positions
    cos = (angle.cos().float() * st["magnitude"])[:, None, :]
    sin = (angle.sin().float() * st["magnitude"])[:, None, :]
    outs = []
    for x in (st["q"], st["k"]):
        y = x.float()
        if case["interleaved"]:
            a, b = y[..., 0:R:2], y[..., 1:R:2]
            turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
        else:
            a, b = y[..., :R // 2], y[..., R // 2:R]
            turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
        outs.append(torch.cat((turned, y[..., R:]), dim=-1).to(x.dtype))
    st["pool"][st["page"], :, 0, st["place"]] = outs[1]
    st["pool"][st["page"], :, 1, st["place"]] = st["v"]
    return outs[0], st["pool"]


def _windowed(q, K, V, first, sink, window):
    """Attention of q [n, hq, D], the tokens at first, first + 1, .., over K and V [L, hkv, D]."""
    n, hkv = q.shape[0], K.shape[1]
    out = []
    for a in range(0, n, 1024):  # a band of queries needs a band of keys
        b = min(n, a + 1024)
        p = torch.arange(first + a, first + b, device=q.device)
        start = max(0, first + a - window + 1) if window else 0
        t = torch.cat((torch.arange(min(sink, start), device=q.device), torch.arange(start, first + b, device=q.device)))
        seen = t[None] <= p[:, None]
        if window:
            seen &= (t[None] > p[:, None] - window) | (t[None] < sink)
        rows = q[a:b].view(b - a, hkv, -1, D).permute(1, 2, 0, 3)  # [hkv, G, band, D]
        s = rows @ K[t].float().permute(1, 2, 0)[:, None] / math.sqrt(D)
        s = s.masked_fill(~seen, -math.inf)
        s = torch.exp(s - s.amax(-1, keepdim=True))
        o = s @ V[t].float().transpose(0, 1)[:, None] / s.sum(-1, keepdim=True)
        out.append(o.permute(2, 0, 1, 3).flatten(1, 2))
    return torch.cat(out)


def _run_window(st):
    if own:
        return st["cache"].attend_window(0, st["q"], out=st["out"])
    case, q = st["case"], st["q"].float()
    out, at = [], 0
    for (K, V), L, n in zip(st["kv"], _context(case), _new(case)):
        out.append(_windowed(q[at:at + n], K, V, L - n, case["sink"], case["window"]))
        at += n
    return torch.cat(out).to(torch.bfloat16)


def _run_int4(st):
    if own:
        return st["cache"].decode(0, st["q"], out=st["out"])
    q, out = st["q"].float(), []
    for i, (k, v) in enumerate(st["kv"]):
        K, V = _values(*k), _values(*v)
        s = q[i].view(K.shape[1], -1, D) @ K.permute(1, 2, 0) / math.sqrt(D)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        out.append((p @ V.transpose(0, 1) / p.sum(-1, keepdim=True)).flatten(0, 1))
    return torch.stack(out).to(torch.bfloat16)


def _run_fill(st):
    case = st["case"]
    if own:
        st["cache"].append(0, st["k"], st["v"])
        return st["cache"].read(0, st["slot"], 0, case["held"] + case["new"], k_out=st["k_out"], v_out=st["v_out"])
    for x, store in zip((st["k"], st["v"]), st["store"]):
        for r, p in zip(store, _quantize(x, case["group"])):
            r[case["held"]:] = p
    return tuple(_values(*store).to(torch.bfloat16) for store in st["store"])


def run(state):
    return {"append": _run_append, "window": _run_window, "int4": _run_int4, "fill": _run_fill}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_append(st):
    case, R = st["case"], st["case"]["rotary"]
    f, magnitude = _frequencies(case)
    angle = st["positions"].double()[:, None] * f.cuda()[None]
    turn = torch.polar(torch.full_like(angle, magnitude), angle)[:, None, :]
    outs = []
    for x in (st["q"], st["k"]):
        y = x.double()
        pair = y[..., :R].unflatten(-1, (R // 2, 2) if case["interleaved"] else (2, R // 2))
        axis = -1 if case["interleaved"] else -2
        z = torch.complex(pair.select(axis, 0), pair.select(axis, 1)) * turn
        y[..., :R] = torch.stack((z.real, z.imag), dim=axis).flatten(-2)
        outs.append(y)
    pool = st["pool"].double()
    rows = torch.stack((outs[1], st["v"].double()), dim=2)  # [rows, hkv, K|V, D]
    flat = pool.permute(0, 3, 1, 2, 4).reshape(-1, case["hkv"], 2, D)
    flat[st["page"] * PAGE + st["place"]] = rows
    return outs[0], flat.view(pool.shape[0], PAGE, case["hkv"], 2, D).permute(0, 2, 3, 1, 4)


def _exact_window(case, st):
    out, at = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda"), 0
    for (K, V), L, n in zip(st["kv"], _context(case), _new(case)):
        G = case["hq"] // case["hkv"]
        for a in range(0, n, 512):
            b = min(n, a + 512)
            p = torch.arange(L - n + a, L - n + b, device="cuda")[:, None]
            t = torch.arange(L - n + b, device="cuda")
            if case["window"]:
                t = t[(t < case["sink"]) | (t > L - n + a - case["window"])]
            off = t > p
            if case["window"]:
                off |= (t <= p - case["window"]) & (t >= case["sink"])
            bias = torch.zeros(off.shape, dtype=torch.float64, device="cuda")
            bias[off] = -math.inf
            for h in range(case["hkv"]):
                k, v = K[t, h].double(), V[t, h].double()
                for j in range(h * G, (h + 1) * G):
                    w = torch.softmax(st["q"][at + a:at + b, j].double() @ k.T * (1.0 / math.sqrt(D)) + bias, dim=-1)
                    out[at + a:at + b, j] = w @ v
        at += n
    return out


def _exact_rows(x, group):
    """What a 4-bit cache holds of rows x, in 64 bits.  (A code is defined by the 32-bit difference and quotient, so that
    halves, which a value next to one becomes there, are the same for everyone.)"""
    y = x.float().unflatten(-1, (-1, group))
    low = y.min(-1, keepdim=True)[0]
    s = ((y.max(-1, keepdim=True)[0] - low).double() / 15.0).float().to(torch.bfloat16)
    t = ((y - low) / s.float()).double()
    codes = torch.floor(t + 0.5)
    ties = (t + 0.5 == codes) & (codes % 2 == 1)  # halves go to the even code
    codes = torch.where(s > 0, (codes - ties.double()).clamp(0, 15), torch.zeros_like(t))
    return (low.double() + codes * s.double()).flatten(-2)


def _exact_int4(case, st, kv):
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    G = case["hq"] // case["hkv"]
    for i, (K, V) in enumerate(kv):
        for h in range(case["hkv"]):
            k, v = _exact_rows(K[:, h], case["group"]), _exact_rows(V[:, h], case["group"])
            w = torch.softmax(st["q"][i, h * G:(h + 1) * G].double() @ k.T * (1.0 / math.sqrt(D)), dim=-1)
            out[i, h * G:(h + 1) * G] = w @ v
    return out


def exact(case, seed):
    global own
    was, own = own, False
    try:
        if case["op"] == "fill":
            old, new = _tokens(case["held"], case["hkv"], seed, 0), _tokens(case["new"], case["hkv"], seed, 1)
            return tuple(_exact_rows(torch.cat(pair), case["group"]) for pair in zip(old, new))
        st = prepare(case, seed)
        if case["op"] == "append":
            return _exact_append(st)
        if case["op"] == "window":
            return _exact_window(case, st)
        return _exact_int4(case, st, [_tokens(L, case["hkv"], seed, i) for i, L in enumerate(_context(case))])
    finally:
        own = was
