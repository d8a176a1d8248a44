"""The operators around the paged cache, in plain torch and as the library's calls.

Four operators of one serving path: rotary positions on queries and new keys, decode
attention in which requests that map the same prefix pages attend them once, decode
attention that accumulates each cached token's attention weight, and eviction of the
tokens with the least accumulated weight.  run() takes the plain form (own = False) or
the library's calls (own = True) on the same inputs.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

D = 128  # head dimension of the cache
PAGE = 64  # tokens per page


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one request's single token on the 8B-shaped layer, far into its context: latency
        dict(name="rope_step", op="rope", rows=1, hq=32, hkv=8, dtype="bf16", rotary=128, interleaved=False,
             base=1000000.0, scaling="none", factor=1.0, start=32768, transpose=False),
        # the serving loop's prefill chunk on the 32B-shaped layer, context scaled past its original length
        dict(name="rope_prefill", op="rope", rows=16384, hq=64, hkv=8, dtype="bf16", rotary=128, interleaved=False,
             base=1000000.0, scaling="yarn", factor=4.0, start=114688, transpose=False),
        # gradients of a fine-tuning batch whose model turns half of each head, interleaved, in 32 bits; odd row count
        dict(name="rope_gradient", op="rope", rows=4099, hq=32, hkv=8, dtype="f32", rotary=64, interleaved=True,
             base=10000.0, scaling="bands", factor=8.0, start=0, transpose=True),
        # a few chats on one short system prompt: the smallest shared step, latency
        dict(name="shared_small", op="shared", groups=1, members=4, hq=8, hkv=2, common=0, prefix=8, tail_lo=1,
             tail_hi=65, mix=1),
        # the ragged shared-prefix mix: 64 requests, groups of 8 on a 16384-token prefix, private tails of their own
        dict(name="shared_ragged", op="shared", groups=8, members=8, hq=32, hkv=8, common=0, prefix=256, tail_lo=1,
             tail_hi=8192, mix=2),
        # many samples of long prompts: a system prompt under two documents, GQA 8, short tails
        dict(name="shared_wide", op="shared", groups=2, members=32, hq=64, hkv=8, common=96, prefix=416, tail_lo=1,
             tail_hi=512, mix=3),
        # short and one-token requests at odd lengths: latency
        dict(name="weights_short", op="weights", requests=5, hq=8, hkv=2, len_lo=1, len_hi=1000, mix=4),
        # the 8B-shaped layer's single request
        dict(name="weights_8b", op="weights", requests=1, hq=32, hkv=8, len_lo=32768, len_hi=32768, mix=5),
        # the long batch: 8 requests of 100000 tokens
        dict(name="weights_batch", op="weights", requests=8, hq=32, hkv=8, len_lo=100000, len_hi=100000, mix=6),
        # two short requests trimmed to a third: latency
        dict(name="evict_short", op="evict", requests=2, hkv=2, len_lo=1400, len_hi=1500, keep=0.35, sink=4, recent=64,
             mix=7),
        # a ragged batch at half its length, as a pool that runs full would ask for
        dict(name="evict_ragged", op="evict", requests=28, hkv=8, len_lo=1024, len_hi=32768, keep=0.5, sink=4,
             recent=128, mix=8),
        # the long batch cut to a quarter
        dict(name="evict_batch", op="evict", requests=8, hkv=8, len_lo=100000, len_hi=100000, keep=0.25, sink=4,
             recent=256, mix=9),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["rope", "shared", "weights", "evict"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([4, 8])
    mix = rng.randrange(1 << 30)
    if op == "rope":
        return dict(op=op, rows=_log_int(rng, 1, 12000), hq=hq, hkv=hkv, dtype=rng.choice(["bf16", "f16", "f32"]),
                    rotary=rng.choice([128, 128, 96, 64, 32, 18, 2]), interleaved=rng.random() < 0.5,
                    base=rng.choice([10000.0, 500000.0, 1000000.0]),
                    scaling=rng.choice(["none", "linear", "bands", "yarn"]), factor=rng.choice([2.0, 4.0, 8.0]),
                    start=_log_int(rng, 1, 1000000) - 1, transpose=rng.random() < 0.5)
    if op == "shared":
        groups = rng.choice([1, 2, 3, 5, 8])
        members = _log_int(rng, 1, 64 // groups)
        hi = _log_int(rng, 1, 4096)
        return dict(op=op, groups=groups, members=members, hq=hq, hkv=hkv,
                    common=rng.choice([0, 0, 1, 7, _log_int(rng, 1, 96)]), prefix=_log_int(rng, 1, 256), tail_lo=1,
                    tail_hi=hi, mix=mix)
    hi = _log_int(rng, 1, 65536)
    n = _log_int(rng, 1, max(1, min(28, 600000 // hi)))
    lo = rng.choice([1, hi, max(1, hi // 3)])
    if op == "weights":
        return dict(op=op, requests=n, hq=hq, hkv=hkv, len_lo=lo, len_hi=hi, mix=mix)
    sink, recent = rng.choice([0, 1, 4, 64]), rng.choice([0, 1, 31, 128, 256])
    return dict(op=op, requests=n, hkv=hkv, len_lo=lo, len_hi=hi, keep=round(rng.uniform(0.05, 1.0), 3), sink=sink,
                recent=recent, mix=mix)


def _lengths(case, n, lo, hi):
    """n seeded lengths in [lo, hi], over their logarithm; the first two are the ends."""
    r = random.Random(case["mix"])
    out = [hi, lo] + [_log_int(r, lo, hi) for _ in range(n)]
    return out[:n]


def _tails(case):
    return _lengths(case, case["groups"] * case["members"], case["tail_lo"], case["tail_hi"])


def _context(case):
    return _lengths(case, case["requests"], case["len_lo"], case["len_hi"])


def _keeps(case):
    """Tokens kept of each request: its share, one at least, and never less than the protected ends."""
    return [min(L, max(1, int(L * case["keep"]), case["sink"] + case["recent"])) for L in _context(case)]


def work(case):
    op = case["op"]
    if op == "rope":
        size = 4 if case["dtype"] == "f32" else 2
        elements = case["rows"] * (case["hq"] + case["hkv"]) * D
        return {"bytes": 2 * elements * size, "flops": 3 * case["rows"] * (case["hq"] + case["hkv"]) * case["rotary"]}
    if op == "shared":
        n = case["groups"] * case["members"]
        tails = _tails(case)
        shared = PAGE * (case["common"] + case["groups"] * case["prefix"])
        attended = PAGE * (case["common"] + case["prefix"]) * n + sum(tails)
        return {"bytes": (shared + sum(tails)) * case["hkv"] * 2 * D * 2 + 2 * n * case["hq"] * D * 2,
                "flops": 4 * attended * case["hq"] * D}
    total = sum(_context(case))
    if op == "weights":
        return {"bytes": total * case["hkv"] * (2 * D * 2 + 8) + 2 * case["requests"] * case["hq"] * D * 2,
                "flops": 4 * total * case["hq"] * D}
    kept = sum(_keeps(case))
    return {"bytes": case["hkv"] * (4 * total + kept * (2 * 2 * D * 2 + 8)), "flops": total * case["hkv"]}


# ------------------------------------------------------------------ inputs
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


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


def _accumulated(n, hkv, L, seed):
    """Accumulated weights of L tokens: heavy-tailed, a fifth never attended (equal: zero), some on a coarse grid."""
    g = _gen(seed, 777, n)
    w = torch.exp(2.5 * torch.randn(hkv, L, generator=g, device="cuda") - 6.0)
    u = torch.rand(hkv, L, generator=g, device="cuda")
    w = torch.where(u < 0.2, torch.zeros_like(w), w)
    return torch.where(u > 0.95, torch.round(w * 64) / 64, w)


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


def _make_cache(hq, hkv, n, lengths, spare):
    """A BF16 cache of one layer with room for n requests and `spare` pages more."""
    from int2_rotated_kv_rotate_gb300 import OSCAR_FORMAT_BF16, KVCache

    per = max(1, max((L + PAGE - 1) // PAGE for L in lengths))
    pages = sum((L + PAGE - 1) // PAGE for L in lengths) + spare
    return KVCache(fmt=OSCAR_FORMAT_BF16, n_q_heads=hq, n_kv_heads=hkv, n_layers=1, max_requests=n,
                   max_pages=max(1, pages), max_pages_per_request=per)


def _stride(lengths):
    """Tokens a row of the weights holds: whole pages of the longest request."""
    return PAGE * max(1, max((L + PAGE - 1) // PAGE for L in lengths))


def _append(cache, slots, counts, K, V):
    cache.reserve(slots, counts)
    cache.append(0, K, V)
    cache.commit()


def _prepare_rope(case, seed):
    g = _gen(seed, 1, case["rows"])
    rows, hq, hkv = case["rows"], case["hq"], case["hkv"]
    # queries and keys are slices of one fused projection's rows
    qkv = torch.randn(rows, (hq + 2 * hkv) * D, generator=g, device="cuda").to(DTYPES[case["dtype"]])
    q = qkv[:, :hq * D].view(rows, hq, D)
    k = qkv[:, hq * D:(hq + hkv) * D].view(rows, hkv, D)
    positions = torch.arange(case["start"], case["start"] + rows, device="cuda", dtype=torch.int32)
    st = dict(case=case, q=q, k=k, positions=positions)
    if own:
        from int2_rotated_kv_rotate_gb300 import RotaryEmbedding

        scaling = None
        if case["scaling"] != "none":
            scaling = dict(type=case["scaling"], factor=case["factor"], original_context=32768)
        st["rotary"] = RotaryEmbedding(head_dim=D, rotary_dim=case["rotary"], base=case["base"],
                                       interleaved=case["interleaved"], scaling=scaling)
        st["q_out"] = torch.empty(rows, hq, D, dtype=q.dtype, device="cuda")
        st["k_out"] = torch.empty(rows, hkv, D, dtype=q.dtype, device="cuda")
    else:
        f, magnitude = _frequencies(case)
        st["freq"], st["magnitude"] = f.cuda(), magnitude
    return st


def _segments(case, seed):
    """The batch's runs of tokens: (requests that attend it, K, V), shared ones first."""
    hkv, members = case["hkv"], case["members"]
    n = case["groups"] * members
    out = []
    if case["common"]:
        out.append((list(range(n)), *_tokens(PAGE * case["common"], hkv, seed, 1)))
    for g in range(case["groups"]):
        out.append((list(range(g * members, (g + 1) * members)), *_tokens(PAGE * case["prefix"], hkv, seed, 100 + g)))
    for i, L in enumerate(_tails(case)):
        out.append(([i], *_tokens(L, hkv, seed, 10000 + i)))
    return out


def _prepare_shared(case, seed):
    hq, hkv, members = case["hq"], case["hkv"], case["members"]
    n = case["groups"] * members
    segs = _segments(case, seed)
    q = torch.randn(n, hq, D, generator=_gen(seed, 2), device="cuda").to(torch.bfloat16)
    st = dict(case=case, q=q)
    if not own:
        st["segments"] = [(torch.tensor(m, device="cuda"), K, V) for m, K, V in segs]
        return st
    from int2_rotated_kv_rotate_gb300 import OSCAR_PLAN_SHARED_PREFIX

    head = PAGE * (case["common"] + case["prefix"])
    tails = _tails(case)
    cache = _make_cache(hq, hkv, n, [head + t for t in tails], 0)
    slots = [cache.alloc() for _ in range(n)]
    at = 0
    if case["common"]:
        _append(cache, [slots[0]], [PAGE * case["common"]], segs[0][1], segs[0][2])
        at = 1
    for g in range(case["groups"]):
        first = slots[g * members]
        if g and case["common"]:
            cache.share_prefix(first, slots[0], PAGE * case["common"])
        _append(cache, [first], [PAGE * case["prefix"]], segs[at + g][1], segs[at + g][2])
        for s in slots[g * members + 1:(g + 1) * members]:
            cache.share_prefix(s, first, head)
    tail = segs[at + case["groups"]:]
    _append(cache, slots, tails, torch.cat([s[1] for s in tail]), torch.cat([s[2] for s in tail]))
    cache.plan(slots, flags=OSCAR_PLAN_SHARED_PREFIX)
    st.update(cache=cache, out=torch.empty_like(q))
    return st


def _prepare_weights(case, seed):
    hq, hkv, lengths = case["hq"], case["hkv"], _context(case)
    n = len(lengths)
    q = torch.randn(n, hq, D, generator=_gen(seed, 3), device="cuda").to(torch.bfloat16)
    weights = torch.zeros(n, hkv, _stride(lengths), device="cuda")
    for i, L in enumerate(lengths):
        weights[i, :, :L] = _accumulated(i, hkv, L, seed)
    st = dict(case=case, q=q, weights=weights, weights_out=torch.zeros_like(weights))
    if own:
        cache = _make_cache(hq, hkv, n, lengths, 0)
        slots = [cache.alloc() for _ in range(n)]
        for i, L in enumerate(lengths):
            _append(cache, [slots[i]], [L], *_tokens(L, hkv, seed, i))
        cache.plan(slots)
        st.update(cache=cache, out=torch.empty_like(q))
    else:
        st["kv"] = [_tokens(L, hkv, seed, i) for i, L in enumerate(lengths)]
    return st


def _prepare_evict(case, seed):
    hkv, lengths, keeps = case["hkv"], _context(case), _keeps(case)
    n = len(lengths)
    weights = torch.zeros(n, hkv, _stride(lengths), device="cuda")
    for i, L in enumerate(lengths):
        weights[i, :, :L] = _accumulated(i, hkv, L, seed)
    st = dict(case=case, weights=weights)
    if own:
        spare = sum((k + PAGE - 1) // PAGE for k in keeps)
        cache = _make_cache(4 * hkv, hkv, n, lengths, spare)
        slots = [cache.alloc() for _ in range(n)]
        for i, L in enumerate(lengths):
            _append(cache, [slots[i]], [L], *_tokens(L, hkv, seed, i))
        cache.evict_begin(slots, keeps, n_sink=case["sink"], n_recent=case["recent"])
        pool = cache.bf16_pages(0)  # [pages, hkv, K|V, 64, D]
        views = []
        for i, k in enumerate(keeps):
            pages = cache.evict_pages(slots[i])
            first, full, rest = pages[0], k // PAGE, k % PAGE
            assert pages == list(range(first, first + len(pages)))  # a fresh pool hands its pages out in order
            views += [pool[first:first + full], pool[first + full:first + full + (rest > 0), :, :, :rest]]
        st.update(cache=cache, views=views, weights_out=torch.zeros_like(weights),
                  kept=torch.full(weights.shape, -1, dtype=torch.int32, device="cuda"))
    else:
        # [hkv, K|V, L, D]: what the pages hold of each head
        st["kv"] = [torch.stack(_tokens(L, hkv, seed, i)).permute(2, 0, 1, 3).contiguous()
                    for i, L in enumerate(lengths)]
    return st


def prepare(case, seed):
    return {"rope": _prepare_rope, "shared": _prepare_shared, "weights": _prepare_weights,
            "evict": _prepare_evict}[case["op"]](case, seed)


# ------------------------------------------------------------------ one pass
def _run_rope(st):
    case, R = st["case"], st["case"]["rotary"]
    if own:
        return st["rotary"].apply(st["positions"], st["q"], st["k"], q_out=st["q_out"], k_out=st["k_out"],
                                  transpose=case["transpose"])
    angle = st["positions"].double()[:, None] * st["freq"][None, :]  # in 64 bits: far positions
    cos = (angle.cos().float() * st["magnitude"])[:, None, :]
    sin = (angle.sin().float() * st["magnitude"])[:, None, :]
    if case["transpose"]:
        sin = -sin
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
    return tuple(outs)


def _run_shared(st):
    if own:
        return st["cache"].decode(0, st["q"], out=st["out"])
    case, q = st["case"], st["q"].float()
    n, hq, hkv = q.shape[0], case["hq"], case["hkv"]
    G = hq // hkv
    q = q.view(n, hkv, G, D).transpose(0, 1)  # [hkv, n, G, D]
    m = torch.full((hkv, n, G, 1), -math.inf, device=q.device)
    l = torch.zeros(hkv, n, G, 1, device=q.device)
    o = torch.zeros(hkv, n, G, D, device=q.device)
    for who, K, V in st["segments"]:  # a run of tokens, once for every request that attends it
        rows = q[:, who].reshape(hkv, -1, D)
        s = rows @ K.float().permute(1, 2, 0) / math.sqrt(D)
        top = s.amax(-1, keepdim=True)
        p = torch.exp(s - top)
        part_l = p.sum(-1, keepdim=True).view(hkv, len(who), G, 1)
        part_o = (p @ V.float().transpose(0, 1)).view(hkv, len(who), G, D)
        top = top.view(hkv, len(who), G, 1)
        new = torch.maximum(m[:, who], top)
        a, b = torch.exp(m[:, who] - new), torch.exp(top - new)
        o[:, who] = o[:, who] * a + part_o * b
        l[:, who] = l[:, who] * a + part_l * b
        m[:, who] = new
    return (o / l).transpose(0, 1).reshape(n, hq, D).to(torch.bfloat16)


def _run_weights(st):
    if own:
        return st["cache"].decode_weights(0, st["q"], st["weights"], weights_out=st["weights_out"], out=st["out"])
    case, q = st["case"], st["q"].float()
    hkv, G = case["hkv"], case["hq"] // case["hkv"]
    out, total = [], st["weights_out"]
    for i, (K, V) in enumerate(st["kv"]):
        s = q[i].view(hkv, G, D) @ K.float().permute(1, 2, 0) / math.sqrt(D)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        out.append((p @ V.float().transpose(0, 1)).view(hkv * G, D))
        total[i, :, :K.shape[0]] = st["weights"][i, :, :K.shape[0]] + p.sum(1)
    return torch.stack(out).to(torch.bfloat16), total


def _run_evict(st):
    case = st["case"]
    if own:
        st["cache"].evict(0, st["weights"], weights_out=st["weights_out"], kept=st["kept"])
        return [st["weights_out"], st["kept"]] + st["views"]
    weights = st["weights"]
    out_w, out_i, pages = torch.zeros_like(weights), torch.full(weights.shape, -1, dtype=torch.int32, device="cuda"), []
    for i, (L, keep) in enumerate(zip(_context(case), _keeps(case))):
        w = weights[i, :, :L].clone()
        w[:, :case["sink"]] = math.inf
        w[:, max(0, L - case["recent"]):] = math.inf
        order = torch.sort(w, dim=-1, descending=True, stable=True)[1][:, :keep]  # ties: the lowest index
        index = torch.sort(order, dim=-1)[0]
        out_w[i, :, :keep] = torch.gather(weights[i, :, :L], 1, index)
        out_i[i, :, :keep] = index.to(torch.int32)
        kv = st["kv"][i]  # [hkv, 2, L, D]
        rows = torch.gather(kv, 2, index[:, None, :, None].expand(-1, 2, -1, D))
        full = keep // PAGE
        pages.append(rows[:, :, :full * PAGE].reshape(rows.shape[0], 2, full, PAGE, D).permute(2, 0, 1, 3, 4).contiguous())
        pages.append(rows[:, :, full * PAGE:].unsqueeze(0)[:int(keep % PAGE > 0)].contiguous())
    return [out_w, out_i] + pages


def run(state):
    return {"rope": _run_rope, "shared": _run_shared, "weights": _run_weights,
            "evict": _run_evict}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_rope(st):
    case, R = st["case"], st["case"]["rotary"]
    f, magnitude = _frequencies(case)
    angle = st["positions"].double()[:, None] * f.cuda()[None]
    turn = torch.polar(torch.full_like(angle, magnitude), -angle if case["transpose"] else angle)[:, None, :]
    outs = []
    for x in (st["q"], st["k"]):
        y = x.double()
        pair = y[..., :R].unflatten(-1, (R // 2, 2) if case["interleaved"] else (2, R // 2))
        axis = -1 if case["interleaved"] else -2
        z = torch.complex(pair.select(axis, 0), pair.select(axis, 1)) * turn
        y[..., :R] = torch.stack((z.real, z.imag), dim=axis).flatten(-2)
        outs.append(y)
    return tuple(outs)


def _exact_attention(q, K, V):
    """q [G, D], K and V [L, D] -> (out [G, D], probabilities [G, L]) in fp64."""
    p = torch.softmax(q.double() @ K.double().T * (1.0 / math.sqrt(D)), dim=-1)
    return p @ V.double(), p


def _exact_shared(case, seed, q):
    n, G = q.shape[0], case["hq"] // case["hkv"]
    segs = _segments(case, seed)
    out = torch.empty(n, case["hq"], D, dtype=torch.float64, device="cuda")
    for i in range(n):
        mine = [s for s in segs if i in s[0]]
        for h in range(case["hkv"]):
            K, V = torch.cat([s[1][:, h] for s in mine]), torch.cat([s[2][:, h] for s in mine])
            out[i, h * G:(h + 1) * G] = _exact_attention(q[i, h * G:(h + 1) * G], K, V)[0]
    return out


def _exact_weights(case, st):
    G = case["hq"] // case["hkv"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    total = torch.zeros(st["weights"].shape, dtype=torch.float64, device="cuda")
    for i, (K, V) in enumerate(st["kv"]):
        for h in range(case["hkv"]):
            o, p = _exact_attention(st["q"][i, h * G:(h + 1) * G], K[:, h], V[:, h])
            out[i, h * G:(h + 1) * G] = o
            total[i, h, :K.shape[0]] = st["weights"][i, h, :K.shape[0]].double() + p.sum(0)
    return out, total


def _exact_evict(case, st):
    """By the threshold: every weight above the keep-th largest, then the lowest indices equal to it."""
    weights = st["weights"].double().cpu().numpy()
    out_w, out_i = np.zeros(weights.shape), np.full(weights.shape, -1, dtype=np.int32)
    pages = []
    for i, (L, keep) in enumerate(zip(_context(case), _keeps(case))):
        kv = st["kv"][i]
        full, rest = keep // PAGE, keep % PAGE
        body = torch.empty(full, kv.shape[0], 2, PAGE, D, dtype=torch.float64, device="cuda")
        last = torch.empty(int(rest > 0), kv.shape[0], 2, rest, D, dtype=torch.float64, device="cuda")
        a, b = min(case["sink"], L), max(min(case["sink"], L), L - case["recent"])
        for h in range(kv.shape[0]):
            take = np.ones(L, dtype=bool)
            need = keep - a - (L - b)
            mid = weights[i, h, a:b]
            if need < mid.size:
                edge = np.partition(mid, mid.size - need)[mid.size - need] if need else np.inf
                above = mid > edge
                equal = np.flatnonzero(mid == edge)[:need - int(above.sum())]
                above[equal] = True
                take[a:b] = above
            index = np.flatnonzero(take)
            out_w[i, h, :keep] = weights[i, h, index]
            out_i[i, h, :keep] = index
            rows = kv[h][:, torch.from_numpy(index).cuda()].double()  # [2, keep, D]
            if full:
                body[:, h] = rows[:, :full * PAGE].reshape(2, full, PAGE, D).transpose(0, 1)
            if rest:
                last[0, h] = rows[:, full * PAGE:]
        pages += [body, last]
    return [torch.from_numpy(out_w).cuda(), torch.from_numpy(out_i).cuda()] + pages


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed) if case["op"] != "shared" else None
        if case["op"] == "rope":
            return _exact_rope(st)
        if case["op"] == "weights":
            return _exact_weights(case, st)
        if case["op"] == "evict":
            return _exact_evict(case, st)
        n = case["groups"] * case["members"]
        q = torch.randn(n, case["hq"], D, generator=_gen(seed, 2), device="cuda").to(torch.bfloat16)
        return _exact_shared(case, seed, q)
    finally:
        own = was
