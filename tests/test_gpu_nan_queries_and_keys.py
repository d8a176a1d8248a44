"""Queries that are NaN, or that attend a key of NaN or a score of +inf, have NaN for an output, however many items, tiles or parts
their tokens are in; a score of -inf is a weight of 0.  Nobody else's output changes by a bit."""
import math

import pytest
import torch

from int2_rotated_kv_rotate_gb300 import (OSCAR_FORMAT_BF16, OSCAR_FORMAT_INT2, OSCAR_FORMAT_INT2_CM, OSCAR_FORMAT_INT4,
                                          OSCAR_PLAN_SHARED_PREFIX, KVCache)
from int2_rotated_kv_rotate_gb300 import _native as N

pytestmark = pytest.mark.gpu
HKV = 2


def rows(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(n, HKV, 128, generator=g, device="cuda").bfloat16() for _ in range(2)]


def filled(fmt, kv, gqa, group=32):
    pages = sum(-(-k.shape[0] // 64) for k, _ in kv)
    c = KVCache(fmt=fmt, n_q_heads=HKV * gqa, n_kv_heads=HKV, group=group, max_requests=len(kv), max_pages=pages, max_pages_per_request=pages)
    if c.is_int2:
        eye, one = torch.eye(128).expand(HKV, 128, 128).contiguous(), torch.full((HKV,), 3.0)
        c.set_layer_params(0, eye, eye, one, one)
    slots = [c.alloc() for _ in kv]
    c.reserve(slots, [k.shape[0] for k, _ in kv])
    c.append(0, torch.cat([k for k, _ in kv]), torch.cat([v for _, v in kv]))
    c.commit()
    return c, slots


def queries(n, gqa, seed=9):
    return torch.randn(n, HKV * gqa, 128, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def both(c, q, run):
    o32 = torch.full(q.shape, 7.0, device="cuda")
    out = run(c, q, o32)
    assert torch.equal(out.isnan(), o32.isnan()) and torch.equal(out[~out.isnan()], o32.bfloat16()[~out.isnan()])
    assert c.status() == (0, 0)
    return o32


def decode(c, q, o32):
    return c.decode(0, q, out_f32=o32)


def attend(c, q, o32):
    return c.attend_window(0, q, out_f32=o32)


@pytest.mark.parametrize("gqa", [4, 8])
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("kind", ["bf16", "int4", "int4_128", "int2", "int2_cm", "window", "weights"])
@pytest.mark.parametrize("split", [0, 2])
def test_a_query_that_is_not_finite(kind, gqa, value, split):
    """One channel of one head of one request, on requests of one item and of several."""
    fmt = dict(int4=OSCAR_FORMAT_INT4, int4_128=OSCAR_FORMAT_INT4, int2=OSCAR_FORMAT_INT2, int2_cm=OSCAR_FORMAT_INT2_CM).get(kind, OSCAR_FORMAT_BF16)
    if kind == "int2_cm" and gqa == 8:
        pytest.skip("group 32 at GQA 4 only")
    lengths = (40, 700, 9000, 1)
    c, slots = filled(fmt, [rows(n, n) for n in lengths], gqa, 128 if kind == "int4_128" else 32)
    run = decode
    if kind == "window":
        c.plan_window(slots, n_sink=3, window=split * 3000)
        run = attend
    else:
        c.plan(slots, max_split_pages=split)
    if kind == "weights":
        run = lambda c, q, o32: c.decode_weights(0, q, c.new_weights(), out_f32=o32)[0]  # noqa: E731
    q = queries(4, gqa)
    want = both(c, q, run)
    assert bool(want.isfinite().all())
    for request, head in ((0, 0), (1, gqa + 1), (2, 2), (2, 2 * gqa - 1), (3, 1)):
        bad = q.clone()
        bad[request, head, 17] = value
        got = both(c, bad, run)
        here = torch.zeros(got.shape, dtype=torch.bool, device="cuda")
        here[request, head] = True
        assert torch.equal(got[~here], want[~here])
        if value == math.inf and not bool(got[here].isnan().all()):  # all scores may be -inf: no weights
            assert request in (0, 3) and bool((got[here] == 0).all())
        else:
            assert bool(got[here].isnan().all()), (request, head)


@pytest.mark.parametrize("gqa", [4, 8])
@pytest.mark.parametrize("new", [1, 5, 100, 300])
@pytest.mark.parametrize("L,window", [(320, 0), (3000, 0), (20000, 0), (3000, 130)])
def test_keys_that_are_not_finite(gqa, new, L, window):
    """Single queries, tiles whole and cut: a NaN, and an infinity that makes scores of +inf or -inf by the query's sign."""
    k, v = rows(L, 5)
    q = queries(new, gqa)
    sink = 2
    p, t = torch.arange(L - new, L, device="cuda")[:, None], torch.arange(L, device="cuda")[None]
    see = (t <= p) & ((t > p - window) | (t < sink) if window else t <= p)
    for at, value in ((1, math.nan), (L - 1 - new // 2, math.nan), (L - 1 - new // 2, math.inf), (0, -math.inf), (L // 2, math.inf)):
        bad = k.clone()
        bad[at, 1, 9] = value
        c, slots = filled(OSCAR_FORMAT_BF16, [(bad, v)], gqa)
        c.plan_window(slots, [new], n_sink=sink, window=window)
        if (new, L, gqa) == (5, 20000, 4):
            assert c.window_info()[2] > 0
        got = both(c, q, attend)
        ref = torch.empty(got.shape, dtype=torch.float64, device="cuda")
        for h in range(HKV):
            kk = bad[:, h].double()
            for a in range(0, new, 50):
                s = q[a:a + 50, h * gqa:(h + 1) * gqa].double() @ kk.T / math.sqrt(128.0)
                ref[a:a + 50, h * gqa:(h + 1) * gqa] = torch.softmax(s.masked_fill(~see[a:a + 50, None], -math.inf), -1) @ v[:, h].double()
        assert torch.equal(got.isnan(), ref.isnan()), (at, value)
        fine = ~ref.isnan()
        # half a step of bf16 of each weight; the scores, under 2^7, and exponentials less than 2^-9
        assert float((got.double() - ref)[fine].abs().max()) <= (2.0 ** -8 + 2.0 ** -9) * float(v.abs().max())


@pytest.mark.parametrize("gqa", [4, 8])
@pytest.mark.parametrize("new,L", [(5, 320), (5, 20000), (100, 700), (100, 20000), (200, 6000)])
def test_a_nan_among_the_queries_of_a_tile(gqa, new, L):
    """The same NaN in a whole tile, in one whose blocks are joined and in one that is cut."""
    c, slots = filled(OSCAR_FORMAT_BF16, [rows(L, 5)], gqa)
    q = queries(new, gqa)
    c.plan_window(slots, [new], n_sink=2)
    want = both(c, q, attend)
    assert bool(want.isfinite().all())
    bad, here = q.clone(), torch.zeros(want.shape, dtype=torch.bool, device="cuda")
    for token, head in ((0, 0), (new - 1, 2 * gqa - 1), (new // 2, gqa)):
        bad[token, head, 127] = math.nan
        here[token, head] = True
    got = both(c, bad, attend)
    assert torch.equal(got.isnan(), here) and torch.equal(got[~here], want[~here])


@pytest.mark.parametrize("gqa", [4, 8])
def test_an_infinite_value_reaches_the_joined_parts(gqa):
    """Where the other parts of a cut tile have all the weight, too."""
    L, new = 20000, 5
    k, v = rows(L, 6)
    k[:] = 0
    k[10] = 1.0  # 2^-1500 and less for every other token
    v[L - new, 0, 3] = math.inf
    q = torch.full((new, HKV * gqa, 128), 90.0, device="cuda").bfloat16()
    c, slots = filled(OSCAR_FORMAT_BF16, [(k, v)], gqa)
    c.plan_window(slots, [new])
    assert c.window_info()[2] > 0
    got = both(c, q, attend)
    odd = torch.zeros(got.shape, dtype=torch.bool, device="cuda")
    odd[:, :gqa, 3] = True
    assert torch.equal(~got.isfinite(), odd)


def test_shared_prefixes():
    """Requests whose first pages are attended in one launch for all."""
    gqa, shared, n = 8, 64 * 64, 6
    k, v = rows(shared, 7)
    tails = [rows(70 + i, 20 + i) for i in range(n)]
    pages = shared // 64 + 4 * n
    c = KVCache(fmt=OSCAR_FORMAT_BF16, n_q_heads=HKV * gqa, n_kv_heads=HKV, max_requests=n, max_pages=pages, max_pages_per_request=pages)
    slots = [c.alloc() for _ in range(n)]
    c.reserve(slots[:1], [shared])
    c.append(0, k, v)
    c.commit()
    for s in slots[1:]:
        c.share_prefix(s, slots[0], shared)
    c.reserve(slots, [t[0].shape[0] for t in tails])
    c.append(0, torch.cat([a for a, _ in tails]), torch.cat([b for _, b in tails]))
    c.commit()
    c.plan(slots, flags=OSCAR_PLAN_SHARED_PREFIX | N.OSCAR_PLAN_SHARED_ALWAYS)
    assert c.shared_info()[0] > 0
    q = queries(n, gqa)
    want = both(c, q, decode)
    bad = q.clone()
    bad[3, 10, 5] = math.nan
    got = both(c, bad, decode)
    here = torch.zeros(got.shape, dtype=torch.bool, device="cuda")
    here[3, 10] = True
    assert torch.equal(got[~here], want[~here]) and bool(got[here].isnan().all())
