"""Attention within a sliding window and over the first tokens, against attention in 64 bits over what
each query sees.

Tolerances of the fp32 output (derived, not fitted).  Scores are exact bf16 products summed in fp32,
off by at most 2^-18 S in all, S = sum |q_c k_c| / sqrt(128); with an exponential's 2^-20 a weight is
off by a factor 1 + 2^-18 S + 2^-20, which moves the output by at most twice that of the largest
value.  Single queries keep 16 bits of a weight (2^-16), several queries of a request its bf16, off by
up to half a step (2^-8) of each, while the denominator keeps all."""
import math

import pytest
import torch

from int2_rotated_kv_rotate_gb300 import (OSCAR_FORMAT_BF16, OSCAR_FORMAT_INT2, OSCAR_FORMAT_INT4, KVCache, OscarError,
                                          RotaryEmbedding)
from int2_rotated_kv_rotate_gb300 import _native as N

pytestmark = pytest.mark.gpu


def make(lengths, hkv=2, gqa=4, layers=1, spare=0):
    pages = sum((n + 63) // 64 for n in lengths) + spare
    c = KVCache(fmt=OSCAR_FORMAT_BF16, n_q_heads=hkv * gqa, n_kv_heads=hkv, n_layers=layers, max_requests=max(1, len(lengths)),
                max_pages=max(1, pages), max_pages_per_request=max(1, pages))
    for layer in range(layers):  # what no token was written to is NaN
        c.bf16_pages(layer).view(torch.int16).fill_(-1)
    return c


def tokens(n, hkv, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn(n, hkv, 128, generator=g, device="cuda") for _ in range(2))
    k[..., 5] *= 8
    v[..., 77] *= 8
    return k.bfloat16(), v.bfloat16()


def filled(lengths, hkv, gqa, layers=1, spare=0, kv=None):
    c = make(lengths, hkv, gqa, layers, spare)
    slots = [c.alloc() for _ in lengths]
    kv = kv or [tokens(n, hkv, 100 + i) for i, n in enumerate(lengths)]
    some = [i for i, n in enumerate(lengths) if n]
    c.reserve([slots[i] for i in some], [lengths[i] for i in some])
    for layer in range(layers):
        c.append(layer, torch.cat([kv[i][0] for i in some]), torch.cat([kv[i][1] for i in some]))
    c.commit()
    return c, slots, kv


def seen(L, n, sink, window):
    """bool [n, L]: what the last n tokens see."""
    p, t = torch.arange(L - n, L)[:, None], torch.arange(L)[None]
    s = t <= p
    return s & ((t < sink) | (t > p - window)) if window else s


def check(out, out32, q, k, v, n, sink, window, label, rows=None):
    """One request's queries [n, H_q, 128] against 64 bits (rows: the ones that are looked at)."""
    L, hkv = k.shape[:2]
    G = q.shape[1] // hkv
    see = seen(L, n, sink, window).cuda()
    rows = torch.arange(n) if rows is None else torch.as_tensor(rows)
    for h in range(hkv):
        kk, vv = k[:, h].double(), v[:, h].double()
        for a in range(0, len(rows), 256):
            i = rows[a:a + 256].cuda()
            qq = q[i, h * G:(h + 1) * G].double()
            s = (qq @ kk.T / math.sqrt(128.0)).masked_fill(~see[i][:, None], -math.inf)
            ref = torch.softmax(s, -1) @ vv
            S = float((qq.abs() @ kk.abs().amax(0)).max()) / math.sqrt(128.0)
            big = float(vv.abs().max())
            tol = (2 * (2.0 ** -18 * S + 2.0 ** -20) + (2.0 ** -16 if n == 1 else 2.0 ** -8)) * big
            err = float((out32[i, h * G:(h + 1) * G].double() - ref).abs().max())
            assert err <= tol, f"{label} head {h}: {err:.3e} > {tol:.3e}"
    assert torch.equal(out, out32.bfloat16())


def run(c, q, layer=0):
    o32 = torch.full(q.shape, math.nan, device="cuda")
    return c.attend_window(layer, q, out_f32=o32), o32


@pytest.mark.parametrize("gqa", [4, 8])
@pytest.mark.parametrize("sink,window", [(0, 1), (4, 1), (4, 64), (0, 0), (1, 63), (65, 130), (130, 40), (4, 1000000), (1000000, 5)])
@pytest.mark.parametrize("lengths", [(1, 2, 63, 64, 65), (130, 200, 700)])
def test_single_queries(gqa, sink, window, lengths):
    c, slots, kv = filled(lengths, 2, gqa)
    q = torch.randn(len(lengths), 2 * gqa, 128, device="cuda").bfloat16()
    assert c.plan_window(slots, n_sink=sink, window=window) == len(lengths)
    out, o32 = run(c, q)
    for i, (k, v) in enumerate(kv):
        check(out[i:i + 1], o32[i:i + 1], q[i:i + 1], k, v, 1, sink, window, f"request {i}")
    assert c.window_info()[1:] == (0, 0) and c.status() == (0, 0)


@pytest.mark.parametrize("gqa", [4, 8])
@pytest.mark.parametrize("sink,window", [(0, 1), (4, 1), (4, 64), (0, 0), (1, 63), (65, 130), (130, 40), (3, 129), (1000000, 5)])
@pytest.mark.parametrize("lengths,new", [((2, 63, 64, 65, 129), (2, 63, 64, 33, 2)), ((130, 200, 700), (5, 1, 300)),
                                         ((500, 333, 3), (500, 0, 3)), ((1030,), (17,))])
def test_several_queries(gqa, sink, window, lengths, new):
    c, slots, kv = filled(lengths, 2, gqa)
    q = torch.randn(sum(new), 2 * gqa, 128, device="cuda").bfloat16()
    c.plan_window(slots, new, n_sink=sink, window=window)
    out, o32 = run(c, q)
    at = 0
    for i, n in enumerate(new):
        if n:
            check(out[at:at + n], o32[at:at + n], q[at:at + n], *kv[i], n, sink, window, f"request {i}")
        at += n
    assert c.status() == (0, 0)


@pytest.mark.parametrize("gqa,hkv,L,n,sink,window", [(4, 8, 6000, 3000, 4, 1024), (8, 1, 20000, 9, 4, 0), (4, 3, 9000, 2000, 0, 0),
                                                     (8, 2, 5000, 5000, 64, 333)])
def test_long(gqa, hkv, L, n, sink, window):
    c, slots, kv = filled([L], hkv, gqa)
    q = torch.randn(n, hkv * gqa, 128, device="cuda").bfloat16()
    c.plan_window(slots, [n], n_sink=sink, window=window)
    out, o32 = run(c, q)
    g = torch.Generator().manual_seed(1)
    rows = sorted(set([0, 1, n - 1, n // 2] + torch.randint(0, n, (200,), generator=g).tolist()))
    check(out, o32, q, *kv[0], n, sink, window, f"{c.window_info()}", rows)
    for _ in range(3):  # the same bits every time
        assert torch.equal(run(c, q)[1], o32)
    assert c.status() == (0, 0)


def test_tiles_are_cut_and_joined():
    c, slots, kv = filled([20000, 300], 1, 4)
    q = torch.randn(7 + 40, 4, 128, device="cuda").bfloat16()
    c.plan_window(slots, [7, 40])
    rows, parts, cut = c.window_info()
    assert rows == 0 and cut >= 1 and parts > 2
    out, o32 = run(c, q)
    check(out[:7], o32[:7], q[:7], *kv[0], 7, 0, 0, "cut")
    check(out[7:], o32[7:], q[7:], *kv[1], 40, 0, 0, "short")


def test_many_small_tiles():
    """More small tiles than SMs: a CTA joins the blocks of several, beside larger and single ones."""
    lengths = [200 + 37 * i for i in range(40)]
    new = [(5, 2, 9, 1, 40)[i % 5] for i in range(40)]
    c, slots, kv = filled(lengths, 8, 4)
    q = torch.randn(sum(new), 32, 128, device="cuda").bfloat16()
    c.plan_window(slots, new, n_sink=4, window=700)
    out, o32 = run(c, q)
    at = 0
    for i, n in enumerate(new):
        if i % 3 == 0:
            check(out[at:at + n], o32[at:at + n], q[at:at + n], *kv[i], n, 4, 700, f"request {i} {c.window_info()}")
        at += n
    assert torch.equal(run(c, q)[1], o32) and c.status() == (0, 0)


@pytest.mark.parametrize("gqa", [4, 8])
@pytest.mark.parametrize("new", [(1, 1), (300, 2)])
def test_infinities_and_nan_reach_only_those_who_see_them(gqa, new):
    """Keys and values outside a query's view are as if they were not there, whatever they hold."""
    lengths, sink, window = (500, 333), 3, 70
    kv = [tokens(n, 2, 100 + i) for i, n in enumerate(lengths)]
    clean = [(k.clone(), v.clone()) for k, v in kv]
    places = {0: (50, 3, 120, 260, 333, 410, 431, 470, 499), 1: (0, 100, 262, 331, 332)}
    for i, ts in places.items():
        for j, t in enumerate(ts):
            kv[i][1][t, :, (7 * j) % 128] = (math.inf, -math.inf, math.nan)[j % 3]
        kv[i][0][10] = math.nan  # a key that only queries near it see
        kv[i][0][40, 1, 3] = math.inf
    c, slots, _ = filled(lengths, 2, gqa, kv=kv)
    q = torch.randn(sum(new), 2 * gqa, 128, device="cuda").bfloat16()
    c.plan_window(slots, new, n_sink=sink, window=window)
    out, o32 = run(c, q)
    at = 0
    for i, n in enumerate(new):
        L = lengths[i]
        see = seen(L, n, sink, window)
        k, v = clean[i]
        v = v.clone()
        bad_key = see[:, 10] | see[:, 40]
        want_bad = torch.zeros(n, 2, 128, dtype=torch.bool)
        for j, t in enumerate(places[i]):
            want_bad[see[:, t], :, (7 * j) % 128] = True
        for h in range(2):
            rows = slice(h * gqa, (h + 1) * gqa)
            got = o32[at:at + n, rows].cpu()
            ok = ~bad_key
            assert torch.equal(~got.isfinite()[ok], want_bad[ok][:, h:h + 1].expand(-1, gqa, -1)), f"request {i} head {h}"
            kk, vv = k[:, h].double().cpu(), kv[i][1][:, h].double().cpu().nan_to_num(0.0, 0.0, 0.0)
            s = (q[at:at + n, rows].double().cpu() @ kk.T / math.sqrt(128.0)).masked_fill(~see[:, None], -math.inf)
            ref = torch.softmax(s, -1) @ vv
            fine = got.isfinite() & ok[:, None, None]
            tol = (2.0 ** -8 + 2.0 ** -9) * float(vv.abs().max())
            assert float((got.double() - ref)[fine].abs().max()) <= tol
        at += n
    assert c.status() == (0, 0)


def test_beside_the_decode_plan():
    """Layers with and without a window take turns under one reservation; the windowless plan is the
    decode's attention."""
    c, slots, kv = filled([700, 65, 3000], 2, 4, layers=2, spare=3)
    k2, v2 = tokens(3, 2, 5)
    q = torch.randn(3, 8, 128, device="cuda").bfloat16()
    c.reserve(slots, [1, 1, 1])
    c.plan(slots)
    c.plan_window(slots, n_sink=4, window=100)
    o32 = torch.empty(q.shape, device="cuda")
    for layer in range(2):
        c.append(layer, k2, v2)
    full = c.decode(0, q, out_f32=o32)
    out, w32 = run(c, q, 1)
    for i in range(3):
        k, v = (torch.cat((a, b[i:i + 1])) for a, b in zip(kv[i], (k2, v2)))
        check(full[i:i + 1], o32[i:i + 1], q[i:i + 1], k, v, 1, 0, 0, f"full {i}")
        check(out[i:i + 1], w32[i:i + 1], q[i:i + 1], k, v, 1, 4, 100, f"window {i}")
    c.commit()
    assert torch.equal(run(c, q, 1)[1], w32)  # a plan made over the reservation outlives its commit
    c.plan_window(slots)
    a = run(c, q, 0)[1]
    assert float((a - o32).abs().max()) <= 2.0 ** -14 * 40  # two orders of the same sums
    c.reserve(slots, [1, 1, 1])
    with pytest.raises(OscarError) as e:
        c.attend_window(0, q)
    assert e.value.status == 7


def test_a_prompt_in_chunks_equals_itself_whole():
    """Chunked prefill with rotated appends: every chunk's queries see the history and themselves."""
    L, sink, window = 1000, 4, 200
    rot = RotaryEmbedding(base=1e6)
    c = make([L, L], 2, 4)
    a, b = c.alloc(), c.alloc()
    k, v = tokens(L, 2, 1)
    q = torch.randn(L, 8, 128, device="cuda").bfloat16()
    c.reserve([a], [L])
    q1 = c.append_rotated(0, rot, k, v, q)
    c.plan_window([a], [L], n_sink=sink, window=window)
    whole, w32 = run(c, q1)
    c.commit()
    qr, kr = rot.apply(torch.arange(L).cuda(), q, k)
    check(whole, w32, qr, kr, v, L, sink, window, "whole")
    at = 0
    for n in (1, 63, 300, 1, 2, 633):
        c.reserve([b], [n])
        qc = c.append_rotated(0, rot, k[at:at + n], v[at:at + n], q[at:at + n])
        c.plan_window([b], [n], n_sink=sink, window=window)
        out, o32 = run(c, qc)
        check(out, o32, qc, kr[:at + n], v[:at + n], n, sink, window, f"chunk at {at}")
        c.commit()
        at += n
    assert c.status() == (0, 0)


def test_captured_launches_serve_later_plans():
    """A graph captured under a plan of single queries is replayed under plans of many, and back."""
    c, slots, kv = filled([900, 300, 2000], 2, 8)
    q = torch.randn(3 + 200, 16, 128, device="cuda").bfloat16()
    plans = [[1, 1, 1], [100, 3, 100], [1, 1, 201], [1, 1, 1]]
    big, big32 = torch.empty_like(q), torch.empty(q.shape, device="cuda")
    c.plan_window(slots, plans[0], n_sink=4, window=128)
    N.oscar_window_attention(c.handle, 0, q, big, c.window_workspace, big32)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        N.oscar_window_attention(c.handle, 0, q, big, c.window_workspace, big32)
    with pytest.raises(OscarError):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            N.oscar_window_attention(c.handle, 0, q, big, c.window_workspace[:c.window_workspace.numel() - 256], big32)
    torch.cuda.synchronize()
    for new in plans:
        n = sum(new)
        c.plan_window(slots, new, n_sink=4, window=128)
        big.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want, w32 = run(c, q[:n])
        assert torch.equal(big[:n], want) and torch.equal(big32[:n], w32)
        assert bool((big[n:] == 0).all())  # rows behind the queries stay
    assert c.status() == (0, 0)


def test_another_stream():
    c, slots, kv = filled([900, 300], 2, 4)
    q = torch.randn(51, 8, 128, device="cuda").bfloat16()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for new in ((1, 50), (50, 1)):
        c.plan_window(slots, new, n_sink=4, window=100, stream=side.cuda_stream)
        out = c.attend_window(0, q, stream=side)
        side.synchronize()
        c.plan_window(slots, new, n_sink=4, window=100)
        assert torch.equal(out, c.attend_window(0, q))
        torch.cuda.synchronize()


def test_bad_page_entry_is_flagged():
    c, slots, _ = filled([900], 2, 4)
    table = c.mem[c.layout.page_table:c.layout.page_table + 64].view(torch.int32)
    keep = table.clone()
    for new in ([1], [100]):
        c.plan_window(slots, new)
        table[3] = -7
        q = torch.randn(new[0], 8, 128, device="cuda").bfloat16()
        c.attend_window(0, q)
        assert c.status() == (4, N.OSCAR_FLAG_BAD_PAGE)
        table.copy_(keep)
        c.attend_window(0, q)
        assert c.status() == (0, 0)


def test_refusals():
    c, slots, _ = filled([100, 30], 2, 4, spare=2)
    q = torch.randn(2, 8, 128, device="cuda").bfloat16()
    with pytest.raises(ValueError):
        c.attend_window(0, q)
    for kw in (dict(n_queries=[1, 31]), dict(n_queries=[-1, 1]), dict(n_sink=-1), dict(window=-1)):
        with pytest.raises(OscarError):
            c.plan_window(slots, **kw)
    with pytest.raises(ValueError):
        c.plan_window(slots, [1])
    with pytest.raises(OscarError):
        c.plan_window([slots[0], slots[0]])
    c.plan_window(slots)
    for bad in (q[:1], q.float(), q.cpu(), q[:, :4]):
        with pytest.raises(ValueError):
            c.attend_window(0, bad)
    with pytest.raises(OscarError):
        c.attend_window(1, q)
    with pytest.raises(ValueError):
        c.attend_window(0, q, out=q.cpu())
    odd = torch.empty(2 * 8 * 128 + 1, device="cuda").bfloat16()[1:].view(2, 8, 128)
    with pytest.raises(OscarError):
        c.attend_window(0, odd)
    with pytest.raises(OscarError):
        N.oscar_window_attention(c.handle, 0, q, q.clone(), c.window_workspace[:256])
    assert c.plan_window(slots, [0, 0]) == 0 and c.attend_window(0, q[:0]).shape == (0, 8, 128)
    c.free(slots[1])
    with pytest.raises(OscarError):
        c.attend_window(0, q[:0].new_zeros(0, 8, 128)) if c._n_window else N.oscar_window_attention(c.handle, 0, q, q, c.window_workspace)
    empty = make([64])
    s = empty.alloc()
    with pytest.raises(OscarError):  # a request without tokens has no query
        empty.plan_window([s])
    for fmt in (OSCAR_FORMAT_INT2, OSCAR_FORMAT_INT4):
        o = KVCache(fmt=fmt, n_q_heads=8, n_kv_heads=2, max_requests=1, max_pages=2, max_pages_per_request=2)
        with pytest.raises(OscarError) as e:
            o.plan_window([o.alloc()])
        assert e.value.status == 7
        assert N.oscar_window_workspace_max_bytes(o.handle) == 0
