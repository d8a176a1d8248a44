"""The 4-bit cache: rows bit for bit against the definition in fp32, decode against attention in 64
bits over the values that the rows stand for, its refusals.

Tolerance of the decode before its rounding to bf16 (derived, not fitted).  A score's products and
sums are in fp32: at most 24 additions of magnitude S = sum |q_c| (15 s + |z|) / sqrt(128), each off
by 2^-23 of it on a tensor core that truncates, so under 2^-18 S; an exponential and its argument add
2^-20.  A weight is thus off by a factor 1 + 2^-18 S + 2^-20, which moves the output by at most
twice that of the largest value.  P' is rounded to 11 bits (2^-12 of code * scale <= the group's
range, and 2^-25 of the largest scale where it is subnormal)."""
import math

import pytest
import torch

import int2_rotated_kv_rotate_gb300 as pkg
from int2_rotated_kv_rotate_gb300 import OSCAR_FORMAT_INT4, KVCache, OscarError, RotaryEmbedding
from int2_rotated_kv_rotate_gb300 import _native as N

pytestmark = pytest.mark.gpu
LIMIT = 2.0 ** 126


def make(lengths, hkv=2, gqa=4, group=32, layers=1, spare=0):
    pages = max(1, sum((n + 63) // 64 for n in lengths) + spare)
    cache = KVCache(fmt=OSCAR_FORMAT_INT4, n_q_heads=hkv * gqa, n_kv_heads=hkv, group=group, n_layers=layers,
                    max_requests=max(1, len(lengths)), max_pages=pages, max_pages_per_request=pages)
    at = cache.layout.codes  # what no token was written to: NaN scales and zeros
    cache.mem[at:at + layers * pages * hkv * cache.layout.codes_page_bytes].fill_(255)
    return cache


def tokens(n, hkv, seed, scale_k=1.0, scale_v=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn(n, hkv, 128, generator=g, device="cuda") for _ in range(2))
    k[..., 5] *= 20
    v[..., 77] *= 8
    norm = torch.exp(0.5 * torch.randn(n, hkv, 1, generator=g, device="cuda"))
    return (k * norm * scale_k).bfloat16(), (v * norm * scale_v).bfloat16()


def quantized(x, group):
    """Codes, scales and zero points of bf16 rows by the definition, fp32 on the host."""
    y = x.float().cpu()
    y = torch.where(y.isnan(), torch.tensor(LIMIT), y).clamp(-LIMIT, LIMIT).unflatten(-1, (-1, group))
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    s = torch.div(hi - lo, torch.full_like(lo, 15.0)).bfloat16()
    t = torch.div(y - lo, s.float())
    codes = torch.where(s == 0, torch.zeros_like(y), t.round().clamp(0, 15))
    return codes.flatten(-2), s, lo


def values(x, group):
    codes, s, lo = quantized(x, group)
    return torch.addcmul(lo, codes.unflatten(-1, (-1, group)), s.float()).flatten(-2)


def fill(cache, slots, kv, step=None):
    for s, (k, v) in zip(slots, kv):
        n, at = k.shape[0], 0
        while at < n:
            m = min(n - at, step or n)
            cache.reserve([s], [m])
            cache.append(0, k[at:at + m], v[at:at + m])
            cache.commit()
            at += m


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("n,step", [(1, None), (17, 1), (64, None), (65, 64), (333, 50), (2000, None)])
def test_rows_are_the_definitions(group, n, step):
    cache = make([n], hkv=3, group=group)
    slot = cache.alloc()
    k, v = tokens(n, 3, n)
    if n > 16:
        k[3] = 0  # constant groups: scale 0
        v[4, 1] = 7.25
        k[5, 0, :32] = torch.arange(32, device="cuda") / 2  # halves of a step: quotients that tie
        v[6] *= 2.0 ** -130
        v[7] *= 2.0 ** 90
    fill(cache, [slot], [(k, v)], step)
    got = cache.read(0, slot, 0, n, dtype=torch.float32)
    for x, y in zip((k, v), got):
        assert torch.equal(y.cpu(), values(x, group))
    for a, b in ((n // 3, n), (n // 2, n - n // 7), (0, 1)):
        for dtype in (torch.bfloat16, torch.float32):
            for x, y in zip(got, cache.read(0, slot, a, b, dtype=dtype)):
                assert torch.equal(y, x[a:b].to(dtype))
    # the stored layout: bits and words as documented
    t = n - 1
    head, ng = cache.layout.codes_page_bytes, 128 // group
    page = cache.pages(slot)[t // 64]
    at = cache.layout.codes + (page * 3 + 2) * head + (t % 64 // 32) * (head // 2)  # the half page of head 2
    assert head == 2 * 2 * 32 * (64 + 4 * ng)
    block = cache.mem[at + 2048:at + 4096].cpu().view(torch.int32).view(32, 16)  # V
    codes, s, z = quantized(v[t, 2], group)
    for c in range(128):
        word = int(block[t % 32, 4 * ((c // 8 % 4) ^ (t % 64 // 2 % 4)) + c // 32])
        assert (word >> (4 * (c % 8))) & 15 == int(codes[c])
    at += 4096 + 32 * ng * 4 + (t % 32) * ng * 4
    sz = cache.mem[at:at + ng * 4].cpu().view(torch.bfloat16).view(ng, 2)
    assert torch.equal(sz[:, 0], s.flatten()) and torch.equal(sz[:, 1].float(), z.flatten())


def test_rows_of_values_that_are_not_finite():
    cache = make([5], hkv=1)
    slot = cache.alloc()
    k, v = tokens(5, 1, 3)
    k[0, 0, 3], k[1, 0, 40], v[2, 0, 9], v[3] = math.inf, -math.inf, math.nan, math.inf
    v[4, 0, 0] = torch.finfo(torch.bfloat16).max
    fill(cache, [slot], [(k, v)])
    for x, y in zip((k, v), cache.read(0, slot, 0, 5, dtype=torch.float32)):
        assert torch.equal(y.cpu(), values(x, 32)) and bool(y.isfinite().all())


def check(out, out32, q, k, v, sv, group, label):
    """One request's decode against 64 bits; k, v: the values [L, hkv, 128] held, sv their largest scales per head."""
    hkv, G = k.shape[1], q.shape[0] // k.shape[1]
    for h in range(hkv):
        qq, kk, vv = (x.double().cpu() for x in (q[h * G:(h + 1) * G], k[:, h], v[:, h]))
        ref = torch.softmax(qq @ kk.T / math.sqrt(128.0), -1) @ vv
        # 15 s + |z| is at most three times a group's largest value
        top = kk.abs().amax(0).unflatten(0, (-1, group)).amax(-1).repeat_interleave(group)
        S = 3 * float((qq.abs() @ top).max()) / math.sqrt(128.0)
        span = 15 * float(sv[h])
        tol = 2 * (2.0 ** -18 * S + 2.0 ** -20) * float(vv.abs().max()) + (2.0 ** -12 + 15 * 2.0 ** -25) * span
        err = float((out32[h * G:(h + 1) * G].double().cpu() - ref).abs().max())
        assert err <= tol, f"{label} head {h}: {err:.3e} > {tol:.3e}"
    assert torch.equal(out, out32.bfloat16())


@pytest.mark.parametrize("gqa", [4, 8])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("lengths,hkv,sk,svs", [((1, 31, 32, 33), 1, 1, 1), ((63, 64, 65, 127, 129), 2, 1, 1),
                                                ((1000, 1, 4097), 3, 1, 1), ((20000,), 2, 1, 1),
                                                ((70, 500), 2, 2.0 ** -60, 2.0 ** 90), ((70, 500), 2, 1e-3, 2.0 ** -100)])
def test_decode(gqa, group, lengths, hkv, sk, svs):
    cache = make(lengths, hkv=hkv, gqa=gqa, group=group)
    slots = [cache.alloc() for _ in lengths]
    kv = [tokens(n, hkv, 10 + i, sk, svs) for i, n in enumerate(lengths)]
    fill(cache, slots, kv)
    held = [cache.read(0, s, 0, n, dtype=torch.float32) for s, n in zip(slots, lengths)]
    q = (torch.randn(len(lengths), hkv * gqa, 128, device="cuda") / sk).bfloat16()
    for split in (0, 1, 3):
        cache.plan(slots, max_split_pages=split)
        o32 = torch.empty(q.shape, device="cuda")
        out = cache.decode(0, q, out_f32=o32)
        again = cache.decode(0, q)
        assert torch.equal(out, again)
        for i, n in enumerate(lengths):
            sv = quantized(kv[i][1], group)[1].float().amax((0, 2, 3))
            check(out[i], o32[i], q[i], held[i][0], held[i][1], sv, group, f"split {split} request {i}")
    assert cache.status() == (0, 0)


def test_many_items_and_empty_requests():
    """Several waves of items, requests without tokens (zeros), queries of zero."""
    lengths = [0] + [3000 + 61 * i for i in range(40)] + [0]
    cache = make(lengths, hkv=8, gqa=8)
    slots = [cache.alloc() for _ in lengths]
    kv = [tokens(n, 8, i) for i, n in enumerate(lengths)]
    fill(cache, slots, kv)
    q = torch.randn(len(lengths), 64, 128, device="cuda").bfloat16()
    q[5] = 0
    cache.plan(slots, max_split_pages=4)
    o32 = torch.empty(q.shape, device="cuda")
    out = cache.decode(0, q, out_f32=o32)
    assert bool((out[0] == 0).all() and (out[-1] == 0).all())
    for i in (1, 5, 40):
        k, v = cache.read(0, slots[i], 0, lengths[i], dtype=torch.float32)
        check(out[i], o32[i], q[i], k, v, quantized(kv[i][1], 32)[1].float().amax((0, 2, 3)), 32, f"request {i}")
    assert cache.status() == (0, 0)


def test_prefix_sharing_a_step_and_a_graph():
    """Append, decode and a sharer's continuation as a serving step uses them, eager and replayed."""
    cache = make([300, 300, 0], hkv=2, gqa=4, layers=2, spare=4)
    a, b = cache.alloc(), cache.alloc()
    k, v = tokens(300, 2, 1)
    for layer in range(2):
        if layer == 0:
            cache.reserve([a], [256])
        cache.append(layer, k[:256], v[:256])
    cache.commit()
    cache.share_prefix(b, a, 256)
    k2, v2 = tokens(2, 2, 2)
    q = torch.randn(2, 8, 128, device="cuda").bfloat16()
    outs = [torch.empty_like(q) for _ in range(2)]

    def step():
        for layer in range(2):
            cache.append(layer, k2, v2)
            cache.decode(layer, q, out=outs[layer])

    cache.reserve([a, b], [1, 1])
    cache.plan([a, b])
    step()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for o in outs:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    cache.commit()
    for i, s in enumerate((a, b)):
        held = cache.read(1, s, 0, 257, dtype=torch.float32)
        full = [torch.cat((x[:256], y[i:i + 1])) for x, y in zip((k, v), (k2, v2))]
        for x, y in zip(full, held):
            assert torch.equal(y.cpu(), values(x, 32))
        o32 = want[1][i].float()  # rounded to 8 bits, 2^-8; S < 64 here, so the rest is under 2^-9
        for h in range(2):
            p = torch.softmax(q[i, 4 * h:4 * h + 4].double() @ held[0][:, h].double().T / math.sqrt(128.0), -1)
            ref = p @ held[1][:, h].double()
            assert float((o32[4 * h:4 * h + 4].double() - ref).abs().max()) <= float(held[1][:, h].abs().max()) * (2.0 ** -8 + 2.0 ** -9)
    # a later plan under the captured launches: longer requests
    cache.reserve([a, b], [1, 1])
    cache.plan([a, b])
    graph.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in outs]
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(got, outs))
    cache.commit()
    assert cache.status() == (0, 0)


def test_another_stream():
    cache = make([500, 3])
    slots = [cache.alloc(), cache.alloc()]
    kv = [tokens(500, 2, 1), tokens(3, 2, 2)]
    q = torch.randn(2, 8, 128, device="cuda").bfloat16()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    cache.reserve(slots, [500, 3], stream=side)
    cache.append(0, torch.cat([x[0] for x in kv]), torch.cat([x[1] for x in kv]), stream=side.cuda_stream)
    side.wait_stream(torch.cuda.current_stream())
    cache.append(0, torch.cat([x[0] for x in kv]), torch.cat([x[1] for x in kv]), stream=side.cuda_stream)
    cache.commit()
    cache.plan(slots, stream=side)
    out = cache.decode(0, q, stream=side)
    k, v = cache.read(0, slots[0], 0, 500, dtype=torch.float32, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(v.cpu(), values(kv[0][1], 32))
    torch.cuda.synchronize()
    cache.plan(slots)
    assert torch.equal(out, cache.decode(0, q))


def test_bad_page_entry_is_flagged():
    cache = make([200])
    slot = cache.alloc()
    fill(cache, [slot], [tokens(200, 2, 1)])
    table = cache.mem[cache.layout.page_table:cache.layout.page_table + 16].view(torch.int32)
    keep = table.clone()
    table[1] = 1 << 20
    cache.plan([slot])
    out = cache.decode(0, torch.randn(1, 8, 128, device="cuda").bfloat16())
    cache.read(0, slot, 0, 200)
    assert cache.status() == (4, N.OSCAR_FLAG_BAD_PAGE) and bool(out.isfinite().all())
    table.copy_(keep)
    cache.plan([slot])
    cache.decode(0, torch.randn(1, 8, 128, device="cuda").bfloat16())
    assert cache.status() == (0, 0)


def test_refusals():
    cache = make([200], spare=2)
    slot = cache.alloc()
    k, v = tokens(10, 2, 1)
    z = torch.zeros(1, 8, 128, device="cuda").bfloat16()
    with pytest.raises(OscarError):  # no reservation
        N.oscar_int4_append(cache.handle, 0, k, v)
    cache.reserve([slot], [10])
    with pytest.raises(ValueError):
        cache.append(0, k[:9], v)
    with pytest.raises(ValueError):
        cache.append(0, k.float(), v)
    for call in (N.oscar_bf16_append, N.oscar_quantize_append):
        with pytest.raises(OscarError) as e:
            call(cache.handle, 0, k, v)
        assert e.value.status == 7
    with pytest.raises(OscarError):
        cache.append(1, k, v)
    cache.append(0, k, v)
    assert cache.read(0, slot, 0, 10)[0].shape == (10, 2, 128)  # reserved tokens, once appended
    for a, b in ((0, 11), (-1, 3), (5, 4)):
        with pytest.raises((OscarError, ValueError)):
            cache.read(0, slot, a, b)
    cache.commit()
    cache.read(0, slot, 3, 3)
    both = torch.empty(20, 2, 128, device="cuda").bfloat16()
    with pytest.raises(OscarError):
        cache.read(0, slot, 0, 10, k_out=both[:10], v_out=both[5:15])
    with pytest.raises(ValueError):
        cache.read(0, slot, 0, 10, dtype=torch.float16)
    with pytest.raises(ValueError):
        cache.read(0, slot, 0, 10, k_out=both[:10].cpu())
    with pytest.raises(OscarError):  # no plan
        N.oscar_int4_decode_attention(cache.handle, 0, z, z.clone(), torch.empty(256, dtype=torch.uint8, device="cuda"))
    cache.plan([slot])
    for call in (N.oscar_bf16_decode_attention, N.oscar_decode_attention):
        with pytest.raises(OscarError) as e:
            call(cache.handle, 0, z, z.clone(), cache.workspace)
        assert e.value.status == 7
    with pytest.raises(OscarError):
        cache.plan([slot], flags=pkg.OSCAR_PLAN_SHARED_PREFIX)
    with pytest.raises(OscarError):
        cache.plan([slot], flags=N.OSCAR_PLAN_FOLDED_ROTATIONS)
    with pytest.raises(OscarError):
        cache.evict_begin([slot], [5])
    with pytest.raises(ValueError):
        cache.new_weights()
    with pytest.raises(ValueError):
        cache.bf16_pages(0)
    with pytest.raises(OscarError):
        cache.set_layer_params(0, torch.eye(128)[None].repeat(2, 1, 1), torch.eye(128)[None].repeat(2, 1, 1), torch.ones(2), torch.ones(2))
    bf = KVCache(fmt=pkg.OSCAR_FORMAT_BF16, n_q_heads=8, n_kv_heads=2, max_requests=1, max_pages=2, max_pages_per_request=2)
    s = bf.alloc()
    bf.reserve([s], [10])
    with pytest.raises(OscarError) as e:
        N.oscar_int4_append(bf.handle, 0, k, v)
    assert e.value.status == 7
    with pytest.raises(OscarError):
        bf.read(0, s, 0, 10)
    with pytest.raises(OscarError):
        make([64], group=64)


def test_rotated_rows_are_those_of_the_two_calls():
    cache, two = make([100, 40], spare=2), make([100, 40], spare=2)
    rot = RotaryEmbedding(base=1e6, rotary_dim=96)
    k, v = tokens(140, 2, 5)
    q = torch.randn(140, 8, 128, device="cuda").bfloat16()
    for c in (cache, two):
        c.reserve([c.alloc(), c.alloc()], [100, 40])
    got = cache.append_rotated(0, rot, k, v, q)
    at = torch.cat((torch.arange(100), torch.arange(40))).cuda()
    q2, k2 = rot.apply(at, q, k)
    two.append(0, k2, v)
    assert torch.equal(got, q2)
    for s, n in ((0, 100), (1, 40)):
        for x, y in zip(cache.read(0, s, 0, n, dtype=torch.float32), two.read(0, s, 0, n, dtype=torch.float32)):
            assert torch.equal(x, y)
