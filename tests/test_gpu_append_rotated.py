"""Appends with rotary positions: the pages and the turned queries are, bit for bit, those of
RotaryEmbedding.apply and an append after it, and within a rounding of the definition in 64 bits."""
import pytest
import torch

from int2_rotated_kv_rotate_gb300 import (OSCAR_FORMAT_BF16, OSCAR_FORMAT_INT2, OSCAR_FORMAT_INT4, KVCache, OscarError,
                                          RotaryEmbedding)
from int2_rotated_kv_rotate_gb300 import _native as N

pytestmark = pytest.mark.gpu


def make(fmt=OSCAR_FORMAT_BF16, hkv=2, gqa=4, pages=80, requests=8, layers=1):
    c = KVCache(fmt=fmt, n_q_heads=hkv * gqa, n_kv_heads=hkv, group=32, n_layers=layers, max_requests=requests, max_pages=pages,
                max_pages_per_request=pages)
    if fmt == OSCAR_FORMAT_BF16:
        for layer in range(layers):
            c.bf16_pages(layer).zero_()
    return c


def held(c, layer=0):
    """Everything that the pages hold."""
    if c.fmt == OSCAR_FORMAT_BF16:
        return c.bf16_pages(layer)
    return torch.cat([torch.stack(c.read(layer, s, 0, c.info(s)[0], dtype=torch.float32)).flatten()
                      for s in range(c.cfg.max_requests - c.stats()[1])])


def grow(c, slots, counts):
    """Tokens held before, whatever they are."""
    c.reserve(slots, counts)
    z = torch.zeros(sum(counts), c.cfg.n_kv_heads, 128, device="cuda").bfloat16()
    c.append(0, z, z)
    c.commit()


def fused(rows, hq, hkv, seed=1, pad=0):
    """q, k, v as slices of a projection's rows (pad: channels in front, off 16 bytes)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, pad + (hq + 2 * hkv) * 128, generator=g, device="cuda").bfloat16()[:, pad:]
    return [t.view(rows, -1, 128) for t in x.split([hq * 128, hkv * 128, hkv * 128], 1)]


@pytest.mark.parametrize("fmt", [OSCAR_FORMAT_BF16, OSCAR_FORMAT_INT4])
@pytest.mark.parametrize("R,interleaved", [(128, False), (128, True), (96, False), (64, True), (48, False), (18, False), (18, True),
                                           (2, False), (2, True), (126, False)])
@pytest.mark.parametrize("before,new,hkv,gqa", [((0,), (1,), 1, 4), ((5, 63, 64, 100), (1, 1, 1, 1), 2, 4),
                                                ((0, 17, 130), (300, 1, 65), 3, 8)])
def test_equals_the_two_calls(fmt, R, interleaved, before, new, hkv, gqa):
    hq, rows = hkv * gqa, sum(new)
    rot = RotaryEmbedding(base=1e6, rotary_dim=R, interleaved=interleaved)
    q, k, v = fused(rows, hq, hkv)
    pair = []
    for _ in range(2):
        c = make(fmt, hkv, gqa)
        slots = [c.alloc() for _ in before]
        if any(before):
            grow(c, [s for s, b in zip(slots, before) if b], [b for b in before if b])
        c.reserve(slots, list(new))
        pair.append(c)
    at = torch.cat([torch.arange(b, b + n) for b, n in zip(before, new)]).cuda()
    got = pair[0].append_rotated(0, rot, k, v, q)
    q2, k2 = rot.apply(at, q, k)
    pair[1].append(0, k2, v.contiguous())
    assert torch.equal(got, q2)
    for c in pair:
        c.commit()
    assert torch.equal(held(pair[0]), held(pair[1]))
    assert pair[0].status() == (0, 0)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("scaling", [None, dict(type="yarn", factor=4.0, original_context=32768)])
def test_positions_given(dtype, scaling):
    """Positions that are not the places (after an eviction), far ones among them; a layer each."""
    rot = RotaryEmbedding(base=5e5, scaling=scaling)
    q, k, v = fused(50, 8, 2)
    pos = (torch.randperm(50, generator=torch.Generator().manual_seed(1)) * 977 + (1 << 20 if dtype == torch.int32 else 1 << 40)).to(dtype).cuda()
    pos[3] = -5
    a, b = make(layers=2), make(layers=2)
    for c in (a, b):
        c.reserve([c.alloc()], [50])
    for layer in range(2):
        q1 = a.append_rotated(layer, rot, k + layer, v, q, positions=pos)
        q2, k2 = rot.apply(pos, q, k + layer)
        b.append(layer, k2, v.contiguous())
        assert torch.equal(q1, q2) and torch.equal(held(a, layer), held(b, layer))


def test_against_64_bits():
    """Turned values are off by half a step of bf16 (8 significant bits, so 2^-8 of the value) and by what
    fp32 sines and products are: 2^-8 + 2^-21 of the pair's norm."""
    rot = RotaryEmbedding(base=1e4)
    q, k, v = fused(70, 4, 1)
    c = make(hkv=1)
    c.reserve([c.alloc()], [70])
    got = c.append_rotated(0, rot, k, v, q)
    f = 1e4 ** (-torch.arange(64, dtype=torch.float64) / 64)
    ang = torch.arange(70, dtype=torch.float64)[:, None] * f
    cos, sin = ang.cos()[:, None].cuda(), ang.sin()[:, None].cuda()
    pages = c.bf16_pages(0)
    kk = torch.cat((pages[0, :, 0], pages[1, :, 0]), 1)[:, :70].transpose(0, 1)
    vv = torch.cat((pages[0, :, 1], pages[1, :, 1]), 1)[:, :70].transpose(0, 1)
    for x, y in ((q, got), (k, kk)):
        a, b = x.double()[..., :64], x.double()[..., 64:]
        want = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        norm = (a * a + b * b).sqrt().repeat(1, 1, 2)
        assert bool(((y.double() - want).abs() <= norm * (2.0 ** -8 + 2.0 ** -21)).all())
    assert torch.equal(vv, v)
    assert bool((pages[1, :, :, 6:] == 0).all())  # rows behind the last token stay


@pytest.mark.parametrize("R", [128, 18])
@pytest.mark.parametrize("pad", [0, 1])
def test_strides_alignment_and_in_place(R, pad):
    """Slices off 16 bytes, heads before rows, q turned in place, other outputs."""
    rot = RotaryEmbedding(base=1e6, rotary_dim=R)
    q, k, v = fused(37, 8, 2, pad=pad)
    at = torch.arange(37).cuda()
    q2, k2 = rot.apply(at, q.contiguous(), k.contiguous())
    want = make()
    want.reserve([want.alloc()], [37])
    want.append(0, k2, v.contiguous())
    kt, vt = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (k, v))  # [heads, rows] in memory
    qt = torch.empty(8, 37 * 3, 128, device="cuda").bfloat16()[:, ::3].transpose(0, 1)
    for kk, vv, kw in ((k, v, {}), (kt, vt, {}), (k, vt, dict(q_out=qt)), (k, v, dict(q_out=None))):
        c = make()
        c.reserve([c.alloc()], [37])
        got = c.append_rotated(0, rot, kk, vv, q, **kw)
        assert torch.equal(got, q2) and torch.equal(held(c), held(want))
    c = make()
    c.reserve([c.alloc()], [37])
    mine = q.clone() if not pad else q
    version = mine._version
    assert c.append_rotated(0, rot, k, v, mine, q_out=mine) is mine
    assert torch.equal(mine, q2) and mine._version > version
    # without queries
    c = make()
    c.reserve([c.alloc()], [37])
    assert c.append_rotated(0, rot, k, v) is None
    assert torch.equal(held(c), held(want))


def test_no_rows_and_broadcast_rows():
    rot = RotaryEmbedding()
    c = make()
    s = c.alloc()
    c.reserve([s], [0])
    e = torch.empty(0, 2, 128, device="cuda").bfloat16()
    assert c.append_rotated(0, rot, e, e, torch.empty(0, 8, 128, device="cuda").bfloat16()).shape == (0, 8, 128)
    c.commit()
    c.reserve([s], [9])
    k = torch.randn(1, 2, 128, device="cuda").bfloat16().expand(9, 2, 128)  # row stride 0
    c.append_rotated(0, rot, k, k)
    assert torch.equal(c.bf16_pages(0)[0, :, 1, :9], k.transpose(0, 1))
    assert c.status() == (0, 0)


def test_streams_and_a_graph():
    rot = RotaryEmbedding(base=1e6)
    q, k, v = fused(3, 8, 2)
    a, b = make(), make()
    for c in (a, b):
        grow(c, [c.alloc(), c.alloc(), c.alloc()], [10, 64, 200])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a.reserve([0, 1, 2], [1, 1, 1], stream=side)
    got = a.append_rotated(0, rot, k, v, q, stream=side.cuda_stream)
    side.synchronize()
    b.reserve([0, 1, 2], [1, 1, 1])
    want = b.append_rotated(0, rot, k, v, q)
    assert torch.equal(got, want) and torch.equal(held(a), held(b))
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.append_rotated(0, rot, k, v, q, q_out=out)
    b.commit()
    a.commit()
    # replayed under a later reservation with more items: places and pages are that one's
    for c in (a, b):
        c.reserve([2, 0, 1], [1, 1, 1])
    graph.replay()
    torch.cuda.synchronize()
    want = a.append_rotated(0, rot, k, v, q)
    assert torch.equal(out, want) and torch.equal(held(a), held(b))


def test_refusals():
    rot = RotaryEmbedding()
    q, k, v = fused(5, 8, 2)
    c = make()
    s = c.alloc()
    with pytest.raises((OscarError, ValueError)):
        c.append_rotated(0, rot, k, v, q)  # no reservation
    c.reserve([s], [5])
    bad = [dict(k_new=k[:4]), dict(v_new=v.float()), dict(q=q[:4]), dict(q=q.cpu()), dict(positions=torch.arange(4).cuda()),
           dict(positions=torch.arange(5)), dict(positions=torch.arange(5.0).cuda()), dict(q=None, q_out=q),
           dict(q_out=q[:, :4]), dict(q=q.detach().float().requires_grad_()), dict(q=q.detach().clone().requires_grad_()),
           dict(k_new=k.transpose(1, 2).contiguous().transpose(1, 2))]
    for kw in bad:
        args = dict(k_new=k, v_new=v, q=q)
        args.update(kw)
        with pytest.raises(ValueError):
            c.append_rotated(0, rot, args.pop("k_new"), args.pop("v_new"), args.pop("q"), **args)
    with pytest.raises(ValueError):
        c.append_rotated(0, RotaryEmbedding(head_dim=64), k, v, q)
    with pytest.raises(OscarError):
        c.append_rotated(1, rot, k, v, q)
    over = torch.empty(5, 1, 128, device="cuda").bfloat16().expand(5, 8, 128)
    with pytest.raises(OscarError):
        c.append_rotated(0, rot, k, v, q, q_out=over)
    with pytest.raises(OscarError):
        N.oscar_append_rotated(c.handle, 0, rot.steps, 130, 1.0, 0, None, None, None, k, v)
    with pytest.raises(OscarError):
        N.oscar_append_rotated(c.handle, 0, rot.steps, 128, 1.0, N.OSCAR_ROPE_TRANSPOSE, None, None, None, k, v)
    i2 = make(OSCAR_FORMAT_INT2)
    i2.reserve([i2.alloc()], [5])
    with pytest.raises(OscarError) as e:
        i2.append_rotated(0, rot, k, v, q)
    assert e.value.status == 7
    assert c.status() == (0, 0)
