"""The operators on the paged caches where a request's pages lie past 4 GiB of the pool.

Tolerances, of the largest value: a score's sums have magnitude S = sum |q k| / sqrt(128) < 16 here,
which moves the output by 2 (2^-18 S + 2^-20) < 2^-12.  Weights of tiles are rounded to bf16 (2^-8);
weights times scales of 4-bit values to 11 bits of at most the group's range, twice the largest
value (2^-11)."""
import math

import pytest
import torch

from int2_rotated_kv_rotate_gb300 import OSCAR_FORMAT_BF16, OSCAR_FORMAT_INT4, KVCache, RotaryEmbedding

pytestmark = pytest.mark.gpu


def far_cache(fmt, page_bytes, tokens):
    """A cache whose second request's pages begin past 4 GiB; the first request holds what is before
    them, never written."""
    before = (1 << 32) // page_bytes + 5
    c = KVCache(fmt=fmt, n_q_heads=32, n_kv_heads=8, group=32, n_layers=1, max_requests=2, max_pages=before + tokens // 64 + 2,
                max_pages_per_request=before + 1)
    a, b = c.alloc(), c.alloc()
    for at in range(0, before, 8192):  # a reservation's items are limited
        c.reserve([a], [64 * min(8192, before - at)])
        c.commit()
    c.reserve([b], [tokens])
    assert min(c.pages(b)) * page_bytes > 1 << 32
    return c, b


def reference(q, k, v, see):
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for h in range(32):
        s = (q[:, h].double() @ k[:, h // 4].double().T / math.sqrt(128.0)).masked_fill(~see, -math.inf)
        out[:, h] = torch.softmax(s, -1) @ v[:, h // 4].double()
    return out


def test_rotated_append_and_window():
    n = 333
    rot = RotaryEmbedding(base=1e6)
    c, slot = far_cache(OSCAR_FORMAT_BF16, 8 * 32768, n)
    k, v = (torch.randn(n, 8, 128, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(n, 32, 128, device="cuda").bfloat16()
    qr = c.append_rotated(0, rot, k, v, q)
    want_q, kr = rot.apply(torch.arange(n).cuda(), q, k)
    assert torch.equal(qr, want_q)
    pages = c.bf16_pages(0)[torch.tensor(c.pages(slot)).cuda()]  # [pages, 8, K|V, 64, 128]
    held = pages.permute(2, 0, 3, 1, 4).reshape(2, -1, 8, 128)[:, :n]
    assert torch.equal(held[0], kr) and torch.equal(held[1], v)
    p, t = torch.arange(n, device="cuda")[:, None], torch.arange(n, device="cuda")[None]
    see = (t <= p) & ((t < 4) | (t > p - 100))
    for queries in (n, 1):
        c.plan_window([slot], [queries], n_sink=4, window=100)
        o32 = torch.empty(queries, 32, 128, device="cuda")
        c.attend_window(0, qr[n - queries:].contiguous(), out_f32=o32)
        ref = reference(qr[n - queries:], kr, v, see[n - queries:])
        assert float((o32.double() - ref).abs().max()) <= (2.0 ** -8 + 2.0 ** -10) * float(v.abs().max())
    assert c.status() == (0, 0)


def test_4_bit_rows():
    n = 333
    c, slot = far_cache(OSCAR_FORMAT_INT4, 8 * 2 * 64 * (64 + 16), n)
    k, v = (torch.randn(n, 8, 128, device="cuda").bfloat16() for _ in range(2))
    c.append(0, k, v)
    held = c.read(0, slot, 0, n, dtype=torch.float32)
    for x, y in zip((k, v), held):
        x = x.float().unflatten(-1, (4, 32))
        s = ((x.amax(-1, keepdim=True) - x.amin(-1, keepdim=True)) / 15).bfloat16().float()
        assert bool(((y.unflatten(-1, (4, 32)) - x).abs() <= s * (0.5 + 15 * 2.0 ** -8)).all())
    c.commit()
    c.plan([slot])
    q = torch.randn(1, 32, 128, device="cuda").bfloat16()
    o32 = torch.empty(1, 32, 128, device="cuda")
    c.decode(0, q, out_f32=o32)
    ref = reference(q, *held, torch.ones(1, n, dtype=torch.bool, device="cuda"))
    assert float((o32.double() - ref).abs().max()) <= (2 * 2.0 ** -12 + 2.0 ** -10) * float(held[1].abs().max())
    assert c.status() == (0, 0)
