"""Infinities and NaN among the values of small tiles, whose even and odd pages go to two blocks that are joined in their CTA
or, where the tile is cut, by the merge: every query that sees one has it in its output, in its channel alone, and no
other query has.

Tolerance of the finite channels: as several queries of a request have it (half a step of bf16, 2^-8, of each weight; the
fp32 sums and exponentials under 2^-9 at these scores), times the largest value."""
import math

import pytest
import torch

from int2_rotated_kv_rotate_gb300 import OSCAR_FORMAT_BF16, KVCache

pytestmark = pytest.mark.gpu
NEW = 5  # queries of a request, the last tokens


def filled(kv, gqa):
    n, hkv = kv[0][0].shape[:2]
    c = KVCache(fmt=OSCAR_FORMAT_BF16, n_q_heads=hkv * gqa, n_kv_heads=hkv, max_requests=len(kv), max_pages=len(kv) * (n // 64),
                max_pages_per_request=n // 64)
    slots = [c.alloc() for _ in kv]
    c.reserve(slots, [n] * len(kv))
    c.append(0, torch.cat([k for k, _ in kv]), torch.cat([v for _, v in kv]))
    c.commit()
    return c, slots


# (pages; page, token and channel of the value): the last page is odd in the list and its query rows differ in what they
# see of it; the first is even; in the pages between every query sees every token
PLACES = [(6, 5, 60, 100), (6, 5, 63, 127), (6, 5, 3, 0), (6, 4, 62, 99), (6, 0, 0, 64), (7, 6, 60, 100), (7, 5, 33, 5),
          (34, 33, 60, 100), (34, 33, 63, 127), (34, 32, 7, 31), (34, 1, 50, 70)]


@pytest.mark.parametrize("gqa", [4, 8])
@pytest.mark.parametrize("pages,page,token,channel", PLACES)
def test_values_of_either_block_reach_the_output(gqa, pages, page, token, channel):
    n, at = 64 * pages, 64 * page + token
    g = torch.Generator(device="cuda").manual_seed(at + channel)
    k, v = (torch.randn(n, 1, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(NEW, gqa, 128, generator=g, device="cuda").bfloat16()
    p = torch.arange(n - NEW, n, device="cuda")[:, None]
    hidden = torch.arange(n, device="cuda")[None] > p
    s = (torch.einsum("qhc,tc->hqt", q.double(), k[:, 0].double()) / math.sqrt(128.0)).masked_fill(hidden, -math.inf)
    for value in (math.inf, -math.inf, math.nan):
        w = v.clone()
        w[at, :, channel] = value
        c, slots = filled([(k, w)], gqa)
        c.plan_window(slots, [NEW])
        assert (c.window_info()[2] > 0) == (pages > 8)  # the long one is cut
        clean = w[:, 0].double()
        clean[at, channel] = 0
        ref = (torch.softmax(s, -1) @ clean).transpose(0, 1)
        odd = torch.zeros(NEW, gqa, 128, dtype=torch.bool, device="cuda")
        odd[~hidden[:, at], :, channel] = True
        for _ in range(20):
            o32 = torch.full(q.shape, 7.0, device="cuda")
            c.attend_window(0, q, out_f32=o32)
            assert torch.equal(~o32.isfinite(), odd)
            if math.isnan(value):
                assert bool(o32[odd].isnan().all())
            tol = (2.0 ** -8 + 2.0 ** -9) * float(clean.abs().max())
            assert float((o32.double() - ref)[~odd].abs().max()) <= tol
        assert c.status() == (0, 0)


def test_many_tiles_with_values_of_all_kinds():
    """As many small tiles as SMs: each joins its blocks while the others do."""
    n, requests, gqa = 6 * 64, torch.cuda.get_device_properties(0).multi_processor_count // 4, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    kv, odd = [], torch.zeros(requests * NEW, 4 * gqa, 128, dtype=torch.bool, device="cuda")
    for i in range(requests):
        k, v = (torch.randn(n, 4, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
        for h in range(4):
            token = n - 1 - (i + h) % 8  # some that every query sees, some of which only the last ones do
            v[token, h, (37 * i + h) % 128] = (math.inf, -math.inf, math.nan)[i % 3]
            odd[i * NEW + max(0, token - (n - NEW)):(i + 1) * NEW, h * gqa:(h + 1) * gqa, (37 * i + h) % 128] = True
        kv.append((k, v))
    c, slots = filled(kv, gqa)
    q = torch.randn(requests * NEW, 4 * gqa, 128, generator=g, device="cuda").bfloat16()
    c.plan_window(slots, [NEW] * requests)
    for _ in range(50):
        o32 = torch.full(q.shape, 7.0, device="cuda")
        c.attend_window(0, q, out_f32=o32)
        assert torch.equal(~o32.isfinite(), odd)
    assert c.status() == (0, 0)
