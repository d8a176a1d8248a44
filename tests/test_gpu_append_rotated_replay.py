"""A rotated append captured under a small reservation and replayed under larger ones: every CTA of the captured grid takes several
items, with a table of sines for each."""
import pytest
import torch

from int2_rotated_kv_rotate_gb300 import OSCAR_FORMAT_BF16, OSCAR_FORMAT_INT4, KVCache, RotaryEmbedding

pytestmark = pytest.mark.gpu
HQ, HKV, SLOTS, ROWS = 32, 4, 5, 700


def make(fmt):
    c = KVCache(fmt=fmt, n_q_heads=HQ, n_kv_heads=HKV, group=32, max_requests=SLOTS, max_pages=64, max_pages_per_request=40)
    for _ in range(SLOTS):
        c.alloc()
    return c


def held(c):
    if c.fmt == OSCAR_FORMAT_BF16:
        out = []
        for s in range(SLOTS):
            n, ids = c.info(s)[0], c.pages(s)
            if n:  # [pages, heads, K|V, 64, 128] as tokens
                out.append(c.bf16_pages(0)[torch.tensor(ids, device="cuda")].permute(0, 3, 1, 2, 4).flatten(0, 1)[:n].flatten())
        return torch.cat(out)
    return torch.cat([torch.stack(c.read(0, s, 0, c.info(s)[0], dtype=torch.float32)).flatten() for s in range(SLOTS) if c.info(s)[0]])


@pytest.mark.parametrize("fmt", [OSCAR_FORMAT_BF16, OSCAR_FORMAT_INT4])
@pytest.mark.parametrize("R,interleaved", [(128, False), (64, True), (18, False)])
@pytest.mark.parametrize("given", [False, True])
def test_more_items_than_the_captured_grid(fmt, R, interleaved, given):
    rot = RotaryEmbedding(base=1e6, rotary_dim=R, interleaved=interleaved)
    g = torch.Generator(device="cuda").manual_seed(R)
    q = torch.randn(ROWS, HQ, 128, generator=g, device="cuda").bfloat16()
    k, v = (torch.randn(ROWS, HKV, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    out = torch.zeros_like(q)
    places = torch.zeros(ROWS, dtype=torch.int64, device="cuda")
    a, b = make(fmt), make(fmt)

    def positions(c, slots, counts):
        p = torch.cat([torch.arange(c.info(s)[0], c.info(s)[0] + n) for s, n in zip(slots, counts)])
        return (p * 3 + 1000 if given else p).cuda()

    graph = None
    for slots, counts in (([0], [3]), ([1, 2, 0], [1, 40, 300]), ([4, 3, 0, 1, 2], [17, 1, 500, 64, 5]), ([3], [1]), ([2, 0], [100, 433])):
        n = sum(counts)
        at = positions(a, slots, counts)
        places[:n] = at
        for c in (a, b):
            c.reserve(slots, counts)
        out.zero_()
        if graph is None:
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                a.append_rotated(0, rot, k[:n], v[:n], q[:n], positions=places[:n] if given else None, q_out=out[:n])
        graph.replay()
        torch.cuda.synchronize()
        q2, k2 = rot.apply(at, q[:n], k[:n])
        b.append(0, k2, v[:n])
        for c in (a, b):
            c.commit()
        assert torch.equal(out[:n], q2) and bool((out[n:] == 0).all())
        assert torch.equal(held(a), held(b))
    assert a.status() == (0, 0)


def test_plain_4_bit_appends_replayed():
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(ROWS, HKV, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    a, b = make(OSCAR_FORMAT_INT4), make(OSCAR_FORMAT_INT4)
    graph = None
    for slots, counts in (([0], [40]), ([1, 2, 0], [1, 40, 300]), ([4, 3, 0, 1, 2], [17, 1, 500, 64, 5])):
        n = sum(counts)
        for c in (a, b):
            c.reserve(slots, counts)
        if graph is None:
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                a.append(0, k[:n], v[:n])
        graph.replay()
        b.append(0, k[:n], v[:n])
        for c in (a, b):
            c.commit()
        assert torch.equal(held(a), held(b))
    assert a.status() == (0, 0)
