"""Rotated appends whose turned queries would be written over rows or positions that are still to be read are refused, and queries
turned in place within a fused projection are not."""
import pytest
import torch

from int2_rotated_kv_rotate_gb300 import OSCAR_FORMAT_BF16, OSCAR_FORMAT_INT4, KVCache, OscarError, RotaryEmbedding

pytestmark = pytest.mark.gpu
HQ, HKV, ROWS = 8, 2, 37


def make(fmt):
    c = KVCache(fmt=fmt, n_q_heads=HQ, n_kv_heads=HKV, group=32, max_requests=1, max_pages=1, max_pages_per_request=1)
    c.reserve([c.alloc()], [ROWS])
    return c


def projection():
    x = torch.randn(ROWS, (HQ + 2 * HKV) * 128, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    return x, [t.view(ROWS, -1, 128) for t in x.split([HQ * 128, HKV * 128, HKV * 128], 1)]


@pytest.mark.parametrize("fmt", [OSCAR_FORMAT_BF16, OSCAR_FORMAT_INT4])
def test_outputs_over_inputs_are_refused(fmt):
    rot = RotaryEmbedding(base=1e6)
    c = make(fmt)
    x, (q, k, v) = projection()
    before = x.clone()
    flat = x.view(-1)
    row = x.shape[1]

    def at(offset, rows=ROWS, heads=HQ):
        return flat.as_strided((rows, heads, 128), (row, 128, 1), offset)

    own = torch.randn(ROWS, HQ, 128, device="cuda").bfloat16()
    other = torch.randn(ROWS + 1, HQ, 128, device="cuda").bfloat16()
    positions = torch.arange(ROWS * 64, device="cuda")
    over = positions.view(torch.bfloat16).view(-1)[:2 * HQ * 128 * 4]
    for kw in (dict(q=own, q_out=at(2 * 128)),  # the last heads of k
               dict(q=own, q_out=at(HKV * 128 * 2)),  # k and v
               dict(q=q, q_out=at(128)),  # itself, a head further
               dict(q=other[1:], q_out=other[:-1]),  # a row further
               dict(q=k[:, :1], q_out=k[:, :1]),  # in place over the keys
               dict(q=v, q_out=v)):
        with pytest.raises(OscarError) as e:
            c.append_rotated(0, rot, k, v, kw["q"], q_out=kw["q_out"])
        assert e.value.status == 1 and "overlaps" in str(e.value)
    # over the positions
    rows_out = over[:ROWS * 128].view(ROWS, 1, 128)
    with pytest.raises(OscarError):
        c.append_rotated(0, rot, k, v, own[:, :1].contiguous(), q_out=rows_out, positions=positions[:ROWS])
    assert torch.equal(x, before)
    # nothing was appended over, and what is allowed works
    q2, k2 = rot.apply(torch.arange(ROWS).cuda(), q.contiguous(), k.contiguous())
    got = c.append_rotated(0, rot, k, v, q, q_out=q)
    assert got is q and torch.equal(q, q2) and torch.equal(x[:, HQ * 128:], before[:, HQ * 128:])
    want = make(fmt)
    want.append(0, k2, v.contiguous())
    n = c.layout.bf16_page_bytes * HKV if fmt == OSCAR_FORMAT_BF16 else 0
    if n:
        assert torch.equal(c.bf16_pages(0)[:, :, :, :ROWS], want.bf16_pages(0)[:, :, :, :ROWS])
    else:
        for a, b in zip(c.read(0, 0, 0, ROWS), want.read(0, 0, 0, ROWS)):
            assert torch.equal(a, b)


def test_outputs_between_the_inputs_rows():
    """Gaps of one buffer: q' beside k and v in the same rows, and heads before rows."""
    rot = RotaryEmbedding(base=1e6)
    c = make(OSCAR_FORMAT_BF16)
    room = torch.zeros(ROWS, 2 * HQ + 2 * HKV, 128, device="cuda").bfloat16()
    q, out, k, v = room[:, 0:2 * HQ:2], room[:, 1:2 * HQ:2], room[:, 2 * HQ:2 * HQ + HKV], room[:, 2 * HQ + HKV:]
    room[:, 0:2 * HQ:2] = torch.randn(ROWS, HQ, 128, device="cuda").bfloat16()
    room[:, 2 * HQ:] = torch.randn(ROWS, 2 * HKV, 128, device="cuda").bfloat16()
    q2, k2 = rot.apply(torch.arange(ROWS).cuda(), q, k)
    c.append_rotated(0, rot, k, v, q, q_out=out)
    assert torch.equal(out, q2)
    pages = c.bf16_pages(0)[0, :, :, :ROWS].permute(2, 0, 1, 3)
    assert torch.equal(pages[:, :, 0], k2) and torch.equal(pages[:, :, 1], v)
    assert c.status() == (0, 0)
