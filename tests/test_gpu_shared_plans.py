"""Shared-prefix plans whose work items are the odd ones: one page, short runs under which longer
ones part ways.  Against fp64 attention, to the tolerance that test_gpu_shared derives."""
import pytest
import torch

from int2_rotated_kv_rotate_gb300 import OSCAR_PLAN_SHARED_PREFIX

from test_gpu_shared import SHARED, Batch

pytestmark = pytest.mark.gpu


def same_again(b, n):
    """Which warp is ahead of which differs from launch to launch; the outputs do not."""
    q = torch.randn(n, b.hq, 128, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda").bfloat16()
    first = b.cache.decode(0, q)
    for _ in range(30):
        assert torch.equal(first, b.cache.decode(0, q))
    assert b.cache.status() == (0, 0)


@pytest.mark.parametrize("gqa", [4, 8])
def test_many_items_of_one_page(gqa):
    """Every CTA of the shared launch takes several items of one page, whose odd pages are none."""
    groups, members, hkv = 60, 5, 8
    b = Batch(hkv, gqa, groups * members, groups * (1 + members), 4)
    slots = []
    for g in range(groups):
        first = b.new(64)
        slots += [first] + [b.new((i * 13 + g) % 40, first, 1) for i in range(1, members)]
    b.check(slots, flags=OSCAR_PLAN_SHARED_PREFIX | SHARED, label="one page each")
    items, pages = b.cache.shared_info()
    assert items == groups * hkv > 3 * 152 and pages == groups
    same_again(b, len(slots))


@pytest.mark.parametrize("seed", range(4))
def test_items_of_one_page_between_longer_ones(seed):
    """Runs of 1 to 70 pages in any order: one-page items alone, as the end of a run, and in rows
    of several a CTA, of one row block and of two."""
    groups, hkv = 48, 8
    g = torch.Generator().manual_seed(seed)
    pick = lambda values: values[int(torch.randint(len(values), (1,), generator=g))]  # noqa: E731
    b = Batch(hkv, 4, groups * 40, groups * 120, 80)
    slots = []
    for k in range(groups):
        pages, members = pick([1, 1, 1, 2, 3, 5, 17, 33, 70]), pick([2, 2, 3, 5, 9, 40] if k % 8 == 0 else [2, 3, 5])
        first = b.new(64 * pages)
        slots += [first] + [b.new(pick([0, 0, 1, 30]), first, pages) for _ in range(members - 1)]
    order = torch.randperm(len(slots), generator=g).tolist()
    b.check([slots[i] for i in order], seed=seed, label="mixed")
    assert b.cache.shared_info()[0] > 2 * 152
    same_again(b, len(slots))


@pytest.mark.parametrize("common", [1, 2])
def test_long_runs_under_a_short_one(common):
    """Two pairs of requests on 512 pages of their own behind one or two common pages, which by
    themselves would save too little: the pairs' pages are attended once for each pair."""
    b = Batch(8, 4, 4, 2 * 512 + common + 8, 520)
    first = b.new(64 * common)
    other = b.new(0, first, common)
    b.append(first, 64 * 512)
    b.append(other, 64 * 512)
    slots = [first, other, b.new(7, first, 512 + common), b.new(70, other, 512 + common)]
    _, launches = b.check(slots, flags=OSCAR_PLAN_SHARED_PREFIX, label="pairs")
    items, pages = b.cache.shared_info()
    assert launches == 2 and items > 0 and 2 * 512 <= pages <= 2 * (512 + common)


@pytest.mark.parametrize("members,pages,tail,shares", [
    (8, 8, 40, False), (4, 32, 40, False), (2, 128, 40, False), (4, 64, 40, True), (32, 8, 40, False), (8, 64, 40, True),
    (32, 32, 40, True), (5, 96, 2000, False), (16, 4, 500, False), (16, 200, 2000, True)])
def test_plans_share_where_it_was_measured_to_pay(members, pages, tail, shares):
    b = Batch(8, 4, members, pages + members * (2 + tail // 64), pages + 2 + tail // 64)
    first = b.cache.alloc()
    b.cache.reserve([first], [64 * pages])
    b.cache.commit()
    slots = [first] + [b.cache.alloc() for _ in range(members - 1)]
    for s in slots[1:]:
        b.cache.share_prefix(s, first, 64 * pages)
    b.cache.reserve(slots, [tail] * members)
    b.cache.commit()
    b.cache.plan(slots, flags=OSCAR_PLAN_SHARED_PREFIX)
    assert (b.cache.shared_info()[0] > 0) == shares
