"""Plans with OSCAR_PLAN_SHARED_PREFIX on the BF16 cache: pages that requests share are attended
once for all of them; against fp64 attention over each request's own tokens.

Tolerance on the fp32 output, relative to sum p |v|: a score is at worst 128 truncating adds
of its products, 2^-16 A with A = sum |q_i k_i| / sqrt(d), so a probability is within
2^-15 max A; p is held in 16 bits or more (2^-17); the value sums add 16 tokens a step in
fp32, hi and lo apart: L / 8 truncating adds of 2^-23; 2^-20 for exponentials and the merge."""
import numpy as np
import pytest
import torch

from int2_rotated_kv_rotate_gb300 import KVCache, OSCAR_PLAN_SHARED_PREFIX, workloads as wl
from int2_rotated_kv_rotate_gb300 import _native as N

from helpers import compare_decode

pytestmark = pytest.mark.gpu

SEED = 515
SHARED = OSCAR_PLAN_SHARED_PREFIX | N.OSCAR_PLAN_SHARED_ALWAYS  # the small cases here would go without


def tokens(hkv, stream, n):
    w = wl.scaled(wl.WORKLOADS["tiny"], name="shared", n_kv_heads=hkv, lognormal_sigma=0.5)
    return wl.gen_kv(w, SEED, 0, stream, 0, n, device="cuda")


class Batch:
    """A cache of requests whose prefixes form a forest: node = (parent, pages, tails...)."""

    def __init__(self, hkv, gqa, max_requests, max_pages, per):
        self.hkv, self.hq = hkv, hkv * gqa
        self.cache = KVCache(fmt=N.OSCAR_FORMAT_BF16, n_q_heads=self.hq, n_kv_heads=hkv, n_layers=1,
                             max_requests=max_requests, max_pages=max_pages, max_pages_per_request=per)
        self.kv = {}  # slot -> (K, V)
        self.stream = 0

    def append(self, slot, n):
        self.stream += 1
        k, v = tokens(self.hkv, self.stream, n)
        self.cache.reserve([slot], [n])
        self.cache.append(0, k, v)
        self.cache.commit()
        old = self.kv.get(slot)
        self.kv[slot] = (k, v) if old is None else (torch.cat((old[0], k)), torch.cat((old[1], v)))

    def new(self, n=0, parent=None, pages=0):
        slot = self.cache.alloc()
        if parent is not None:
            self.cache.share_prefix(slot, parent, 64 * pages)
            self.kv[slot] = (self.kv[parent][0][:64 * pages], self.kv[parent][1][:64 * pages])
        else:
            self.kv[slot] = tokens(self.hkv, 0, 0)
        if n:
            self.append(slot, n)
        return slot

    def reference(self, slot, q):
        """fp64 (out [hq, 128], tolerance)."""
        K, V = self.kv[slot]
        L, G = K.shape[0], self.hq // self.hkv
        if L == 0:
            return torch.zeros(self.hq, 128, dtype=torch.float64), torch.zeros(self.hq, 128, dtype=torch.float64)
        outs, tols = [], []
        for h in range(self.hkv):
            k, v, qq = K[:, h].double(), V[:, h].double(), q[h * G:(h + 1) * G].double()
            p = torch.softmax(qq @ k.T / np.sqrt(128.0), -1)
            A = float((qq.abs() @ k.abs().T).max()) / np.sqrt(128.0)
            outs.append(p @ v)
            tols.append((p @ v.abs()) * (2.0**-15 * A + 2.0**-17 + L / 8 * 2.0**-23 + 2.0**-20))
        return torch.cat(outs).cpu(), torch.cat(tols).cpu()

    def check(self, slots, seed=1, msp=0, flags=SHARED, q=None, label=""):
        n = len(slots)
        if q is None:
            q = torch.randn(n, self.hq, 128, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()
        self.cache.plan(slots, max_split_pages=msp, flags=flags)
        out32 = torch.full((n, self.hq, 128), float("nan"), device="cuda")
        out = self.cache.decode(0, q, out_f32=out32)
        launches = N.oscar_last_launch_count()
        torch.cuda.synchronize()
        assert self.cache.status() == (0, 0), label
        for i, s in enumerate(slots):
            want, tol = self.reference(s, q[i])
            d = (out32[i].cpu().double() - want).abs()
            assert (d <= tol).all(), f"{label} request {i}: {float((d - tol).max()):.3e} over the tolerance"
            compare_decode(out32[i], out[i], want.numpy(), f"{label} request {i}")
        return out32, launches


@pytest.mark.parametrize("gqa", [4, 8])
@pytest.mark.parametrize("members,pages", [(2, 1), (2, 3), (3, 40), (16, 7), (17, 5), (33, 2), (40, 9), (65, 4), (100, 1)])
def test_one_group(gqa, members, pages):
    """Row counts around a block's 128 and an item's 256, with tails of nothing, one token, a
    page's edge and more."""
    b = Batch(2, gqa, members, pages + 3 * members + 8, pages + 8)
    first = b.new(64 * pages)
    slots = [first] + [b.new(parent=first, pages=pages) for _ in range(members - 1)]
    for i, s in enumerate(slots):
        tail = [0, 1, 63, 64, 65, 130][i % 6]
        if tail:
            b.append(s, tail)
    shared, launches = b.check(slots, label=f"{gqa} x {members} x {pages}")
    items, attended = b.cache.shared_info()
    assert launches == 2 and attended == pages and items > 0
    plain, launches = b.check(slots, flags=0, label="without the flag")
    assert launches == 1 and b.cache.shared_info() == (0, 0)
    b.check(slots[::-1], msp=1, label="other order, short private items")


def test_forest_of_prefixes():
    """A prefix under longer ones, requests that part ways inside, one that ends inside it, one
    on its own, an empty one; several of one plan in any order."""
    b = Batch(2, 4, 16, 200, 64)
    root = b.new(64 * 12)
    kids = [b.new(64 * 9, root, 12), b.new(64 * 4 + 5, root, 12), b.new(30, root, 7)]
    grand = [b.new(100, kids[0], 21), b.new(64, kids[0], 21), b.new(1, kids[0], 20), b.new(200, kids[0], 15)]
    short = b.new(0, root, 3)
    alone, empty = b.new(500), b.new()
    other = b.new(64 * 5)
    pair = [b.new(11, other, 5), b.new(0, other, 5)]
    every = [root, *kids, *grand, short, alone, empty, other, *pair]
    b.check(every, label="all")
    assert b.cache.shared_info()[1] > 12
    g = torch.Generator().manual_seed(4)
    for k in range(4):
        pick = [every[i] for i in torch.randperm(len(every), generator=g).tolist()[:5 + 2 * k]]
        b.check(pick, seed=k, label=f"subset {k}")
    b.check([alone], label="one request")
    assert b.cache.shared_info() == (0, 0)
    b.check([alone, empty], label="nothing shared")
    assert b.cache.shared_info() == (0, 0)


def test_long_prefix_and_many_heads():
    b = Batch(8, 4, 8, 420, 320)
    first = b.new(64 * 300)
    slots = [first] + [b.new(20 * i + 1, first, 300) for i in range(1, 8)]
    b.check(slots, label="long")
    items, pages = b.cache.shared_info()
    assert pages == 300 and items <= 152


@pytest.mark.parametrize("gqa,members,pages", [(4, 2, 9), (8, 17, 4)])
def test_more_items_than_multiprocessors(gqa, members, pages):
    """Every CTA of the shared launch takes several items, of one row block and of two, with even
    and odd numbers of pages (its warps pass barriers of one item to the next)."""
    groups, hkv = 41, 8
    b = Batch(hkv, gqa, groups * members, groups * (pages + 2) + groups * members, pages + 4)
    slots = []
    for g in range(groups):
        first = b.new(64 * (pages - g % 3))
        slots += [first] + [b.new(1 + (7 * i) % 50 if i % 2 else 0, first, pages - g % 3) for i in range(members - 1)]
    b.check(slots, label="many")
    items, shared = b.cache.shared_info()
    assert items > 2 * 152 and shared == sum(pages - g % 3 for g in range(groups))


def test_sharing_only_where_it_pays():
    """A short prefix goes without the shared launch unless told otherwise, a long one has it; a
    decode captured under the first is right under the second."""
    b = Batch(8, 4, 16, 300, 80)
    short = b.new(64 * 4)
    few = [short, b.new(9, short, 4)]
    q = torch.randn(16, b.hq, 128, device="cuda").bfloat16()
    _, launches = b.check(few, flags=OSCAR_PLAN_SHARED_PREFIX, label="short")
    assert launches == 1 and b.cache.shared_info() == (0, 0)
    _, launches = b.check(few, label="short, always")
    assert launches == 2 and b.cache.shared_info()[1] == 4
    first = b.new(64 * 64)
    many = [first] + [b.new(5 * i, first, 64) for i in range(1, 12)]
    _, launches = b.check(many, flags=OSCAR_PLAN_SHARED_PREFIX, label="long")
    assert launches == 2 and b.cache.shared_info()[1] == 64
    b.cache.plan(few, flags=OSCAR_PLAN_SHARED_PREFIX)
    out, out32 = torch.empty_like(q), torch.empty(q.shape, device="cuda")
    call = lambda: N.oscar_bf16_decode_attention(b.cache.handle, 0, q, out, b.cache.workspace, out32)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    b.cache.plan(many, flags=OSCAR_PLAN_SHARED_PREFIX)
    graph.replay()
    torch.cuda.synchronize()
    for i, s in enumerate(many):
        want, tol = b.reference(s, q[i])
        assert ((out32[i].cpu().double() - want).abs() <= tol).all(), f"request {i}"


def test_peaked_scores_move_the_reference():
    """Scores that grow along the prefix by far more than the lazy reference allows, and fall."""
    b = Batch(1, 4, 3, 60, 20)
    first = b.new(64 * 16)
    slots = [first, b.new(3, first, 16), b.new(90, first, 16)]
    K = b.kv[first][0]
    grow = torch.linspace(0.01, 3.0, 64 * 16, device="cuda")
    grow[512:] = grow[512:].flip(0)
    scaled = (K.float() * grow[:, None, None]).bfloat16()
    pages = b.cache.bf16_pages(0)
    for i, p in enumerate(b.cache.pages(first)[:16]):
        pages[p, 0, 0] = scaled[64 * i:64 * (i + 1), 0]
    for s in slots:
        k, v = b.kv[s]
        b.kv[s] = (torch.cat((scaled, k[1024:])), v)
    for seed in range(3):
        b.check(slots, seed=seed, label="peaked")


def test_infinite_keys_in_the_prefix():
    b = Batch(1, 4, 2, 20, 8)
    first = b.new(64 * 4)
    slots = [first, b.new(10, first, 4)]
    pages = b.cache.bf16_pages(0)
    q = torch.randn(2, 4, 128, device="cuda").bfloat16()
    q[..., 0] = 1.0
    ids = b.cache.pages(first)
    pages[ids[0], 0, 0, :, 0] = float("-inf")  # the first page has no weight at all
    pages[ids[2], 0, 0, 7, 0] = float("-inf")
    for s in slots:
        K = b.kv[s][0].clone()
        K[:64, 0, 0] = float("-inf")
        K[128 + 7, 0, 0] = float("-inf")
        keep = torch.isfinite(K[:, 0, 0])
        b.kv[s] = (K[keep], b.kv[s][1][keep])
    b.check(slots, q=q, label="part")
    for p in ids:
        pages[p, 0, 0, :, 0] = float("-inf")
    b.kv[slots[1]] = tuple(x[-10:] for x in b.kv[slots[1]])
    b.kv[first] = tuple(x[:0] for x in b.kv[first])
    b.check(slots, q=q, label="all of it")


def test_appends_beside_the_prefix_and_replays():
    """Steps planned while their tokens are reserved, and one captured decode replayed under later
    plans: longer, with other members, and without anything shared."""
    b = Batch(2, 8, 6, 120, 30)
    first = b.new(64 * 10)
    slots = [first] + [b.new(5 + i, first, 10) for i in range(3)]
    alone = b.new(70)
    for step in range(3):
        n = len(slots)
        k, v = tokens(2, 900 + step, n)
        q = torch.randn(n, b.hq, 128, device="cuda").bfloat16()
        b.cache.reserve(slots, [1] * n)
        b.cache.plan(slots, flags=SHARED)
        b.cache.append(0, k, v)
        out32 = torch.empty(n, b.hq, 128, device="cuda")
        out = b.cache.decode(0, q, out_f32=out32)
        b.cache.commit()
        for i, s in enumerate(slots):
            b.kv[s] = (torch.cat((b.kv[s][0], k[i:i + 1])), torch.cat((b.kv[s][1], v[i:i + 1])))
            want, tol = b.reference(s, q[i])
            assert ((out32[i].cpu().double() - want).abs() <= tol).all(), f"step {step} request {i}"
            compare_decode(out32[i], out[i], want.numpy())
    q = torch.randn(4, b.hq, 128, device="cuda").bfloat16()
    out, out32 = torch.empty_like(q), torch.empty(q.shape, device="cuda")
    b.cache.plan(slots, flags=SHARED)
    b.cache.decode(0, q, out=out, out_f32=out32)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.cache.decode(0, q, out=out, out_f32=out32)
    b.append(slots[2], 300)
    for pick, flags in ((slots, SHARED), ([alone, slots[1], slots[3], slots[2]], SHARED), ([alone, slots[0]], SHARED),
                        (slots, 0)):
        b.cache.plan(pick, flags=flags)
        out32.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for i, s in enumerate(pick):
            want, tol = b.reference(s, q[i])
            assert ((out32[i].cpu().double() - want).abs() <= tol).all(), f"replay {len(pick)} {flags} request {i}"
    assert b.cache.status() == (0, 0)


def test_sharing_survives_an_eviction():
    b = Batch(1, 4, 4, 60, 16)
    first = b.new(64 * 8)
    slots = [first] + [b.new(40, first, 8) for _ in range(3)]
    w = b.cache.new_weights()
    w.uniform_(generator=torch.Generator(device="cuda").manual_seed(1))
    b.cache.evict_begin([slots[1]], [200], n_sink=4, n_recent=32)
    _, kept = b.cache.evict(0, w)
    b.cache.evict_commit()
    t = kept[slots[1], 0, :200].long()
    b.kv[slots[1]] = tuple(x[t] for x in b.kv[slots[1]])
    b.check(slots, label="after")
    assert b.cache.shared_info()[1] == 8  # the other three still share


def test_a_bad_page_is_flagged_and_skipped():
    b = Batch(1, 4, 2, 20, 8)
    first = b.new(64 * 4)
    slots = [first, b.new(5, first, 4)]
    b.cache.plan(slots, flags=SHARED)
    table = b.cache.mem[b.cache.layout.page_table:b.cache.layout.page_table + 4 * 2 * 8].view(torch.int32).view(2, 8)
    keep = table.clone()
    table[:, 2] = 1 << 20
    q = torch.randn(2, 4, 128, device="cuda").bfloat16()
    out = b.cache.decode(0, q)
    st, flags = b.cache.status()
    assert st == 4 and flags == N.OSCAR_FLAG_BAD_PAGE and torch.isfinite(out.float()).all()
    table.copy_(keep)
    b.check(slots, label="mended")


def test_more_runs_than_the_plan_has_room_for():
    """A plan whose runs would fill the partial slots goes without some or all of the sharing."""
    b = Batch(1, 4, 96, 400, 100)
    first = b.new(64 * 90)
    slots = [first]
    for i in range(95):  # every request leaves the prefix one page further on
        slots.append(b.new(1 + i % 40, first, 90 - i % 85))
    b.check(slots, label="comb")
    assert b.cache.shared_info()[1] > 0
    b.check(slots, msp=1, label="comb, one page an item")


def test_refusals():
    b = Batch(1, 4, 2, 20, 8)
    first = b.new(64 * 4)
    slots = [first, b.new(5, first, 4)]
    for flags in (0x10, N.OSCAR_PLAN_SHARED_ALWAYS):
        with pytest.raises(N.OscarError) as e:
            b.cache.plan(slots, flags=flags)
        assert e.value.status == 1
    with pytest.raises(N.OscarError) as e:
        b.cache.plan([slots[0], slots[0]], flags=SHARED)
    assert e.value.status == 1
    b.cache.plan(slots, flags=SHARED)
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(N.OscarError) as e:
        b.cache.decode_weights(0, q, b.cache.new_weights())
    assert e.value.status == 7
    int2 = KVCache(n_q_heads=4, n_kv_heads=1, max_pages=4, max_pages_per_request=4)
    with pytest.raises(N.OscarError) as e:
        int2.plan([int2.alloc()], flags=SHARED)
    assert e.value.status == 1
