"""Accumulated attention weights and eviction on the BF16 cache, against fp64 attention and a
selection written from the definition.

Tolerance of the weights: a score is 128 exact products added in fp32, at worst one
truncating addition each, 128 * 2^-23 = 2^-16 of A = sum |q_i k_i| / sqrt(d); numerator and
denominator of a probability so differ by at most 2^-15 max A relative, plus 2^-20 for the
exponentials and the scaling; the sum with the accumulated weight rounds once.  Kept
positions, kept weights and rows have to be equal bit for bit."""
import numpy as np
import pytest
import torch

from int2_rotated_kv_rotate_gb300 import KVCache, workloads as wl
from int2_rotated_kv_rotate_gb300 import _native as N

from helpers import compare_decode

pytestmark = pytest.mark.gpu

SEED = 4242


def make(hq, hkv, lens, layers=1, spare=0, max_requests=None, per=None):
    n = max_requests or len(lens)
    per = per or max(1, max(-(-L // 64) for L in lens))
    cache = KVCache(fmt=N.OSCAR_FORMAT_BF16, n_q_heads=hq, n_kv_heads=hkv, n_layers=layers, max_requests=n,
                    max_pages=max(1, sum(-(-L // 64) for L in lens) + spare), max_pages_per_request=per)
    return cache, [cache.alloc() for _ in lens]


def fill(cache, slots, lens, layers=1):
    """Seeded tokens appended to every slot; K and V [layer][request], [L, hkv, 128]."""
    w = wl.scaled(wl.WORKLOADS["tiny"], name="evict", n_kv_heads=cache.cfg.n_kv_heads, lognormal_sigma=0.5)
    kv = [[wl.gen_kv(w, SEED, la, i, 0, L, device="cuda") for i, L in enumerate(lens)] for la in range(layers)]
    cache.reserve(slots, lens)
    for la in range(layers):
        cache.append(la, torch.cat([k for k, _ in kv[la]]), torch.cat([v for _, v in kv[la]]))
    cache.commit()
    return kv


def queries(n, hq, seed):
    return torch.randn(n, hq, 128, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def attention(q, K, V):
    """fp64 of q [G, 128] over K, V [L, 128]: (out, p, largest sum |q k| / sqrt d)."""
    q, K, V = q.double(), K.double(), V.double()
    p = torch.softmax(q @ K.T / np.sqrt(128.0), -1)
    a = q.abs() @ K.abs().T
    return p @ V, p, float(a.max()) / np.sqrt(128.0) if a.numel() else 0.0


def check_weights(got, before, q, kv, hkv, label):
    """One request: got, before [hkv, stride]; q [hq, 128]; kv (K, V) [L, hkv, 128].  -> fp64 out."""
    K, V = kv
    L, G = K.shape[0], q.shape[0] // hkv
    outs = []
    for h in range(hkv):
        o, p, A = attention(q[h * G:(h + 1) * G], K[:, h], V[:, h])
        outs.append(o)
        want = before[h, :L].double() + p.sum(0)
        tol = p.sum(0) * (2.0**-15 * A + 2.0**-20) + 2.0**-24 * want.abs()
        assert ((got[h, :L].double() - want).abs() <= tol).all(), f"{label} head {h}: weights"
        assert torch.equal(got[h, L:], before[h, L:]), f"{label} head {h}: entries past the request changed"
    return torch.cat(outs)


@pytest.mark.parametrize("gqa", [4, 8])
@pytest.mark.parametrize("msp", [0, 1, 3])
def test_decode_weights(gqa, msp):
    hkv, lens = 2, [1, 63, 0, 64, 65, 1000, 2500]
    cache, slots = make(hkv * gqa, hkv, lens)
    kv = fill(cache, slots, lens)[0]
    n = len(lens)
    q = queries(n, hkv * gqa, 1)
    g = torch.Generator(device="cuda").manual_seed(2)
    before = torch.rand(cache.new_weights().shape, generator=g, device="cuda") * 3
    order = [5, 2, 0, 6, 1, 4, 3]  # the plan's order is not the slots'
    cache.plan([slots[i] for i in order], max_split_pages=msp)
    plain = torch.empty(n, hkv * gqa, 128, device="cuda")
    cache.decode(0, q, out_f32=plain)
    out32 = torch.empty_like(plain)
    after = torch.full_like(before, 7.0)
    out, w = cache.decode_weights(0, q, before, weights_out=after, out_f32=out32)
    assert w is after and N.oscar_last_launch_count() == 2
    assert torch.equal(out32, plain)  # the attention itself is the plain decode's
    for pos, i in enumerate(order):
        full = before[slots[i]].clone()
        full[:, lens[i]:] = 7.0
        ref = check_weights(after[slots[i]], torch.where(torch.arange(full.shape[1], device="cuda") < lens[i],
                                                         before[slots[i]], full), q[pos], kv[i], hkv, f"request {i}")
        if lens[i]:
            compare_decode(out32[pos], out[pos], ref.cpu().numpy(), f"request {i}")
    # in place, and from nothing
    inplace = before.clone()
    cache.decode_weights(0, q, inplace)
    zero = torch.full_like(before, -1.0)
    N.oscar_bf16_decode_weights(cache.handle, 0, q, out, None, zero, cache.weights_workspace)
    for i, L in enumerate(lens):
        assert torch.equal(inplace[slots[i], :, :L], after[slots[i], :, :L])
        assert torch.equal(inplace[slots[i], :, L:], before[slots[i], :, L:])
        if L:
            total = zero[slots[i], :, :L].double().sum(-1)  # the probabilities of a head add up to one
            assert ((total - gqa).abs() <= gqa * (L * 2.0**-24 + 2.0**-12)).all()
    assert cache.status() == (0, 0)


def test_decode_weights_with_masked_scores():
    """Keys of -inf take no weight; a request whose every score is -inf takes none at all."""
    hkv, lens = 1, [130, 70]
    cache, slots = make(4, hkv, lens)
    kv = fill(cache, slots, lens)[0]
    pages = cache.bf16_pages(0)
    q = queries(2, 4, 3)
    q[..., 0] = 1.0
    pages[cache.pages(slots[0])[0], 0, 0, 5:9, 0] = float("-inf")
    for p in cache.pages(slots[1]):
        pages[p, 0, 0, :, 0] = float("-inf")
    cache.plan(slots)
    out, w = cache.decode_weights(0, q, cache.new_weights())
    assert (w[0, 0, 5:9] == 0).all() and abs(float(w[0, 0].double().sum()) - 4) < 4 * 2.0**-12
    assert (w[1] == 0).all() and (out[1] == 0).all()
    assert torch.isfinite(out.float()).all() and torch.isfinite(w).all()


def select(w, L, keep, sink, recent):
    """Positions that stay, by the definition: w fp32 numpy [L]."""
    if keep >= L:
        return np.arange(L)
    s = min(sink, L)
    r = min(recent, L - s)
    protected = np.zeros(L, dtype=bool)
    protected[:s] = True
    protected[L - r:] = True
    value = np.where(np.isnan(w), -np.inf, w.astype(np.float64))
    nan_last = np.isnan(w)
    order = np.lexsort((np.arange(L), nan_last, -value, ~protected))
    return np.sort(order[:keep])


def draw_weights(kind, shape, g):
    u = torch.rand(shape, generator=g, device="cuda")
    if kind == "heavy":
        w = torch.exp(3 * torch.randn(shape, generator=g, device="cuda"))
        return torch.where(u < 0.2, torch.zeros_like(w), w)
    if kind == "zero":
        return torch.zeros(shape, device="cuda")
    if kind == "few":
        return torch.floor(u * 3)
    if kind == "near":  # neighbours in the last bits, across the digits of a key
        return (torch.floor(u * 5000).to(torch.int32) + 0x3F7FF000).view(torch.float32)
    special = torch.tensor([float("nan"), float("inf"), float("-inf"), -0.0, 0.0, 1e-45, -1e-45, 3.4e38, -3.4e38, 1.0,
                            -1.0], device="cuda")
    return special[(u * 11).long().clamp(max=10)]


def check_evicted(cache, i, slot, kv, pages, w, w_out, kept, keep, sink, recent, L, label):
    """One request of one layer; pages: its pages after the eviction.  -> kept positions per head."""
    hkv = cache.cfg.n_kv_heads
    n = min(keep, L)
    picks = []
    for h in range(hkv):
        want = select(w[slot, h, :L].cpu().numpy(), L, keep, sink, recent)
        idx = kept[slot, h, :n].cpu().numpy()
        assert np.array_equal(idx, want), f"{label} request {i} head {h}: positions"
        t = torch.from_numpy(want).cuda()
        assert torch.equal(w_out[slot, h, :n].view(torch.int32), w[slot, h][t].view(torch.int32)), label
        assert (w_out[slot, h, n:].view(torch.int32) == 0).all(), f"{label}: no zeros behind the kept weights"
        rows = pages[:, h].transpose(0, 1).reshape(2, -1, 128)[:, :n]
        assert torch.equal(rows[0].view(torch.int16), kv[0][:, h][t].view(torch.int16)), f"{label}: K rows"
        assert torch.equal(rows[1].view(torch.int16), kv[1][:, h][t].view(torch.int16)), f"{label}: V rows"
        picks.append(t)
    return picks


@pytest.mark.parametrize("kind", ["heavy", "zero", "few", "near", "special"])
def test_evict_against_the_definition(kind):
    lens = [1, 2, 64, 65, 0, 1500, 5000, 20000, 63]
    keeps = [1, 1, 63, 65, 3, 700, 129, 19999, 0]
    hkv, layers, sink, recent = 2, 2, 0, 0
    g = torch.Generator(device="cuda").manual_seed(11)
    cache, slots = make(8, hkv, lens, layers=layers, spare=400)
    kv = fill(cache, slots, lens, layers)
    free = cache.stats()[0]
    W = [draw_weights(kind, cache.new_weights().shape, g) for _ in range(layers)]
    cache.evict_begin(slots, keeps)
    moved = sum(-(-k // 64) for k, L in zip(keeps, lens) if k < L)
    assert cache.stats()[0] == free - moved
    outs = []
    for la in range(layers):
        pool = cache.bf16_pages(la)
        old = pool.clone()
        w_out, kept = cache.evict(la, W[la])
        assert kept.dtype == torch.int32
        for i, s in enumerate(slots):
            pages = pool[torch.tensor(cache.evict_pages(s), dtype=torch.long, device="cuda")]
            check_evicted(cache, i, s, kv[la][i], pages, W[la], w_out, kept, keeps[i], sink, recent, lens[i], kind)
            assert (kept[s, :, min(keeps[i], lens[i]):] == -1).all()
        new = {p for s, k, L in zip(slots, keeps, lens) if k < L for p in cache.evict_pages(s)}
        rest = torch.tensor([p for p in range(pool.shape[0]) if p not in new], device="cuda")
        assert torch.equal(pool[rest].view(torch.int16), old[rest].view(torch.int16))  # old pages stay until the commit
        outs.append((w_out, kept))
    cache.evict_commit()
    for s, k, L in zip(slots, keeps, lens):
        assert cache.info(s)[0] == min(k, L) and cache.info(s)[2] == -(-min(k, L) // 64)
    assert cache.stats()[0] == free + sum(-(-L // 64) - -(-k // 64) for k, L in zip(keeps, lens) if k < L)
    # the decode over what is left is the attention over each head's kept tokens
    q = queries(len(lens), 8, 5)
    cache.plan(slots)
    for la in range(layers):
        out32 = torch.empty(len(lens), 8, 128, device="cuda")
        out = cache.decode(la, q, out_f32=out32)
        for i, s in enumerate(slots):
            n = min(keeps[i], lens[i])
            ref = torch.zeros(8, 128, dtype=torch.float64, device="cuda")
            for h in range(hkv):
                t = outs[la][1][s, h, :n].long()
                if n:
                    ref[h * 4:h * 4 + 4] = attention(q[i, h * 4:h * 4 + 4], kv[la][i][0][:, h][t], kv[la][i][1][:, h][t])[0]
            compare_decode(out32[i], out[i], ref.cpu().numpy(), f"{kind} request {i}")
    assert cache.status() == (0, 0)


@pytest.mark.parametrize("sink,recent", [(4, 128), (0, 1), (64, 0), (1, 300)])
def test_evict_protects_the_ends(sink, recent):
    lens = [100, 700, 3000, sink + recent + 1]
    keeps = [max(100, sink + recent), sink + recent, sink + recent + 1000, sink + recent]
    g = torch.Generator(device="cuda").manual_seed(sink + recent)
    cache, slots = make(4, 1, lens, spare=200)
    kv = fill(cache, slots, lens)[0]
    W = draw_weights("heavy", cache.new_weights().shape, g)
    cache.evict_begin(slots, keeps, n_sink=sink, n_recent=recent)
    w_out, kept = cache.evict(0, W)
    for i, s in enumerate(slots):
        pages = cache.bf16_pages(0)[torch.tensor(cache.evict_pages(s), dtype=torch.long, device="cuda")]
        check_evicted(cache, i, s, kv[i], pages, W, w_out, kept, keeps[i], sink, recent, lens[i], f"{sink}/{recent}")


def test_evict_a_long_row_and_many_heads():
    """A row longer than the cluster's tiles, 32-bit offsets left behind by far."""
    lens, hkv = [131072, 90001], 8
    cache, slots = make(32, hkv, lens, spare=2200)
    kv = fill(cache, slots, lens)[0]
    g = torch.Generator(device="cuda").manual_seed(3)
    for kind, keep in (("heavy", [32768, 90000]), ("few", [131071, 64]), ("zero", [70000, 1])):
        W = draw_weights(kind, cache.new_weights().shape, g)
        cache.evict_begin(slots, keep)
        w_out, kept = cache.evict(0, W)
        for i, s in enumerate(slots):
            pages = cache.bf16_pages(0)[torch.tensor(cache.evict_pages(s), dtype=torch.long, device="cuda")]
            check_evicted(cache, i, s, kv[i], pages, W, w_out, kept, keep[i], 0, 0, lens[i], kind)
        cache.evict_cancel()


@pytest.mark.parametrize("lens", [[30000] * 3 + [9000, 20481, 100], [90000] + [33000] * 4 + [5], [25000] * 2 + [3000] * 8])
def test_evict_rows_of_one_and_of_several_ctas(lens):
    """Row counts and lengths on either side of the CTAs a row gets and of what they hold."""
    hkv = 8
    cache, slots = make(32, hkv, lens, spare=sum(-(-L // 64) for L in lens))
    kv = fill(cache, slots, lens)[0]
    g = torch.Generator(device="cuda").manual_seed(17)
    for kind, share in (("heavy", 0.3), ("few", 0.62)):
        keep = [max(1, int(L * share)) for L in lens]
        W = draw_weights(kind, cache.new_weights().shape, g)
        cache.evict_begin(slots, keep, n_sink=1)
        w_out, kept = cache.evict(0, W)
        for i, s in enumerate(slots):
            pages = cache.bf16_pages(0)[torch.tensor(cache.evict_pages(s), dtype=torch.long, device="cuda")]
            check_evicted(cache, i, s, kv[i], pages, W, w_out, kept, keep[i], 1, 0, lens[i], kind)
        cache.evict_cancel()


def test_evict_leaves_shared_pages_and_other_slots_alone():
    lens = [640, 0, 200]
    cache, slots = make(4, 1, [640, 640, 200], spare=20)
    kv = fill(cache, slots, lens)[0]
    cache.share_prefix(slots[1], slots[0], 640)
    free = cache.stats()[0]
    g = torch.Generator(device="cuda").manual_seed(8)
    W = draw_weights("heavy", cache.new_weights().shape, g)
    w_out, kept = torch.full_like(W, 5.0), torch.full(W.shape, 9, dtype=torch.int32, device="cuda")
    before = cache.bf16_pages(0).clone()
    cache.evict_begin([slots[1]], [100])
    cache.evict(0, W, weights_out=w_out, kept=kept)
    new = cache.evict_pages(slots[1])
    cache.evict_commit()
    assert cache.pages(slots[1]) == new and cache.stats()[0] == free - 2  # the prefix is still the holder's
    old = torch.tensor(cache.pages(slots[0]) + cache.pages(slots[2]), device="cuda")
    assert torch.equal(cache.bf16_pages(0)[old].view(torch.int16), before[old].view(torch.int16))
    check_evicted(cache, 1, slots[1], kv[0], cache.bf16_pages(0)[torch.tensor(new, device="cuda")], W, w_out, kept, 100, 0,
                  0, 640, "sharer")
    for s in (slots[0], slots[2]):
        assert (w_out[s] == 5).all() and (kept[s] == 9).all()
    assert (kept[slots[1], :, 100:] == 9).all()
    # freed for good once the holder goes too
    cache.free(slots[0])
    cache.free(slots[1])
    cache.free(slots[2])
    assert cache.stats()[0] == cache.cfg.max_pages


def test_pages_past_four_gib():
    """Every operator on pages whose byte offsets in the pool pass 32 bits."""
    hkv, far = 8, 17000  # 256 KB a page
    cache = KVCache(fmt=N.OSCAR_FORMAT_BF16, n_q_heads=32, n_kv_heads=hkv, n_layers=1, max_requests=4, max_pages=far + 60,
                    max_pages_per_request=far)
    below = cache.alloc()  # holds the pages below
    for _ in range(2):
        cache.reserve([below], [32 * far])
        cache.commit()
    w = wl.scaled(wl.WORKLOADS["tiny"], name="far", n_kv_heads=hkv)
    first = cache.alloc()
    K, V = wl.gen_kv(w, SEED, 0, 1, 0, 700, device="cuda")
    cache.reserve([first], [700])
    cache.append(0, K, V)
    cache.commit()
    assert min(cache.pages(first)) * cache.cfg.n_kv_heads * cache.layout.bf16_page_bytes > 1 << 32
    second = cache.alloc()
    cache.share_prefix(second, first, 640)
    q = queries(2, 32, 8)
    for flags in (0, N.OSCAR_PLAN_SHARED_PREFIX | N.OSCAR_PLAN_SHARED_ALWAYS):
        cache.plan([first, second], flags=flags)
        out32 = torch.empty(2, 32, 128, device="cuda")
        out = cache.decode(0, q, out_f32=out32)
        for i, n in ((0, 700), (1, 640)):
            ref = torch.cat([attention(q[i, 4 * h:4 * h + 4], K[:n, h], V[:n, h])[0] for h in range(hkv)])
            compare_decode(out32[i], out[i], ref.cpu().numpy(), f"flags {flags} request {i}")
    cache.plan([first, second])
    weights = cache.new_weights()
    before = weights.clone()
    cache.decode_weights(0, q, weights)
    check_weights(weights[second], before[second], q[1], (K[:640], V[:640]), hkv, "far")
    cache.evict_begin([first], [130])
    w_out, kept = cache.evict(0, weights)
    pages = cache.bf16_pages(0)[torch.tensor(cache.evict_pages(first), dtype=torch.long, device="cuda")]
    check_evicted(cache, 0, first, (K, V), pages, weights, w_out, kept, 130, 0, 0, 700, "far")
    cache.evict_commit()
    assert cache.status() == (0, 0)


@pytest.mark.parametrize("handle", [False, True])
def test_another_stream(handle):
    """Weights' decode and eviction on a stream that is not the current one, which is kept busy:
    what the calls make is made in their stream's order."""
    lens = [3000, 700]
    cache, slots = make(4, 1, lens, spare=40)
    kv = fill(cache, slots, lens)[0]
    q = queries(2, 4, 3)
    cache.plan(slots)
    want = cache.decode_weights(0, q, cache.new_weights())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    w = cache.new_weights()
    out = torch.empty_like(q)
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        busy = busy @ busy * 1e-3
    cache.decode_weights(0, q, w, out=out, stream=stream)
    cache.evict_begin(slots, [1000, 699], stream=stream)
    w_out, kept = cache.evict(0, w, stream=stream)
    side.synchronize()
    assert torch.equal(w.cpu(), want[1].cpu()) and torch.equal(out.cpu(), want[0].cpu())
    torch.cuda.synchronize()
    for i, s in enumerate(slots):
        pages = cache.bf16_pages(0)[torch.tensor(cache.evict_pages(s), dtype=torch.long, device="cuda")]
        check_evicted(cache, i, s, kv[i], pages, w, w_out, kept, [1000, 699][i], 0, 0, lens[i], "side stream")
    cache.evict_commit(stream=stream)
    side.synchronize()


def test_a_captured_eviction_serves_later_plans():
    """Captured where nothing moves, replayed where it does, for more requests and longer rows."""
    lens = [100, 700, 300]
    cache, slots = make(4, 1, lens, spare=30)
    kv = fill(cache, slots, lens)[0]
    W = draw_weights("heavy", cache.new_weights().shape, torch.Generator(device="cuda").manual_seed(5))
    w_out, kept = torch.zeros_like(W), torch.zeros(W.shape, dtype=torch.int32, device="cuda")
    cache.evict_begin([slots[0]], [100])
    cache.evict(0, W, weights_out=w_out, kept=kept)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.evict(0, W, weights_out=w_out, kept=kept)
    cache.evict_cancel()
    keeps = [64, 333, 300]
    cache.evict_begin(slots, keeps)
    graph.replay()
    for i, s in enumerate(slots):
        pages = cache.bf16_pages(0)[torch.tensor(cache.evict_pages(s), dtype=torch.long, device="cuda")]
        check_evicted(cache, i, s, kv[i], pages, W, w_out, kept, keeps[i], 0, 0, lens[i], "replay")
    cache.evict_commit()
    assert cache.status() == (0, 0)


def test_cancel_and_state_rules():
    lens = [500, 300]
    cache, slots = make(4, 1, lens, spare=8, max_requests=3)
    fill(cache, slots, lens)
    free = cache.stats()[0]
    W = cache.new_weights()
    with pytest.raises(N.OscarError) as e:
        cache.evict(0, W)
    assert e.value.status == 7
    for call in (cache.evict_commit, cache.evict_cancel, lambda: cache.evict_pages(slots[0])):
        with pytest.raises(N.OscarError) as e:
            call()
        assert e.value.status == 7
    bad = [([slots[0], slots[0]], [1, 1], {}), ([9], [1], {}), ([2], [1], {}), ([slots[0]], [-1], {}),
           ([slots[0]], [100], dict(n_sink=64, n_recent=64)), ([slots[0]], [100], dict(n_sink=-1)), ([], [], {})]
    for s, k, kw in bad:
        with pytest.raises(N.OscarError) as e:
            cache.evict_begin(s, k, **kw)
        assert e.value.status == 1
    with pytest.raises(N.OscarError) as e:
        cache.evict_begin(slots, [499, 299])  # 8 + 5 pages, 8 spare
    assert e.value.status == 3 and cache.stats()[0] == free
    cache.evict_begin(slots, [200, 100])
    for call in (lambda: cache.evict_begin(slots, [200, 100]), lambda: cache.reserve(slots, [1, 1]),
                 lambda: cache.free(slots[0]), lambda: cache.share_prefix(cache.alloc(), slots[0], 64)):
        with pytest.raises(N.OscarError) as e:
            call()
        assert e.value.status == 7
    for args in (dict(weights_out=W), dict(kept=W.view(torch.int32)), dict(layer=1)):
        with pytest.raises(N.OscarError) as e:
            cache.evict(args.pop("layer", 0), W, **args)
        assert e.value.status == 1
    for w in (W[:1], W.double(), W.cpu(), W.transpose(0, 1)):
        with pytest.raises(ValueError):
            cache.evict(0, w)
    cache.evict_cancel()
    assert cache.stats()[0] == free and cache.info(slots[0])[0] == 500
    q = queries(1, 4, 1)
    cache.plan([slots[0]])
    cache.decode(0, q)
    cache.reserve([slots[0]], [1])
    with pytest.raises(N.OscarError) as e:
        cache.evict_begin(slots, [200, 100])
    assert e.value.status == 7
    cache.append(0, torch.zeros(1, 1, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 1, 128, dtype=torch.bfloat16, device="cuda"))
    cache.commit()
    cache.evict_begin(slots, [200, 100])
    cache.evict(0, W)
    cache.evict_commit()
    with pytest.raises(N.OscarError) as e:  # lengths changed: the plan went with them
        N.oscar_bf16_decode_attention(cache.handle, 0, q, torch.empty_like(q), cache.workspace)
    assert e.value.status == 7


def test_int2_caches_are_refused():
    cache = KVCache(n_q_heads=4, n_kv_heads=1, max_pages=4, max_pages_per_request=4)
    s = cache.alloc()
    assert cache.weights_stride == 0
    with pytest.raises(N.OscarError) as e:
        cache.evict_begin([s], [0])
    assert e.value.status == 7
    for call in (cache.new_weights, lambda: cache.bf16_pages(0)):
        with pytest.raises(ValueError):
            call()
    t = torch.zeros(64, device="cuda")
    with pytest.raises(N.OscarError) as e:
        N.oscar_bf16_decode_weights(cache.handle, 0, t, t, t, t, t)
    assert e.value.status == 7


def test_decode_weights_refusals():
    cache, slots = make(4, 1, [100])
    fill(cache, slots, [100])
    cache.plan(slots)
    q, w = queries(1, 4, 1), cache.new_weights()
    out = torch.empty_like(q)
    ws = torch.empty(N.oscar_decode_weights_workspace_bytes(cache.handle), dtype=torch.uint8, device="cuda")
    args = dict(q=q, out=out, weights_in=w, weights_out=w, workspace=ws)
    for kw in (dict(q=None), dict(out=None), dict(weights_out=None), dict(workspace=ws[:-1]), dict(workspace=ws[128:]),
               dict(layer=1), dict(layer=-1)):
        a = dict(args, layer=0)
        a.update(kw)
        with pytest.raises(N.OscarError) as e:
            N.oscar_bf16_decode_weights(cache.handle, a["layer"], a["q"], a["out"], a["weights_in"], a["weights_out"],
                                        a["workspace"])
        assert e.value.status == 1 and N.oscar_last_launch_count() == 0
    two = torch.zeros(2 * w.numel(), device="cuda")
    half = two[w.numel() // 2:].data_ptr()
    assert N.lib().oscar_bf16_decode_weights(cache.handle, 0, q.data_ptr(), out.data_ptr(), two.data_ptr(), half,
                                             ws.data_ptr(), ws.numel(), None, None) == 1
    for bad in (w[..., :-1], w.double(), w.cpu()):
        with pytest.raises(ValueError):
            cache.decode_weights(0, q, bad)
    for bad in (q[:, :2], q.float(), q.cpu()):
        with pytest.raises(ValueError):
            cache.decode_weights(0, bad, w)


def test_decode_weights_in_a_graph_under_later_plans():
    """A captured decode replays under later plans of more requests and other lengths, on one
    workspace of every plan's size; two captured layers share it."""
    hkv, layers = 1, 2
    cache, slots = make(4, hkv, [300, 900, 64], layers=layers, spare=8, per=20)
    kv = fill(cache, slots, [300, 900, 64], layers)
    W = [cache.new_weights() for _ in range(layers)]
    q = queries(3, 4, 6)
    out = [torch.empty_like(q) for _ in range(layers)]
    cache.plan(slots[:1])
    stream = torch.cuda.Stream()
    call = lambda la: N.oscar_bf16_decode_weights(cache.handle, la, q, out[la], W[la], W[la],  # noqa: E731
                                                  cache.weights_workspace)
    cache.weights_workspace = torch.empty(N.oscar_decode_weights_workspace_max_bytes(cache.handle), dtype=torch.uint8,
                                          device="cuda")
    with torch.cuda.stream(stream):
        for la in range(layers):
            call(la)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for la in range(layers):
            call(la)
    for w in W:
        w.zero_()
    cache.plan([slots[1], slots[2], slots[0]], max_split_pages=1)
    graph.replay()
    graph.replay()
    for la in range(layers):
        for pos, i in enumerate([1, 2, 0]):
            one = torch.zeros_like(W[la][slots[i]])
            half = W[la][slots[i]] / 2  # two equal passes
            check_weights(half, one, q[pos], kv[la][i], hkv, f"layer {la} request {i}")
