"""The serving loop's pages and buffers with eviction: what it admits fits until the end."""
import pytest
import torch

from int2_rotated_kv_rotate_gb300 import OSCAR_FORMAT_BF16, _native as N, serving, workloads as wl

pytestmark = pytest.mark.gpu

SEED = 77


def shape(**kw):
    return wl.scaled(wl.WORKLOADS["qwen3_8b_layer"], name="serving_pages", **{**dict(n_layers=2, n_q_heads=8, n_kv_heads=2, window=64,
                                                                                     calib_tokens=512), **kw})


def loop_of(pages, w, tokens, **kw):
    """A loop whose pool has just so many pages."""
    def make(budget):
        try:
            return serving.ServingLoop(w, OSCAR_FORMAT_BF16, budget, tokens, **kw)
        except ValueError:  # holds no page
            return None

    lo, hi = 0, 1 << 32
    while lo < hi:  # the least budget with them
        mid = (lo + hi) // 2
        loop = make(mid)
        if loop is not None and loop.cache.cfg.max_pages >= pages:
            hi = mid
        else:
            lo = mid + 1
        if loop is not None:
            loop.close()
    loop = make(lo)
    assert loop.cache.cfg.max_pages == pages
    return loop


@pytest.mark.parametrize("pages", [11, 13, 15, 16, 19])
def test_sharers_that_evict_twice_fit(pages):
    """Requests behind a shared prefix of three pages (192 tokens) move to pages of their own at
    the first eviction and need five and three of them at the second."""
    w = shape()
    tokens = serving.TokenSource(w, SEED, pool_tokens=2048)
    loop = loop_of(pages, w, tokens, max_requests=4, max_len=600, prefix_tokens=192, evict_above=300, evict_to=180, n_sink=4,
                   n_recent=32)
    reqs = [serving.Request(rid=i, prompt=200 + 10 * i, gen=400, group=0) for i in range(3)]
    st = loop.run(reqs)
    assert st["completed"] == 3 and st["prefix_hits"] == 3 and st["evictions"] >= 6
    assert loop.cache.status() == (0, 0)
    loop.close()


def test_eviction_keeps_within_the_budget():
    """The default slots and lengths in 1 GiB: cache, weights and what a run allocates besides (the
    decode's partial sums aside, which every format's loop has) stay within it."""
    w = shape(n_layers=4, n_q_heads=32, n_kv_heads=8)
    tokens = serving.TokenSource(w, SEED, pool_tokens=2048)
    budget = 1 << 30
    torch.cuda.empty_cache()
    before = torch.cuda.memory_allocated()
    loop = serving.ServingLoop(w, OSCAR_FORMAT_BF16, budget, tokens, evict_above=700, evict_to=300)
    assert torch.cuda.memory_allocated() - before <= budget
    assert loop.cache.nbytes > budget // 4  # and most of it is not given away
    st = loop.run([serving.Request(rid=i, prompt=600 + 50 * i, gen=150) for i in range(6)])
    assert st["completed"] == 6 and st["evictions"] >= 6
    scores = loop.cache.weights_workspace.numel() - (N.oscar_decode_weights_workspace_max_bytes(loop.cache.handle)
                                                     - 4 * 128 * 32 * loop.cache.weights_stride)
    kept = sum(t.numel() * 4 for t in [*loop.weights, loop._weights_out, loop._kept])
    assert loop.cache.nbytes + kept + scores <= budget
    loop.close()
