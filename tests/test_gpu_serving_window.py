"""The serving loop with the operators on the paged caches together, as they are used: keys turned as
they are appended, attention within a window and over the first tokens, and the 4-bit cache."""
import math

import pytest
import torch

from int2_rotated_kv_rotate_gb300 import (OSCAR_FORMAT_BF16, OSCAR_FORMAT_INT2, OSCAR_FORMAT_INT4, RotaryEmbedding, serving,
                                          workloads as wl)

pytestmark = pytest.mark.gpu
SEED = 2718


def shape():
    return wl.scaled(wl.WORKLOADS["qwen3_8b_layer"], name="serving_window", n_layers=2, n_q_heads=8, n_kv_heads=2, group=32,
                     window=64, calib_tokens=512)


def rows(w, tokens, prefix, rotary, r, layer, n):
    """K (turned) and V rows of r's first n positions."""
    idx = tokens.index(layer, [(serving.TokenSource.stream(r, p, prefix), p, 1) for p in range(n)])
    K, V = tokens.K.index_select(0, idx), tokens.V.index_select(0, idx)
    return (K if rotary is None else rotary.apply(torch.arange(n, dtype=torch.int32, device="cuda"), K)), V


def attention(q, k, v):
    """fp64 attention of q [H_q, 128] over k, v [n, H_kv, 128]."""
    G = q.shape[0] // k.shape[1]
    out = []
    for h in range(k.shape[1]):
        p = torch.softmax(q[h * G:(h + 1) * G].double() @ k[:, h].double().T / math.sqrt(128.0), -1)
        out.append(p @ v[:, h].double())
    return torch.cat(out)


@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("sinks,window", [(4, 100), (0, 1), (130, 64)])
def test_window_in_the_loop(sinks, window, rotated):
    w, prefix = shape(), 128
    tokens = serving.TokenSource(w, SEED, pool_tokens=4096)
    rotary = RotaryEmbedding(base=1e6) if rotated else None
    reqs = serving.make_requests(9, (129, 400), (2, 5), n_groups=2, seed=SEED)
    loop = serving.ServingLoop(w, OSCAR_FORMAT_BF16, 64 << 20, tokens, max_requests=8, max_len=600, prefix_tokens=prefix,
                               prefill_chunk=300, rotary=rotary, window=window, window_sinks=sinks)
    checked = [0]

    def on_output(step, layer, reqs_, K, V, q, out, o32):
        for i, r in enumerate(reqs_):
            n = r.position + 1
            k, v = rows(w, tokens, prefix, rotary, r, layer, n)
            assert torch.equal(K[i], k[-1]) and torch.equal(V[i], v[-1])
            t = torch.arange(n, device="cuda")
            see = (t < sinks) | (t > n - 1 - window)
            ref = attention(q[i], k[see], v[see])
            # (single queries keep 16 bits of a weight; the scores of these rows stay under 2^7)
            tol = (2.0 ** -16 + 2 * (2.0 ** -11 + 2.0 ** -20)) * float(v.abs().max())
            assert float((o32[i].double() - ref).abs().max()) <= tol, f"step {step} layer {layer} request {r.rid}"
            assert torch.equal(out[i], o32[i].bfloat16())
            checked[0] += 1

    st = loop.run(reqs, on_output=on_output)
    assert st["completed"] == len(reqs) and st["prefix_hits"] > 0 and checked[0] == 2 * st["generated"]
    assert loop.cache.status() == (0, 0)
    loop.close()


@pytest.mark.parametrize("rotated", [False, True])
def test_the_4_bit_cache_in_the_loop(rotated):
    """Every output is attention over the values that the cache holds, which are the quantised rows."""
    w, prefix = shape(), 128
    tokens = serving.TokenSource(w, SEED, pool_tokens=4096)
    rotary = RotaryEmbedding(base=1e6, rotary_dim=64, interleaved=True) if rotated else None
    reqs = serving.make_requests(9, (129, 400), (2, 5), n_groups=2, seed=SEED)
    loop = serving.ServingLoop(w, OSCAR_FORMAT_INT4, 24 << 20, tokens, max_requests=8, max_len=600, prefix_tokens=prefix,
                               prefill_chunk=300, rotary=rotary)

    def on_output(step, layer, reqs_, K, V, q, out, o32):
        for i, r in enumerate(reqs_):
            n = r.position + 1
            held = loop.cache.read(layer, r.slot, 0, n, dtype=torch.float32)
            for x, y in zip(rows(w, tokens, prefix, rotary, r, layer, n), held):
                x = x.float().unflatten(-1, (-1, 32))
                s = ((x.amax(-1, keepdim=True) - x.amin(-1, keepdim=True)) / 15).bfloat16().float()
                # half a step, and what the scale's rounding cuts off the top code (15 * 2^-9 of a step)
                assert bool(((y.unflatten(-1, (-1, 32)) - x).abs() <= s * (0.5 + 15 * 2.0 ** -8)).all())
            ref = attention(q[i], *held)
            tol = (2.0 ** -12 + 2 * (2.0 ** -10 + 2.0 ** -20)) * 2 * float(held[1].abs().max())
            assert float((o32[i].double() - ref).abs().max()) <= tol, f"step {step} layer {layer} request {r.rid}"

    st = loop.run(reqs, on_output=on_output)
    assert st["completed"] == len(reqs) and st["prefix_hits"] > 0
    assert loop.cache.status() == (0, 0)
    loop.close()


def test_the_4_bit_cache_holds_more():
    """At one budget the 4-bit cache has over three times the pages of the BF16 cache."""
    w = shape()
    pages = [serving.cache_for_budget(w, fmt, 512 << 20, 8, 600, "cuda").cfg.max_pages for fmt in (OSCAR_FORMAT_BF16, OSCAR_FORMAT_INT4)]
    assert pages[1] > 3 * pages[0]


def test_refusals():
    w = shape()
    tokens = serving.TokenSource(w, SEED, pool_tokens=64)
    make = lambda fmt, **kw: serving.ServingLoop(w, fmt, 16 << 20, tokens, max_requests=2, max_len=200, **kw)  # noqa: E731
    for fmt, kw in ((OSCAR_FORMAT_INT4, dict(window=10)), (OSCAR_FORMAT_INT2, dict(window=10)), (OSCAR_FORMAT_INT4, dict(share_decode=True)),
                    (OSCAR_FORMAT_INT4, dict(evict_above=100, evict_to=80)), (OSCAR_FORMAT_BF16, dict(window=-1)),
                    (OSCAR_FORMAT_BF16, dict(window_sinks=3)), (OSCAR_FORMAT_BF16, dict(window=10, share_decode=True)),
                    (OSCAR_FORMAT_BF16, dict(window=10, evict_above=100, evict_to=80))):
        with pytest.raises(ValueError):
            make(fmt, **kw)
