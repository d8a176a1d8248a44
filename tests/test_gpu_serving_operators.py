"""The serving loop with the operators around its attention, as they are used together: rotary
positions, the decode with shared prefixes, accumulated weights and eviction, against
attention in plain torch over the tokens that each head still holds."""
import numpy as np
import pytest
import torch

from int2_rotated_kv_rotate_gb300 import OSCAR_FORMAT_BF16, OSCAR_FORMAT_INT2, RotaryEmbedding, serving, workloads as wl
from int2_rotated_kv_rotate_gb300 import _native as N
from oracle import calibration as ocal

from helpers import compare_decode

pytestmark = pytest.mark.gpu

SEED = 3141


def shape():
    return wl.scaled(wl.WORKLOADS["qwen3_8b_layer"], name="serving_ops", n_layers=2, n_q_heads=8, n_kv_heads=2, window=64,
                     calib_tokens=512)


class Mirror:
    """What every (request, layer, head) holds: rotated K and V rows, by the positions kept."""

    def __init__(self, w, tokens, prefix, rotary):
        self.w, self.tokens, self.prefix, self.rotary = w, tokens, prefix, rotary
        self.held = {}  # (rid, layer, head) -> positions; missing: all so far

    def rows(self, r, layer, n):
        pieces = [(serving.TokenSource.stream(r, p, self.prefix), p, 1) for p in range(n)]
        idx = self.tokens.index(layer, pieces)
        K, V = self.tokens.K.index_select(0, idx), self.tokens.V.index_select(0, idx)
        if self.rotary is not None:
            K = self.rotary.apply(torch.arange(n, dtype=torch.int32, device="cuda"), K)
        return K, V

    def attention(self, r, layer, q, n):
        """fp64 attention of q [H_q, 128] over what r holds once position n - 1 is appended."""
        K, V = self.rows(r, layer, n)
        G = self.w.gqa
        out = []
        for h in range(self.w.n_kv_heads):
            at = self.held.get((r.rid, layer, h))
            t = torch.arange(n, device="cuda") if at is None else torch.cat((at, torch.arange(self.since[r.rid], n, device="cuda")))
            k, v = K[t, h].double(), V[t, h].double()
            p = torch.softmax(q[h * G:(h + 1) * G].double() @ k.T / np.sqrt(128.0), -1)
            out.append(p @ v)
        return torch.cat(out).cpu().numpy()

    since = {}


@pytest.mark.parametrize("rotated", [False, True])
def test_shared_decode_in_the_loop(rotated):
    w, prefix = shape(), 64 * 40
    tokens = serving.TokenSource(w, SEED, pool_tokens=4096)
    rotary = RotaryEmbedding(base=1e6) if rotated else None
    reqs = serving.make_requests(40, (prefix + 1, prefix + 90), (2, 4), n_groups=1, seed=SEED)
    loop = serving.ServingLoop(w, OSCAR_FORMAT_BF16, 64 << 20, tokens, max_requests=64, max_len=3000, prefix_tokens=prefix,
                               rotary=rotary, share_decode=True)
    mirror = Mirror(w, tokens, prefix, rotary)
    shared = []

    def on_output(step, layer, reqs_, K, V, q, out, o32):
        torch.cuda.synchronize()
        shared.append(loop.cache.shared_info()[1])
        for i in range(0, len(reqs_), 7):
            ref = mirror.attention(reqs_[i], layer, q[i], reqs_[i].position + 1)
            compare_decode(o32[i], out[i], ref, f"step {step} layer {layer} request {reqs_[i].rid}")

    st = loop.run(reqs, on_output=on_output)
    assert st["completed"] == len(reqs) and st["prefix_hits"] > 0
    assert max(shared) == prefix // 64  # the group's prefix was attended once
    assert loop.cache.status() == (0, 0)
    loop.close()


def test_eviction_in_the_loop():
    w, prefix = shape(), 128
    tokens = serving.TokenSource(w, SEED, pool_tokens=4096)
    rotary = RotaryEmbedding(rotary_dim=64, base=10000.0, interleaved=True)
    reqs = serving.make_requests(7, (150, 420), (4, 60), n_groups=2, seed=SEED)
    above, to, sink, recent = 300, 180, 4, 32
    # a pool of 30 pages: two or three requests at once
    budget = N.oscar_cache_device_bytes(N.oscar_config(OSCAR_FORMAT_BF16, 128, w.n_q_heads, w.n_kv_heads, w.group, 64, 0, 0,
                                                       w.n_layers, 8, 1, 12)) + 29 * w.n_layers * w.n_kv_heads * 32768
    loop = serving.ServingLoop(w, OSCAR_FORMAT_BF16, budget, tokens, max_requests=8, max_len=600, prefix_tokens=prefix,
                               prefill_chunk=500, rotary=rotary, evict_above=above, evict_to=to, n_sink=sink, n_recent=recent)
    free0 = loop.cache.stats()
    mirror = Mirror(w, tokens, prefix, rotary)
    mirror.since = {}
    checked = [0]

    def on_output(step, layer, reqs_, K, V, q, out, o32):
        torch.cuda.synchronize()
        for i, r in enumerate(reqs_):
            assert r.length <= max(r.prompt, above) + 1
            compare_decode(o32[i], out[i], mirror.attention(r, layer, q[i], r.position + 1),
                           f"step {step} layer {layer} request {r.rid} (position {r.position}, holds {r.length})")
            checked[0] += 1

    def on_evict(layer, reqs_, weights, kept):
        torch.cuda.synchronize()
        for r in reqs_:
            L = r.length
            for h in range(w.n_kv_heads):
                t = kept[r.slot, h, :to].long()
                # each step gave the weights one unit a query head; what stays holds the ends
                total = float(weights[r.slot, h, :L].double().sum())
                assert total > 0 and bool((weights[r.slot, h, L:] == 0).all())
                assert t[:sink].tolist() == list(range(sink)) and t[-recent:].tolist() == list(range(L - recent, L))
                key = (r.rid, layer, h)
                last = mirror.since.get(r.rid, 0)
                before = torch.cat((mirror.held[key], torch.arange(last, r.position, device="cuda"))) if key in mirror.held \
                    else torch.arange(L, device="cuda")
                mirror.held[key] = before[t]
        if layer == w.n_layers - 1:
            for r in reqs_:
                mirror.since[r.rid] = r.position

    st = loop.run(reqs, on_output=on_output, on_evict=on_evict)
    assert st["completed"] == len(reqs) and st["evictions"] > 2
    assert checked[0] == st["generated"] * w.n_layers
    for s in list(loop.holders.values()):
        loop.cache.free(s)
    loop.holders = {}
    assert loop.cache.stats() == free0 and loop.cache.status() == (0, 0)
    loop.close()


def test_rotary_before_the_int2_cache():
    """The INT2 cache's loop takes the same rotated rows: against attention over what it stored is
    the parity tests' matter; here the loop with positions equals the loop over rows rotated
    beforehand."""
    w = shape()
    tokens = serving.TokenSource(w, SEED, pool_tokens=4096)
    params = [[], [], [], []]
    for layer in range(w.n_layers):
        q, k, v = wl.gen_calibration(w, SEED, layer)
        for i, a in enumerate(ocal.calibrate_layer(q.float().numpy(), k.float().numpy(), v.float().numpy(), w.clip_percentile)):
            params[i].append(a)
    params = [np.stack(a) for a in params]
    rotary = RotaryEmbedding(base=1e6)
    outs = []

    def run(rot):
        loop = serving.ServingLoop(w, OSCAR_FORMAT_INT2, 32 << 20, tokens, layer_params=params, max_requests=4, max_len=600,
                                   rotary=rot)
        got = []
        loop.run(serving.make_requests(2, (150, 300), (3, 3), 0, SEED),
                 on_output=lambda s, la, rs, K, V, q, out, o32: got.append((q.clone(), K.clone(), out.clone())))
        loop.close()
        return got

    for (q, K, out), (q0, K0, _) in zip(run(rotary), run(None)):
        outs.append(out)
        assert not torch.equal(q, q0) and not torch.equal(K, K0)
        # a rotation keeps the norms, up to the rounding of 128 bf16 channels
        assert torch.allclose(q.float().norm(dim=-1), q0.float().norm(dim=-1), rtol=2.0**-8)
    assert all(torch.isfinite(o.float()).all() for o in outs)


def test_refusals():
    w = shape()
    tokens = serving.TokenSource(w, SEED, pool_tokens=64)
    make = lambda fmt, **kw: serving.ServingLoop(w, fmt, 8 << 20, tokens, max_requests=2, max_len=200, **kw)  # noqa: E731
    for fmt, kw in ((OSCAR_FORMAT_INT2, dict(share_decode=True)), (OSCAR_FORMAT_INT2, dict(evict_above=100, evict_to=80)),
                    (OSCAR_FORMAT_BF16, dict(share_decode=True, evict_above=100, evict_to=80)),
                    (OSCAR_FORMAT_BF16, dict(evict_above=100, evict_to=120)), (OSCAR_FORMAT_BF16, dict(evict_above=100)),
                    (OSCAR_FORMAT_BF16, dict(evict_above=100, evict_to=60, n_recent=64))):
        with pytest.raises(ValueError):
            make(fmt, **kw)
    assert N.oscar_weights_stride(make(OSCAR_FORMAT_BF16).cache.handle) > 0
