"""The workspace of the weights' decode goes with the tokens of the plan, not with the longest
rows that the cache could hold; against fp64 by the tolerances of test_gpu_evict."""
import pytest
import torch

from int2_rotated_kv_rotate_gb300 import _native as N

from test_gpu_evict import check_weights, fill, make, queries

pytestmark = pytest.mark.gpu


def test_workspace_grows_with_the_plans():
    hkv, hq, lens = 2, 8, [100, 3000, 1, 700]
    cache, slots = make(hq, hkv, lens, max_requests=64, per=2048, spare=4000)
    kv = fill(cache, slots, lens)[0]
    full = N.oscar_decode_weights_workspace_max_bytes(cache.handle)
    q = queries(4, hq, 1)
    sizes = []
    for pick in ([0], [2, 0], [0, 1, 2, 3], [3]):
        need = cache.plan([slots[i] for i in pick])
        need = N.oscar_decode_weights_workspace_bytes(cache.handle)
        rest = full - 64 * hq * 2048 * 64 * 4  # all but the scores
        assert need == rest + 4 * hq * sum(lens[i] for i in pick)
        before = torch.rand(cache.new_weights().shape, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
        _, after = cache.decode_weights(0, q[:len(pick)], before, weights_out=before.clone())
        assert need <= cache.weights_workspace.numel() <= need + need // 4 < full
        sizes.append(cache.weights_workspace.numel())
        for pos, i in enumerate(pick):
            check_weights(after[slots[i]], before[slots[i]], q[pos], kv[i], hkv, f"{pick} request {i}")
    assert sizes[2] == sizes[3]  # what there is serves a smaller plan
    assert cache.status() == (0, 0)


def test_a_captured_launch_gets_room_for_every_plan():
    """Captured under a short plan by the cache's own call, replayed under longer ones, with eager
    calls of other plans between."""
    hkv, hq, lens = 1, 4, [64, 900, 1300]
    cache, slots = make(hq, hkv, lens, spare=8, per=24)
    kv = fill(cache, slots, lens)[0]
    full = N.oscar_decode_weights_workspace_max_bytes(cache.handle)
    q, W = queries(3, hq, 2), cache.new_weights()
    cache.plan(slots[:1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cache.decode_weights(0, q[:1], W)
    torch.cuda.current_stream().wait_stream(side)
    assert cache.weights_workspace.numel() < full
    out = torch.empty_like(q)  # (the launch takes its requests from the plan of its replay)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.decode_weights(0, q[:1], W, out=out[:1])
    assert cache.weights_workspace.numel() >= full
    at = cache.weights_workspace.data_ptr()
    cache.plan([slots[2], slots[1]])
    cache.decode_weights(0, q[:2], cache.new_weights())
    assert cache.weights_workspace.data_ptr() == at
    W.zero_()
    cache.plan([slots[1], slots[2], slots[0]])
    graph.replay()
    for pos, i in enumerate([1, 2, 0]):
        check_weights(W[slots[i]], torch.zeros_like(W[slots[i]]), q[pos], kv[i], hkv, f"request {i}")
    assert cache.status() == (0, 0)


def test_growing_beside_pending_launches_of_another_stream():
    """The old workspace is not handed out again while a launch on another stream waits to use it."""
    hkv, hq, lens = 1, 4, [40000, 60000]
    cache, slots = make(hq, hkv, lens, max_requests=2)
    kv = fill(cache, slots, lens)[0]
    q = queries(2, hq, 4)
    torch.cuda.empty_cache()
    cache.plan(slots[:1])
    first, second = cache.new_weights(), cache.new_weights()
    cache.decode_weights(0, q[:1], first.clone())
    size = cache.weights_workspace.numel()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(40):
            busy = busy @ busy * 1e-3
        cache.decode_weights(0, q[:1], first, out=torch.empty_like(q[:1]))
    held = cache.weights_workspace.data_ptr()
    cache.weights_workspace = cache._score_space(None)  # (as the next call would take it)
    cache._weights_need = size + 1  # a longer plan's
    cache._score_space(None)
    again = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    assert again.data_ptr() != held
    torch.cuda.synchronize()
    check_weights(first[slots[0]], torch.zeros_like(first[slots[0]]), q[0], kv[0], hkv, "side")
    cache.plan(slots[1:])
    cache.decode_weights(0, q[1:], second)
    check_weights(second[slots[1]], torch.zeros_like(second[slots[1]]), q[1], kv[1], hkv, "after")
