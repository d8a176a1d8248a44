"""What the operators' calls make themselves is made on the stream of their launch: the caching
allocator hands a block out again in the order of the stream it belongs to."""
import pytest
import torch

from int2_rotated_kv_rotate_gb300 import OSCAR_FORMAT_BF16, KVCache, RotaryEmbedding

pytestmark = pytest.mark.gpu


def pool_stream(t):
    """The stream whose pool the tensor's memory belongs to."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the caching allocator's")


def keep_busy():
    x = torch.randn(4096, 4096, device="cuda")
    for _ in range(40):
        x = x @ x * 1e-3


@pytest.mark.parametrize("handle", [False, True])
def test_rotary_outputs_on_another_stream(handle):
    """A block that pending work of the current stream still reads is not the output's."""
    rot = RotaryEmbedding(base=1e6)
    q = torch.randn(2048, 16, 128, device="cuda").bfloat16()
    k = torch.randn(2048, 4, 128, device="cuda").bfloat16()
    positions = torch.arange(2048, device="cuda")
    want = rot.apply(positions, q, k)
    side = torch.cuda.Stream()
    keep_busy()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    read = torch.zeros_like(q)  # (q_out's size: the block that its allocation would get)
    kept = torch.empty_like(q)
    torch.cuda.synchronize()
    keep_busy()
    kept.copy_(read)
    del read
    got = rot.apply(positions, q, k, stream=side.cuda_stream if handle else side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    torch.cuda.synchronize()
    assert bool((kept == 0).all())
    assert pool_stream(got[0]) == pool_stream(got[1]) == side.cuda_stream


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("call", ["decode", "decode_weights"])
def test_decode_outputs_and_workspaces_on_another_stream(call, handle):
    cache = KVCache(fmt=OSCAR_FORMAT_BF16, n_q_heads=4, n_kv_heads=1, n_layers=1, max_requests=2, max_pages=64,
                    max_pages_per_request=32)
    slots = [cache.alloc(), cache.alloc()]
    cache.reserve(slots, [100, 1500])
    cache.append(0, torch.randn(1600, 1, 128, device="cuda").bfloat16(), torch.randn(1600, 1, 128, device="cuda").bfloat16())
    cache.commit()
    q = torch.randn(2, 4, 128, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    w = cache.new_weights()
    torch.cuda.synchronize()
    cache.plan(slots, stream=stream)
    if call == "decode":
        out = cache.decode(0, q, stream=stream)
    else:
        out, _ = cache.decode_weights(0, q, w, stream=stream)
        assert pool_stream(cache.weights_workspace) == side.cuda_stream
    assert pool_stream(out) == pool_stream(cache.workspace) == side.cuda_stream
    side.synchronize()
    cache.plan(slots)
    assert torch.equal(out, cache.decode(0, q))
    assert pool_stream(cache.decode(0, q)) == torch.cuda.current_stream().cuda_stream


def test_outputs_on_another_device_are_refused():
    cache = KVCache(fmt=OSCAR_FORMAT_BF16, n_q_heads=4, n_kv_heads=1, n_layers=1, max_requests=1, max_pages=2,
                    max_pages_per_request=2)
    slot = cache.alloc()
    cache.reserve([slot], [3])
    cache.append(0, *(torch.zeros(3, 1, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    cache.commit()
    cache.plan([slot])
    q, host = torch.zeros(1, 4, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 4, 128)
    for kw in (dict(out=host.bfloat16()), dict(out_f32=host)):
        with pytest.raises(ValueError):
            cache.decode_weights(0, q, cache.new_weights(), **kw)
        with pytest.raises(ValueError):
            cache.decode(0, q, **kw)
