"""Rotary positions whose angles are small: their sines in full precision."""
import pytest
import torch

from int2_rotated_kv_rotate_gb300 import RotaryEmbedding

from test_gpu_rope import reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
def test_small_angles_keep_their_bits(interleaved):
    """Channels whose partner is zero are b sin and a cos alone.  A pair's phase is converted with
    2^-24 relative, sines and cosines are within one ulp (2^-23), the product rounds once
    (2^-24): 2^-22 relative, however small the angle."""
    rot = RotaryEmbedding(base=1e6, interleaved=interleaved, scaling=dict(type="linear", factor=8.0))
    positions = torch.tensor([1, 2, 3, 7, 100, 5000, -1, -64], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(8, 2, 128, generator=g, device="cuda")
    first = torch.arange(128, device="cuda") % 2 == 0 if interleaved else torch.arange(128, device="cuda") < 64
    x[:, 0, first] = 0.0  # head 0: a = 0; head 1: b = 0
    x[:, 1, ~first] = 0.0
    want, _ = reference(rot, positions, x)
    got = rot.apply(positions, x).cpu().double()
    assert (want.abs() > 0).all()
    assert ((got - want).abs() <= (2.0**-22 + 2.0**-40) * want.abs()).all()
