"""Rotary positions on the GPU against fp64, from the definition: phases of the table in
exact integer arithmetic, pairs as complex numbers.

Tolerance, from the arithmetic: sines and cosines are within 1 ulp (2^-23) of those of a
phase that is within 2^-24 of its value (at most pi / 4), and are rounded once with the
magnitude; the two products and the sum round once each: an absolute error of at most
3 * 2^-23 * magnitude * (|a| + |b|) before the one rounding to the dtype, of half a step."""
import numpy as np
import pytest
import torch

from int2_rotated_kv_rotate_gb300 import RotaryEmbedding
from int2_rotated_kv_rotate_gb300 import _native as N

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def reference(rot, positions, x, transpose=False):
    """(fp64 result, absolute error bound before the final rounding)."""
    R = rot.rotary_dim
    steps = rot.steps.cpu().numpy().view(np.uint64)
    pos = positions.cpu().numpy().astype(np.int64).view(np.uint64)
    phase = (pos[:, None] * steps[None, :]).view(np.int64).astype(np.float64) * (2 * np.pi / 2.0**64)
    turn = torch.from_numpy(rot.magnitude * np.exp((-1j if transpose else 1j) * phase))[:, None, :]
    y = x.detach().cpu().double()
    if rot.interleaved:
        pair = y[..., :R].unflatten(-1, (R // 2, 2))
        a, b = pair[..., 0], pair[..., 1]
    else:
        a, b = y[..., :R // 2], y[..., R // 2:R]
    z = torch.complex(a, b) * turn
    bound = 3 * 2.0**-23 * rot.magnitude * (a.abs() + b.abs())
    err = torch.zeros_like(y)
    y = y.clone()
    if rot.interleaved:
        y[..., :R] = torch.stack((z.real, z.imag), -1).flatten(-2)
        err[..., :R] = torch.stack((bound, bound), -1).flatten(-2)
    else:
        y[..., :R] = torch.cat((z.real, z.imag), -1)
        err[..., :R] = torch.cat((bound, bound), -1)
    return y, err


def check(got, want, err, dtype):
    half = torch.finfo(dtype).eps / 2
    tol = half * want.abs() + (1 + half) * err + (2.0**-25 if dtype == torch.float16 else 0.0)
    d = (got.cpu().double() - want).abs()
    assert torch.isfinite(got).all()
    assert (d <= tol).all(), f"off by {float((d - tol).max()):.3e} over the tolerance"


def inputs(rows, hq, hkv, d, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, hq, d, generator=g, device="cuda").to(dtype),
            torch.randn(rows, hkv, d, generator=g, device="cuda").to(dtype))


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,hq,hkv,d,R", [
    (1, 32, 8, 128, 128), (1, 1, 1, 2, 2), (3, 8, 2, 128, 64), (17, 5, 3, 128, 96), (33, 64, 8, 128, 18),
    (2500, 8, 8, 128, 128), (7, 40, 1, 80, 20), (5, 3, 2, 512, 512), (4, 2, 1, 511, 510), (2, 7, 1, 512, 2)])
def test_against_fp64(dtype, interleaved, rows, hq, hkv, d, R):
    t = DTYPES[dtype]
    rot = RotaryEmbedding(head_dim=d, rotary_dim=R, base=10000.0, interleaved=interleaved)
    q, k = inputs(rows, hq, hkv, d, t, rows + hq)
    g = torch.Generator(device="cuda").manual_seed(7)
    for positions in (torch.arange(rows, device="cuda", dtype=torch.int32) + 131000,
                      torch.randint(0, 1 << 20, (rows,), generator=g, device="cuda")):
        for transpose in (False, True):
            q2, k2 = rot.apply(positions, q, k, transpose=transpose)
            for x, y in ((q, q2), (k, k2)):
                want, err = reference(rot, positions, x, transpose)
                check(y, want, err, t)
                assert torch.equal(y[..., R:], x[..., R:])


@pytest.mark.parametrize("scaling", [dict(type="linear", factor=8.0), dict(type="bands", factor=8.0, original_context=8192),
                                     dict(type="yarn", factor=4.0, original_context=32768)])
def test_scaled_frequencies(scaling):
    rot = RotaryEmbedding(base=1e6, scaling=scaling)
    q, k = inputs(9, 4, 1, 128, torch.float32, 3)
    positions = torch.tensor([0, 1, 2, 8191, 8192, 32768, 100000, 131071, 1 << 20], device="cuda")
    for x, y in zip((q, k), rot.apply(positions, q, k)):
        check(y, *reference(rot, positions, x), torch.float32)
    # and the angles of the formula itself, from fp64 frequencies (positions up to 2^20: the
    # two sides' frequencies differ by under 2^-49 relative, 2^-29 of an angle)
    if scaling["type"] == "linear":
        f = 1e6 ** (-np.arange(64) * 2 / 128) / 8.0
        ang = positions.cpu().numpy()[:, None] * f
        a, b = q.cpu().double()[:, 0, :64].numpy(), q.cpu().double()[:, 0, 64:].numpy()
        want = a * np.cos(ang) - b * np.sin(ang)
        got = rot.apply(positions, q)[:, 0, :64].cpu().double().numpy()
        assert (np.abs(got - want) <= 2.0**-24 * np.abs(want) + 4 * 2.0**-23 * (np.abs(a) + np.abs(b))).all()


def test_far_and_negative_positions():
    rot = RotaryEmbedding(base=10000.0)
    positions = torch.tensor([-1, -(1 << 31), (1 << 31) - 1, 1 << 40, -(1 << 62), (1 << 63) - 1], device="cuda")
    q, _ = inputs(6, 3, 1, 128, torch.float32, 5)
    check(rot.apply(positions, q), *reference(rot, positions, q), torch.float32)
    p32 = positions[:3].to(torch.int32)
    assert torch.equal(rot.apply(p32, q[:3]), rot.apply(positions[:3], q[:3]))


def test_strides_alignment_and_in_place():
    rot = RotaryEmbedding(rotary_dim=64, base=1e6)
    g = torch.Generator(device="cuda").manual_seed(1)
    rows, hq, hkv = 11, 8, 2
    positions = torch.randint(0, 1 << 17, (rows,), generator=g, device="cuda")
    for extra in (0, 1, 8):  # a fused projection's rows: 1 breaks the 16-byte alignment
        qkv = torch.randn(rows, (hq + 2 * hkv) * 128 + extra, generator=g, device="cuda").to(torch.bfloat16)
        q = qkv[:, extra:extra + hq * 128].view(rows, hq, 128)
        k = qkv[:, extra + hq * 128:extra + (hq + hkv) * 128].view(rows, hkv, 128)
        keep = qkv.clone()
        want = rot.apply(positions, q.clone(), k.clone())
        got = rot.apply(positions, q, k)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(qkv, keep)
        # in place, inside the fused rows; values and padding stay as they were
        rot.apply(positions, q, k, q_out=q, k_out=k)
        assert torch.equal(q, want[0]) and torch.equal(k, want[1])
        keep[:, extra:extra + (hq + hkv) * 128] = qkv[:, extra:extra + (hq + hkv) * 128]
        assert torch.equal(qkv, keep)
    # head-major storage [H, rows, d], in and out; one row broadcast to all
    x = torch.randn(hq, rows, 128, generator=g, device="cuda")
    out = torch.empty(hq, rows, 128, device="cuda")
    rot.apply(positions, x.transpose(0, 1), q_out=out.transpose(0, 1))
    assert torch.equal(out.transpose(0, 1), rot.apply(positions, x.transpose(0, 1).contiguous()))
    one = x[:, :1].transpose(0, 1).expand(rows, hq, 128)
    assert torch.equal(rot.apply(positions, one), rot.apply(positions, one.contiguous()))


def test_gradient_is_the_transpose():
    """<g, rope(x)> has the gradient rope^T(g): against autograd of the fp64 definition, against
    differences, and rope^T(rope(x)) = magnitude^2 x."""
    rot = RotaryEmbedding(rotary_dim=32, head_dim=64, interleaved=True, base=10000.0,
                          scaling=dict(type="yarn", factor=4.0, original_context=4096))
    q, g = inputs(5, 3, 3, 64, torch.float32, 9)
    positions = torch.tensor([0, 5, 4095, 4096, 77777], device="cuda")
    grad = rot.apply(positions, g, transpose=True)
    x = q.cpu().double().requires_grad_()
    steps = rot.steps.cpu().numpy().view(np.uint64)
    phase = (positions.cpu().numpy().view(np.uint64)[:, None] * steps).view(np.int64) * (2 * np.pi / 2.0**64)
    c = torch.from_numpy(rot.magnitude * np.cos(phase))[:, None]
    s = torch.from_numpy(rot.magnitude * np.sin(phase))[:, None]
    a, b = x[..., 0:32:2], x[..., 1:32:2]
    y = torch.cat((torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2), x[..., 32:]), -1)
    (y * g.cpu().double()).sum().backward()
    _, err = reference(rot, positions, g, True)
    check(grad, x.grad, err, torch.float32)
    # differences: the map is linear, so its step is any size; h = 2 keeps sums exact in scale
    for row, ch in ((1, 0), (2, 7), (4, 63)):
        e = torch.zeros_like(q)
        e[row, 1, ch] = 2.0
        diff = (rot.apply(positions, q + e).double() - rot.apply(positions, q - e).double()) / 4.0
        got = float((diff * g.double()).sum())
        # each output within 2^-24 |y| + 3 * 2^-23 mag (|a| + |b|), |y| and the inputs under 8
        tol = 2 * 64 * 3 * 64 * 2.0**-22 / 4.0
        assert abs(got - float(grad[row, 1, ch])) <= tol
    back = rot.apply(positions, rot.apply(positions, q), transpose=True)
    m2 = torch.ones(64, dtype=torch.float64)
    m2[:32] = rot.magnitude**2
    assert ((back.cpu().double() - q.cpu().double() * m2).abs() <= 8 * 8 * 2.0**-22).all()


def test_empty_and_special_values():
    rot = RotaryEmbedding()
    none = torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    assert rot.apply(torch.empty(0, dtype=torch.int32, device="cuda"), none).shape == none.shape
    assert N.oscar_last_launch_count() == 0
    x = torch.zeros(2, 1, 128, device="cuda")
    x[0, 0, 3], x[1, 0, 5] = float("nan"), float("inf")
    y = rot.apply(torch.tensor([1, 0], device="cuda"), x)
    bad = torch.isnan(y[0, 0]).nonzero().flatten().tolist()
    assert bad == [3, 67]  # a NaN stays in its pair
    assert y[1, 0, 5] == float("inf") and torch.isnan(y[1, 0, 69])  # inf * cos, inf * 0
    assert torch.isfinite(y[1, 0, torch.arange(128) % 64 != 5]).all()


def test_streams_and_graph():
    rot = RotaryEmbedding(base=1e6)
    q, k = inputs(6, 8, 2, 128, torch.bfloat16, 4)
    positions = torch.arange(6, device="cuda", dtype=torch.int32)
    want = rot.apply(positions, q, k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = rot.apply(positions, q, k, q_out=torch.empty_like(q), k_out=torch.empty_like(k), stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rot.apply(positions, q, k, q_out=q_out, k_out=k_out)
    positions += 1000
    q.mul_(2)
    graph.replay()
    again = rot.apply(positions, q, k)
    assert torch.equal(q_out, again[0]) and torch.equal(k_out, again[1])


def test_refusals():
    rot = RotaryEmbedding()
    q, k = inputs(4, 8, 2, 128, torch.bfloat16, 2)
    p = torch.arange(4, device="cuda")
    bad = [(p[:3], q, k, {}), (p.float(), q, k, {}), (p.cpu(), q, k, {}), (p, q[..., :64], k, {}), (p, q.double(), k, {}),
           (p, q, k.float(), {}), (p, q, k[:3], {}), (p, q.cpu(), None, {}), (p, q, None, dict(k_out=k)),
           (p, q, k, dict(q_out=q.float())), (p, q.transpose(1, 2), None, {}), (p[::2], q[:2], None, {}),
           (p, q, k, dict(q_out=q[:, :4]))]
    for positions, a, b, kw in bad:
        with pytest.raises(ValueError):
            rot.apply(positions, a, b, **kw)
    with pytest.raises(N.OscarError):  # every row the same memory
        rot.apply(p, q, q_out=q[:1].clone().expand(4, 8, 128))
