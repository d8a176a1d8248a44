"""Decode over 4-bit pages whose values differ widely in scale from token to token and group to group: what is hardly attended
costs the others nothing, whatever its scale.

Tolerance per head and channel of the fp32 output (derived, not fitted), with w the weights in 64 bits, v, s, z the values, scales
and zero points held, N the tokens.  A weight is off by a factor 1 + d, d = 2^-18 S + 2^-20, S = sum |q_c| (15 s + |z|) /
sqrt(128) (tests of the decode at uniform scales have the derivation), which moves an output by 2 d sum w |v| at most.  The
products of weight and scale are rounded to the 11 bits of fp16, 2^-11 of each at most, or, where they are subnormal there, to
2^-25 of a 64th of the largest product: 15 sum w s 2^-11 + 15 N 2^-31 max w s.  The fp32 sums add N 2^-26 sum w (15 s + |z|) (some N / 128
additions one after the other, 2^-23 each and a few more)."""
import math

import pytest
import torch

from int2_rotated_kv_rotate_gb300 import OSCAR_FORMAT_INT4, KVCache

pytestmark = pytest.mark.gpu


def decode(log2_weights, k, v, gqa, group, split):
    """Outputs and references of queries to whose scores k's rows, a[t] u with u of +-1, are proportional."""
    n = v.shape[0]
    c = KVCache(fmt=OSCAR_FORMAT_INT4, n_q_heads=gqa, n_kv_heads=1, group=group, max_requests=1, max_pages=-(-n // 64),
                max_pages_per_request=-(-n // 64))
    slot = c.alloc()
    c.reserve([slot], [n])
    c.append(0, k, v)
    c.commit()
    # heads with scores 1, 0.97, .. times the weights asked for
    span = float(log2_weights.abs().max())
    unit = k[int(log2_weights.abs().argmax()), 0].float().sign()
    q = (-unit * (span * math.log(2.0) * math.sqrt(128.0) / 128.0 / 8.0))[None] * (1 - 0.03 * torch.arange(gqa, device="cuda"))[:, None]
    q = q.bfloat16()
    c.plan([slot], max_split_pages=split)
    o32 = torch.empty(1, gqa, 128, device="cuda")
    c.decode(0, q[None], out_f32=o32)
    assert c.status() == (0, 0)
    held = [x[:, 0].double() for x in c.read(0, slot, 0, n, dtype=torch.float32)]
    return o32[0].double(), q.double(), held


def scales(x, group):
    y = x[:, 0].float().unflatten(-1, (-1, group))
    lo, hi = y.amin(-1), y.amax(-1)
    return ((hi - lo) / 15).bfloat16().double().repeat_interleave(group, -1), lo.double().abs().repeat_interleave(group, -1)


def check(log2_weights, v_scale, gqa, group, split, seed, v_group=None, label=""):
    n = log2_weights.shape[0]
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = torch.where(torch.arange(128, device="cuda") % 2 == 0, 1.0, -1.0)
    span = float(log2_weights.abs().max())
    k = (8.0 * log2_weights.abs().cuda() / span)[:, None, None] * u  # 0 at the peak, 8 at the least weight
    v = (1 + 0.5 * torch.randn(n, 1, 128, generator=g, device="cuda")) * v_scale.cuda()[:, None, None]
    if v_group is not None:
        v = v * v_group.cuda()
    k, v = k.bfloat16(), v.bfloat16()
    got, q, (kk, vv) = decode(log2_weights, k, v, gqa, group, split)
    sk, zk = scales(k, group)
    s, z = scales(v, group)
    w = torch.softmax(q @ kk.T / math.sqrt(128.0), -1)
    S = float((q.abs() @ (15 * sk + zk).T).max()) / math.sqrt(128.0)
    d = 2.0 ** -18 * S + 2.0 ** -20
    ws = w @ s
    most = (w[:, :, None] * s[None, :, ::group]).amax((1, 2))
    tol = 2 * d * (w @ vv.abs()) + 15 * 2.0 ** -11 * ws + 15 * n * 2.0 ** -31 * most[:, None] + n * 2.0 ** -26 * (15 * ws + w @ z)
    err = (got - w @ vv).abs()
    at = int((err / tol).argmax())
    assert bool((err <= tol).all()), f"{label} at {at // 128, at % 128}: {float(err.flatten()[at]):.3e} > {float(tol.flatten()[at]):.3e}"


CASES = pytest.mark.parametrize("gqa,group", [(4, 32), (4, 128), (8, 32), (8, 128)])


@CASES
@pytest.mark.parametrize("split", [0, 1000])
@pytest.mark.parametrize("n,light,ratio", [(1300, -16, 9), (1300, -13, 12), (12000, -15, 9), (1300, -11, 18), (5000, -12, 30)])
@pytest.mark.parametrize("every", [32, 100000])
def test_large_values_that_are_hardly_attended(gqa, group, split, n, light, ratio, every):
    """A peak of weight 1, many light tokens, and, first in their half pages, tokens of weight 2^-60 and 2^ratio times the scale."""
    lw = torch.full((n,), float(light))
    lw[0::every] = -60
    lw[min(40, n - 1)] = 0
    vs = torch.ones(n)
    vs[lw == -60] = 2.0 ** ratio
    check(lw, vs, gqa, group, split, n + ratio, label=f"2^{ratio}")


@CASES
@pytest.mark.parametrize("ratio", [6, 12, 20])
def test_large_values_that_lose_their_weight(gqa, group, ratio):
    """Scores that rise by 2^60 in steps while the values' scales fall, and steeply at once."""
    n = 4000
    lw = -60 + 60 * (torch.arange(n) / (n - 1.0))
    check(lw, 2.0 ** (ratio * (-lw / 60)), gqa, group, 1000, ratio)
    lw = torch.where(torch.arange(n) < 300, -45.0, torch.where(torch.arange(n) % 97 == 50, 0.0, -10.0))
    lw[5] = -60
    check(lw, torch.where(torch.arange(n) < 300, 2.0 ** ratio, 1.0), gqa, group, 1000, ratio + 1)


@CASES
@pytest.mark.parametrize("ratio", [8, 20, 40])
def test_a_heavy_token_of_small_values(gqa, group, ratio):
    """A first token that takes half the weight and has next to no values; the others' are far above it."""
    n = 3000
    lw = torch.full((n,), -11.0)
    lw[0], lw[1] = 0, -60
    vs = torch.ones(n)
    vs[0] = 2.0 ** -ratio
    for split in (0, 1000):
        check(lw, vs, gqa, group, split, ratio)


@pytest.mark.parametrize("gqa", [4, 8])
@pytest.mark.parametrize("ratio", [5, 9, 12])
def test_groups_of_different_scales(gqa, ratio):
    """A group of channels 2^ratio times the others in every token."""
    n = 4000
    lw = torch.full((n,), -13.0)
    lw[100], lw[7] = 0, -60
    vg = torch.ones(128)
    vg[64:96] = 2.0 ** ratio
    check(lw, torch.ones(n), gqa, 32, 1000, ratio, v_group=vg)
    check(lw, torch.ones(n), gqa, 32, 0, ratio, v_group=vg)


@CASES
def test_values_without_a_range(gqa, group):
    """Scales of zero (constant groups) before and between tokens that have one."""
    n = 700
    g = torch.Generator(device="cuda").manual_seed(3)
    lw = torch.full((n,), -6.0)
    lw[650], lw[3] = 0, -30
    u = torch.where(torch.arange(128, device="cuda") % 2 == 0, 1.0, -1.0)
    k = ((8.0 * lw.abs().cuda() / 30)[:, None, None] * u).bfloat16()
    v = (1 + 0.5 * torch.randn(n, 1, 128, generator=g, device="cuda"))
    v[:300], v[400:500] = 2.0, -1.0
    v = v.bfloat16()
    got, q, (kk, vv) = decode(lw, k, v, gqa, group, 1000)
    w = torch.softmax(q @ kk.T / math.sqrt(128.0), -1)
    # S < 2^7 here, so d < 2^-10; and 2^-11 of the ranges
    assert float((got - w @ vv).abs().max()) <= (2 * 2.0 ** -10 + 2.0 ** -11) * 2 * float(vv.abs().max())
