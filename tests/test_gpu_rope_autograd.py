"""Rotary positions under autograd: gradients by the transposed map, and refusals."""
import pytest
import torch

from int2_rotated_kv_rotate_gb300 import RotaryEmbedding

from test_gpu_rope import DTYPES, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_autograd(dtype, interleaved):
    """Inputs that need gradients get them: those of the transposed map, bit for bit, for queries
    and keys, broadcast and strided ones too; a second pass through the gradient as well."""
    rot = RotaryEmbedding(rotary_dim=96, base=1e6, interleaved=interleaved,
                          scaling=dict(type="yarn", factor=4.0, original_context=4096))
    q, k = inputs(7, 6, 2, 128, DTYPES[dtype], 31)
    gq, gk = inputs(7, 6, 2, 128, DTYPES[dtype], 32)
    positions = torch.arange(7, device="cuda") + 5000
    want = rot.apply(positions, gq, gk, transpose=True)
    q.requires_grad_()
    k.requires_grad_()
    oq, ok = rot.apply(positions, q, k)
    with torch.no_grad():
        assert torch.equal(oq, rot.apply(positions, q)) and torch.equal(ok, rot.apply(positions, k))
    a, b = torch.autograd.grad((oq, ok), (q, k), (gq, gk))
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    # one of the two, a gradient that is one number for all, channels that are not contiguous
    a, = torch.autograd.grad(rot.apply(positions, q, k.detach())[0].sum(), (q,))
    assert torch.equal(a, rot.apply(positions, torch.ones_like(q), transpose=True))
    turned = gq.transpose(1, 2).contiguous().transpose(1, 2)
    a, = torch.autograd.grad(rot.apply(positions, q), (q,), (turned,))
    assert torch.equal(a, want[0])
    # the keys alone reach the loss: the queries' gradient is zero
    oq, ok = rot.apply(positions, q, k)
    a, b = torch.autograd.grad((ok * gk).sum(), (q, k), allow_unused=True)
    assert torch.equal(b, want[1]) and (a is None or bool((a == 0).all()))
    # the gradient's gradient is the map itself
    g = gq.clone().requires_grad_()
    a, = torch.autograd.grad(rot.apply(positions, q), (q,), (g,), create_graph=True)
    again, = torch.autograd.grad(a, (g,), (gq,))
    assert torch.equal(again, rot.apply(positions, gq))


def test_autograd_on_another_stream_and_refusals():
    rot = RotaryEmbedding()
    q, k = inputs(5, 4, 2, 128, torch.float32, 8)
    positions = torch.arange(5, device="cuda")
    g = torch.randn_like(q)
    want = rot.apply(positions, g, transpose=True)
    q.requires_grad_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = rot.apply(positions, q, stream=side)
    side.synchronize()
    a, = torch.autograd.grad(out, (q,), (g,))
    torch.cuda.synchronize()
    assert torch.equal(a, want)
    leaf = q.detach().clone().requires_grad_()
    for args, kw in (((leaf,), dict(q_out=leaf)), ((leaf,), dict(q_out=torch.empty_like(leaf))),
                     ((leaf, k), dict(k_out=k)), ((k.detach(), leaf), dict(q_out=k))):
        before = leaf.detach().clone()
        with pytest.raises(ValueError, match="grad"):
            rot.apply(positions, *args, **kw)
        assert torch.equal(leaf, before)
    with torch.no_grad():
        rot.apply(positions, leaf, q_out=leaf)
    # a positions tensor that changes before the backward pass is an error, not a wrong gradient
    p = positions.clone()
    out = rot.apply(p, q)
    p.add_(1)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(out, (q,), (g,))


def test_given_outputs_count_as_written():
    """A graph that saved a tensor which a later call overwrites fails instead of using it."""
    rot = RotaryEmbedding()
    q, k = inputs(5, 4, 2, 128, torch.float32, 9)
    positions = torch.arange(5, device="cuda") + 3
    w = torch.ones_like(q).requires_grad_()
    loss = (w * q).sum()
    rot.apply(positions, q, k, q_out=q)
    with pytest.raises(RuntimeError):
        loss.backward()
    version = k._version
    rot.apply(positions, q, k)
    assert k._version == version


def test_gradients_against_differences():
    """<g, rope(x)> by central differences of the linear map: the two outputs round within
    2^-24 |y| + 3 * 2^-23 * (|a| + |b|) each, |x| and |g| under 6, h = 1."""
    rot = RotaryEmbedding(head_dim=16, rotary_dim=8, base=10.0)
    q, g = inputs(3, 2, 2, 16, torch.float32, 5)
    positions = torch.tensor([0, 3, 900], device="cuda")
    q.requires_grad_()
    (rot.apply(positions, q) * g).sum().backward()
    with torch.no_grad():
        for row, head, ch in ((0, 0, 0), (1, 1, 5), (2, 0, 7), (2, 1, 12)):
            e = torch.zeros_like(q)
            e[row, head, ch] = 1.0
            d = ((rot.apply(positions, q + e).double() - rot.apply(positions, q - e).double()) * g.double()).sum() / 2
            # two channels of either output change: 2 * 2 * (2^-24 * 12 + 3 * 2^-23 * 14) * 6 / 2, and q +- e round
            assert abs(float(d) - float(q.grad[row, head, ch])) <= 12 * (2.0**-24 * 12 + 3 * 2.0**-23 * 14) + 24 * 2.0**-22


def test_a_captured_step_with_its_gradient():
    """Forward and backward captured into one graph, replayed on other inputs."""
    rot = RotaryEmbedding(base=1e6)
    q, k = inputs(9, 4, 2, 128, torch.float32, 6)
    gq, gk = inputs(9, 4, 2, 128, torch.float32, 7)
    positions = torch.arange(9, device="cuda")
    q.requires_grad_()
    k.requires_grad_()

    def step():
        return torch.autograd.grad(rot.apply(positions, q, k), (q, k), (gq, gk))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    gq.mul_(-3)
    gk.add_(1)
    positions.add_(77)
    graph.replay()
    want = rot.apply(positions, gq, gk, transpose=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
