"""The 64-bit references of layer norm, linear and cross attention on the CPU: their gradients against autograd
of the definitions and against differences of their own forward passes."""
import pytest
import torch

import dit_reference as ref

D = torch.float64


def rnd(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed + sum(shape)), dtype=D)


def numeric(f, x, dy, h=1e-6):
    """Central differences of sum(f(x) * dy)."""
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        e = torch.zeros_like(x).view(-1)
        e[i] = h
        e = e.view_as(x)
        g.view(-1)[i] = ((f(x + e) - f(x - e)) * dy).sum() / (2 * h)
    return g


@pytest.mark.parametrize("per_batch", [False, True])
def test_norm_gradients(per_batch):
    x, dy = rnd(2, 3, 5), rnd(2, 3, 5, seed=1)
    w, b = (rnd(2, 5, seed=2), rnd(2, 5, seed=3)) if per_batch else (rnd(5, seed=2), rnd(5, seed=3))
    y, mean, rstd, *_ = ref.norm_forward(x, w, b, 1e-6)
    if not per_batch:
        assert torch.allclose(y, torch.nn.functional.layer_norm(x, (5,), w, b, 1e-6), atol=1e-12)
    (dx, _), (dw, _), (db, _) = ref.norm_backward(dy, x, w, mean, rstd, per_batch)
    for got, f, at in ((dx, lambda t: ref.norm_forward(t, w, b, 1e-6)[0], x),
                       (dw, lambda t: ref.norm_forward(x, t, b, 1e-6)[0], w),
                       (db, lambda t: ref.norm_forward(x, w, t, 1e-6)[0], b)):
        assert torch.allclose(got, numeric(f, at, dy), atol=1e-7)


@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu"])
def test_linear_gradients(name):
    x, w, b, res, dy = rnd(4, 3), rnd(5, 3, seed=1), rnd(5, seed=2), rnd(4, 5, seed=3), rnd(4, 5, seed=4)
    y, z, _, _ = ref.linear_forward(x, w, b, name, res)
    t = torch.nn.functional.linear(x, w, b)
    want = {"none": lambda a: a, "relu": torch.relu, "silu": torch.nn.functional.silu,
            "gelu": lambda a: torch.nn.functional.gelu(a, approximate="tanh")}[name](t) + res
    assert torch.allclose(y, want, atol=1e-12)
    (dx, _), (dw, _), (db, _) = ref.linear_backward(dy, x, w, z, name, D)
    for got, f, at in ((dx, lambda t: ref.linear_forward(t, w, b, name, res)[0], x),
                       (dw, lambda t: ref.linear_forward(x, t, b, name, res)[0], w),
                       (db, lambda t: ref.linear_forward(x, w, t, name, res)[0], b)):
        assert torch.allclose(got, numeric(f, at, dy), atol=1e-7)


def test_cross_gradients():
    q, k, v, dy = rnd(3, 2, 2, 3), rnd(3, 4, 2, 3, seed=1), rnd(3, 4, 2, 3, seed=2), rnd(3, 2, 2, 3, seed=3)
    lens, scale, f32 = [4, 0, 2], 0.7, torch.float32
    out, lse, _, _ = ref.cross_forward(q, k, v, lens, scale, f32)
    for b, n in enumerate(lens):
        if n:
            want = torch.nn.functional.scaled_dot_product_attention(
                *(t[b].transpose(0, 1) for t in (q, k[:, :n], v[:, :n])), scale=scale).transpose(0, 1)
            assert torch.allclose(out[b], want, atol=1e-12)
    assert out[1].abs().max() == 0 and torch.isinf(lse[1]).all()
    grads = [g for g, _ in ref.cross_backward(q, k, v, out, lse, dy, lens, scale, f32)]
    fwd = lambda *a: ref.cross_forward(*a, lens, scale, f32)[0]  # noqa: E731
    for got, f, at in ((grads[0], lambda t: fwd(t, k, v), q), (grads[1], lambda t: fwd(q, t, v), k),
                       (grads[2], lambda t: fwd(q, k, t), v)):
        assert torch.allclose(got, numeric(f, at, dy), atol=1e-7)
    assert grads[0][1].abs().max() == 0 and grads[1][1].abs().max() == 0 and grads[2][2, 2:].abs().max() == 0
