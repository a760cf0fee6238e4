"""GPU parity of la_layer_norm_forward / _backward against the 64-bit reference, with the bounds of
dit_reference.py: every vector path (widths that are and are not whole vectors, one channel, wider than a
CTA's registers), one row and many, weights per channel and per batch element, absent ones, large offsets."""
import pytest
import torch

import dit_reference as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def la():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_causal_linear_b200 import build

    build.build()
    from block_causal_linear_b200 import la as _la

    return _la


def draw(B, N, C, dtype, vec, seed, offset=0.5):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(B, N, C, generator=g) + offset * torch.randn(C, generator=g)).to(dtype).cuda()
    dy = torch.randn(B, N, C, generator=g).to(dtype).cuda()
    shape = {"channel": (C,), "batch": (B, C)}.get(vec)
    w = b = None
    if shape:
        w = (1 + 0.2 * torch.randn(shape, generator=g)).to(dtype).cuda()
        b = (0.2 * torch.randn(shape, generator=g)).to(dtype).cuda()
    return x, dy, w, b


CASES = [  # B, N, C, dtype, vectors
    (1, 1, 1, BF, "channel"), (1, 1, 1, F32, "none"), (3, 5, 2, F32, "batch"),
    (2, 1, 2048, BF, "channel"), (2, 3, 32, BF, "batch"), (2, 130, 64, F32, "channel"),
    (1, 77, 250, BF, "channel"), (2, 33, 1001, F32, "batch"), (3, 19, 1001, BF, "none"),
    (2, 301, 2048, BF, "batch"), (1, 190, 2048, F32, "channel"), (2, 65, 2056, BF, "batch"),
    (1, 40, 5120, BF, "channel"), (2, 21, 5119, BF, "batch"), (1, 9, 8200, F32, "channel"),
    (1, 3, 20000, BF, "channel"), (2, 2, 33333, F32, "batch"), (4, 700, 96, BF, "batch"),
    (1, 7200, 2048, BF, "channel"), (2400, 3, 1024, BF, "batch"), (3, 2500, 768, F32, "batch"),     # rings of rows
    (1, 40, 8192, F32, "channel"), (2, 70, 4096, BF, "batch"), (3, 1, 8192, BF, "batch"),
    (1, 5000, 40, BF, "none"), (5, 260, 512, F32, "none"), (1, 2500, 1152, BF, "channel"),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_norm_matches_reference(la, case):
    B, N, C, dtype, vec = case
    x, dy, w, b = draw(B, N, C, dtype, vec, seed=B * 1000 + N + C)
    eps = 1e-6
    y, mean, rstd = la.layer_norm_forward(x, w, b, eps, return_stats=True)
    ry, rm, rr, sy, sm, sr = ref.norm_forward(x, w, b, eps)
    ref.check("y", y, ry, sy, dtype)
    ref.check("mean", mean, rm, sm, F32)
    ref.check("rstd", rstd, rr, sr, F32)
    assert torch.equal(la.layer_norm_forward(x, w, b, eps), y)
    per_batch = vec == "batch"
    got = la.layer_norm_backward(dy, x, w, mean, rstd)
    want = ref.norm_backward(dy, x, w, mean, rstd, per_batch)
    for name, g, (r, s) in zip(("dx", "dw", "db"), got, want):
        ref.check(name, g, r, s, dtype)
    again = la.layer_norm_backward(dy, x, w, mean, rstd)
    assert all(torch.equal(a, c) for a, c in zip(got, again))


def test_norm_parts_alone(la):
    """A bias without a weight, a gradient of one vector alone, sums per batch element without a weight, and a
    two-dimensional input."""
    x, dy, w, b = draw(3, 50, 264, BF, "channel", 5)
    y, mean, rstd = la.layer_norm_forward(x, None, b, return_stats=True)
    ry, _, _, sy, _, _ = ref.norm_forward(x, None, b, 1e-6)
    ref.check("y", y, ry, sy, BF)
    full = la.layer_norm_backward(dy, x, w, mean, rstd)
    dx, dw, none = la.layer_norm_backward(dy, x, w, mean, rstd, bias_grad=False)
    assert none is None and torch.equal(dx, full[0]) and torch.equal(dw, full[1])
    dx, none, db = la.layer_norm_backward(dy, x, w, mean, rstd, weight_grad=False)
    assert none is None and torch.equal(dx, full[0]) and torch.equal(db, full[2])
    dx, n1, n2 = la.layer_norm_backward(dy, x, w, mean, rstd, weight_grad=False, bias_grad=False)
    assert n1 is None and n2 is None and torch.equal(dx, full[0])
    got = la.layer_norm_backward(dy, x, None, mean, rstd, per_batch=True)
    for name, g, (r, s) in zip(("dx", "dw", "db"), got, ref.norm_backward(dy, x, None, mean, rstd, True)):
        ref.check(name, g, r, s, BF)
    flat = la.layer_norm_forward(x.view(150, 264), None, b)
    assert torch.equal(flat.view_as(y), y)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_of_constant_and_far_rows(la, dtype):
    """Equal channels (variance 0, y = bias), one huge outlier, and a mean 100 times the deviation."""
    x, dy, w, b = draw(1, 4, 512, dtype, "channel", 9, offset=0.0)
    x[0, 0] = 3.0
    x[0, 1, 7] = 30000.0
    x[0, 2] += 100.0
    y, mean, rstd = la.layer_norm_forward(x, w, b, return_stats=True)
    ry, _, _, sy, _, _ = ref.norm_forward(x, w, b, 1e-6)
    ref.check("y", y, ry, sy, dtype)
    assert torch.equal(y[0, 0], b)
    for name, g, (r, s) in zip(("dx", "dw", "db"), la.layer_norm_backward(dy, x, w, mean, rstd),
                               ref.norm_backward(dy, x, w, mean, rstd, False)):
        ref.check(name, g, r, s, dtype)


def test_norm_writes_only_its_rows(la):
    x, dy, w, b = draw(1, 37, 72, BF, "channel", 3)
    buf = torch.full((39, 72), 7.0, dtype=BF, device="cuda")
    la.layer_norm_forward(x, w, b, out=buf[1:38].view(1, 37, 72))
    assert (buf[0] == 7).all() and (buf[38] == 7).all()
