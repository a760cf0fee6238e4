"""GPU parity of la_linear_forward / _backward against the 64-bit reference, with the bounds of
dit_reference.py: one row to many, widths of one, odd widths, tile edges, every activation with and without
bias and residual, the residual updated in place."""
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


def draw(R, K, N, dtype, bias, res, seed):
    g = torch.Generator().manual_seed(seed)
    t = lambda *s, std=1.0: (std * torch.randn(s, generator=g)).to(dtype).cuda()  # noqa: E731
    return (t(R, K), t(N, K, std=K ** -0.5), t(N, std=0.3) if bias else None, t(R, N) if res else None, t(R, N))


CASES = [  # R, K, N, dtype, act, bias, residual
    (1, 1, 1, BF, "none", True, False), (1, 1, 1, F32, "silu", True, True), (3, 2, 5, BF, "gelu", False, True),
    (1, 2048, 512, BF, "none", True, False), (2, 2048, 1000, BF, "silu", True, False),
    (4, 512, 96, BF, "gelu", True, True), (8, 256, 264, BF, "relu", False, False), (9, 264, 136, BF, "silu", True, True),
    (2, 513, 77, BF, "none", True, True), (7, 65, 300, BF, "relu", True, False),
    (127, 64, 128, BF, "none", False, False), (128, 64, 256, BF, "silu", True, False),
    (129, 72, 264, BF, "gelu", True, True), (300, 2048, 192, BF, "none", True, True),
    (257, 1000, 520, BF, "relu", True, True), (640, 320, 72, BF, "silu", False, True),
    (100, 63, 65, BF, "gelu", True, True), (333, 130, 1, BF, "none", True, False), (333, 1, 130, BF, "silu", True, True),
    (1030, 264, 776, BF, "silu", True, True), (2500, 128, 64, BF, "none", True, False),
    (2700, 640, 2048, BF, "silu", True, True), (2305, 264, 2056, BF, "gelu", True, True),   # whole waves and tail tiles
    (40, 4104, 200, BF, "gelu", True, False), (20, 200, 4104, BF, "none", False, True),
    (1, 70, 300, F32, "gelu", True, False), (5, 33, 17, F32, "relu", True, True), (130, 127, 129, F32, "silu", True, True),
    (300, 256, 384, F32, "none", True, True), (513, 100, 64, F32, "gelu", False, True), (64, 2000, 40, F32, "none", True, False),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_linear_matches_reference(la, case):
    R, K, N, dtype, act, bias, res = case
    x, w, b, r, dy = draw(R, K, N, dtype, bias, res, seed=R + 3 * K + 7 * N)
    y, pre = la.linear_forward(x, w, b, act=act, residual=r, return_pre=True)
    ry, rz, sy, sz = ref.linear_forward(x, w, b, act, r)
    ref.check("y", y, ry, sy, dtype)
    assert (pre is None) == (act == "none")
    if pre is not None:
        assert pre.dtype == (torch.float16 if dtype is BF else F32)
        ref.check("pre", pre, rz, sz + ref.PRE_ABS, pre.dtype)
    assert torch.equal(la.linear_forward(x, w, b, act=act, residual=r), y)
    got = la.linear_backward(dy, x, w, pre=pre, act=act)
    for name, g, (want, s) in zip(("dx", "dw", "db"), got, ref.linear_backward(dy, x, w, pre, act, dtype)):
        ref.check(name, g, want, s, dtype)
    again = la.linear_backward(dy, x, w, pre=pre, act=act)
    assert all(torch.equal(a, c) for a, c in zip(got, again))


@pytest.mark.parametrize("R", [3, 200])
def test_linear_parts(la, R):
    """One gradient alone, z asked for without an activation, the residual updated in place, and an input of
    more dimensions."""
    x, w, b, r, dy = draw(R, 136, 200, BF, True, True, 11)
    y, pre = la.linear_forward(x, w, b, act="silu", residual=r, return_pre=True)
    full = la.linear_backward(dy, x, w, pre=pre, act="silu")
    for i in range(3):
        want = [j == i for j in range(3)]
        got = la.linear_backward(dy, x, w, pre=pre, act="silu", input_grad=want[0], weight_grad=want[1],
                                 bias_grad=want[2])
        assert [g is not None for g in got] == want and torch.equal(got[i], full[i])
    z = torch.empty_like(y, dtype=torch.float16)
    la.linear_forward(x, w, b, return_pre=True, pre=z)
    _, rz, _, sz = ref.linear_forward(x, w, b, "none", None)
    ref.check("pre", z, rz, sz + ref.PRE_ABS, z.dtype)
    inplace = r.clone()
    la.linear_forward(x, w, b, act="silu", residual=inplace, out=inplace)
    assert torch.equal(inplace, y)
    more = la.linear_forward(x.view(1, R, 1, 136), w, b, act="silu", residual=r.view(1, R, 1, 200))
    assert more.shape == (1, R, 1, 200) and torch.equal(more.view_as(y), y)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_activations_far_out(la, act, dtype):
    """z from -90 to 90 through an identity: the activations' tails and slopes neither overflow nor turn to NaN."""
    z = torch.linspace(-90, 90, 721).to(dtype).cuda()
    x, w = z[:, None].contiguous(), torch.ones(1, 1, dtype=dtype, device="cuda")
    y, pre = la.linear_forward(x, w, act=act, return_pre=True)
    ry, _, sy, _ = ref.linear_forward(x, w, None, act, None)
    ref.check("y", y, ry, sy, dtype)
    dx, _, _ = la.linear_backward(torch.ones_like(y), x, w, pre=pre, act=act)
    (rdx, sdx), _, _ = ref.linear_backward(torch.ones_like(y), x, w, pre, act, dtype)
    ref.check("dx", dx, rdx, sdx, dtype)


def test_fp32_over_the_whole_range(la):
    """fp32 operands from 1e-30 to the largest finite value: exponents far apart in one row, and products that
    come back to order one."""
    g = torch.Generator().manual_seed(5)
    R, K, N = 150, 48, 70
    e = torch.randint(-30, 31, (R, 1), generator=g).double()
    x = (torch.randn(R, K, generator=g).double() * 10.0 ** e).to(F32).cuda()
    w = torch.randn(N, K, generator=g).to(F32).cuda()
    y = la.linear_forward(x, w)
    ry, _, sy, _ = ref.linear_forward(x, w, None, "none", None)
    ref.check("y", y, ry, sy, F32)
    big = torch.zeros(R, K, device="cuda")
    big[:, 0] = torch.finfo(F32).max
    small = torch.zeros(N, K, device="cuda")
    small[:, 0] = 2.0 ** -100
    y = la.linear_forward(big, small)
    ry, _, sy, _ = ref.linear_forward(big, small, None, "none", None)
    ref.check("y", y, ry, sy, F32)


def test_slopes_of_huge_inputs(la):
    """Activations and slopes at +-1e30: the identity or zero, never NaN."""
    x, w = torch.tensor([[1e30], [-1e30]], device="cuda"), torch.ones(1, 1, device="cuda")
    for act in ("relu", "silu", "gelu"):
        y, pre = la.linear_forward(x, w, act=act, return_pre=True)
        dx, _, _ = la.linear_backward(torch.ones_like(y), x, w, pre=pre, act=act)
        assert y[0] == 1e30 and y[1] == 0 and dx[0] == 1 and dx[1] == 0


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_slopes_at_the_ends_of_fp16(la, act, rows):
    """bf16 z beyond fp16's range, and below its smallest number: the slopes are those of z."""
    z = torch.tensor([1e30, 1e6, 7e4, 6e4, 1e-9, 1e-30, 0.0, -0.0, -1e-30, -1e-9, -6e4, -7e4, -1e6, -1e30],
                     dtype=BF, device="cuda")
    x, w = torch.ones(rows, 1, dtype=BF, device="cuda"), z[:, None].contiguous()
    y, pre = la.linear_forward(x, w, act=act, return_pre=True)
    assert pre.isfinite().all() and pre.abs().max() == 65504
    got = la.linear_backward(torch.ones_like(y), x, w, pre=pre, act=act)[2]      # db: the slopes' sums over the rows
    slope = ref.act(z.double().clamp(-100, 100), act)[1]
    ref.check("db", got, rows * slope, rows * (ref.half(BF) + ref.ACT_REL + 1e-6), BF)


def test_linear_writes_only_its_outputs(la):
    x, w, b, r, _ = draw(130, 64, 72, BF, True, True, 4)
    buf = torch.full((132, 72), 7.0, dtype=BF, device="cuda")
    la.linear_forward(x, w, b, out=buf[1:131])
    assert (buf[0] == 7).all() and (buf[131] == 7).all()
