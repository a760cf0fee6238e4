"""GPU parity of la_cross_attention_forward / _backward against the 64-bit reference, with the bounds of
dit_reference.py: one query and many, one state and many, lengths of zero, one, tile edges and out of range,
k and v as views of one tensor, NaN behind the lengths, large scores."""
import math

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


def draw(B, N, M, H, d, dtype, fused, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    t = lambda *s: (std * torch.randn(s, generator=g)).to(dtype).cuda()  # noqa: E731
    q, dout = t(B, N, H, d), (torch.randn(B, N, H, d, generator=g)).to(dtype).cuda()
    if fused:
        kv = t(B, M, 2, H, d)
        return q, kv[:, :, 0], kv[:, :, 1], dout
    return q, t(B, M, H, d), t(B, M, H, d), dout


def run_case(la, q, k, v, dout, lens, dtype, scale=None):
    B, N, H, d = q.shape
    M = k.shape[1]
    sc = d ** -0.5 if scale is None else scale
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    held = [M] * B if lens is None else [min(max(n, 0), M) for n in lens]
    out, lse = la.cross_attention_forward(q, k, v, kv_len=ln, scale=scale, return_lse=True)
    # what lies behind the lengths is never used: the reference gets zeros there
    kz, vz = k.clone(), v.clone()
    for b, n in enumerate(held):
        kz[b, n:] = 0
        vz[b, n:] = 0
    ro, rl, so, sl = ref.cross_forward(q, kz, vz, held, sc, dtype)
    ref.check("out", out, ro, so, dtype)
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), empty) and (lse[empty] < 0).all()
    ref.check("lse", lse.masked_fill(empty, 0), rl.masked_fill(empty, 0), sl, F32)
    assert torch.equal(la.cross_attention_forward(q, k, v, kv_len=ln, scale=scale), out)
    if dout is None:
        return out, lse, None
    got = la.cross_attention_backward(q, k, v, out, lse, dout, kv_len=ln, scale=scale)
    want = ref.cross_backward(q, kz, vz, out, lse.masked_fill(empty, 0), dout, held, sc, dtype)
    for name, g, (r, s) in zip(("dq", "dk", "dv"), got, want):
        ref.check(name, g, r, s, dtype)
    for b, n in enumerate(held):
        assert not got[1][b, n:].any() and not got[2][b, n:].any()
        if n == 0:
            assert not out[b].any() and not got[0][b].any()
    again = la.cross_attention_backward(q, k, v, out, lse, dout, kv_len=ln, scale=scale)
    assert all(torch.equal(a, c) for a, c in zip(got, again))
    return out, lse, got


CASES = [  # B, N, M, H, d, dtype, fused, lengths
    (1, 1, 1, 1, 32, BF, False, None), (1, 1, 1, 1, 64, F32, False, None), (2, 1, 300, 4, 32, BF, True, [300, 17]),
    (1, 1, 4096, 8, 32, BF, True, None), (1, 3, 1030, 4, 64, BF, False, None), (2, 2, 700, 3, 64, BF, True, [0, 513]),
    (1, 128, 128, 2, 32, BF, False, None), (1, 129, 129, 2, 64, BF, True, None), (2, 130, 64, 3, 32, BF, True, [64, 63]),
    (3, 257, 300, 4, 32, BF, True, [300, 0, 1]), (2, 300, 77, 5, 64, BF, False, [76, 65]),
    (4, 200, 512, 2, 32, BF, True, [512, 385, 384, 128]), (2, 390, 513, 2, 32, BF, False, [513, 512]),
    (2, 500, 1100, 1, 64, BF, True, [1100, 700]), (1, 1000, 33, 4, 32, BF, True, [-5]), (2, 64, 40, 2, 64, BF, False, [99, 7]),
    (1, 2000, 300, 1, 64, BF, True, None), (2, 31, 16, 2, 32, BF, True, [15, 16]), (3, 700, 2, 3, 64, BF, True, [2, 0, 1]), (2, 1300, 17, 30, 32, BF, False, [0, 17]), (1, 260, 257, 20, 32, BF, True, None),
    (1, 8, 200, 2, 32, BF, True, None), (1, 9, 200, 2, 64, BF, True, None), (2, 5, 260, 3, 64, BF, False, [260, 0]),
    (1, 385, 150, 3, 32, BF, True, None), (1, 769, 65, 2, 64, BF, True, None), (2, 100, 2100, 2, 32, BF, True, [2100, 900]),
    (1, 300, 3000, 1, 64, BF, True, None), (3, 1300, 130, 2, 32, BF, True, [130, 128, 2]), (40, 130, 66, 1, 32, BF, True, None),
    (2, 77, 40, 3, 32, F32, True, [40, 9]), (1, 391, 77, 8, 64, F32, False, None), (2, 130, 70, 2, 64, F32, True, [0, 70]),
    (1, 1, 500, 4, 32, F32, True, None), (3, 64, 5, 2, 32, F32, False, [5, 1, 12]),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_cross_matches_reference(la, case):
    B, N, M, H, d, dtype, fused, lens = case
    q, k, v, dout = draw(B, N, M, H, d, dtype, fused, seed=N + 3 * M + H)
    run_case(la, q, k, v, dout, lens, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,M", [(2, 150), (140, 150), (140, 90)])
def test_nothing_behind_the_lengths_is_used(la, dtype, N, M):
    q, k, v, dout = draw(3, N, M, 2, 32, dtype, True, 1)
    lens = [M, 2 * M // 3, 3]
    k, v = k.clone(), v.clone()
    plain = run_case(la, q, k, v, dout, lens, dtype)
    for b, n in enumerate(lens):
        k[b, n:] = math.nan
        v[b, n:] = math.inf
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = la.cross_attention_forward(q, k, v, kv_len=ln, return_lse=True)
    got = la.cross_attention_backward(q, k, v, out, lse, dout, kv_len=ln)
    assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])
    assert all(torch.equal(a, c) for a, c in zip(got, plain[2]))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [1, 150])
def test_large_scores(la, dtype, N):
    """Scores of hundreds, rising along the states so that the running maximum keeps moving, falling so that the
    first state wins, and all equal."""
    q, k, v, dout = draw(1, N, 200, 2, 32, dtype, False, 2)
    q.fill_(4.0)
    ramp = torch.linspace(-6, 6, 200, device="cuda").to(dtype)[None, :, None, None]
    for kk in (ramp, -ramp, torch.zeros_like(ramp)):
        run_case(la, q, kk.expand_as(k).contiguous(), v, dout, None, dtype, scale=0.5)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradients_into_a_wider_tensor(la, dtype):
    """dk and dv written into one [B, M, 2, H, d] tensor, as the fused projection's backward pass takes it."""
    q, k, v, dout = draw(2, 140, 90, 2, 64, dtype, True, 3)
    out, lse = la.cross_attention_forward(q, k, v, return_lse=True)
    want = la.cross_attention_backward(q, k, v, out, lse, dout)
    dkv = torch.full((2, 91, 2, 2, 64), 7.0, dtype=dtype, device="cuda")[:, :90]
    with pytest.raises(ValueError):     # batch elements 91 states apart: not this layout
        la.cross_attention_backward(q, k, v, out, lse, dout, grads=(torch.empty_like(q), dkv[:, :, 0], dkv[:, :, 1]))
    dkv = torch.full((2, 90, 3, 2, 64), 7.0, dtype=dtype, device="cuda")
    dq = torch.empty_like(q)
    la.cross_attention_backward(q, k, v, out, lse, dout, grads=(dq, dkv[:, :, 0], dkv[:, :, 2]))
    assert torch.equal(dq, want[0]) and torch.equal(dkv[:, :, 0], want[1]) and torch.equal(dkv[:, :, 2], want[2])
    assert (dkv[:, :, 1] == 7).all()


@pytest.mark.parametrize("scale", [1e-20, 1e-4, 30.0])
def test_scales(la, scale):
    """Scales from the smallest taken (all states alike) to one that leaves one state a query."""
    q, k, v, dout = draw(2, 140, 130, 2, 32, BF, True, 9)
    run_case(la, q, k, v, dout, [130, 77], BF, scale=scale)


def test_gradient_against_differences(la):
    """fp32: the loss's change along random directions against the gradients."""
    q, k, v, dout = draw(1, 40, 30, 2, 32, F32, False, 6)
    out, lse = la.cross_attention_forward(q, k, v, return_lse=True)
    grads = la.cross_attention_backward(q, k, v, out, lse, dout)
    for i, g in enumerate(grads):
        dirn = torch.randn(g.shape, generator=torch.Generator().manual_seed(i)).cuda()
        h, loss = 1e-2, []
        for sgn in (1, -1):
            t = [q, k, v]
            t[i] = t[i] + sgn * h * dirn
            loss.append((la.cross_attention_forward(*t).double() * dout.double()).sum())
        num, ana = (loss[0] - loss[1]) / (2 * h), (g.double() * dirn.double()).sum()
        # second-order differences: h^2 / 6 of the third derivative, which scores of order one keep below 100
        # times the gradient's norm; fp32 outputs of order one, 2560 of them, over 2h
        assert abs(num - ana) <= 100 * h * h / 6 * g.double().norm() + 2560 ** 0.5 * 2.0 ** -22 / h


def test_one_sample_at_a_time(la):
    """Each batch element's results are those of a call of its own, whatever the others hold."""
    q, k, v, dout = draw(3, 150, 140, 2, 32, BF, True, 8)
    ln = torch.tensor([140, 13, 77], dtype=torch.int32, device="cuda")
    out, lse = la.cross_attention_forward(q, k, v, kv_len=ln, return_lse=True)
    for b in range(3):
        s = slice(b, b + 1)
        o, ls = la.cross_attention_forward(q[s], k[s], v[s], kv_len=ln[s], return_lse=True)
        assert torch.equal(o, out[s]) and torch.equal(ls, lse[s])
