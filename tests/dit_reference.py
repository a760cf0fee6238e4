"""64-bit references of layer norm, linear and cross attention, and the error
bounds that their kernels are held to.

Every bound is |got - ref| <= h |ref| + slack, element by element: h is half a
step of the output's type (its one rounding), and slack counts the arithmetic
before it.  A sum of n products in fp32, in any order, is off by at most
n u sum|terms| with u = 2^-24 (Higham, Accuracy and Stability of Numerical
Algorithms, ch. 3); tensor-core sums may cut instead of rounding, so u = 2^-23
is used throughout.  Operands that are rounded to bf16 first (the softmax's p
and ds, and dz behind an activation) add half a bf16 step of each term.
"""
import math

import torch

U = 2.0 ** -23


def half(dtype):
    return torch.finfo(dtype).eps / 2


def check(name, got, ref, slack, dtype):
    """Asserts the bound above; NaN anywhere in got fails."""
    got = got.detach().double().cpu()
    ref, slack = ref.cpu(), slack.cpu() if torch.is_tensor(slack) else slack
    assert got.shape == ref.shape, f"{name}: shape {tuple(got.shape)}, not {tuple(ref.shape)}"
    room = half(dtype) * ref.abs() * (1 + half(dtype)) + slack + 1e-37
    off = (got - ref).abs()
    bad = ~(off <= room)
    if bad.any():
        i = (off / room).nan_to_num(math.inf).argmax().item()
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst at {i}: got "
                             f"{got.flatten()[i]}, ref {ref.flatten()[i]}, room {room.flatten()[i]}")


# ---------------------------------------------------------------- layer norm

def norm_forward(x, w, b, eps):
    """y, mean, rstd and y's slack; x [B, N, C], w and b [C], [B, C] or None."""
    x = x.double()
    C = x.shape[-1]
    w, b = (None if t is None else (t.double()[:, None] if t.dim() == 2 else t.double()) for t in (w, b))
    mean = x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((x - mean).square().mean(-1, keepdim=True) + eps)
    xh = (x - mean) * rstd
    y = xh if w is None else xh * w
    y = y if b is None else y + b
    # the mean is off by at most (its longest chain of additions) u mean|x|: a chain of C / 32 + 16 covers
    # every split of the row over at least a warp; the deviation inherits that, and a relative error of the
    # variance (same chain, and twice the deviations') half of it
    chain = C / 32 + 16
    dmean = chain * U * x.abs().mean(-1, keepdim=True)
    dxh = (dmean + U * x.abs()) * rstd
    rel = (chain * U + 2 * dmean * rstd)
    slack = (dxh + xh.abs() * (rel + 4 * U)) * (1 if w is None else w.abs())
    if b is not None:
        slack = slack + 2 * U * (b.abs() + y.abs())
    return y, mean[..., 0], rstd[..., 0], slack, dmean[..., 0], (rstd * rel)[..., 0] + 2 * U * rstd[..., 0]


def norm_backward(dy, x, w, mean, rstd, per_batch):
    """dx, dw, db and their slacks from the given mean and rstd (fp32 inputs of the call)."""
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[..., None], rstd.double()[..., None]
    w = None if w is None else (w.double()[:, None] if w.dim() == 2 else w.double())
    B, N, C = x.shape
    xh = (x - mean) * rstd
    exh = 3 * U * (x.abs() + mean.abs()) * rstd          # the difference's rounding
    g = dy if w is None else dy * w
    m1, m2 = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    dx = rstd * (g - m1 - xh * m2)
    chain = C / 32 + 16
    e1 = chain * U * g.abs().mean(-1, keepdim=True)
    e2 = chain * U * (g * xh).abs().mean(-1, keepdim=True) + (g.abs() * exh).mean(-1, keepdim=True)
    sdx = rstd * (e1 + xh.abs() * e2 + exh * m2.abs() + 4 * U * (g.abs() + m1.abs() + (xh * m2).abs()))
    dims = 1 if per_batch else (0, 1)
    n = N if per_batch else B * N
    dw, db = (dy * xh).sum(dims), dy.sum(dims)
    sdw = (n + 4) * U * (dy * xh).abs().sum(dims) + (dy.abs() * exh).sum(dims)
    return (dx, sdx), (dw, sdw), (db, (n + 4) * U * dy.abs().sum(dims))


# ---------------------------------------------------------------- linear

def act(z, name):
    """act(z), act'(z) in 64 bits."""
    if name == "relu":
        return z.clamp_min(0), (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu":
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)
    return z, torch.ones_like(z)


# fp32 exponentials and divisions of act and act': __expf's relative error is 2^-21 (1 + |x| / 2) and moves a
# sigmoid by at most s (1 - s) of that, below 2^-20 for every x; the same for the products around it
ACT_REL = 2.0 ** -19


def linear_forward(x, w, b, name, res):
    """y, z and their slacks (x [R, K])."""
    x, w = x.double(), w.double()
    K = x.shape[1]
    z, sz = x @ w.T, x.abs() @ w.abs().T
    if b is not None:
        z, sz = z + b.double(), sz + b.double().abs()
    sz = (K + 2) * U * sz
    y, _ = act(z, name)
    sy = sz if name in ("none", "relu") else 1.13 * sz + ACT_REL * y.abs() + 1e-7   # |act'| < 1.13
    if res is not None:
        y = y + res.double()
        sy = sy + 2 * U * (y.abs() + res.double().abs())
    return y, z, sy, sz


# half the distance of fp16's subnormal numbers, which hold a small z of bf16 products
PRE_ABS = 2.0 ** -25


def linear_backward(dy, x, w, pre, name, dtype):
    """dx, dw, db and their slacks, from the given pre (an input of the call)."""
    dy, x, w = dy.double(), x.double(), w.double()
    dz, e = dy, torch.zeros_like(dy)
    if name != "none":
        slope = act(pre.double(), name)[1]
        dz = dy * slope
        e = half(dtype) * dz.abs() + ACT_REL * dy.abs() * (slope.abs() + pre.double().abs().clamp_max(8) + 1)
    R, N = dz.shape
    a = dz.abs()
    return ((dz @ w, (N + 2) * U * (a @ w.abs()) + e @ w.abs()),
            (dz.T @ x, (R + 2) * U * (a.T @ x.abs()) + e.T @ x.abs()),
            (dz.sum(0), (R + 2) * U * a.sum(0) + e.sum(0)))


# ---------------------------------------------------------------- cross attention

# exponentials: in bf16 calls, whose p is rounded to 2^-8 anyway, an approximation of 2^-12 is allowed
EXP_REL = {torch.bfloat16: 2.0 ** -12, torch.float32: 2.0 ** -20}
# what fp32's smallest normal number bounds: a p (or ds) below it may become zero, which is off by less than 2^-126
# in that term whatever its relative error (p = 1e-38 times dp - D = 10 and q = 4 misses 4e-37 of dk that way)
FLUSH = 2.0 ** -126


def _heads(t):
    return t.double().transpose(1, 2)      # [B, H, tokens, d]


def cross_forward(q, k, v, lens, scale, dtype):
    """out, lse, and out's and lse's slacks; k, v [B, M, H, d], lens a list."""
    B, N, H, d = q.shape
    M = k.shape[1]
    outs, lses, so, sl = [], [], [], []
    qh, kh, vh = _heads(q), _heads(k), _heads(v)
    for b in range(B):
        n = lens[b]
        if n == 0:
            z = torch.zeros(H, N, d, dtype=torch.float64, device=q.device)
            outs.append(z), so.append(z)
            lses.append(torch.full((H, N), -math.inf, dtype=torch.float64, device=q.device)), sl.append(z[..., 0])
            continue
        kk, vv = kh[b, :, :n], vh[b, :, :n]
        s = scale * (qh[b] @ kk.transpose(-1, -2))
        es = scale * (d + 4) * U * (qh[b].abs() @ kk.abs().transpose(-1, -2))     # error of a score
        # the scores are scaled, and the maximum taken off, in fp32 in a base-2 exponent
        es = es + 4 * U * (s.abs() + s.abs().amax(-1, keepdim=True))
        p = torch.softmax(s, -1)
        e = es.amax(-1, keepdim=True)
        rel = 2 * e + EXP_REL[dtype] * 2 + (n + 8) * U
        outs.append(p @ vv)
        ph = half(torch.bfloat16) if dtype == torch.bfloat16 else 0.0
        so.append((rel + ph) * (p @ vv.abs()) + FLUSH * vv.abs().sum(-2, keepdim=True))
        lses.append(torch.logsumexp(s, -1))
        sl.append((e + EXP_REL[dtype] + (n + 8) * U)[..., 0] + 4 * U * lses[-1].abs())
    st = [torch.stack(t) for t in (outs, lses, so, sl)]
    return st[0].transpose(1, 2), st[1], st[2].transpose(1, 2), st[3]


def cross_backward(q, k, v, out, lse, dout, lens, scale, dtype):
    """(dq, dk, dv) with their slacks from the given out and lse (inputs of the call)."""
    B, N, H, d = q.shape
    M = k.shape[1]
    qh, kh, vh, oh, gh = (_heads(t) for t in (q, k, v, out, dout))
    res = [[torch.zeros(B, H, n, d, dtype=torch.float64, device=q.device) for _ in range(2)] for n in (N, M, M)]
    ph = half(torch.bfloat16) if dtype == torch.bfloat16 else 0.0
    for b in range(B):
        n = lens[b]
        if n == 0:
            continue
        Q, K, V, G = qh[b], kh[b, :, :n], vh[b, :, :n], gh[b]
        T = lambda t: t.transpose(-1, -2)  # noqa: E731
        s = scale * (Q @ T(K))
        es = scale * (d + 4) * U * (Q.abs() @ T(K.abs())) + 4 * U * (s.abs() + lse[b].double()[..., None].abs())
        p = torch.exp(s - lse[b].double()[..., None])
        ep = p * (es + EXP_REL[dtype]) + FLUSH
        dp, edp = G @ T(V), (d + 4) * U * (G.abs() @ T(V.abs()))
        if dtype == torch.bfloat16 and M <= 128:       # the call takes D from the states, else from out
            D = (p * dp).sum(-1, keepdim=True)
            eD = (ep * dp.abs() + p * edp + (n + 4) * U * (p * dp).abs()).sum(-1, keepdim=True)
        else:
            D = (G * oh[b]).sum(-1, keepdim=True)
            eD = (d + 4) * U * (G * oh[b]).abs().sum(-1, keepdim=True)
        ds = p * (dp - D)
        eds = ep * (dp - D).abs() + p * (edp + eD + U * (dp.abs() + D.abs())) + (ph + 2 * U) * ds.abs() + FLUSH
        epr = ep + ph * p
        res[0][0][b] = scale * (ds @ K)
        res[0][1][b] = scale * (eds @ K.abs() + (n + 8) * U * (ds.abs() @ K.abs()))
        res[1][0][b, :, :n] = scale * (T(ds) @ Q)
        res[1][1][b, :, :n] = scale * (T(eds) @ Q.abs() + (N + 8) * U * (T(ds.abs()) @ Q.abs()))
        res[2][0][b, :, :n] = T(p) @ G
        res[2][1][b, :, :n] = T(epr) @ G.abs() + (N + 8) * U * (T(p) @ G.abs())
    return [(a.transpose(1, 2), c.transpose(1, 2)) for a, c in res]
