"""The operators of a Linear DiT block around the block-causal linear attention:
layer norm, the projections (matrix products with bias, activation and residual)
and cross attention to a text encoder's states, forward and training.

A case is a dict: "op" is "layer_norm", "linear" or "cross_attention", "dtype" is
"bf16" or "fp32", "train" says whether the pass runs backward too; the other
entries are sizes and options of the operator.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # A timestep embedding's norm: two rows, only latency counts.
        dict(name="norm, 2 rows", op="layer_norm", dtype="bf16", train=False, B=2, N=1, C=2048, per_batch=False),
        # The modulated norm (a scale and shift per sample) before attention, 21 latent frames at 720p.
        dict(name="norm 720p modulated", op="layer_norm", dtype="bf16", train=False, B=1, N=75600, C=2048, per_batch=True),
        # The same in training on a batch of 480p clips, gradients of scale and shift per sample.
        dict(name="norm 480p train", op="layer_norm", dtype="bf16", train=True, B=4, N=8190, C=2048, per_batch=True),
        # A plain affine norm in fp32 of an odd width, trained.
        dict(name="norm fp32 odd train", op="layer_norm", dtype="fp32", train=True, B=3, N=1170, C=1001, per_batch=False),
        # The modulation's projection: one row a sample against 6 C outputs; the weight's bytes are the time.
        dict(name="linear, 2 rows", op="linear", dtype="bf16", train=False, R=2, K=2048, N=12288, act="none", bias=True, residual=False),
        # The Mix-FFN's first pointwise convolution on 21 frames at 480p (5120 channels, as the depthwise benchmark).
        dict(name="linear 480p silu", op="linear", dtype="bf16", train=False, R=8190, K=2048, N=5120, act="silu", bias=True, residual=False),
        # Its last one with the residual, trained on one 480p streaming block of 15600 tokens.
        dict(name="linear 15600 train", op="linear", dtype="bf16", train=True, R=15600, K=5120, N=2048, act="none", bias=True, residual=True),
        # The text states' projection trained in fp32, nothing a multiple of anything.
        dict(name="linear fp32 odd train", op="linear", dtype="fp32", train=True, R=1201, K=1023, N=517, act="gelu", bias=True, residual=False),
        # A single query token over a long encoder sequence: K and V are streamed once.
        dict(name="cross, 1 query", op="cross_attention", dtype="bf16", train=False, B=1, N=1, M=4096, H=64, d=32, ragged=False, fused=True),
        # 21 latent frames at 720p against a caption of 300 states.
        dict(name="cross 720p", op="cross_attention", dtype="bf16", train=False, B=1, N=75600, M=300, H=64, d=32, ragged=False, fused=True),
        # A training batch at 480p, captions of different lengths.
        dict(name="cross 480p train", op="cross_attention", dtype="bf16", train=True, B=4, N=8190, M=512, H=64, d=32, ragged=True, fused=True),
        # fp32 on odd lengths.
        dict(name="cross fp32 odd train", op="cross_attention", dtype="fp32", train=True, B=2, N=391, M=77, H=8, d=64, ragged=True, fused=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width over its logarithm; two in three are multiples of 8."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 1 / 3 else max(8, n // 8 * 8)


def draw(rng):
    caps = {}
    for c in listed():
        w = work(c)
        k = (c["op"], c["dtype"])
        caps[k] = (max(caps.get(k, (0, 0))[0], w["bytes"]), max(caps.get(k, (0, 0))[1], w["flops"]))
    while True:
        op = rng.choice(("layer_norm", "linear", "cross_attention"))
        dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
        train = rng.random() < 0.5
        case = dict(op=op, dtype=dtype, train=train)
        if op == "layer_norm":
            case.update(B=rng.randint(1, 4), N=_log(rng, 1, 75600), C=_width(rng, 64, 5120), per_batch=rng.random() < 0.5)
        elif op == "linear":
            case.update(R=_log(rng, 1, 15600), K=_width(rng, 64, 5120), N=_width(rng, 64, 12288),
                        act=rng.choice(("none", "relu", "silu", "gelu")), bias=rng.random() < 0.7, residual=rng.random() < 0.5)
        else:
            case.update(B=rng.randint(1, 4), N=_log(rng, 1, 75600), M=_log(rng, 1, 4096), H=rng.choice((4, 8, 16, 20, 32, 64)),
                        d=rng.choice((32, 64)), ragged=rng.random() < 0.6, fused=rng.random() < 0.5)
        w = work(case)
        if w["bytes"] <= caps[op, dtype][0] and w["flops"] <= caps[op, dtype][1]:
            return case


def _lengths(case):
    """Valid encoder states of each sample: all M, or falling to about a third of it."""
    B, M = case["B"], case["M"]
    return [M - (2 * M * b) // (3 * B) if case["ragged"] else M for b in range(B)]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    train = case["train"]
    if case["op"] == "layer_norm":
        n, wn = case["B"] * case["N"] * case["C"], (case["B"] if case["per_batch"] else 1) * case["C"]
        # forward: x in, y out, both vectors in; training: dy in, dx out, both vectors' gradients out
        return {"bytes": e * ((4 if train else 2) * n + (4 if train else 2) * wn), "flops": (19 if train else 8) * n}
    if case["op"] == "linear":
        R, K, N = case["R"], case["K"], case["N"]
        words = R * K + N * K + R * N * (2 if case["residual"] else 1) + (N if case["bias"] else 0)
        if train:  # dy in; dx, dw and db out
            words += R * N + R * K + N * K + (N if case["bias"] else 0)
        return {"bytes": e * words, "flops": (6 if train else 2) * R * K * N}
    B, N, H, d = case["B"], case["N"], case["H"], case["d"]
    keys = sum(_lengths(case))
    words = (2 * B * N + 2 * keys) * H * d
    if train:  # dout in; dq, dk and dv out (rows past a sample's length too)
        words += (2 * B * N + 2 * B * case["M"]) * H * d
    return {"bytes": e * words + (4 * B if case["ragged"] else 0), "flops": (14 if train else 4) * N * keys * H * d}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).add_(mean).to(dt)

    st = {"case": case}
    if case["op"] == "layer_norm":
        B, N, C = case["B"], case["N"], case["C"]
        vec = (B, C) if case["per_batch"] else (C,)
        x = torch.randn((B, N, C), generator=g, device="cuda")
        x += torch.randn((C,), generator=g, device="cuda").mul_(0.5)    # channels with offsets, as hidden states have
        st.update(x=x.to(dt), w=normal(*vec, std=0.2, mean=1.0), b=normal(*vec, std=0.2))
        if case["train"]:
            st["dy"] = normal(B, N, C)
    elif case["op"] == "linear":
        R, K, N = case["R"], case["K"], case["N"]
        st.update(x=normal(R, K), w=normal(N, K, std=K ** -0.5), b=normal(N, std=0.2) if case["bias"] else None,
                  res=normal(R, N) if case["residual"] else None)
        if case["train"]:
            st["dy"] = normal(R, N)
    else:
        B, N, M, H, d = (case[s] for s in ("B", "N", "M", "H", "d"))
        st["q"] = normal(B, N, H, d)
        if case["fused"]:  # one projection's output holds both
            kv = normal(B, M, 2, H, d)
            st["k"], st["v"] = kv[:, :, 0], kv[:, :, 1]
        else:
            st["k"], st["v"] = normal(B, M, H, d), normal(B, M, H, d)
        st["len"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
        if case["train"]:
            st["dy"] = normal(B, N, H, d)
    return st


# ---------------------------------------------------------------- plain forms (fp32, rounded once at the end)

def _plain_norm(st):
    c, dt = st["case"], st["x"].dtype
    x, w, b = st["x"].float(), st["w"].float(), st["b"].float()
    if c["per_batch"]:
        w, b = w[:, None], b[:, None]
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    rstd = (xc.square().mean(-1, keepdim=True) + EPS).rsqrt()
    xh = xc * rstd
    y = (xh * w + b).to(dt)
    if not c["train"]:
        return y
    dy = st["dy"].float()
    g = dy * w
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    dims = 1 if c["per_batch"] else (0, 1)
    return {"y": y, "dx": dx.to(dt), "dw": (dy * xh).sum(dims).to(dt), "db": dy.sum(dims).to(dt)}


def _plain_act(z, act):
    """act(z) and its derivative."""
    if act == "relu":
        return z.clamp_min(0), (z > 0).float()
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu":
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z * z * z))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)
    return z, None


def _plain_linear(st):
    c, dt = st["case"], st["x"].dtype
    x, w = st["x"].float(), st["w"].float()
    z = x @ w.t()
    if st["b"] is not None:
        z = z + st["b"].float()
    y, slope = _plain_act(z, c["act"])
    if st["res"] is not None:
        y = y + st["res"].float()
    y = y.to(dt)
    if not c["train"]:
        return y
    dz = st["dy"].float()
    if slope is not None:
        dz = dz * slope
    out = {"y": y, "dx": (dz @ w).to(dt), "dw": (dz.t() @ x).to(dt)}
    if st["b"] is not None:
        out["db"] = dz.sum(0).to(dt)
    return out


def _plain_cross(st):
    c, dt = st["case"], st["q"].dtype
    q, k, v = (st[s].float().transpose(1, 2) for s in ("q", "k", "v"))    # [B, H, tokens, d]
    scale = c["d"] ** -0.5
    s = (q @ k.transpose(-1, -2)).mul_(scale)
    if st["len"] is not None:
        hidden = torch.arange(c["M"], device=s.device) >= st["len"][:, None]
        s.masked_fill_(hidden[:, None, None], float("-inf"))
    p = (s - s.amax(-1, keepdim=True)).exp_()
    p /= p.sum(-1, keepdim=True)
    o = p @ v
    if not c["train"]:
        return o.transpose(1, 2).contiguous().to(dt)
    do = st["dy"].float().transpose(1, 2)
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    outs = {"out": o, "dq": ds @ k, "dk": ds.transpose(-1, -2) @ q, "dv": p.transpose(-1, -2) @ do}
    return {n: t.transpose(1, 2).contiguous().to(dt) for n, t in outs.items()}


# ---------------------------------------------------------------- the framework's operators

def _own_norm(la, st):
    if not st["case"]["train"]:
        return la.layer_norm_forward(st["x"], st["w"], st["b"], eps=EPS)
    y, mean, rstd = la.layer_norm_forward(st["x"], st["w"], st["b"], eps=EPS, return_stats=True)
    dx, dw, db = la.layer_norm_backward(st["dy"], st["x"], st["w"], mean, rstd)
    return {"y": y, "dx": dx, "dw": dw, "db": db}


def _own_linear(la, st):
    act = st["case"]["act"]
    if not st["case"]["train"]:
        return la.linear_forward(st["x"], st["w"], st["b"], act=act, residual=st["res"])
    y, pre = la.linear_forward(st["x"], st["w"], st["b"], act=act, residual=st["res"], return_pre=True)
    dx, dw, db = la.linear_backward(st["dy"], st["x"], st["w"], pre=pre, act=act, bias_grad=st["b"] is not None)
    return {"y": y, "dx": dx, "dw": dw} if db is None else {"y": y, "dx": dx, "dw": dw, "db": db}


def _own_cross(la, st):
    q, k, v, ln = st["q"], st["k"], st["v"], st["len"]
    if not st["case"]["train"]:
        return la.cross_attention_forward(q, k, v, kv_len=ln)
    out, lse = la.cross_attention_forward(q, k, v, kv_len=ln, return_lse=True)
    dq, dk, dv = la.cross_attention_backward(q, k, v, out, lse, st["dy"], kv_len=ln)
    return {"out": out, "dq": dq, "dk": dk, "dv": dv}


def run(state):
    op = state["case"]["op"]
    if own:
        from block_causal_linear_b200 import la

        return {"layer_norm": _own_norm, "linear": _own_linear, "cross_attention": _own_cross}[op](la, state)
    return {"layer_norm": _plain_norm, "linear": _plain_linear, "cross_attention": _plain_cross}[op](state)


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    st = {n: t.double() if torch.is_tensor(t) and t.is_floating_point() else t for n, t in prepare(case, seed).items()}
    if case["op"] == "layer_norm":
        return _exact_norm(case, st)
    return _exact_linear(case, st) if case["op"] == "linear" else _exact_cross(case, st)


def _exact_norm(case, st):
    x, C = st["x"], case["C"]
    w, b = (t.reshape(-1, 1, C) for t in (st["w"], st["b"]))
    var, mean = torch.var_mean(x, dim=2, correction=0, keepdim=True)
    sd = torch.sqrt(var + EPS)
    y = w * ((x - mean) / sd) + b
    if not case["train"]:
        return y
    dy = st["dy"]
    xh = (x - mean) / sd
    t = dy * w / sd
    dx = t - t.sum(2, keepdim=True) / C - xh * (t * xh).sum(2, keepdim=True) / C
    dw, db = torch.einsum("bnc,bnc->bc", dy, xh), torch.einsum("bnc->bc", dy)
    if not case["per_batch"]:
        dw, db = dw.sum(0), db.sum(0)
    return {"y": y, "dx": dx, "dw": dw, "db": db}


def _exact_linear(case, st):
    x, w = st["x"], st["w"]
    z = torch.einsum("rk,nk->rn", x, w) + (0 if st["b"] is None else st["b"])
    act = case["act"]
    if act == "relu":
        y, slope = torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0)
    elif act == "silu":
        sg = torch.sigmoid(z)
        y, slope = z * sg, sg + z * sg * torch.sigmoid(-z)
    elif act == "gelu":
        # z sigmoid(2u), u = sqrt(2/pi) (z + 0.044715 z^3): the tanh form written with the sigmoid
        r = math.sqrt(8 / math.pi)
        sg = torch.sigmoid(r * (z + 0.044715 * z ** 3))
        y, slope = z * sg, sg + z * sg * (1 - sg) * r * (1 + 0.134145 * z ** 2)
    else:
        y, slope = z, torch.ones_like(z)
    if st["res"] is not None:
        y = y + st["res"]
    if not case["train"]:
        return y
    dz = st["dy"] * slope
    out = {"y": y, "dx": torch.einsum("rn,nk->rk", dz, w), "dw": torch.einsum("rn,rk->nk", dz, x)}
    if st["b"] is not None:
        out["db"] = torch.einsum("rn->n", dz)
    return out


def _exact_cross(case, st):
    q, k, v = st["q"], st["k"], st["v"]
    B, H = case["B"], case["H"]
    scale = 1 / math.sqrt(case["d"])
    outs = {"out": torch.zeros_like(q)}
    if case["train"]:
        outs.update(dq=torch.zeros_like(q), dk=torch.zeros(k.shape, dtype=k.dtype, device=k.device),
                    dv=torch.zeros(v.shape, dtype=v.dtype, device=v.device))
    for b, n in enumerate(_lengths(case)):
        for h in range(H):
            qh, kh, vh = q[b, :, h], k[b, :n, h], v[b, :n, h]
            p = torch.softmax(scale * torch.mm(qh, kh.T), dim=1)
            outs["out"][b, :, h] = torch.mm(p, vh)
            if case["train"]:
                doh = st["dy"][b, :, h]
                dp = torch.mm(doh, vh.T)
                ds = p * (dp - (p * dp).sum(1, keepdim=True))
                outs["dq"][b, :, h] = scale * torch.mm(ds, kh)
                outs["dk"][b, :n, h] = scale * torch.mm(ds.T, qh)
                outs["dv"][b, :n, h] = torch.mm(p.T, doh)
    return outs if case["train"] else outs["out"]
