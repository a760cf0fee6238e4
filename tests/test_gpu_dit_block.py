"""Layer norm, the projections, linear attention, cross attention and the Mix-FFN's convolutions run together as
one Linear DiT block, forward and backward, through the public entry points: against the same block in 64-bit
torch (gradients by autograd), on a stream of the caller's, captured into a graph and replayed on new inputs,
and from two graphs and two streams."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
B, T, HG, WG, M, H, D = 2, 2, 5, 13, 40, 4, 32
N, C, CT, CF = T * HG * WG, H * D, 96, 192      # tokens, channels, text channels, Mix-FFN channels
SHAPES = {"wq": (C, C), "wk": (C, C), "wv": (C, C), "wo": (C, C), "xq": (C, C), "xkv": (2 * C, CT), "xo": (C, C),
          "w1": (CF, C), "w2": (C, CF)}


@pytest.fixture(scope="module")
def la():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_causal_linear_b200 import build

    build.build()
    from block_causal_linear_b200 import la as _la

    return _la


def inputs(dtype, seed):
    g = torch.Generator().manual_seed(seed)
    t = lambda *s, std=1.0: (std * torch.randn(s, generator=g)).to(dtype).cuda()  # noqa: E731
    p = {n: t(*s, std=s[1] ** -0.5) for n, s in SHAPES.items()}
    p.update(b1=t(CF, std=0.2), b2=t(C, std=0.2), s1=1 + t(B, C, std=0.2), h1=t(B, C, std=0.2), s2=1 + t(B, C, std=0.2),
             h2=t(B, C, std=0.2), conv=t(CF, 1, 3, 3, std=0.3).float())
    return {"x": t(B, N, C), "text": t(B, M, CT), "dy": t(B, N, C), "p": p,
            "len": torch.tensor([M, 17], dtype=torch.int32, device="cuda")}


def block(la, st, ffn=True):
    """The block's output, and what its backward pass needs (without the Mix-FFN, whose convolution has none)."""
    x, p = st["x"], st["p"]
    n1, m1, r1 = la.layer_norm_forward(x, p["s1"], p["h1"], return_stats=True)
    q, k, v = (la.linear_forward(n1, p[n]).view(B, N, H, D) for n in ("wq", "wk", "wv"))
    a = la.full_forward(q, k, v)
    x1 = la.linear_forward(a.view(B, N, C), p["wo"], residual=x)
    xq = la.linear_forward(x1, p["xq"]).view(B, N, H, D)
    kv = la.linear_forward(st["text"], p["xkv"]).view(B, M, 2, H, D)
    c, lse = la.cross_attention_forward(xq, kv[:, :, 0], kv[:, :, 1], kv_len=st["len"], return_lse=True)
    x2 = la.linear_forward(c.view(B, N, C), p["xo"], residual=x1)
    saved = (n1, m1, r1, q, k, v, a, x1, xq, kv, c, lse, x2)
    if not ffn:
        return x2, saved
    n2 = la.layer_norm_forward(x2, p["s2"], p["h2"])
    f = la.linear_forward(n2, p["w1"], p["b1"], act="silu")
    f = la.dwconv3d(f.view(B, T, HG, WG, CF), p["conv"])
    return la.linear_forward(f.view(B, N, CF), p["w2"], p["b2"], residual=x2), saved


def backward(la, st, saved):
    """Gradients of sum(x2 * dy) for x, the text, and the parameters up to x2."""
    x, p = st["x"], st["p"]
    n1, m1, r1, q, k, v, a, x1, xq, kv, c, lse, _ = saved
    g, dx2 = {}, st["dy"]
    dc, g["xo"], _ = la.linear_backward(dx2, c.view(B, N, C), p["xo"], bias_grad=False)
    dkv = torch.empty_like(kv)
    dxq, _, _ = la.cross_attention_backward(xq, kv[:, :, 0], kv[:, :, 1], c, lse, dc.view_as(c), kv_len=st["len"],
                                            grads=(torch.empty_like(xq), dkv[:, :, 0], dkv[:, :, 1]))
    g["text"], g["xkv"], _ = la.linear_backward(dkv.view(B, M, 2 * C), st["text"], p["xkv"], bias_grad=False)
    dx1, g["xq"], _ = la.linear_backward(dxq.view(B, N, C), x1, p["xq"], bias_grad=False)
    dx1 = dx1 + dx2
    da, g["wo"], _ = la.linear_backward(dx1, a.view(B, N, C), p["wo"], bias_grad=False)
    parts = la.full_backward(q, k, v, da.view_as(a))
    dn1 = 0
    for n, d in zip(("wq", "wk", "wv"), parts):
        t, g[n], _ = la.linear_backward(d.view(B, N, C), n1, p[n], bias_grad=False)
        dn1 = dn1 + t
    dx, g["s1"], g["h1"] = la.layer_norm_backward(dn1, x, p["s1"], m1, r1)
    g["x"] = dx + dx1
    return g


def reference(st, ffn):
    """The block in 64-bit torch and, without the Mix-FFN, autograd's gradients."""
    dbl = lambda t: t.double().requires_grad_(not ffn)  # noqa: E731
    x, text, p = dbl(st["x"]), dbl(st["text"]), {n: dbl(t) for n, t in st["p"].items()}
    norm = lambda t, s, h: torch.nn.functional.layer_norm(t, (C,), eps=1e-6) * s[:, None] + h[:, None]  # noqa: E731
    heads = lambda t: t.view(B, -1, H, D).transpose(1, 2)  # noqa: E731
    n1 = norm(x, p["s1"], p["h1"])
    q, k, v = (heads(n1 @ p[n].T) for n in ("wq", "wk", "wv"))
    fq, fk = q.relu(), k.relu()
    a = (fq @ (fk.transpose(-1, -2) @ v)) / (fq @ fk.sum(2)[..., None] + 1e-6)
    x1 = x + a.transpose(1, 2).reshape(B, N, C) @ p["wo"].T
    kv = (text @ p["xkv"].T).view(B, M, 2, C)
    s = heads(x1 @ p["xq"].T) @ heads(kv[:, :, 0]).transpose(-1, -2) * D ** -0.5
    hidden = torch.arange(M, device="cuda") >= st["len"][:, None]
    c = torch.softmax(s.masked_fill(hidden[:, None, None], float("-inf")), -1) @ heads(kv[:, :, 1])
    x2 = x1 + c.transpose(1, 2).reshape(B, N, C) @ p["xo"].T
    if not ffn:
        (x2 * st["dy"].double()).sum().backward()
        return x2.detach(), {"x": x.grad, "text": text.grad, **{n: t.grad for n, t in p.items() if t.grad is not None}}
    f = norm(x2, p["s2"], p["h2"]) @ p["w1"].T + p["b1"]
    f = (f * torch.sigmoid(f)).view(B, T, HG, WG, CF).permute(0, 4, 1, 2, 3)
    f = torch.nn.functional.conv3d(f, p["conv"][:, None], padding=(0, 1, 1), groups=CF)
    return x2 + f.permute(0, 2, 3, 4, 1).reshape(B, N, CF) @ p["w2"].T + p["b2"], None


# Every tensor between two operators is rounded once (half a step: 2^-9 rms of a value in bf16, 2^-25 in fp32), and
# the block chains at most 12 such tensors behind one another; each operator passes an error on amplified by at most
# about 2 in the norm (weights of unit gain; the linear attention's quotient and the softmax move less than their
# scores).  In norm: 12 roundings, 4 for the amplification and the sum of branches.
TOL = {BF: 12 * 4 * 2.0 ** -9, torch.float32: 12 * 4 * 2.0 ** -20}


def near(name, got, want, dtype):
    rel = ((got.double() - want).norm() / want.norm()).item()
    assert rel <= TOL[dtype], f"{name}: {rel}"


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_block_forward(la, dtype):
    st = inputs(dtype, 1)
    y, _ = block(la, st)
    near("y", y, reference(st, True)[0], dtype)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_block_gradients(la, dtype):
    st = inputs(dtype, 2)
    x2, saved = block(la, st, ffn=False)
    g = backward(la, st, saved)
    want, grads = reference(st, False)
    near("x2", x2, want, dtype)
    for n, t in g.items():
        near(n, t, grads[n], dtype)


def flat(la, st):
    y, saved = block(la, st)
    return [y, *(t for _, t in sorted(backward(la, st, saved).items()))]


def copy_into(a, b):
    for n in ("x", "text", "dy", "len"):
        a[n].copy_(b[n])
    for n in a["p"]:
        a["p"][n].copy_(b["p"][n])


def test_block_on_another_stream(la):
    """The same bits on a stream of the caller's, given as the current stream."""
    st = inputs(BF, 3)
    want = flat(la, st)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = flat(la, st)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_stream_argument(la):
    """stream= alone: outputs and workspaces belong to that stream."""
    st = inputs(BF, 4)
    x, w = st["x"], st["p"]["w1"]
    want = la.linear_backward(la.linear_forward(x, w), x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        y = la.linear_forward(x, w, stream=s)
        got = la.linear_backward(y, x, w, stream=s)
        n, mean, rstd = la.layer_norm_forward(x, return_stats=True, stream=s)
        la.layer_norm_backward(n, x, None, mean, rstd, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs_of_the_block(la):
    """Two captured graphs of the same block on their own inputs, replayed in turn and on two streams at once,
    on new inputs: the bits of the eager calls."""
    keep, graphs = [inputs(BF, 5), inputs(BF, 6)], []
    for st in keep:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            flat(la, st)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = flat(la, st)
        graphs.append((g, outs))
    fresh = [inputs(BF, 7), inputs(BF, 8)]
    want = [flat(la, st) for st in fresh]
    for st, new in zip(keep, fresh):
        copy_into(st, new)
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for (_, outs), w in zip(graphs, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, w))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (_, outs), w in zip(graphs, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, w))
    la.device_status()


CONSUMERS = {
    "block_apply": lambda la, t, o: la.block_apply(t(600, 64, 32), o["sums"], o["state"], commit=False),
    "full_forward": lambda la, t, o: la.full_forward(t(600, 64, 32), o["k"], t(600, 64, 32), tokens_per_block=200),
    "full_backward": lambda la, t, o: la.full_backward(o["k"], t(600, 64, 32), o["k"], t(600, 64, 32)),
    "dwconv": lambda la, t, o: la.dwconv3d(t(10, 6, 10, 2048), o["filter"]),
    "norm": lambda la, t, o: la.layer_norm_forward(t(600, 2048), return_stats=True),
    "norm of few rows": lambda la, t, o: la.layer_norm_forward(t(2, 2048)),
    "norm of many rows": lambda la, t, o: la.layer_norm_forward(t(8000, 2048)),
    "norm of odd rows": lambda la, t, o: la.layer_norm_forward(t(2048, 1000).view(-1)[:2048 * 999].view(2048, 999)),
    "norm backward": lambda la, t, o: la.layer_norm_backward(t(600, 2048), o["k"].view(600, 2048), o["w"][0], *o["stats"]),
    "linear": lambda la, t, o: la.linear_forward(t(600, 2048), o["w"]),
    "linear of few rows": lambda la, t, o: la.linear_forward(t(2, 2048), o["w"]),
    "linear of odd rows": lambda la, t, o: la.linear_forward(t(600, 1000).view(-1)[:600 * 999].view(600, 999), o["odd"]),
    "linear backward": lambda la, t, o: la.linear_backward(t(600, 2048), o["k"].view(600, 2048), o["sq"], o["pre"], "silu"),
    "cross": lambda la, t, o: la.cross_attention_forward(t(600, 64, 32), o["k"], o["k"], return_lse=True),
    "cross of few queries": lambda la, t, o: la.cross_attention_forward(t(2, 64, 32), o["k"], o["k"]),
    "cross backward": lambda la, t, o: la.cross_attention_backward(o["k"], o["k"], o["k"], o["k"], o["lse"], t(600, 64, 32)),
    "cross backward, few states": lambda la, t, o: la.cross_attention_backward(
        o["k"], o["k"][:, :100], o["k"][:, :100], o["k"], o["lse"], t(600, 64, 32)),
}


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("name", CONSUMERS)
def test_each_call_waits_for_the_one_before(la, name, dtype):
    """What a long call writes last is read by the next call of the stream: the kernels of one call may be let
    in while the kernel before them still runs, its results must not be."""
    g = torch.Generator().manual_seed(3)
    t = lambda *s: torch.randn(s, generator=g).to(dtype).cuda()  # noqa: E731
    x, w = t(20000, 2048), t(2048, 448) / 20
    narrow = x.view(-1)[:20000 * 448].view(20000, 448)      # too few products to cut the last tiles, which end late
    o = {"k": t(1, 600, 64, 32), "w": t(256, 2048), "odd": t(256, 999), "sq": t(2048, 2048), "filter": t(2048, 1, 3, 3).float(),
         "pre": torch.zeros(600, 2048, dtype=torch.float16 if dtype is BF else dtype, device="cuda"),
         "sums": la.block_reduce(t(1, 600, 64, 32), t(1, 600, 64, 32))[None].contiguous()}
    o["state"] = la.State(1, 64)
    o["stats"] = la.layer_norm_forward(o["k"].view(600, 2048), return_stats=True)[1:]
    o["lse"] = la.cross_attention_forward(o["k"], o["k"], o["k"], return_lse=True)[1]
    buf, other = torch.empty_like(x), torch.empty_like(x)

    def tail(*shape):
        n = torch.Size(shape).numel()
        flat = buf.view(-1)[buf.numel() - n:]
        return flat.view(shape if len(shape) == 2 else (1, *shape))

    def run():
        r = CONSUMERS[name](la, tail, o)
        return [r] if torch.is_tensor(r) else list(r)

    for _ in range(5):
        buf.zero_()
        torch.cuda.synchronize()
        for out in [other] * 12 + [buf]:                    # (the first ones while the host queues the rest)
            if dtype is BF:
                la.linear_forward(narrow, w, out=out)
            else:
                la.layer_norm_forward(x, out=out)
        got = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, run()))
        la.device_status()
