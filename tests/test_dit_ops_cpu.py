"""Refusals of layer norm, linear and cross attention without a GPU: bad arguments of the C entry points (every
call fails validation, so no pointer is followed) and of the Python wrappers."""
import pytest
import torch

from block_causal_linear_b200 import build as la_build

FAKE, NAN, INF = 1 << 20, float("nan"), float("inf")
BIG = 1 << 60


@pytest.fixture(scope="module")
def la():
    la_build.build()
    from block_causal_linear_b200 import la as _la

    return _la


def caller(fn, args):
    """fn called with the named args in order, some replaced."""
    def call(**kw):
        a = dict(args)
        assert set(kw) <= set(a)
        a.update(kw)
        return fn(*a.values())
    return call


def expect(la, call, table):
    names = {"inval": la.LA_EINVAL, "unsup": la.LA_EUNSUPPORTED, "ws": la.LA_EWORKSPACE}
    for want, kw in table:
        assert call(**kw) == names[want], kw


def test_norm_refusals(la):
    L = la.lib()
    fwd = caller(L.la_layer_norm_forward, dict(x=FAKE, w=FAKE, b=FAKE, y=FAKE, mean=FAKE, rstd=FAKE, dt=la.LA_BF16,
                                               B=2, N=3, C=8, pb=0, eps=1e-6, stream=None))
    expect(la, fwd, [("inval", k) for k in (
        dict(x=None), dict(y=None), dict(x=FAKE + 8), dict(w=FAKE + 2), dict(b=FAKE + 4), dict(y=FAKE + 8),
        dict(mean=FAKE + 4), dict(rstd=FAKE + 4), dict(dt=2), dict(B=0), dict(N=-1), dict(C=0),
        dict(B=1 << 30, N=1 << 30), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF))])
    assert fwd(B=65536, pb=1) == la.LA_EUNSUPPORTED
    assert fwd(B=1 << 20, N=1 << 12, C=8) == la.LA_EUNSUPPORTED      # rows past 2^31
    need = L.la_layer_norm_backward_workspace_size(2, 3, 8, 0)
    assert need > 0 and need % 256 == 0 and L.la_layer_norm_backward_workspace_size(0, 3, 8, 0) == 0
    bwd = caller(L.la_layer_norm_backward, dict(dy=FAKE, x=FAKE, w=FAKE, mean=FAKE, rstd=FAKE, dx=FAKE, dw=FAKE,
                                                db=FAKE, dt=la.LA_F32, B=2, N=3, C=8, pb=0, ws=FAKE, n=need,
                                                stream=None))
    expect(la, bwd, [("inval", {k: None}) for k in ("dy", "x", "mean", "rstd", "dx")] +
           [("inval", {k: FAKE + 8}) for k in ("dy", "x", "w", "mean", "rstd", "dx", "dw", "db")] +
           [("inval", dict(dt=-1)), ("inval", dict(C=-8)), ("ws", dict(ws=None)), ("ws", dict(n=need - 1)),
            ("ws", dict(ws=FAKE + 16)), ("unsup", dict(B=65536, pb=1))])


def test_linear_refusals(la):
    L = la.lib()
    need = L.la_linear_workspace_size(5, 16, 24, la.LA_BF16)
    assert need > 0 and need % 256 == 0
    assert L.la_linear_workspace_size(0, 16, 24, la.LA_BF16) == 0 and L.la_linear_workspace_size(5, 16, 24, 7) == 0
    fwd = caller(L.la_linear_forward, dict(x=FAKE, w=FAKE, b=FAKE, res=FAKE, y=FAKE, pre=FAKE, dt=la.LA_BF16, act=2,
                                           R=5, K=16, N=24, ws=FAKE, n=need, stream=None))
    expect(la, fwd, [("inval", {k: None}) for k in ("x", "w", "y")] +
           [("inval", {k: FAKE + 8}) for k in ("x", "w", "b", "res", "y", "pre")] +
           [("inval", k) for k in (dict(dt=2), dict(act=4), dict(act=-1), dict(R=0), dict(K=0), dict(N=-3),
                                   dict(R=1 << 30, N=1 << 30))] +
           [("ws", dict(ws=None)), ("ws", dict(n=need - 1)), ("ws", dict(ws=FAKE + 128))])
    need = L.la_linear_backward_workspace_size(5, 16, 24, la.LA_BF16, 2)
    assert need > 0 and need % 256 == 0 and L.la_linear_backward_workspace_size(5, 16, 24, la.LA_BF16, 9) == 0
    bwd = caller(L.la_linear_backward, dict(dy=FAKE, x=FAKE, w=FAKE, pre=FAKE, dx=FAKE, dw=FAKE, db=FAKE,
                                            dt=la.LA_BF16, act=2, R=5, K=16, N=24, ws=FAKE, n=need, stream=None))
    expect(la, bwd, [("inval", {k: None}) for k in ("dy", "x", "w", "pre")] +
           [("inval", {k: FAKE + 8}) for k in ("dy", "x", "w", "pre", "dx", "dw", "db")] +
           [("inval", dict(dt=3)), ("inval", dict(act=5)), ("inval", dict(N=0)), ("ws", dict(ws=None)),
            ("ws", dict(n=need - 1)), ("ws", dict(ws=FAKE + 64))])


def test_cross_refusals(la):
    L = la.lib()
    need = L.la_cross_attention_workspace_size(la.LA_BF16, 2, 5, 7, 4, 32)
    assert need > 0 and need % 256 == 0
    assert L.la_cross_attention_workspace_size(la.LA_BF16, 2, 5, 0, 4, 32) == 0
    args = dict(q=FAKE, k=FAKE, v=FAKE, kv_len=FAKE, out=FAKE, lse=FAKE)
    sizes = dict(dt=la.LA_BF16, B=2, N=5, M=7, H=4, d=32, ldk=128, ldv=128)
    fwd = caller(L.la_cross_attention_forward, dict(**args, **sizes, scale=0.2, ws=FAKE, n=need, stream=None))
    common = ([("inval", k) for k in (
        dict(dt=2), dict(B=0), dict(N=0), dict(M=0), dict(H=0), dict(d=0), dict(ldk=127), dict(ldv=124),
        dict(ldk=132), dict(ldk=BIG), dict(kv_len=FAKE + 2), dict(scale=0.0), dict(scale=1e-21), dict(scale=-1.0), dict(scale=NAN),
        dict(scale=INF))] +
        [("unsup", dict(d=48)), ("unsup", dict(d=128, ldk=512, ldv=512)),
         ("unsup", dict(B=1 << 14)), ("ws", dict(ws=None)), ("ws", dict(n=need - 1)), ("ws", dict(ws=FAKE + 32))])
    expect(la, fwd, [("inval", {k: None}) for k in ("q", "k", "v", "out")] +
           [("inval", {k: FAKE + 8}) for k in ("q", "k", "v", "out", "lse")] + common)
    need = L.la_cross_attention_backward_workspace_size(la.LA_BF16, 2, 5, 7, 4, 32)
    assert need > 0 and need % 256 == 0
    ptrs = dict(args, dout=FAKE, dq=FAKE, dk=FAKE, dv=FAKE)
    bwd = caller(L.la_cross_attention_backward, dict(**ptrs, **sizes, lddk=128, lddv=128, scale=0.2, ws=FAKE, n=need,
                                                     stream=None))
    expect(la, bwd, [("inval", {k: None}) for k in ptrs if k != "kv_len"] +
           [("inval", {k: FAKE + 8}) for k in ptrs if k != "kv_len"] +
           [("inval", dict(lddk=64)), ("inval", dict(lddv=129)), ("ws", dict(n=need - 1))] +
           [c for c in common if "n" not in c[1]])


def test_wrappers_refuse(la):
    x, w = torch.zeros(2, 3, 8), torch.zeros(4, 8)
    q = torch.zeros(1, 4, 2, 32)
    for f in (lambda: la.layer_norm_forward(x), lambda: la.linear_forward(x, w),
              lambda: la.cross_attention_forward(q, q, q)):
        with pytest.raises(ValueError):     # not CUDA tensors
            f()


class FakeCuda(torch.Tensor):
    """A CPU tensor that says it is a CUDA tensor: the wrappers' shape checks come before any launch."""
    is_cuda = True


def fake(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(FakeCuda)


def test_wrappers_refuse_shapes_and_types(la):
    x = fake(2, 3, 8)
    bad = [
        (ValueError, lambda: la.layer_norm_forward(fake(2, 3, 8, 1))),
        (ValueError, lambda: la.layer_norm_forward(fake(2, 0, 8))),
        (ValueError, lambda: la.layer_norm_forward(x.transpose(0, 1))),
        (TypeError, lambda: la.layer_norm_forward(fake(2, 8, dtype=torch.float16))),
        (ValueError, lambda: la.layer_norm_forward(x, fake(7))),
        (ValueError, lambda: la.layer_norm_forward(x, fake(3, 8))),
        (ValueError, lambda: la.layer_norm_forward(x, fake(2, 8), fake(8))),
        (TypeError, lambda: la.layer_norm_forward(x, fake(8, dtype=torch.float32))),
        (ValueError, lambda: la.layer_norm_forward(x, out=fake(2, 3, 9))),
        (ValueError, lambda: la.layer_norm_backward(x, x, None, None, None)),
        (ValueError, lambda: la.layer_norm_backward(x, x, fake(8), fake(2, 3), fake(2, 3), per_batch=True)),
        (TypeError, lambda: la.layer_norm_backward(x, x, None, fake(2, 3), fake(2, 3))),
        (ValueError, lambda: la.linear_forward(x, fake(4, 9))),
        (ValueError, lambda: la.linear_forward(x, fake(8))),
        (TypeError, lambda: la.linear_forward(x, fake(4, 8, dtype=torch.float32))),
        (ValueError, lambda: la.linear_forward(x, fake(4, 8), fake(5))),
        (ValueError, lambda: la.linear_forward(x, fake(4, 8), act="tanh")),
        (ValueError, lambda: la.linear_forward(x, fake(4, 8), residual=fake(2, 3, 5))),
        (ValueError, lambda: la.linear_backward(fake(2, 3, 4), x, fake(4, 8), act="silu")),
        (ValueError, lambda: la.linear_backward(fake(2, 3, 5), x, fake(4, 8))),
    ]
    q = fake(2, 4, 2, 32)
    kv = fake(2, 5, 2, 2, 32)
    k, v = kv[:, :, 0], kv[:, :, 1]
    bad += [
        (ValueError, lambda: la.cross_attention_forward(q, fake(2, 5, 2, 64), v)),
        (ValueError, lambda: la.cross_attention_forward(q, fake(1, 5, 2, 32), v)),
        (ValueError, lambda: la.cross_attention_forward(q, k, fake(2, 6, 2, 32))),
        (ValueError, lambda: la.cross_attention_forward(q, k[:, ::2], v[:, ::2])),
        (ValueError, lambda: la.cross_attention_forward(q, fake(2, 2, 5, 32).transpose(1, 2), v)),
        (ValueError, lambda: la.cross_attention_forward(q, fake(2, 5, 2, 64)[..., ::2], v)),
        (TypeError, lambda: la.cross_attention_forward(q, k, fake(2, 5, 2, 32, dtype=torch.float32))),
        (TypeError, lambda: la.cross_attention_forward(q, k, v, kv_len=fake(2, dtype=torch.int64))),
        (ValueError, lambda: la.cross_attention_forward(q, k, v, kv_len=fake(3, dtype=torch.int32))),
        (ValueError, lambda: la.cross_attention_backward(q, k, v, q, fake(2, 2, 5, dtype=torch.float32), q)),
        (ValueError, lambda: la.cross_attention_backward(q, k, v, fake(2, 4, 2, 31), fake(2, 2, 4, dtype=torch.float32), q)),
    ]
    for i, (kind, f) in enumerate(bad):
        with pytest.raises(kind):
            f()
            pytest.fail(f"call {i} was not refused")


def test_head_dimension_is_named(la):
    q = fake(1, 4, 2, 48)
    with pytest.raises(la.LAError) as e:
        la.cross_attention_forward(q, q, q)
    assert e.value.status == la.LA_EUNSUPPORTED
