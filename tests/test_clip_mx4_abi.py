"""Argument checks of the clipping and MXFP4 entry points that need no GPU:
every refusal comes back before anything is enqueued (fake aligned addresses:
nothing is dereferenced)."""
import ctypes as C

import pytest

from implicit_attribute_decode_amd import ia

P = 1 << 20
BAD, UNSUPPORTED, SMALL = ia.IA_ERR_INVALID_ARG, ia.IA_ERR_UNSUPPORTED, ia.IA_ERR_WORKSPACE_TOO_SMALL


def _clip(max_norm=1.0, ws=P, ws_bytes=1 << 30, stats=P, count=1, **kw):
    d = dict(data=P, out=None, rows=10, dim=1, stride=1, out_stride=1, dtype=ia.IA_DTYPE_F32)
    d.update(kw)
    arr = (ia.Grad * 1)(ia.Grad(**d))
    L = ia.load()
    return {fn(arr, count, max_norm, ws, ws_bytes, stats, None) for fn in (L.ia_clip_grad_norm,)}


@pytest.mark.parametrize("kw,status", [
    (dict(max_norm=-1.0), BAD), (dict(max_norm=float("nan")), BAD), (dict(ws=None), BAD), (dict(ws=P + 16), BAD),
    (dict(ws_bytes=64), SMALL), (dict(stats=None), BAD), (dict(stats=P + 2), BAD), (dict(count=-1), BAD),
    (dict(data=None), BAD), (dict(data=P + 2), BAD), (dict(out=P + 1, dtype=ia.IA_DTYPE_F16), BAD),
    (dict(rows=-1), BAD), (dict(dim=0), BAD), (dict(dim=4, stride=3), BAD), (dict(out=P + 400, dim=4, stride=4, out_stride=3), BAD),
    (dict(rows=1 << 40, dim=2, stride=2), BAD), (dict(dtype=3), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED),
    (dict(out=P + 36), BAD),  # overlaps its gradient
    (dict(out=P, rows=3, dim=2, stride=2, out_stride=3), BAD),  # the same start, another stride
])
def test_clip_refuses(kw, status):
    assert _clip(**kw) == {status}
    assert ia.ia_last_error() != ""


def _adam(max_norm=1.0, beta1=0.9, beta2=0.999, eps=1e-15, step=1, ws=P, ws_bytes=1 << 30, stats=P, **kw):
    d = dict(param=P, grad=P, m=P, v=P, param_f16=None, rows=10, dim=1, param_stride=1, lr=1e-3)
    d.update(kw)
    arr = (ia.AdamGroup * 1)(ia.AdamGroup(**d))
    return ia.load().ia_adam_clip_step(arr, 1, max_norm, beta1, beta2, eps, step, ws, ws_bytes, stats, None)


@pytest.mark.parametrize("kw,status", [
    (dict(max_norm=-0.5), BAD), (dict(step=0), BAD), (dict(beta1=1.0), BAD), (dict(beta2=-0.1), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(lr=-1.0), BAD), (dict(lr=float("nan")), BAD),
    (dict(param=None), BAD), (dict(grad=P + 2), BAD), (dict(param_f16=P + 1), BAD), (dict(rows=-1), BAD),
    (dict(dim=0), BAD), (dict(dim=4, param_stride=3), BAD), (dict(rows=1 << 40, dim=2, param_stride=2), BAD),
    (dict(ws_bytes=64), SMALL), (dict(stats=None), BAD),
])
def test_adam_clip_refuses(kw, status):
    assert _adam(**kw) == status


def test_workspace_sizes():
    assert ia.ia_clip_workspace_size(0) > 0
    assert ia.ia_clip_workspace_size(1000) > ia.ia_clip_workspace_size(10)
    assert ia.ia_clip_workspace_size(2 ** 31 - 1) > 0
    for bad in (-1,):
        with pytest.raises(ia.IAError):
            ia.ia_clip_workspace_size(bad)
    for fn in (ia.ia_mx4_matmul_workspace_size, ia.ia_mx4_linear_workspace_size,
               ia.ia_mx4_linear_backward_workspace_size):
        assert fn(0, 0, 0) >= 0 and fn(300_000, 256, 256) >= 0
        for args in ((-1, 1, 1), (1, -1, 1), (1, 1, -1), (1 << 31, 1, 1), (1, 1 << 31, 1), (1, 1, 1 << 31)):
            with pytest.raises(ia.IAError) as e:
                fn(*args)
            assert e.value.status == BAD


def _q(**kw):
    d = dict(codes=P, scales=P, rows=8, cols=64)
    d.update(kw)
    return ia.Mx4(**d)


@pytest.mark.parametrize("kw,q,status", [
    (dict(x=None), {}, BAD), (dict(x=P + 2), {}, BAD), (dict(dtype=3), {}, UNSUPPORTED), (dict(rows=-1), {}, BAD),
    (dict(ld=63), {}, BAD), (dict(ld=-64), {}, BAD), (dict(rows=1 << 40), dict(rows=1 << 40), BAD),
    ({}, dict(codes=None), BAD), ({}, dict(codes=P + 8), BAD), ({}, dict(scales=None), BAD), ({}, dict(rows=9), BAD),
    ({}, dict(cols=65), BAD), (dict(transpose=1), {}, BAD), (dict(ld=1 << 40), {}, BAD),
])
def test_quantize_refuses(kw, q, status):
    d = dict(x=P, dtype=ia.IA_DTYPE_F32, rows=8, cols=64, ld=64, transpose=0)
    d.update(kw)
    L = ia.load()
    assert L.ia_mx4_quantize(d["x"], d["dtype"], d["rows"], d["cols"], d["ld"], d["transpose"], C.byref(_q(**q)),
                             None) == status
    assert L.ia_mx4_quantize(P, 0, 8, 64, 64, 0, None, None) == BAD


def test_dequantize_refuses():
    L = ia.load()
    q = _q()
    assert L.ia_mx4_dequantize(C.byref(q), 0, P, 63, None) == BAD
    assert L.ia_mx4_dequantize(C.byref(q), 0, P, 0, None) == BAD  # one output row for all
    assert L.ia_mx4_dequantize(C.byref(q), 0, None, 64, None) == BAD
    assert L.ia_mx4_dequantize(C.byref(q), 7, P, 64, None) == UNSUPPORTED
    assert L.ia_mx4_dequantize(None, 0, P, 64, None) == BAD


@pytest.mark.parametrize("kw,status", [
    (dict(a=_q(cols=32)), BAD), (dict(a=None), BAD), (dict(b=_q(codes=P + 4)), BAD), (dict(act=1), UNSUPPORTED),
    (dict(dtype=5), UNSUPPORTED), (dict(ldc=7), BAD), (dict(ldc=0), BAD), (dict(c=None), BAD), (dict(c=P + 2), BAD),
    (dict(bias=P + 1), BAD), (dict(a=_q(rows=1 << 31, cols=64)), BAD),
])
def test_matmul_refuses(kw, status):
    d = dict(a=_q(rows=4), b=_q(), bias=None, act=ia.IA_ACT_NONE, dtype=0, c=P, ldc=8, ws=P, ws_bytes=1 << 40)
    d.update(kw)
    ref = lambda q: None if q is None else C.byref(q)  # noqa: E731
    assert ia.load().ia_mx4_matmul(ref(d["a"]), ref(d["b"]), d["bias"], d["act"], d["dtype"], d["c"], d["ldc"], d["ws"],
                                   d["ws_bytes"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(w=None), BAD), (dict(x=None), BAD), (dict(ldx=63), BAD), (dict(ldy=7), BAD), (dict(M=-1), BAD),
    (dict(M=1 << 31), BAD), (dict(act=1), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED), (dict(y=None), BAD),
])
def test_linear_refuses(kw, status):
    d = dict(x=P, dtype=0, M=4, ldx=64, w=_q(), bias=None, act=-1, y=P, ldy=8, ws=P, ws_bytes=1 << 40)
    d.update(kw)
    assert ia.load().ia_mx4_linear(d["x"], d["dtype"], d["M"], d["ldx"], None if d["w"] is None else C.byref(d["w"]),
                                   d["bias"], d["act"], d["y"], d["ldy"], d["ws"], d["ws_bytes"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), BAD), (dict(lddy=7), BAD), (dict(y=P + 2), BAD), (dict(ldy=7), BAD), (dict(x=None), BAD),
    (dict(ldx=63), BAD), (dict(wt=None), BAD), (dict(wt=_q()), BAD), (dict(lddx=0), BAD), (dict(dtype=4), UNSUPPORTED),
    (dict(M=-1), BAD), (dict(K=1 << 31), BAD), (dict(db=P + 2), BAD), (dict(dw=P + 2), BAD), (dict(ws_bytes=16), SMALL),
])
def test_linear_backward_refuses(kw, status):
    d = dict(dy=P, lddy=8, y=P, ldy=8, x=P, ldx=64, dtype=0, M=4, N=8, K=64, wt=_q(rows=64, cols=8), dx=P, lddx=64,
             dw=P, db=P, ws=P, ws_bytes=1 << 40)
    d.update(kw)
    wt = None if d["wt"] is None else C.byref(d["wt"])
    assert ia.load().ia_mx4_linear_backward(d["dy"], d["lddy"], d["y"], d["ldy"], d["x"], d["ldx"], d["dtype"], d["M"],
                                            d["N"], d["K"], wt, d["dx"], d["lddx"], d["dw"], d["db"], d["ws"],
                                            d["ws_bytes"], None) == status
