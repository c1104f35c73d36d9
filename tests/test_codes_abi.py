"""Argument checks of the lookup, dropout and group-scaled 4-bit entry points
that need no GPU: every refusal comes back before anything is enqueued (fake
aligned addresses: nothing is dereferenced)."""
import ctypes as C

import pytest
import torch

from implicit_attribute_decode_amd import ia, pipeline

P = 1 << 20
BAD, UNSUPPORTED, SMALL = ia.IA_ERR_INVALID_ARG, ia.IA_ERR_UNSUPPORTED, ia.IA_ERR_WORKSPACE_TOO_SMALL
NAN, INF = float("nan"), float("inf")


def _drop(p=0.5, seed=1, offset=0, step=None):
    return ia.Drop(p, seed, offset, step)


def _ref(s):
    return None if s is None else C.byref(s)


def _far(k):
    return P + (k << 32)  # places that cannot overlap


@pytest.mark.parametrize("kw,status", [
    (dict(drop=None), BAD), (dict(drop=_drop(-0.1)), BAD), (dict(drop=_drop(1.5)), BAD), (dict(drop=_drop(NAN)), BAD),
    (dict(drop=_drop(step=P + 4)), BAD), (dict(x=None), BAD), (dict(x=P + 2), BAD), (dict(out=None), BAD), (dict(rows=-1), BAD),
    (dict(rows=1 << 31), BAD), (dict(cols=1 << 31, ldx=1 << 31, ldo=1 << 31), BAD), (dict(ldx=63), BAD), (dict(ldo=0), BAD),
    (dict(ldo=63), BAD), (dict(dtype=3), UNSUPPORTED), (dict(out=P + 4), BAD), (dict(out=P, ldo=65), BAD),
    (dict(drop=_drop(step=_far(1) + 8)), BAD),  # the call's number lies where the output is written
])
def test_dropout_refuses(kw, status):
    d = dict(x=P, dtype=0, rows=8, cols=64, ldx=64, drop=_drop(), out=_far(1), ldo=64)
    d.update(kw)
    assert ia.load().ia_dropout(d["x"], d["dtype"], d["rows"], d["cols"], d["ldx"], _ref(d["drop"]), d["out"], d["ldo"],
                                None) == status
    assert ia.ia_last_error() != ""


LOOKUP = [
    (dict(index=None), BAD), (dict(index=_far(1) + 2), BAD), (dict(index_bytes=2), UNSUPPORTED), (dict(n=-1), BAD),
    (dict(n=1 << 31), BAD), (dict(stride=-1), BAD), (dict(stride=1 << 40), BAD), (dict(scale=NAN), BAD), (dict(scale=INF), BAD),
    (dict(scale=1e39), BAD), (dict(scale=1e38, drop=_drop(0.9)), BAD), (dict(drop=_drop(2.0)), BAD), (dict(out=None), BAD),
    (dict(out=_far(2) + 1), BAD), (dict(ldo=63), BAD), (dict(ldo=0), BAD), (dict(out_dtype=5), UNSUPPORTED),
    (dict(out=_far(1) - 8), BAD), (dict(out=P), BAD),
]


@pytest.mark.parametrize("kw,status", LOOKUP + [
    (dict(table=None), BAD), (dict(table=P + 2), BAD), (dict(dtype=7), UNSUPPORTED), (dict(entries=-1), BAD),
    (dict(entries=1 << 31), BAD), (dict(dim=1 << 31), BAD), (dict(ld=63), BAD),
])
def test_embedding_refuses(kw, status):
    d = dict(table=P, dtype=0, entries=100, dim=64, ld=64, index=_far(1), index_bytes=8, n=10, stride=1, scale=1.0, drop=None,
             out_dtype=0, out=_far(2), ldo=64)
    d.update(kw)
    assert ia.load().ia_embedding(d["table"], d["dtype"], d["entries"], d["dim"], d["ld"], d["index"], d["index_bytes"], d["n"],
                                  d["stride"], d["scale"], _ref(d["drop"]), d["out_dtype"], d["out"], d["ldo"], None) == status


@pytest.mark.parametrize("kw,status", LOOKUP + [
    (dict(table=None), BAD), (dict(table=ia.Mx4(P + 8, _far(4), 100, 64)), BAD), (dict(table=ia.Mx4(P, None, 100, 64)), BAD),
    (dict(table=ia.Mx4(P, _far(4), 1 << 31, 64)), BAD), (dict(out=_far(4)), BAD),
])
def test_embedding_mx4_refuses(kw, status):
    d = dict(table=ia.Mx4(P, _far(4), 100, 64), index=_far(1), index_bytes=8, n=10, stride=1, scale=1.0, drop=None, out_dtype=0,
             out=_far(2), ldo=64)
    d.update(kw)
    assert ia.load().ia_embedding_mx4(_ref(d["table"]), d["index"], d["index_bytes"], d["n"], d["stride"], d["scale"],
                                      _ref(d["drop"]), d["out_dtype"], d["out"], d["ldo"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), BAD), (dict(dy=P + 2), BAD), (dict(dtype=3), UNSUPPORTED), (dict(lddy=63), BAD), (dict(dim=1 << 31), BAD),
    (dict(index=None), BAD), (dict(index_bytes=1), UNSUPPORTED), (dict(n=-1), BAD), (dict(stride=-3), BAD),
    (dict(entries=-1), BAD), (dict(entries=1 << 31), BAD), (dict(scale=NAN), BAD), (dict(drop=_drop(-1.0)), BAD),
    (dict(grad=None), BAD), (dict(grad=_far(2) + 2), BAD), (dict(ws=None), BAD), (dict(ws=_far(3) + 16), BAD),
    (dict(ws_bytes=100), SMALL), (dict(grad=P + 64), BAD), (dict(ws=_far(2)), BAD), (dict(grad=_far(1)), BAD),
])
def test_embedding_backward_refuses(kw, status):
    d = dict(dy=P, dtype=0, dim=64, lddy=64, index=_far(1), index_bytes=8, n=10, stride=1, entries=100, scale=1.0, drop=None,
             grad=_far(2), ws=_far(3), ws_bytes=1 << 30)
    d.update(kw)
    assert ia.load().ia_embedding_backward(d["dy"], d["dtype"], d["dim"], d["lddy"], d["index"], d["index_bytes"], d["n"],
                                           d["stride"], d["entries"], d["scale"], _ref(d["drop"]), d["grad"], d["ws"],
                                           d["ws_bytes"], None) == status


def test_workspace_sizes():
    size = ia.ia_embedding_backward_workspace_size
    assert size(0, 10, 10) == size(10, 0, 10) == size(10, 10, 0) == 0
    assert 0 < size(1, 1, 1) < size(100_000, 150, 64) < size(300_000, 150, 64)
    for args in ((-1, 1, 1), (1, -1, 1), (1, 1, -1), (1 << 31, 1, 1), (1, 1 << 31, 1), (1 << 30, 1, 1 << 30)):
        with pytest.raises(ia.IAError) as e:
            size(*args)
        assert e.value.status == BAD
    linear = ia.ia_q4_linear_workspace_size
    assert linear(0, 0, 0, 0) == 0 and all(linear(d, 300_000, 256, 256) >= linear(d, 1, 256, 256) for d in (0, 1, 2))
    for args in ((0, -1, 1, 1), (0, 1, -1, 1), (1, 1, 1, -1), (2, 1 << 31, 1, 1), (0, 1, 1 << 31, 1), (0, 1, 1, 1 << 31),
                 (0, 1 << 30, 1 << 30, 1)):
        with pytest.raises(ia.IAError) as e:
            linear(*args)
        assert e.value.status == BAD
    with pytest.raises(ia.IAError) as e:
        linear(3, 1, 1, 1)
    assert e.value.status == UNSUPPORTED


def _q(**kw):
    d = dict(codes=_far(1), words=_far(2), rows=8, cols=130, group=64)
    d.update(kw)
    return ia.Q4(**d)


Q4 = [(dict(codes=None), BAD), (dict(codes=_far(1) + 8), BAD), (dict(words=None), BAD), (dict(words=_far(2) + 4), BAD),
      (dict(rows=-1), BAD), (dict(cols=-1), BAD), (dict(rows=1 << 31, cols=1), BAD), (dict(rows=1, cols=1 << 31), BAD),
      (dict(rows=1 << 30, cols=1 << 11), BAD), (dict(group=16), UNSUPPORTED),
      (dict(group=0), UNSUPPORTED), (dict(group=256), UNSUPPORTED)]


@pytest.mark.parametrize("q,status", Q4)
def test_q4_matrices_refused(q, status):
    L, ref = ia.load(), C.byref(_q(**q))
    assert L.ia_q4_quantize(P, 0, 130, ref, None) == status
    assert L.ia_q4_dequantize(ref, 0, P, 130, None) == status
    assert L.ia_q4_linear(P, 0, 4, 130, ref, None, -1, _far(3), 8, _far(4), 1 << 40, None) == status


def test_q4_conversions_refuse():
    L, ref = ia.load(), C.byref(_q())
    for x, dtype, ld, status in ((None, 0, 130, BAD), (P + 2, 0, 130, BAD), (P, 3, 130, UNSUPPORTED), (P, 0, 129, BAD),
                                 (_far(1) + 16, 0, 130, BAD), (_far(2), 0, 130, BAD)):
        assert L.ia_q4_quantize(x, dtype, ld, ref, None) == status
        assert L.ia_q4_dequantize(ref, dtype, x, ld, None) == status
    assert L.ia_q4_dequantize(ref, 0, P, 0, None) == BAD  # one output row for all
    assert L.ia_q4_quantize(P, 0, 130, None, None) == L.ia_q4_dequantize(None, 0, P, 130, None) == BAD


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), BAD), (dict(x=P + 2), BAD), (dict(ldx=129), BAD), (dict(ldy=7), BAD), (dict(ldy=0), BAD), (dict(M=-1), BAD),
    (dict(M=1 << 31), BAD), (dict(act=1), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED), (dict(y=None), BAD),
    (dict(bias=P + 1), BAD), (dict(w=None), BAD), (dict(y=P + 16), BAD), (dict(y=_far(1)), BAD), (dict(y=_far(2)), BAD),
    (dict(bias=_far(3)), BAD), (dict(w=_q(rows=1 << 31, cols=32)), BAD),
])
def test_q4_linear_refuses(kw, status):
    d = dict(x=P, dtype=0, M=4, ldx=130, w=_q(), bias=None, act=-1, y=_far(3), ldy=8, ws=_far(4), ws_bytes=1 << 40)
    d.update(kw)
    assert ia.load().ia_q4_linear(d["x"], d["dtype"], d["M"], d["ldx"], _ref(d["w"]), d["bias"], d["act"], d["y"], d["ldy"],
                                  d["ws"], d["ws_bytes"], None) == status


# ------------------------------------------------------------- Python calls


@pytest.mark.parametrize("args", [(-0.1, 0), (1.1, 0), (NAN, 0), (0.5, -1), (0.5, 2 ** 64), (0.5, 0, -1), (0.5, 0, 2 ** 64),
                                  (0.5, 0, 0, torch.zeros(1, dtype=torch.int64)), (0.5, 0, 0, torch.zeros(1))])
def test_dropouts_refused(args):
    with pytest.raises(ValueError):
        pipeline.Dropout(*args)


def test_tensors_off_the_gpu_are_refused():
    x, i = torch.zeros((3, 4)), torch.zeros(3, dtype=torch.int64)
    codes, words = torch.zeros((3, 16), dtype=torch.uint8), torch.zeros((3, 4), dtype=torch.int32)
    for call in (lambda: pipeline.Dropout(0.5, 1)(x), lambda: pipeline.embedding(x, i), lambda: pipeline.embedding_backward(x, i, 3),
                 lambda: pipeline.q4_quantize(x), lambda: pipeline.Q4Tensor(codes, words, 32, 32)):
        with pytest.raises(ValueError):
            call()


@pytest.fixture
def calls(monkeypatch):
    """{entry point: arguments of its last call}; tensors off the GPU pass for GPU ones."""
    seen = {}
    monkeypatch.setattr(pipeline, "_dtype", lambda t: pipeline._DTYPES[t.dtype])
    monkeypatch.setattr(pipeline, "_here", lambda *t: None)
    monkeypatch.setattr(pipeline, "_index", lambda i: (pipeline._INDEX_BYTES[i.dtype], i.shape[0], i.stride(0)))
    for name in ("ia_dropout", "ia_embedding", "ia_embedding_backward"):
        monkeypatch.setattr(ia, name, lambda *a, _n=name: seen.__setitem__(_n, a))
    return seen


def test_shapes_types_and_strides_that_do_not_fit(calls):
    x, i = torch.zeros((6, 4)), torch.zeros(6, dtype=torch.int64)
    d = pipeline.Dropout(0.5, 1)
    for call in (lambda: d(x, out=torch.zeros((6, 5))), lambda: d(x, out=x.half()), lambda: d(x[0]), lambda: d(x.t()),
                 lambda: pipeline.embedding(x, i, out=torch.zeros((5, 4))),
                 lambda: pipeline.embedding(x, i, dtype=torch.float16, out=torch.zeros((6, 4))),
                 lambda: pipeline.embedding(x.t(), i), lambda: pipeline.embedding(x[0], i),
                 lambda: pipeline.embedding_backward(x, i[:5], 9), lambda: pipeline.embedding_backward(x.t(), i[:4], 9),
                 lambda: pipeline.embedding_backward(x, i, 9, out=torch.zeros((9, 5))),
                 lambda: pipeline.embedding_backward(x, i, 9, out=torch.zeros((9, 4), dtype=torch.float16))):
        with pytest.raises(ValueError):
            call()
    assert not calls


def test_outputs_have_the_types_asked_for_under_another_default_type(calls):
    x, i = torch.zeros((6, 4), dtype=torch.float16), torch.zeros(6, dtype=torch.int32)
    torch.set_default_dtype(torch.float64)
    try:
        assert pipeline.embedding_backward(x, i, 9).dtype == torch.float32
        assert pipeline.embedding(x, i).dtype == torch.float16
        assert pipeline.embedding(x, i, dtype=torch.bfloat16).dtype == torch.bfloat16
    finally:
        torch.set_default_dtype(torch.float32)


@pytest.mark.parametrize("zeros", [torch.tensor([[16]]), torch.tensor([[-1]]), torch.tensor([[1.0]]), 16, 0.5])
def test_zeros_out_of_range_are_refused(zeros):
    with pytest.raises(ValueError, match="zeros"):
        pipeline.Q4Tensor.from_parts(torch.zeros((1, 16), dtype=torch.uint8), torch.ones((1, 1)), zeros, 32, 32)


def test_index_types_refused():
    for i in (torch.zeros(3), torch.zeros((2, 2), dtype=torch.int64), torch.zeros(3, dtype=torch.int16),
              torch.zeros(3, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            pipeline._index(i)
