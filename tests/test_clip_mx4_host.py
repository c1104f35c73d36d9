"""What the Python calls of clipping and MXFP4 hand to the C ABI, checked on the
host: the library's entry points are replaced by recorders, so nothing is
dereferenced and no GPU is needed."""
import pytest
import torch

from implicit_attribute_decode_amd import ia, pipeline as P


@pytest.fixture
def calls(monkeypatch):
    """{entry point: arguments of its last call}; tensors off the GPU pass for GPU ones."""
    seen = {}
    monkeypatch.setattr(P, "_dtype", lambda t: P._DTYPES[t.dtype])
    for name in ("ia_grad_norm", "ia_clip_grad_norm", "ia_adam_clip_step", "ia_mx4_linear_backward"):
        monkeypatch.setattr(ia, name, lambda *a, _n=name: seen.__setitem__(_n, a))
    return seen


@pytest.fixture(params=[torch.bfloat16, torch.float16, torch.float64], ids=str)
def default_type(request):
    before = torch.get_default_dtype()
    torch.set_default_dtype(request.param)
    yield request.param
    torch.set_default_dtype(before)


def test_outputs_are_float32_under_another_default_type(calls, default_type):
    """The kernels write 32-bit gradients, moments and statistics whatever torch's default type is."""
    x, dy = (torch.zeros(s, dtype=torch.float32) for s in ((6, 40), (6, 8)))
    got = P.mx4_linear_backward(dy, x, None, want_x=False)
    passed = calls["ia_mx4_linear_backward"]
    assert passed[13] is got["weight"] and passed[14] is got["bias"]
    assert got["weight"].dtype == got["bias"].dtype == torch.float32
    clip = P.GradClip([x])
    assert clip(1.0).dtype == clip.norm().dtype == torch.float32
    opt = P.Adam({"x": {"param": x, "lr": 1e-3}}, warmup=0, total=1)
    assert all(t.dtype == torch.float32 and t.shape == x.shape for t in opt.state["x"])
    assert opt.state["x"][0].data_ptr() != opt.state["x"][1].data_ptr()


def _far(rows, dim, stride):
    """A tensor without memory whose rows are `stride` elements apart."""
    return torch.empty_strided((rows, dim), (stride, 1), dtype=torch.float32, device="meta")


def test_row_strides_past_32_bits_are_refused(calls):
    """A stride of 2^32 + 100 would reach the library as 100: rows of 100 values as a dense tensor."""
    near = _far(3, 100, 2 ** 31 - 1)
    assert P.GradClip([near])._arr[0].stride == 2 ** 31 - 1
    for stride in (2 ** 31, 2 ** 32 + 100, 2 ** 33 + 104):
        far = _far(3, 100, stride)
        for args in (([far],), ([near, far],), ([near], [far]), ([torch.empty((3, 100), device="meta")], [far])):
            with pytest.raises(ValueError):
                P.GradClip(*args)
    wide = _far(2, 2 ** 32 + 5, 2 ** 32 + 6)
    with pytest.raises(ValueError):
        P.GradClip([wide])


def test_adam_row_strides_past_32_bits_are_refused(monkeypatch):
    class Entry:
        @staticmethod
        def ia_adam_step_strided(*a):
            raise AssertionError("reached the library")

    monkeypatch.setattr(ia, "load", lambda: Entry)
    dense = torch.empty((3, 100), dtype=torch.float32, device="meta")
    with pytest.raises(ValueError):
        ia.ia_adam_step_strided(_far(3, 100, 2 ** 32 + 100), dense, dense, dense, 1e-3, 0.9, 0.999, 1e-15, 1)
