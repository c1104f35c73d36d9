"""What the Python calls of clipping and MXFP4 hand to the C ABI, checked on the
host: the library's entry points are replaced by recorders, so nothing is
dereferenced and no GPU is needed."""
import copy
import pickle

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


def _adam(**kw):
    """(an optimiser of one group with a mirror, its gradients), host tensors."""
    d = dict(param=torch.zeros(6, 4), grad=torch.zeros(6, 4), m=torch.zeros(6, 4), v=torch.zeros(6, 4),
             f16=torch.zeros(24, dtype=torch.int16))
    d.update(kw)
    opt = P.Adam({"w": {"param": d["param"], "lr": 1e-3, "f16": d["f16"]}}, warmup=0, total=10)
    opt.state["w"] = (d["m"], d["v"])
    return opt, {"w": d["grad"]}


@pytest.mark.parametrize("kw,what", [
    ({}, "one GPU"),  # all of it on the host
    (dict(m=torch.zeros(6, 3)), "moments"), (dict(v=torch.zeros(23)), "moments"), (dict(m=torch.zeros(0)), "moments"),
    (dict(m=torch.zeros(6, 3), v=torch.zeros(6, 3)), "moments"), (dict(m=torch.zeros(25), v=torch.zeros(25)), "moments"),
    (dict(m=torch.zeros(6, 4, dtype=torch.float16)), "moments"), (dict(v=torch.zeros(3, 4, dtype=torch.float64)), "moments"),
    (dict(m=torch.zeros(4, 6).t()), "moments"), (dict(v=torch.zeros(6, 8)[:, ::2]), "moments"),
    (dict(m=torch.empty(6, 4, device="meta")), "moments"),
    (dict(f16=torch.zeros(23, dtype=torch.float16)), "mirror"), (dict(f16=torch.zeros(24, dtype=torch.float32)), "mirror"),
    (dict(f16=torch.zeros(12, dtype=torch.float32)), "mirror"), (dict(f16=torch.zeros(24, dtype=torch.uint8)), "mirror"),
    (dict(f16=torch.zeros(48, dtype=torch.float16)[::2]), "mirror"),
    (dict(grad=torch.zeros(24)), "one shape"), (dict(grad=torch.zeros(6, 4, dtype=torch.float16)), "one shape"),
    (dict(param=torch.zeros(4, 6).t()), "contiguous"),
])
def test_adam_refuses_arrays_that_the_kernel_would_pass_the_end_of(calls, monkeypatch, kw, what):
    """Host arrays, and moments or mirrors of another size, type or layout: refused before their addresses are taken."""
    if what == "contiguous":  # the check after the device's
        monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    with pytest.raises(ValueError, match=what):
        opt, grads = _adam(**kw)
        opt.step(grads, max_norm=1.0)
    assert "ia_adam_clip_step" not in calls


def test_adam_refuses_moments_on_another_device(calls, monkeypatch):
    opt, grads = _adam()
    m = opt.state["w"][0]
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    opt.step(grads, max_norm=1.0)
    assert calls.pop("ia_adam_clip_step")
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: int(t is m))
    with pytest.raises(ValueError, match="moments"):
        opt.step(grads, max_norm=1.0)
    assert "ia_adam_clip_step" not in calls


@pytest.mark.parametrize("put", [
    lambda opt, mv: opt.state.__setitem__("w", mv), lambda opt, mv: opt.state.update(w=mv),
    lambda opt, mv: opt.state.update({"w": mv}), lambda opt, mv: opt.state.setdefault("x", mv),
    lambda opt, mv: setattr(opt, "state", {"w": mv}), lambda opt, mv: opt.state.__ior__({"w": mv}),
    lambda opt, mv: copy.deepcopy(opt).state.update(w=mv), lambda opt, mv: pickle.loads(pickle.dumps(opt.state)).update(w=mv),
])
def test_every_way_to_put_moments_in_checks_them(put):
    opt, _ = _adam()
    put(opt, [torch.ones(6, 4), torch.ones(6, 4)])
    with pytest.raises(ValueError, match="moments"):
        put(_adam()[0], (torch.ones(6, 4), torch.ones(6, 4).half()))


def test_adam_refuses_groups_on_several_devices(calls, monkeypatch):
    opt, grads = _adam()
    opt.groups["b"] = {"param": torch.zeros(5), "lr": 1e-3}
    opt.state["b"] = (torch.zeros(5), torch.zeros(5))
    grads["b"] = torch.zeros(5)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    opt.step(grads, max_norm=1.0)
    assert len(calls.pop("ia_adam_clip_step")[0]) == 2
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: int(t.numel() == 5))
    with pytest.raises(ValueError, match="one GPU"):
        opt.step(grads, max_norm=1.0)
    assert "ia_adam_clip_step" not in calls


@pytest.mark.parametrize("M,N,K,most", [(8_000_000, 256, 256, 340e6), (8_000_000, 64, 64, 140e6), (300_000, 256, 192, 80e6)])
def test_workspace_of_narrow_gradients(M, N, K, most):
    """Mask words and the blocks' sums; not the 4-bit copies of all rows that wider layers need (3.3 GB for the first)."""
    assert ia.ia_mx4_linear_backward_workspace_size(M, N, K) <= most


class _Packed:
    """Stands for an Mx4Tensor with memory on the host."""

    def __init__(self, rows, cols):
        self._codes = self.codes = torch.zeros((rows, (cols + 31) // 32 * 16), dtype=torch.uint8)
        self.rows, self.cols, self.c = rows, cols, None


@pytest.mark.parametrize("far", ["x", "w", "bias", "out", "dy", "y", "wt", "a", "b", "q", "grad", "codes"])
def test_tensors_on_several_devices_are_refused(calls, monkeypatch, far):
    """One argument on another GPU: no entry point is reached."""
    for name in ("ia_mx4_quantize", "ia_mx4_dequantize", "ia_mx4_matmul", "ia_mx4_linear"):
        monkeypatch.setattr(ia, name, lambda *a, _n=name: calls.__setitem__(_n, a))
    monkeypatch.setattr(P, "_bias", lambda bias, n: bias)
    t = dict(x=torch.zeros(6, 40), bias=torch.zeros(8), out=torch.zeros(6, 8), dy=torch.zeros(6, 8), y=torch.zeros(6, 8),
             grad=torch.zeros(9), codes=torch.zeros(6, 32, dtype=torch.uint8), w=_Packed(8, 40), wt=_Packed(40, 8),
             a=_Packed(6, 40), b=_Packed(8, 40), q=_Packed(6, 40))
    uses = {
        "linear": (("x", "w", "bias", "out"), lambda: P.mx4_linear(t["x"], t["w"], t["bias"], out=t["out"])),
        "backward": (("dy", "x", "y", "wt"), lambda: P.mx4_linear_backward(t["dy"], t["x"], t["wt"], t["y"])),
        "matmul": (("a", "b", "bias", "out"), lambda: P.mx4_matmul(t["a"], t["b"], t["bias"], out=t["out"])),
        "quantize": (("x", "q"), lambda: P.mx4_quantize(t["x"], out=t["q"])),
        "dequantize": (("x", "q"), lambda: P.Mx4Tensor.dequantize(t["q"], out=t["x"])),
        "clip": (("x", "grad"), lambda: P.GradClip([t["x"], t["grad"]])),
        "tensor": (("codes",), None),
    }
    for args, call in uses.values():
        if call:
            call()
    assert len(calls) == 5
    calls.clear()
    other = t[far]._codes if isinstance(t[far], _Packed) else t[far]
    monkeypatch.setattr(torch.Tensor, "get_device", lambda u: int(u is other))
    refused = 0
    for args, call in uses.values():
        if call and far in args:
            with pytest.raises(ValueError, match="several devices"):
                call()
            refused += 1
    assert refused or far == "codes"
    if far == "codes":
        monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda u: True), raising=False)
        with pytest.raises(ValueError, match="several devices"):
            P.Mx4Tensor(t["codes"], torch.zeros(6, 2, dtype=torch.uint8), 40)
    assert not calls


def test_the_current_stream_by_either_way(monkeypatch):
    """torch's raw handle is not part of its public interface: without it the public call serves."""
    class Stream:
        cuda_stream = 4711

    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 100 + device, raising=False)
    assert ia._stream() == 103 and ia._stream(Stream) == 4711
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    assert ia._stream() == 4711


def test_the_count_of_steps_left_out_is_made_with_the_optimiser(calls, monkeypatch):
    """Not within the first step, where a captured graph would clear it in every replay."""
    opt, grads = _adam()
    count = opt.skipped
    assert count.dtype == torch.int32 and count.tolist() == [0] and count.device == grads["w"].device
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    opt.step(grads, max_norm=1.0)
    assert opt.skipped is count and calls["ia_adam_clip_step"][-1] is count
    empty = P.Adam({}, warmup=0, total=1)
    assert empty.skipped is None
