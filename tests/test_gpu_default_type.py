"""Results under another torch default type: the framework's outputs stay
32-bit floats, equal bit for bit to those under float32."""
import numpy as np
import pytest
import torch

from implicit_attribute_decode_amd import scenes as S
from implicit_attribute_decode_amd.pipeline import Adam, Decoder, GradClip, mx4_linear_backward, mx4_quantize

from gpu_util import cuda

pytestmark = pytest.mark.gpu


def _results():
    rng = np.random.default_rng(1)
    x, dy, w = (cuda(rng.normal(0, 1, s).astype(np.float32)) for s in ((300, 70), (300, 40), (40, 70)))
    out = {f"layer_{k}": v for k, v in mx4_linear_backward(dy, x, mx4_quantize(w, transpose=True)).items()}
    out["norm"] = GradClip([x, dy]).norm(1.0)
    opt = Adam({"w": {"param": w, "lr": 1e-3}}, warmup=0, total=10)
    for _ in range(2):
        out["stats"] = opt.step({"w": out["layer_weight"]}, max_norm=0.5)
    opt.step({"w": out["layer_weight"]})
    out.update(w=w, m=opt.state["w"][0], v=opt.state["w"][1])
    D = Decoder(S.single_decoder())
    pos = cuda(rng.uniform(0, 1, (2000, 4)).astype(np.float32))
    attrs = D.decode_xyzt(pos)
    out.update(attrs)
    out["pos"] = D.backward(pos, {k: torch.ones_like(v) for k, v in attrs.items()})["pos"]
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float64], ids=str)
def test_results_do_not_depend_on_the_default_type(dtype):
    want = _results()
    before = torch.get_default_dtype()
    torch.set_default_dtype(dtype)
    try:
        got = _results()
    finally:
        torch.set_default_dtype(before)
    torch.cuda.synchronize()
    for k in want:
        assert got[k].dtype == torch.float32 and torch.equal(got[k], want[k]), k
