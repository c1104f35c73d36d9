"""The 4-bit training example end to end: layers, gradients, clipped Adam,
quantising again, and a decoder's tables stored in 4 bits."""
import os
import sys

import pytest
import torch

from oracle import mx4 as O
from implicit_attribute_decode_amd import scenes as S
from implicit_attribute_decode_amd.pipeline import Decoder

from gpu_util import host, say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_training_in_four_bits_lowers_the_loss():
    import mx4_training as E

    net, losses, norms, factors = E.train(steps=40, rows=4000)
    say("losses", [round(v, 3) for v in losses[::8]], "factors", [round(v, 3) for v in factors[::8]])
    assert losses[-1] < 0.5 * losses[0]
    assert all(0.0 < f <= 1.0 for f in factors) and min(factors) < 1.0
    assert all((f == 1.0) == (n <= 0.5) for f, n in zip(factors, norms))
    for layer in net:  # the 4-bit forms are the masters'
        codes, scales = O.quantize(host(layer.weight))
        assert (host(layer.w.codes) == codes).all() and (host(layer.w.scales) == scales).all()
        codes, scales = O.quantize(host(layer.weight).T)
        assert (host(layer.wt.codes) == codes).all() and (host(layer.wt.scales) == scales).all()


def test_tables_stored_in_four_bits():
    import mx4_training as E

    D, ref = Decoder(S.single_decoder()), Decoder(S.single_decoder())
    before = D._tables.clone()
    a, b = E.store_tables(D)
    assert b * 64 == a * 17  # 17 bytes for 32 values of 2 bytes
    flat = before.view(before.shape[0], -1)[:2, :4096]
    want = torch.as_tensor(O.values(host(flat.float()))).half()
    assert torch.equal(D._tables.view(before.shape[0], -1)[:2, :4096].cpu(), want)
    x = torch.rand((500, 4), device="cuda")
    assert not torch.equal(D.decode_xyzt(x)["colors"], ref.decode_xyzt(x)["colors"])
