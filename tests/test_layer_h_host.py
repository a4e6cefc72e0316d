"""CPU: what the inputs of layer_ref.py can tell: an h of one bf16 term between the layer's two products is
seen, one of two terms or of fp32 passes."""
import pytest
import torch

import layer_ref as layer
from test_gpu_layer_h import OWN, SHARED, overs


def one_term(h):
    return h.to(torch.bfloat16).double()


def two_terms(h):
    top = h.float().to(torch.bfloat16)
    return top.double() + (h.float() - top.float()).to(torch.bfloat16).double()


def shifted(h):
    """The second term of another slot."""
    top = one_term(h)
    return top + (h - top).roll(1, 0)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("shape", OWN[:2] + SHARED[:2], ids=lambda s: "-".join(map(str, s)))
def test_one_term_is_seen(shape, fmt):
    idx, w, x, (_, _, v1), (_, _, v2) = layer.make(fmt, *shape, seed=sum(shape))

    def count(hold, step):
        out = layer.layer(idx, w, x, v1, v2, shape[3], step, hold)[0].float().to(torch.bfloat16)
        return overs(out, *layer.layer(idx, w, x, v1, v2, shape[3], step))

    assert count(lambda h: h.float().double(), 0.0) == 0 and count(two_terms, 2.0 ** -16) == 0
    assert count(one_term, 0.0) > 20 and count(one_term, 2.0 ** -16) > 20
    if shape in SHARED:
        assert count(shifted, 2.0 ** -16) > 20


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp4"])
def test_sums_are_exact(fmt):
    """Gate and up in fp32, summed forwards and backwards, are the 64-bit ones."""
    _, _, x, (_, _, v1), _ = layer.make(fmt, 3, 2, 4, 0, 4, 2048, 128, seed=1)
    want = x.double() @ v1[0].T
    for order in (range(2048), range(2047, -1, -1)):
        y = torch.zeros(want.shape)
        for c in order:
            y += x[:, c:c + 1].float() * v1[0][:, c].float()
        assert torch.equal(y.double(), want)
    assert 0.3 < want.std() < 6
