"""GPU: h of the layer for a few tokens on its way between the two products: fp32, or two bf16 terms where
slots share experts.  The inputs and the bounds are layer_ref.py's; test_layer_h_host.py shows that they tell one
bf16 term from two."""
import pytest
import torch

import layer_ref as layer
from combine_topk_idx_multihot_amd import binding as B

FORMATS = ("bf16", "fp8", "mxfp4")
OWN = [  # T, k, E, lb, EL, H, I: at most one slot per eight experts, every slot on its own
    (1, 8, 64, 0, 64, 512, 256), (3, 4, 96, 16, 64, 256, 128), (1, 1, 8, 0, 8, 256, 128), (2, 6, 96, 0, 96, 768, 384),
]
SHARED = [  # more than 16 slots, and at least one per expert
    (24, 4, 8, 0, 8, 512, 256), (17, 2, 16, 4, 8, 256, 128), (40, 8, 16, 0, 16, 768, 384), (70, 3, 4, 0, 4, 512, 128),
    (256, 4, 6, 0, 6, 256, 128), (33, 4, 128, 0, 128, 256, 640),
]


def overs(got, want, bound):
    """How many values lie outside the bound and one rounding to bf16."""
    return int(((got.double() - want).abs() > bound + 2.0 ** -8 * (want.abs() + bound)).sum())


def run(fmt, shape, h_step):
    T, k, E, lb, EL, H, I = shape
    idx, w, x, (w1, s1, v1), (w2, s2, v2) = layer.make(fmt, *shape, seed=sum(shape))
    want, bound = layer.layer(idx, w, x, v1, v2, lb, h_step)
    d = B.make_desc(T, k, E, lb, EL)
    idx, w, x, w1, s1, w2, s2 = (None if t is None else t.cuda() for t in (idx, w, x, w1, s1, w2, s2))
    got = B.layer_tokens(d, idx, w, x, w1, w2, s1, s2).cpu()
    assert torch.isfinite(got).all() and overs(got, want, bound) == 0, (overs(got, want, bound), got.numel())


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", SHARED, ids=lambda s: "-".join(map(str, s)))
def test_slots_that_share_experts_keep_two_terms_of_h(shape, fmt):
    run(fmt, shape, 2.0 ** -16)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", OWN, ids=lambda s: "-".join(map(str, s)))
def test_slots_on_their_own_keep_h_in_fp32(shape, fmt):
    run(fmt, shape, 0.0)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [OWN[0], SHARED[0]], ids=lambda s: "-".join(map(str, s)))
def test_an_infinite_weight_stays_in_its_output(shape):
    """Infinite or NaN for the tokens of that expert in that column, nothing else changed."""
    T, k, E, lb, EL, H, I = shape
    idx, w, x, (w1, _, _), (w2, _, _) = layer.make("bf16", *shape, seed=5)
    d = B.make_desc(T, k, E, lb, EL)
    idx, w, x, w1, w2 = (t.cuda() for t in (idx, w, x, w1, w2))
    want = B.layer_tokens(d, idx, w, x, w1, w2)
    e = int(idx[0, 0])
    w2[e - lb, 7, 33] = float("inf")
    got = B.layer_tokens(d, idx, w, x, w1, w2)
    mine = (idx == e).any(1)
    assert not torch.isfinite(got[mine, 7]).any()
    got[mine, 7] = want[mine, 7]
    assert torch.equal(got, want)
