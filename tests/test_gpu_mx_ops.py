"""GPU: the torch ops of the MXFP4 path and of the layer for a few tokens: torch's own checks of the registrations,
and whole layers under torch.compile, with a changing number of tokens too."""
import pytest
import torch

import mx_ref as mx
from combine_topk_idx_multihot_amd import ops
from test_gpu_layer_tokens import FORMATS, weights

pytestmark = pytest.mark.gpu

T, K, E, H, I = 48, 2, 8, 256, 128
CHECKS = ("test_schema", "test_faketensor")


def inputs(T=T, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    idx = torch.rand((T, E), generator=g, device="cuda").topk(K, 1).indices
    w = torch.rand((T, K), generator=g, device="cuda")
    return torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16), idx, w, g


def test_ops_pass_torchs_checks():
    x, idx, w, g = inputs()
    for v in (x, x.float()):
        torch.library.opcheck(ops.quantize_mxfp4, (v,), test_utils=CHECKS)
    q, s = ops.quantize_mxfp4(x)
    for f32 in (False, True):
        torch.library.opcheck(ops.dequantize_mxfp4, (q, s, f32), test_utils=CHECKS)
    *handle, host = ops.route(idx, E, 0, E, 1, 0)
    where, R = (*handle, E, 0, 1, 0), int(host[0])
    torch.library.opcheck(ops.dispatch_mxfp4, (x, w, *where, R), test_utils=CHECKS)
    rows, scale, *_ = ops.dispatch_mxfp4(x, w, *where, R)
    w1, w2 = mx.make_weights(E, 2 * I, H, g), mx.make_weights(E, 264, H, g)
    torch.library.opcheck(ops.expert_swiglu_mxfp4, (rows, scale, *w1, *where), test_utils=CHECKS)
    torch.library.opcheck(ops.expert_gemm_mxfp4, (rows, scale, *w2, *where), test_utils=CHECKS)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [3, 48])
def test_layer_op_passes_torchs_checks(T, fmt):
    x, idx, w, g = inputs(T)
    w1, s1 = weights(fmt, E, 2 * I, H, g)
    w2, s2 = weights(fmt, E, H, I, g)
    # (the schema check multiplies its inputs, which torch has not for E4M3)
    torch.library.opcheck(torch.ops.moe_mi355x.layer_tokens.default, (x, idx, w, w1, w2, s1, s2, E, 0),
                          test_utils=CHECKS[1:] if fmt == "fp8" else CHECKS)


def test_mxfp4_layer_compiled():
    x, idx, w, g = inputs()
    all_of = (*mx.make_weights(E, 2 * I, H, g), *mx.make_weights(E, H, I, g))
    for capacity in (T * K + 8, 0):
        fn = lambda *a: ops.moe_layer_mxfp4(*a, E, 0, 2, capacity)  # noqa: E731,B023
        want = fn(x, idx, w, *all_of)
        assert torch.isfinite(want).all() and want.any()
        if capacity:  # (without one the row count is read on the host: no full graph)
            fn = torch.compile(fn, backend="aot_eager", fullgraph=True)
        assert torch.equal(fn(x, idx, w, *all_of), want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_token_layer_compiled(fmt):
    """One graph for every number of tokens, on both sides of the choice of kernels."""
    g = torch.Generator(device="cuda").manual_seed(1)
    w1, s1 = weights(fmt, E, 2 * I, H, g)
    w2, s2 = weights(fmt, E, H, I, g)
    fn = lambda x, idx, w: ops.moe_layer_tokens(x, idx, w, w1, w2, E, s1, s2)  # noqa: E731
    compiled = torch.compile(fn, backend="aot_eager", fullgraph=True, dynamic=True)
    for T in (2, 3, 40, 500, 8):
        x, idx, w, _ = inputs(T, T)
        assert torch.equal(compiled(x, idx, w), fn(x, idx, w)), T


def test_layer_op_takes_strided_inputs():
    """Views that are not contiguous are laid out by the op."""
    x, idx, w, g = inputs()
    w1, w2 = weights("bf16", E, 2 * I, H, g)[0], weights("bf16", E, H, I, g)[0]
    want = ops.moe_layer_tokens(x, idx, w, w1, w2, E)
    wide = torch.zeros((T, 2 * H), dtype=x.dtype, device="cuda")
    wide[:, ::2] = x
    t1, t2 = w1.transpose(1, 2).contiguous().transpose(1, 2), w2.transpose(0, 2).contiguous().transpose(0, 2)
    both = torch.stack((idx, idx), -1)
    got = ops.moe_layer_tokens(wide[:, ::2], both[..., 0], w.t().contiguous().t(), t1, t2, E)
    assert torch.equal(got, want)
