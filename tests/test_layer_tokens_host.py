"""CPU: argument rules of the layer for a few tokens and the fake shapes of its torch op.  Every call
below fails validation before any HIP call; nothing is launched."""
import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from combine_topk_idx_multihot_amd import binding as B
from combine_topk_idx_multihot_amd import ops

FAKE = 0x100000  # 16-byte aligned, never dereferenced by validation
FP8 = B.MOE_WEIGHTS_FP8


def _desc(**kw):
    base = dict(T=4, k=8, E=128, local_begin=0, num_local=128, pad_multiple=16, mode=B.MOE_EAGER)
    return B.make_desc(**{**base, **kw})


def layer(d=None, idx=FAKE, w=FAKE, x=FAKE, H=512, I=256, fmt=FP8, w1=FAKE, s1=FAKE, w2=FAKE, s2=FAKE, ws=FAKE,
          n=1 << 30, out=FAKE, flags=None):
    return B.lib().moe_layer_tokens(ctypes.byref(d or _desc()), idx, w, x, H, I, fmt, w1, s1, w2, s2, ws, n, out,
                                    flags, None)


def test_description():
    for d in (_desc(k=65), _desc(num_local=129), _desc(T=-1), _desc(pad_multiple=0), _desc(mode=2)):
        assert layer(d) == B.MOE_ERR_ARG
    assert layer(_desc(mode=B.MOE_SYNC_FREE, capacity=10)) == B.MOE_ERR_CAPACITY
    assert layer(_desc(T=129)) == B.MOE_ERR_ARG and "1024" in B.last_error()
    assert layer(_desc(T=1025, k=1)) == B.MOE_ERR_ARG
    assert B.lib().moe_layer_tokens_workspace_size(ctypes.byref(_desc(T=129)), 512, 256) == 0


def test_sizes():
    for H in (0, -256, 128, 384):
        assert layer(H=H) == B.MOE_ERR_HIDDEN
        assert B.lib().moe_layer_tokens_workspace_size(ctypes.byref(_desc()), H, 256) == 0
    assert layer(H=65792) == B.MOE_ERR_ARG
    for I in (0, -128, 64, 200, 65664):
        assert layer(I=I) == B.MOE_ERR_ARG, I
        assert B.lib().moe_layer_tokens_workspace_size(ctypes.byref(_desc()), 512, I) == 0
    for fmt in (-1, 3):
        assert layer(fmt=fmt) == B.MOE_ERR_ARG and "w_format" in B.last_error()


def test_pointers():
    for n in ("idx", "w"):
        assert layer(**{n: None}) == B.MOE_ERR_ARG and n in B.last_error()
    for n in ("x", "w1", "w2", "s1", "s2", "out"):
        assert layer(**{n: None}) == B.MOE_ERR_ARG, n
        assert layer(**{n: FAKE + 8}) == B.MOE_ERR_ARG, n
        assert "aligned" in B.last_error()
    for s1, s2 in ((FAKE, None), (None, FAKE), (FAKE, FAKE)):
        assert layer(fmt=B.MOE_WEIGHTS_BF16, s1=s1, s2=s2) == B.MOE_ERR_ARG and "no scales" in B.last_error()


def test_workspace():
    need = B.moe_layer_tokens_workspace_size(_desc(), 512, 256)
    assert need >= 4 * 8 * 256 * 2
    # slots that share experts' weights: fp32 rows of them too
    assert B.moe_layer_tokens_workspace_size(_desc(T=17), 512, 256) >= 17 * 8 * (256 * 2 + 512 * 4)
    assert layer(ws=None) == B.MOE_ERR_WORKSPACE and layer(ws=FAKE + 8) == B.MOE_ERR_WORKSPACE
    assert layer(n=need - 1) == B.MOE_ERR_WORKSPACE and str(need) in B.last_error()
    assert B.moe_layer_tokens_workspace_size(_desc(T=0), 256, 128) > 0


def test_no_tokens_launch_nothing():
    assert layer(_desc(T=0), idx=None, w=None, x=None, w1=None, w2=None, s1=None, s2=None, ws=None, n=0,
                 out=None) == B.MOE_OK


def tensors(fmt, T=4, k=2, EL=3, H=512, I=128):
    u8, e8 = dict(dtype=torch.uint8), dict(dtype=torch.float8_e4m3fn)
    idx, w = torch.zeros((T, k), dtype=torch.int32), torch.zeros((T, k))
    x = torch.zeros((T, H), dtype=torch.bfloat16)
    if fmt == "bf16":
        z = dict(dtype=torch.bfloat16)
        return [idx, w, x, torch.zeros((EL, 2 * I, H), **z), torch.zeros((EL, H, I), **z), None, None]
    if fmt == "fp8":
        return [idx, w, x, torch.zeros((EL, 2 * I, H), **e8), torch.zeros((EL, H, I), **e8),
                torch.zeros((EL, 2 * I // 128, H // 128)), torch.zeros((EL, H // 128, I // 128))]
    return [idx, w, x, torch.zeros((EL, 2 * I, H // 2), **u8), torch.zeros((EL, H, I // 2), **u8),
            torch.zeros((EL, 2 * I, H // 32), **u8), torch.zeros((EL, H, I // 32), **u8)]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp4"])
def test_binding_refusals(fmt):
    d = B.make_desc(4, 2, 8, 1, 3)

    def call(*a, d=d):
        idx, w, x, w1, w2, s1, s2 = a
        return B.layer_tokens(d, idx, w, x, w1, w2, s1, s2)

    good = tensors(fmt)
    with pytest.raises(B.MoeError, match="GPU tensor"):
        call(*good)
    for i, bad in ((3, good[3][:, :128]), (3, good[3][:2]), (4, good[4][:, :256]), (4, good[4][:2]),
                   (3, good[3][..., :64])):
        with pytest.raises(B.MoeError, match="must be"):
            call(*good[:i], bad, *good[i + 1:])
    with pytest.raises(B.MoeError, match="T=5"):
        call(*good, d=B.make_desc(5, 2, 8, 1, 3))
    with pytest.raises(B.MoeError, match="1024"):
        call(*tensors(fmt, T=513), d=B.make_desc(513, 2, 8, 1, 3))
    if fmt == "bf16":
        with pytest.raises(B.MoeError, match="without scales"):
            call(*good[:6], torch.zeros(1))
        return
    for i in (5, 6):
        with pytest.raises(B.MoeError, match="must be|both"):
            call(*good[:i], good[i][:, :1], *good[i + 1:])
        with pytest.raises(B.MoeError, match="both|must be"):
            call(*good[:i], None, *good[i + 1:])


def test_prepared_products_refuse_sizes_before_anything_else():
    q = torch.zeros((8, 64), dtype=torch.uint8)
    for K, I in ((128, 0), (128, -128), (0, 128), (-128, 128)):
        for out, scale in ((torch.zeros((8, 128), dtype=torch.bfloat16), None), (q, q)):
            with pytest.raises(B.MoeError, match="positive"):
                B.PreparedExpertSwigluMxfp4(B.make_desc(4, 2, 8), None, q, q, K, q, q, I, out, scale)


def test_op_fake_shape_and_registration():
    schema = str(torch.ops.moe_mi355x.layer_tokens.default._schema)
    assert schema.startswith("moe_mi355x::layer_tokens(") and "!" not in schema
    for fmt in ("bf16", "fp8", "mxfp4"):
        with FakeTensorMode():
            idx, w, x, w1, w2, s1, s2 = (None if t is None else torch.empty(t.shape, dtype=t.dtype, device="cuda")
                                         for t in tensors(fmt))
            out = ops.moe_layer_tokens(x, idx, w, w1, w2, 8, s1, s2, 1)
            assert out.shape == (4, 512) and out.dtype == torch.bfloat16 and out.device.type == "cuda"
