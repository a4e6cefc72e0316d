"""CPU: argument rules of the MXFP4 operators and the fake shapes of their torch ops.  Every call below
fails validation before any HIP call; nothing is launched."""
import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from combine_topk_idx_multihot_amd import binding as B
from combine_topk_idx_multihot_amd import ops

FAKE = 0x100000  # 16-byte aligned, never dereferenced by validation


def _desc(**kw):
    base = dict(T=100, k=8, E=128, local_begin=0, num_local=128, pad_multiple=16, mode=B.MOE_EAGER)
    return B.make_desc(**{**base, **kw})


def _handle(**kw):
    base = dict(routing_map=FAKE, tokens_per_expert=FAKE, padded_offsets=FAKE, row_of_slot=FAKE,
                status=FAKE, workspace=FAKE, workspace_bytes=1 << 30)
    return B._Handle(**{**base, **kw})


def quantize(x=FAKE, f32=0, n=10, K=64, q=FAKE, s=FAKE):
    return B.lib().moe_quantize_mxfp4(x, f32, n, K, q, s, None)


def dequantize(x=FAKE, f32=0, n=10, K=64, q=FAKE, s=FAKE):
    return B.lib().moe_dequantize_mxfp4(q, s, n, K, x, f32, None)


def dispatch(d=None, h=None, x=FAKE, H=512, w=None, R=10, q=FAKE, s=FAKE, rw=None):
    return B.lib().moe_dispatch_mxfp4(ctypes.byref(d or _desc()), ctypes.byref(h or _handle()), x, H, w, R, q,
                                      s, rw, None, None, None)


def gemm(d=None, h=None, a=FAKE, sa=FAKE, K=512, R=10, w=FAKE, sw=FAKE, N=256, out=FAKE):
    return B.lib().moe_expert_gemm_mxfp4(ctypes.byref(d or _desc()), ctypes.byref(h or _handle()), a, sa, K, R,
                                         w, sw, N, out, None)


def swiglu(d=None, h=None, a=FAKE, sa=FAKE, K=512, R=10, w=FAKE, sw=FAKE, I=256, out=FAKE, os=FAKE):
    return B.lib().moe_expert_swiglu_mxfp4(ctypes.byref(d or _desc()), ctypes.byref(h or _handle()), a, sa, K,
                                           R, w, sw, I, out, os, None)


@pytest.mark.parametrize("call", (quantize, dequantize))
def test_quantization(call):
    for K in (0, -32, 16, 33, 48):
        assert call(K=K) == B.MOE_ERR_ARG and "32" in B.last_error()
    assert call(n=-1) == B.MOE_ERR_ARG and call(n=1 << 31) == B.MOE_ERR_ARG
    assert call(f32=2) == B.MOE_ERR_ARG and call(f32=-1) == B.MOE_ERR_ARG
    for name in ("x", "q", "s"):
        for bad in (None, FAKE + 8):
            assert call(**{name: bad}) == B.MOE_ERR_ARG and "aligned" in B.last_error()
    assert call(n=0, x=None, q=None, s=None) == B.MOE_OK
    assert call(n=(1 << 31) - 1, K=(1 << 31) - 32) == B.MOE_ERR_ARG and "too large" in B.last_error()


@pytest.mark.parametrize("call", (dispatch, gemm, swiglu))
def test_description_handle_and_rows(call):
    assert call(d=_desc(k=65)) == B.MOE_ERR_ARG
    assert call(d=_desc(num_local=129)) == B.MOE_ERR_ARG
    assert call(d=_desc(mode=B.MOE_SYNC_FREE, capacity=100)) == B.MOE_ERR_CAPACITY
    sf = _desc(mode=B.MOE_SYNC_FREE, capacity=5000)
    assert call(d=sf, R=10) == B.MOE_ERR_ARG and "capacity" in B.last_error()
    assert call(R=-1) == B.MOE_ERR_ARG and call(R=1 << 31) == B.MOE_ERR_ARG
    assert call(h=_handle(padded_offsets=None)) == B.MOE_ERR_ARG
    assert call(h=_handle(row_of_slot=None)) == B.MOE_ERR_ARG


@pytest.mark.parametrize("call,names", [(dispatch, ("x", "q", "s")), (gemm, ("a", "sa", "w", "sw", "out")),
                                        (swiglu, ("a", "sa", "w", "sw", "out"))])
def test_null_and_misaligned_pointers(call, names):
    for n in names:
        assert call(**{n: None}) == B.MOE_ERR_ARG, n
        assert call(**{n: FAKE + 8}) == B.MOE_ERR_ARG, n
        assert "aligned" in B.last_error()
    assert swiglu(os=FAKE + 4) == B.MOE_ERR_ARG


def test_sizes():
    for H in (0, -256, 128, 384):
        assert dispatch(H=H) == B.MOE_ERR_HIDDEN
    for K in (0, -128, 64, 200, (1 << 23) + 128):
        assert gemm(K=K) == B.MOE_ERR_ARG and swiglu(K=K) == B.MOE_ERR_ARG
    for N in (0, -8, 4, 12, (1 << 30) + 8):
        assert gemm(N=N) == B.MOE_ERR_ARG, N
    for I in (0, -128, 64, 136, 1 << 30):
        assert swiglu(I=I) == B.MOE_ERR_ARG, I
    assert dispatch(w=FAKE) == B.MOE_ERR_ARG and dispatch(rw=FAKE) == B.MOE_ERR_ARG
    big = _desc(T=(1 << 31) - 1, k=1, E=1, num_local=1, pad_multiple=1)
    assert gemm(d=big, R=(1 << 31) - 1, N=1 << 30) == B.MOE_ERR_ARG and "too large" in B.last_error()
    assert swiglu(d=big, R=(1 << 31) - 1, I=1 << 29) == B.MOE_ERR_ARG
    assert gemm(R=0, a=None, sa=None, w=None, sw=None, out=None) == B.MOE_OK
    assert swiglu(R=0, a=None, sa=None, w=None, sw=None, out=None, os=None) == B.MOE_OK


def test_binding_refusals():
    d = B.make_desc(4, 2, 8, 2, 4)
    u8 = dict(dtype=torch.uint8)
    q, s = torch.zeros((9, 128), **u8), torch.zeros((9, 8), **u8)
    w, ws = torch.zeros((4, 256, 128), **u8), torch.zeros((4, 256, 8), **u8)
    for call in (B.expert_gemm_mxfp4, B.expert_swiglu_mxfp4):
        for bad in ((q, s, torch.zeros((8, 256, 128), **u8), ws), (q, s, w, ws[:, :, :4]), (q, s, w, ws[:, :8]),
                    (q, s.T, w, ws), (q, s[:7], w, ws), (q[:, :64], s, w, ws)):
            with pytest.raises(B.MoeError, match="must be"):
                call(d, None, *bad)
    x = torch.zeros((4, 64))
    with pytest.raises(B.MoeError, match="GPU tensor"):
        B.quantize_mxfp4(x)
    with pytest.raises(B.MoeError, match="multiple of 32"):
        B.quantize_mxfp4(x[:, :40])
    with pytest.raises(B.MoeError, match="must be"):
        B.dequantize_mxfp4(q, s[:, :4])
    with pytest.raises(B.MoeError, match="GPU tensor"):
        B.dequantize_mxfp4(q, s)
    with pytest.raises(B.MoeError, match="out_scale"):
        B._swiglu_out(torch.zeros((8, 128), dtype=torch.bfloat16), s, 8, 128, True)
    with pytest.raises(B.MoeError, match="MXFP4"):
        B._swiglu_out(q, None, 8, 128, True)


def test_fake_shapes():
    T, k, E, EL, H, I, P = 70, 4, 64, 24, 512, 384, 4
    C = T * k + EL * (P - 1)
    u8 = torch.uint8
    with FakeTensorMode():
        x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        w = torch.empty((T, k), device="cuda")
        idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
        where = (*ops.route(idx, E, 8, EL, P, C)[:6], E, 8, P, C)
        q, sc, rw, rt, re = ops.dispatch_mxfp4(x, w, *where, C)
        assert q.shape == (C, H // 2) and sc.shape == (C, H // 32) and q.dtype == sc.dtype == u8
        assert rw.shape == rt.shape == re.shape == (C,)
        w1, s1 = ops.quantize_mxfp4(torch.empty((EL, 2 * I, H), device="cuda"))
        assert w1.shape == (EL, 2 * I, H // 2) and s1.shape == (EL, 2 * I, H // 32) and w1.dtype == s1.dtype == u8
        assert ops.dequantize_mxfp4(w1, s1, True).dtype == torch.float32
        assert ops.dequantize_mxfp4(w1, s1, False).shape == (EL, 2 * I, H)
        h, hs = ops.expert_swiglu_mxfp4(q, sc, w1, s1, *where)
        assert h.shape == (C, I // 2) and hs.shape == (C, I // 32) and h.dtype == hs.dtype == u8
        w2, s2 = ops.quantize_mxfp4(torch.empty((EL, H, I), device="cuda"))
        Y = ops.expert_gemm_mxfp4(h, hs, w2, s2, *where)
        assert Y.shape == (C, H) and Y.dtype == torch.bfloat16
        out = ops.moe_layer_mxfp4(x, idx, w, w1, s1, w2, s2, E, 8, P, C)
        assert out.shape == (T, H) and out.dtype == torch.bfloat16
