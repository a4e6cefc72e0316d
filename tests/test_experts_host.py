"""CPU: argument rules of the weighted combine and of the experts' products.  Every call below fails
validation before any HIP call; nothing is launched."""
import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.fx.experimental.proxy_tensor import make_fx

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


def combine(d=None, h=None, Y=FAKE, H=2048, w=FAKE, R=10, out=FAKE, f32=0):
    return B.lib().moe_combine_weighted(ctypes.byref(d or _desc()), ctypes.byref(h or _handle()), Y,
                                        H, w, R, out, f32, None)


def combine_bwd(d=None, h=None, g=FAKE, Y=FAKE, H=2048, w=FAKE, R=10, gr=FAKE, dw=FAKE):
    return B.lib().moe_combine_weighted_bwd(ctypes.byref(d or _desc()), ctypes.byref(h or _handle()),
                                            g, Y, H, w, R, gr, dw, None)


def gemm(d=None, h=None, a=FAKE, sa=FAKE, K=512, R=10, w=FAKE, sw=FAKE, N=256, out=FAKE):
    return B.lib().moe_expert_gemm_fp8(ctypes.byref(d or _desc()), ctypes.byref(h or _handle()), a,
                                       sa, K, R, w, sw, N, out, None)


def swiglu(d=None, h=None, a=FAKE, sa=FAKE, K=512, R=10, w=FAKE, sw=FAKE, I=256, out=FAKE, os=FAKE):
    return B.lib().moe_expert_swiglu_fp8(ctypes.byref(d or _desc()), ctypes.byref(h or _handle()), a,
                                         sa, K, R, w, sw, I, out, os, None)


ALL = (combine, combine_bwd, gemm, swiglu)


@pytest.mark.parametrize("call", ALL)
def test_description_handle_and_rows(call):
    assert call(d=_desc(k=65)) == B.MOE_ERR_ARG
    assert call(d=_desc(num_local=129)) == B.MOE_ERR_ARG
    assert call(d=_desc(mode=B.MOE_SYNC_FREE, capacity=100)) == B.MOE_ERR_CAPACITY
    sf = _desc(mode=B.MOE_SYNC_FREE, capacity=5000)
    assert call(d=sf, R=10) == B.MOE_ERR_ARG and "capacity" in B.last_error()
    assert call(R=-1) == B.MOE_ERR_ARG and call(R=1 << 31) == B.MOE_ERR_ARG
    assert call(h=_handle(padded_offsets=None)) == B.MOE_ERR_ARG
    assert call(h=_handle(row_of_slot=None)) == B.MOE_ERR_ARG


@pytest.mark.parametrize("call", (combine, combine_bwd))
@pytest.mark.parametrize("H", [0, -256, 128, 384])
def test_hidden(call, H):
    assert call(H=H) == B.MOE_ERR_HIDDEN


@pytest.mark.parametrize("call,names", [
    (combine, ("Y", "out")), (combine_bwd, ("g", "Y", "gr")),
    (gemm, ("a", "sa", "w", "sw", "out")), (swiglu, ("a", "sa", "w", "sw", "out"))])
def test_null_and_misaligned_pointers(call, names):
    for n in names:
        assert call(**{n: None}) == B.MOE_ERR_ARG, n
        assert call(**{n: FAKE + 8}) == B.MOE_ERR_ARG, n
        assert "aligned" in B.last_error()


def test_weights_are_required():
    assert combine(w=None) == B.MOE_ERR_ARG and "topk_w" in B.last_error()
    assert combine_bwd(w=None) == B.MOE_ERR_ARG and combine_bwd(dw=None) == B.MOE_ERR_ARG


@pytest.mark.parametrize("K", [0, -128, 64, 200, (1 << 23) + 128])
def test_product_depth(K):
    assert gemm(K=K) == B.MOE_ERR_ARG and swiglu(K=K) == B.MOE_ERR_ARG
    assert "128" in B.last_error()


def test_product_columns_and_flags():
    for N in (0, -8, 4, 12, (1 << 30) + 8):
        assert gemm(N=N) == B.MOE_ERR_ARG, N
    for I in (0, -128, 64, 136, 1 << 30):
        assert swiglu(I=I) == B.MOE_ERR_ARG, I
    assert combine(f32=2) == B.MOE_ERR_ARG and combine(f32=-1) == B.MOE_ERR_ARG
    assert swiglu(os=FAKE + 4) == B.MOE_ERR_ARG


def test_too_large_for_one_launch():
    big = _desc(T=(1 << 31) - 1, k=1, E=1, num_local=1, pad_multiple=1)
    assert gemm(d=big, R=(1 << 31) - 1, N=1 << 30) == B.MOE_ERR_ARG
    assert "too large" in B.last_error()
    assert swiglu(d=big, R=(1 << 31) - 1, I=1 << 29) == B.MOE_ERR_ARG


def test_no_rows_launch_nothing():
    assert gemm(R=0, a=None, sa=None, w=None, sw=None, out=None) == B.MOE_OK
    assert swiglu(R=0, a=None, sa=None, w=None, sw=None, out=None, os=None) == B.MOE_OK
    assert combine(d=_desc(T=0), R=0, Y=None, w=None, out=None) == B.MOE_OK


def test_binding_rejects_cpu_tensors_and_bad_types():
    d = B.make_desc(4, 2, 4)
    t = dict(dtype=torch.int32)
    h = B.Handle(d, None, torch.zeros(4, **t), torch.zeros(5, **t), torch.zeros((4, 2), **t),
                 torch.zeros(4, **t), torch.zeros(4, **t), None)
    q, s = torch.zeros((8, 128), dtype=torch.uint8), torch.zeros((8, 1))
    w = torch.zeros((4, 128, 128), dtype=torch.uint8)
    ws = torch.zeros((4, 1, 1))
    out = torch.zeros((8, 128), dtype=torch.bfloat16)
    with pytest.raises(B.MoeError, match="GPU tensor"):
        B.moe_expert_gemm_fp8(d, h, q, s, 128, 8, w, ws, 128, out)
    with pytest.raises(B.MoeError, match="GPU tensor"):
        B.combine_weighted(d, h, out, torch.zeros((4, 2)))
    with pytest.raises(B.MoeError, match="K=128"):
        B.expert_gemm_fp8(d, h, q, s, torch.zeros((4, 128, 256), dtype=torch.uint8), ws)
    with pytest.raises(B.MoeError, match="out_scale"):
        B._swiglu_out(out, s, 8, 128)
    with pytest.raises(B.MoeError, match="out_scale"):
        B._swiglu_out(q, None, 8, 128)
    with pytest.raises(B.MoeError, match="another description"):
        B.moe_expert_gemm_fp8(B.make_desc(5, 2, 4), h, q, s, 128, 8, w, ws, 128, out)
    with pytest.raises(B.MoeError, match="positive"):
        B.PreparedExpertGemmFp8(d, h, q, s, 0, w, ws, 128, out)


def test_convenience_shapes():
    """Weights of other experts than the local ones, or scales of another layout, are refused."""
    d = B.make_desc(4, 2, 8, 2, 4)
    q, s = torch.zeros((8, 256), dtype=torch.uint8), torch.zeros((8, 2))
    w, ws = torch.zeros((4, 256, 256), dtype=torch.uint8), torch.zeros((4, 2, 2))
    for call in (B.expert_gemm_fp8, B.expert_swiglu_fp8):
        for bad in ((q, s, torch.zeros((8, 256, 256), dtype=torch.uint8), torch.zeros((8, 2, 2))),
                    (q, s, w, torch.zeros((4, 2, 1))), (q, s, w, torch.zeros((4, 4))),
                    (q, s.T, w, ws), (q, s[:7], w, ws)):
            with pytest.raises(B.MoeError, match="must be"):
                call(d, None, *bad)


def test_outputs_apart():
    buf = torch.zeros(64, dtype=torch.uint8)
    a, b, c = buf[:32], buf[16:48], buf[32:]
    B._apart((a, c), (None, torch.zeros(4)))
    B._apart((a[:0],), (a,))
    for outs, ins in (((a,), (b,)), ((a, b), ()), ((c,), (a, b)), ((a,), (a,)), ((a, None), (buf,))):
        with pytest.raises(B.MoeError, match="overlaps"):
            B._apart(outs, ins)


# ---------------------------------------------------------------------------
# the torch ops, traced with fake tensors
# ---------------------------------------------------------------------------
def test_ops_are_registered():
    for name in ("combine_weighted", "combine_weighted_bwd", "expert_gemm_fp8", "expert_swiglu_fp8"):
        schema = str(getattr(torch.ops.moe_mi355x, name).default._schema)
        assert schema.startswith(f"moe_mi355x::{name}(") and "!" not in schema


def test_fake_shapes():
    T, k, E, EL, H, I, P = 70, 4, 64, 24, 512, 384, 4
    C = T * k + EL * (P - 1)
    e8 = torch.float8_e4m3fn
    with FakeTensorMode():
        x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        w = torch.empty((T, k), device="cuda")
        meta = ops.route(torch.empty((T, k), dtype=torch.int32, device="cuda"), E, 8, EL, P, C)[:6]
        where = (*meta, E, 8, P, C)
        q, sc, *_ = ops.dispatch_fp8(x, w, *where, C)
        w1, s1 = torch.empty((EL, 2 * I, H), dtype=e8, device="cuda"), torch.empty((EL, 6, 4), device="cuda")
        h, hs = ops.expert_swiglu_fp8(q, sc, w1, s1, *where)
        assert h.shape == (C, I) and h.dtype == e8 and h.device.type == "cuda"
        assert hs.shape == (C, I // 128) and hs.dtype == torch.float32
        w2, s2 = torch.empty((EL, H, I), dtype=e8, device="cuda"), torch.empty((EL, 4, 3), device="cuda")
        Y = ops.expert_gemm_fp8(h, hs, w2, s2, *where)
        assert Y.shape == (C, H) and Y.dtype == torch.bfloat16
        out = ops.combine_weighted(Y, w, *where)
        assert out.shape == (T, H) and out.dtype == torch.bfloat16
        gr, dw = ops.combine_weighted_bwd(out, Y, w, *where)
        assert gr.shape == (C, H) and gr.dtype == torch.bfloat16
        assert dw.shape == (T, k) and dw.dtype == torch.float32
        out = ops.moe_layer_fp8(x, torch.empty((T, k), dtype=torch.int64, device="cuda"), w, w1, s1, w2, s2,
                                E, 8, P, C)
        assert out.shape == (T, H) and out.dtype == torch.bfloat16


def test_weighted_backward_traces_to_its_op():
    T, k, E, H, P = 32, 2, 8, 256, 1
    C = T * k

    def step(Y, w, idx, G):
        Y, w = Y.detach().requires_grad_(True), w.detach().requires_grad_(True)
        meta = ops.route(idx, E, 0, E, P, C)[:6]
        out = ops.combine_weighted(Y, w, *meta, E, 0, P, C)
        return torch.autograd.grad((out.float() * G).sum(), (Y, w))

    g = make_fx(step, tracing_mode="fake")(torch.zeros((C, H), dtype=torch.bfloat16), torch.zeros((T, k)),
                                           torch.zeros((T, k), dtype=torch.int32), torch.zeros((T, H)))
    names = [str(n.target) for n in g.graph.nodes if "moe_mi355x" in str(n.target)]
    assert names == [f"moe_mi355x.{n}.default" for n in ("route", "combine_weighted", "combine_weighted_bwd")]
    outs = [n for n in g.graph.nodes if n.op == "output"][0].args[0]
    assert [tuple(o.meta["val"].shape) for o in outs] == [(C, H), (T, k)]
