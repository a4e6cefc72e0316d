"""GPU: calls that are given a stream take their memory from it: outputs and hidden workspaces are in its order,
not in that of the current stream, whose queued work may still use a block that was freed there."""
import pytest
import torch

from combine_topk_idx_multihot_amd import binding as B

pytestmark = pytest.mark.gpu

T, K, E, H, I = 40, 4, 16, 512, 256


def weights(g):
    w1 = (torch.randn((E, 2 * I, H), generator=g, device="cuda") * H ** -0.5).to(torch.bfloat16)
    w2 = (torch.randn((E, H, I), generator=g, device="cuda") * I ** -0.5).to(torch.bfloat16)
    return w1, w2


def inputs(T=T):
    g = torch.Generator(device="cuda").manual_seed(T)
    idx = torch.rand((T, E), generator=g, device="cuda").topk(K, 1).indices.int()
    w = torch.rand((T, K), generator=g, device="cuda")
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    return idx, w, x, *weights(g)


def owner(t):
    """The stream whose memory a tensor lies in."""
    p = t.data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= p < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's")


@pytest.mark.parametrize("prepared", [False, True])
@pytest.mark.parametrize("T", [2, 40])
def test_no_block_that_the_current_stream_still_uses(T, prepared):
    idx, w, x, w1, w2 = inputs(T)
    d = B.make_desc(T, K, E)
    want = B.layer_tokens(d, idx, w, x, w1, w2)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        torch.cuda._sleep(1000)
    sizes = [B.moe_layer_tokens_workspace_size(d, H, I), want.nbytes]
    got = torch.empty_like(want)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    seen = [torch.zeros_like(t) for t in old]
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    for a, b in zip(seen, old):
        a.copy_(b)  # behind the sleep
        b.fill_(0xA5)
    del old, a, b
    if prepared:
        B.PreparedLayerTokens(d, idx, w, x, w1, w2, got, stream=st)()
    else:
        got = B.layer_tokens(d, idx, w, x, w1, w2, stream=st)
    st.synchronize()
    assert not torch.cuda.current_stream().query(), "the current stream should still be asleep"
    torch.cuda.synchronize()
    assert all((t == 0x5A).all() for t in seen)
    assert torch.equal(got, want)


def test_outputs_lie_in_the_given_streams_memory():
    idx, w, x, w1, w2 = inputs()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    raw = st.cuda_stream
    d = B.make_desc(T, K, E, 0, E, 1, B.MOE_SYNC_FREE, False, T * K)

    def mine(out):
        for t in out if isinstance(out, tuple) else (out,):
            for v in vars(t).values() if isinstance(t, B.Handle) else (t,):
                if isinstance(v, torch.Tensor) and v.is_cuda and v.numel():
                    assert owner(v) == raw
        return out

    for s in (st, raw):
        h, _ = mine(B.route(d, idx, w, stream=s))
        rows, *_ = mine(B.dispatch(d, h, x, w, stream=s))
        mine(B.combine(d, h, rows, stream=s))
        mine(B.combine_weighted(d, h, rows, w, stream=s))
        mine(B.combine_weighted_bwd(d, h, x, rows, w, stream=s))
        mine(B.combine_bwd(d, h, x, T * K, rows, stream=s))
        mine(B.dispatch_bwd(d, h, rows, stream=s))
        mine(B.dispatch_fp8(d, h, x, w, stream=s))
        q, sc, *_ = mine(B.dispatch_mxfp4(d, h, x, w, stream=s))
        st.wait_stream(torch.cuda.current_stream())
        q1, s1 = mine(B.quantize_mxfp4(w1, stream=s))
        q2, s2 = mine(B.quantize_mxfp4(w2, s))
        mine(B.dequantize_mxfp4(q1, s1, stream=s))
        a, b = mine(B.expert_swiglu_mxfp4(d, h, q, sc, q1, s1, stream=s))
        y = mine(B.expert_gemm_mxfp4(d, h, a, b, q2, s2, stream=s))
        out = mine(B.layer_tokens(d, idx, w, x, q1, q2, s1, s2, stream=s))
        torch.cuda.synchronize()
        chain = B.combine_weighted(d, h, y, w)
        assert (chain.float() - out.float()).norm() < 0.5 * out.float().norm()


def test_outputs_wait_for_the_callers_stream():
    """A result dropped while the caller's stream still reads it is not handed out again on the given one."""
    idx, w, x, w1, w2 = inputs()
    d = B.make_desc(T, K, E)
    want = B.layer_tokens(d, idx, w, x, w1, w2)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = B.layer_tokens(d, idx, w, x, w1, w2, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda._sleep(400_000_000)
    copy = torch.empty_like(out)
    copy.copy_(out)
    del out
    with torch.cuda.stream(st):
        for _ in range(4):
            torch.full_like(want, 7.0)
    st.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert torch.equal(copy, want)


def test_on_a_side_stream_of_a_capture():
    """A captured call on a stream that the capture has forked: its memory is the graph's."""
    idx, w, x, w1, w2 = inputs()
    d = B.make_desc(T, K, E)
    want = B.layer_tokens(d, idx, w, x, w1, w2)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        out = B.layer_tokens(d, idx, w, x, w1, w2, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        twice = out + out
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(twice, want + want)
        B.layer_tokens(d, idx, w, x, w1, w2)
