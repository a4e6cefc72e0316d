"""GPU: the whole layer for a few tokens (moe_layer_tokens) against 64-bit references, with bf16, E4M3
and MXFP4 weights: one token and the most slots, every slot on its own and slots of an expert together,
experts with no and with all slots, repeated, empty, foreign and bad ids, NaN where nothing may look;
streams, graphs, two calls at once.

Bounds (u = 2^-24): products of bf16 with the weights' values are exact in fp32; a sum of n of them, in
whatever order the matrix instructions take, is off by at most one step (2u) of the sum of magnitudes S
per addition; the additions on a product's way are at most the n products', one per instruction of 32
columns or one per 16 columns with E4M3 weights, and those of up to 64 partial sums in a tree:
n + n / 16 + 8 <= 1.1 n + 8.  silu as in expert_ref.swiglu.  h is rounded to bf16 (half a step, 2^-8).
The combine adds k products of fp32 with one rounding each, or multiplies each lane's run of 8 to 32
products with its slot's weight: those runs leave most of the 1.1 n above for the k I / 512 of them at
most that a lane adds up, as k I / 512 <= I / 8 for k <= 64."""
import pytest
import torch

import expert_ref as ref
import mx_ref as mx
from combine_topk_idx_multihot_amd import binding as B
from combine_topk_idx_multihot_amd import ops

pytestmark = pytest.mark.gpu

FORMATS = ("bf16", "fp8", "mxfp4")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.moe_device_check(0)
    yield


def weights(fmt, EL, n, K, g):
    if fmt == "bf16":
        return (torch.randn((EL, n, K), generator=g, device="cuda") * K ** -0.5).to(torch.bfloat16), None
    if fmt == "fp8":
        return ref.make_weights(EL, n, K, g)
    return mx.make_weights(EL, n, K, g)


def plain(fmt, q, s, e):
    """fp64 [n, K] of expert e."""
    if fmt == "bf16":
        return q[e].double()
    if fmt == "mxfp4":
        return mx.values(q[e], s[e])
    n, K = q[e].shape
    return q[e].double() * s[e].double()[torch.arange(n) // 128][:, torch.arange(K) // 128]


def exact(fmt, x, idx, w, w1, s1, w2, s2, lb):
    """fp64 (out, bound) of an fp32 evaluation."""
    T, k = idx.shape
    out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(out)
    mag = torch.zeros_like(out)
    H, EL = x.shape[1], w1.shape[0]
    for e in range(EL):
        t, j = (idx == lb + e).nonzero(as_tuple=True)
        if not len(t):
            continue
        a, W = x[t].double(), plain(fmt, w1, s1, e)
        h, eh = ref.swiglu(a @ W.T, (1.1 * H + 8) * 2 * ref.U * (a.abs() @ W.abs().T) + ref.TINY)
        eh = eh + 2.0 ** -8 * (h.abs() + eh)
        W = plain(fmt, w2, s2, e)
        z = h @ W.T
        ez = eh @ W.abs().T + (1.1 * h.shape[1] + 8) * 2 * ref.U * ((h.abs() + eh) @ W.abs().T)
        wt = w[t, j].double()[:, None]
        out.index_add_(0, t, z * wt)
        bound.index_add_(0, t, ez * wt.abs())
        mag.index_add_(0, t, (z.abs() + ez) * wt.abs())
    return out, bound + (k + 1) * ref.U * mag + ref.TINY


def make(fmt, T, k, E, lb, EL, H, I, seed=0, empty=0.1, i64=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.Generator().manual_seed(seed)
    idx = torch.rand((T, E), generator=c).topk(k, 1).indices
    idx[torch.rand((T, k), generator=c) < empty] = -1
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.rand((T, k), generator=g, device="cuda") - 0.2
    w1, s1 = weights(fmt, EL, 2 * I, H, g)
    w2, s2 = weights(fmt, EL, H, I, g)
    d = B.make_desc(T, k, E, lb, EL, 1, B.MOE_EAGER, i64)
    return d, idx.to(torch.int64 if i64 else torch.int32).cuda(), w, x, w1, s1, w2, s2


def check(fmt, d, idx, w, x, w1, s1, w2, s2, what):
    T, H, lb = d.T, x.shape[1], d.local_begin
    I = w2.shape[2] * (2 if fmt == "mxfp4" else 1)
    out = torch.full((T + 1, H), -12345.0, dtype=torch.bfloat16, device="cuda")
    n = B.moe_layer_tokens_workspace_size(d, H, I)
    ws = torch.full((n + 64,), 0x55, dtype=torch.uint8, device="cuda")
    flags = torch.full((2,), 77, dtype=torch.int32, device="cuda")
    B.moe_layer_tokens(d, idx, w, x, w1, w2, out, ws[:n], s1, s2, flags)
    torch.cuda.synchronize()
    ref.check_bf16(out[:T], *exact(fmt, x, idx.long(), w, w1, s1, w2, s2, lb), what)
    assert (out[T:] == torch.tensor(-12345.0, dtype=torch.bfloat16)).all() and (ws[n:] == 0x55).all()
    ids = idx.long()
    bad = ((ids < -1) | (ids >= d.E)).any()
    same = (ids[:, :, None] == ids[:, None, :]) & (ids >= 0)[:, :, None] & (ids < d.E)[:, :, None]
    dup = (same.sum((1, 2)) > ((ids >= 0) & (ids < d.E)).sum(1)).any()
    assert flags.tolist() == [int(bad) * B.MOE_FLAG_BAD_ID + int(dup) * B.MOE_FLAG_DUPLICATE, 77], what
    none = ((ids < lb) | (ids >= lb + d.num_local)).all(1)
    assert not out[:T][none].view(torch.int16).any()  # +0, in bits
    return out[:T].clone()


SHAPES = [
    # T, k, E, lb, EL, H, I
    (1, 1, 1, 0, 1, 256, 128), (1, 2, 4, 0, 4, 512, 128), (1, 8, 128, 0, 128, 2048, 768), (1, 7, 16, 3, 9, 768, 384),
    (2, 8, 64, 0, 64, 1280, 256), (3, 5, 8, 2, 5, 512, 640), (16, 1, 4, 0, 4, 256, 256), (1, 16, 32, 0, 32, 4096, 128),
    (1, 17, 32, 0, 32, 256, 256), (1, 64, 100, 0, 100, 256, 128), (5, 6, 64, 16, 32, 2048, 768),
    (9, 4, 300, 100, 200, 512, 384), (33, 8, 128, 0, 128, 1024, 256), (64, 4, 4, 0, 4, 768, 128),
    (100, 3, 1024, 0, 1024, 256, 128), (128, 8, 16, 0, 16, 512, 256), (1024, 1, 8, 4, 4, 256, 128),
    (31, 33, 64, 0, 64, 256, 128), (8, 4, 32, 0, 32, 1280, 384), (3, 11, 32, 0, 32, 768, 128), (2, 9, 16, 8, 8, 256, 640),
    (40, 2, 16, 0, 16, 4096, 128), (17, 1, 4, 1, 3, 2304, 1152),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_layer(shape, fmt):
    check(fmt, *make(fmt, *shape, seed=sum(shape), i64=sum(shape) % 2 == 1), f"{shape} {fmt}")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,k", [(1, 8), (2, 8), (100, 4), (1024, 1), (128, 8)])
def test_every_slot_to_one_expert(T, k, fmt):
    """The same id in every slot (repeats flagged), on the last local expert."""
    d, idx, *rest = make(fmt, T, k, 32, 4, 20, 512, 256, seed=T)
    idx.fill_(23)
    check(fmt, d, idx, *rest, f"{T} x {k} {fmt}")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,k", [(1, 4), (3, 5), (40, 4)])
def test_no_local_slot_and_bad_ids(T, k, fmt):
    d, idx, w, x, *rest = make(fmt, T, k, 32, 8, 8, 512, 128, seed=T)
    idx[0] = 3  # not local
    idx[-1, -1] = 32  # out of range
    idx[-1, 0] = -2
    w[idx < 8] = float("nan")  # weights of empty slots are not used
    w[idx >= 16] = float("inf")
    clean = torch.where((idx < 8) | (idx >= 16), 0.0, w)
    x[0] = float("nan")  # nor is a token without a local slot
    out = torch.empty((T, 512), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(B.moe_layer_tokens_workspace_size(d, 512, 128), dtype=torch.uint8, device="cuda")
    B.moe_layer_tokens(d, idx, w, x, rest[0], rest[2], out, ws, rest[1], rest[3])
    x = torch.where(torch.isnan(x), 0.0, x)
    want, bound = exact(fmt, x, idx.long(), clean, rest[0], rest[1], rest[2], rest[3], 8)
    ref.check_bf16(out, want, bound, f"{T} {k} {fmt}")
    assert not out[0].view(torch.int16).any()
    idx.fill_(-1)
    B.moe_layer_tokens(d, idx, w, x, rest[0], rest[2], out, ws, rest[1], rest[3])
    assert not out.view(torch.int16).any()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [2, 30])
def test_nan_token_and_nan_expert_stay_alone(T, fmt):
    d, idx, w, x, w1, s1, w2, s2 = make(fmt, T, 4, 16, 0, 16, 512, 256, seed=T, empty=0.0)
    idx[0] = torch.arange(0, 4)
    idx[1] = torch.arange(4, 8)
    idx[2:] = idx[2:].clamp_max(11)
    clean = B.layer_tokens(d, idx, w, x, w1, w2, s1, s2)
    x2 = x.clone()
    x2[1, 77] = float("nan")
    out = B.layer_tokens(d, idx, w, x2, w1, w2, s1, s2)
    keep = torch.arange(T, device="cuda") != 1
    assert torch.isnan(out[1]).all() and torch.equal(out[keep], clean[keep])
    # a NaN weight of expert 13 (its down projection's row 5), which only token 0 has
    idx[0, 3] = 13
    clean = B.layer_tokens(d, idx, w, x, w1, w2, s1, s2)
    bad = w2.clone()
    s_bad = None if s2 is None else s2.clone()
    if fmt == "mxfp4":
        s_bad[13, 5, 3] = 255
    elif fmt == "fp8":
        bad.view(torch.uint8)[13, 5, 100] = 0x7F
    else:
        bad[13, 5, 100] = float("nan")
    out = B.layer_tokens(d, idx, w, x, w1, bad, s1, s_bad)
    assert torch.isnan(out[0, 5])
    out[0, 5] = clean[0, 5]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("fmt", FORMATS)
def test_forms_agree_on_a_token(fmt):
    """A token alone, and among others that make the slots share experts: within the bounds of both."""
    d, idx, w, x, w1, s1, w2, s2 = make(fmt, 40, 4, 8, 0, 8, 768, 256, seed=3)
    many = B.layer_tokens(d, idx, w, x, w1, w2, s1, s2)
    want, bound = exact(fmt, x, idx.long(), w, w1, s1, w2, s2, 0)
    for t in (0, 17):
        d1 = B.make_desc(1, 4, 8)
        one = B.layer_tokens(d1, idx[t:t + 1].contiguous(), w[t:t + 1].contiguous(), x[t:t + 1].contiguous(), w1,
                             w2, s1, s2)
        ref.check_bf16(one, want[t:t + 1], bound[t:t + 1], fmt)
    ref.check_bf16(many, want, bound, fmt)


def test_no_tokens():
    d, idx, w, x, w1, s1, w2, s2 = make("fp8", 0, 4, 8, 0, 8, 256, 128)
    assert B.layer_tokens(d, idx, w, x, w1, w2, s1, s2).shape == (0, 256)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 3, 50])
def test_repeats_prepared_and_op_give_equal_bits(T, fmt):
    d, idx, w, x, w1, s1, w2, s2 = make(fmt, T, 6, 32, 5, 20, 1024, 384, seed=T)
    a = B.layer_tokens(d, idx, w, x, w1, w2, s1, s2)
    out = torch.empty_like(a)
    call = B.PreparedLayerTokens(d, idx, w, x, w1, w2, out, s1, s2)
    for _ in range(4):
        out.fill_(3.0)
        call()
        assert torch.equal(out, a)
    assert torch.equal(ops.moe_layer_tokens(x, idx, w, w1, w2, 32, s1, s2, 5), a)
    assert torch.equal(ops.moe_layer_tokens(x, idx.long(), w, w1, w2, 32, s1, s2, 5), a)


@pytest.mark.parametrize("fmt", FORMATS)
def test_two_calls_at_once(fmt):
    """Two streams, each with its own workspace, and the convenience call given a stream."""
    cases = [make(fmt, T, 4, 16, 0, 16, 1024, 512, seed=T) for T in (2, 60)]
    want = [B.layer_tokens(d, idx, w, x, w1, w2, s1, s2) for d, idx, w, x, w1, s1, w2, s2 in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(10):
        for i, (d, idx, w, x, w1, s1, w2, s2) in enumerate(cases):
            got[i].append(B.layer_tokens(d, idx, w, x, w1, w2, s1, s2, stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(g, want[i]) for g in got[i])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 40])
def test_in_a_graph(T, fmt):
    """Two layers captured in one graph, replayed with new tokens and routes between eager calls."""
    d, idx, w, x, w1, s1, w2, s2 = make(fmt, T, 4, 16, 0, 16, 512, 256)

    def two(v):
        y = ops.moe_layer_tokens(v, idx, w, w1, w2, 16, s1, s2)
        return y, ops.moe_layer_tokens(y, idx, w, w1, w2, 16, s1, s2)

    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        two(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = two(x)
    for step in range(3):
        _, i2, wt, x2, *_ = make(fmt, T, 4, 16, 0, 16, 512, 256, seed=20 + step)
        idx.copy_(i2)
        w.copy_(wt)
        x.copy_(x2)
        graph.replay()
        first = B.layer_tokens(d, idx, w, x, w1, w2, s1, s2)
        assert torch.equal(out[0], first)
        assert torch.equal(out[1], B.layer_tokens(d, idx, w, first, w1, w2, s1, s2))


@pytest.mark.parametrize("T", [1, 2, 30])
@pytest.mark.parametrize("i64", [False, True])
def test_ids_far_out_of_range(i64, T):
    """Ids whose distance from local_begin passes 31 bits, and 64-bit ones whose low half is an expert."""
    d, idx, w, x, w1, s1, w2, s2 = make("mxfp4", T, 6, 16, 5, 9, 512, 256, seed=T, i64=i64)
    far = [-(1 << 31), (1 << 31) - 1, 16, -2]
    far += [(1 << 32) + 7, -(1 << 32) + 7, (1 << 40) + 5, -(1 << 63)] if i64 else [4 - (1 << 31), -(1 << 30)]
    for n, v in enumerate(far):
        idx[n % T, n % 6] = v
    check("mxfp4", d, idx, w, x, w1, s1, w2, s2, f"{T} {i64}")


def test_prepared_let_go_while_its_stream_is_busy():
    """The workspace of an object that is gone is not handed out before its stream is done."""
    d, idx, w, x, w1, s1, w2, s2 = make("mxfp4", 40, 4, 16, 0, 16, 512, 256)
    want = B.layer_tokens(d, idx, w, x, w1, w2, s1, s2)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    call = B.PreparedLayerTokens(d, idx, w, x, w1, w2, out, s1, s2, stream=st)
    n = B.moe_layer_tokens_workspace_size(d, 512, 256)
    where = next(t for t in call._keep if t is not None and t.dtype == torch.uint8 and t.numel() == n).data_ptr()
    with torch.cuda.stream(st):
        torch.cuda._sleep(100_000_000)
    call()
    del call
    again = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert where not in [t.data_ptr() for t in again] or st.query()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("T", [2, 40])
@pytest.mark.parametrize("fmt", FORMATS)
def test_weights_past_32_bits(fmt, T):
    """The first and the last expert of weights of more than 2^32 bytes each."""
    H, I = 4096, 4096
    EL = {"bf16": 130, "fp8": 258, "mxfp4": 514}[fmt]
    g = torch.Generator(device="cuda").manual_seed(T)
    few1, few2 = weights(fmt, 2, 2 * I, H, g), weights(fmt, 2, H, I, g)

    def spread(t):
        if t is None:
            return None
        big = torch.empty((EL, *t.shape[1:]), dtype=t.dtype, device="cuda")
        big[0], big[-1] = t[0], t[1]
        return big

    w1, s1, w2, s2 = (spread(t) for t in (*few1, *few2))
    assert w2.nbytes > 1 << 32 and w1.nbytes > 1 << 33
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.rand((T, 14), generator=g, device="cuda")
    ids = torch.full((T, 14), -1, dtype=torch.int32, device="cuda")
    ids[:, 3], ids[::2, 9] = EL - 1, 0
    d = B.make_desc(T, 14, EL)
    out = B.layer_tokens(d, ids, w, x, w1, w2, s1, s2)
    small = torch.where(ids == EL - 1, 1, ids).long()
    ref.check_bf16(out, *exact(fmt, x, small, w, few1[0], few1[1], few2[0], few2[1], 0), fmt)


def test_beside_the_fp8_layer():
    """One token: the E4M3 layer that quantizes rows and h lies as near as those roundings let it."""
    d, idx, w, x, w1, s1, w2, s2 = make("fp8", 1, 8, 64, 0, 64, 1024, 512, empty=0.0)
    a = ops.moe_layer_tokens(x, idx, w, w1, w2, 64, s1, s2)
    b = ops.moe_layer_fp8(x, idx, w, w1, s1, w2, s2, 64, capacity=8)
    # E4M3 rounds by up to 2^-4 of a value, twice on the way; independent errors add up far below that
    assert (a.double() - b.double()).norm() <= 2 * 2.0 ** -4 * a.double().norm()


def test_times_of_a_call():
    d, idx, w, x, w1, s1, w2, s2 = make("mxfp4", 3, 4, 16, 0, 16, 512, 256)
    t = B.KernelTimer()
    t.arm()
    B.layer_tokens(d, idx, w, x, w1, w2, s1, s2)
    torch.cuda.synchronize()
    assert 0 < t.elapsed_ms() < 50
