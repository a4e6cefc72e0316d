"""GPU: MXFP4 quantization and back, the MXFP4 dispatch and the experts' products on MXFP4 rows against
64-bit references: every bf16 value, odd sizes, block borders, NaN and infinities; group sizes around
the kernels' tiles, empty groups, odd column counts, depths that are no multiple of a step, one token
and none, eager and sync-free; rows past the total left as they were; streams, graphs and the layer."""
import pytest
import torch

import expert_ref as ref
import mx_ref as mx
from combine_topk_idx_multihot_amd import binding as B
from combine_topk_idx_multihot_amd import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.moe_device_check(0)
    yield


# ---------------------------------------------------------------------------
# quantization and back
# ---------------------------------------------------------------------------
def check_quantized(x):
    q, s = B.quantize_mxfp4(x)
    want_q, want_s = mx.make(x)
    assert torch.equal(s, want_s) and torch.equal(q, want_q)
    for dtype in (torch.bfloat16, torch.float32):
        y = B.dequantize_mxfp4(q, s, dtype)
        assert y.dtype == dtype and torch.equal(y.double(), mx.values(q, s).view(x.shape))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 32), (1, 64), (3, 96), (7, 2048), (1000, 160), (5, 8192), (4, 17, 64),
                                   (1023, 1056)])
def test_quantize(shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(shape[-1])
    x = torch.randn(shape, generator=g, device="cuda")
    x *= torch.exp(3 * torch.randn(shape[-1], generator=g, device="cuda"))
    x[..., ::3] *= 2.0 ** -20
    check_quantized(x.to(dtype))


def test_quantize_every_bf16():
    """Every finite bf16 value, beside a largest one of each power of two from 0 to 2^9 times its own."""
    x = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = x[torch.isfinite(x)]
    for up in range(0, 10):
        rows = torch.zeros((len(x), 32), dtype=torch.bfloat16, device="cuda")
        rows[:, 5] = x
        top = torch.where(x == 0, 1.0, x.abs().double() * 2.0 ** up)
        rows[:, 9] = torch.where(top < 3e38, top, x.abs().double()).to(torch.bfloat16)
        check_quantized(rows)


def test_quantize_ties_and_borders():
    """fp32 values on and beside every border between codes, and largest magnitudes beside a power of two."""
    at = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 0.0, 1e-30], device="cuda")
    near = torch.stack((at, torch.nextafter(at, at + 9), torch.nextafter(at, at - 9)), 1).view(-1)
    for power in (-126, -60, 0, 60, 120):
        x = torch.zeros((2, len(near), 32), device="cuda")
        x[0, :, 3], x[1, :, 3] = near, -near
        x[:, :, 8] = 4.0
        check_quantized(x * 2.0 ** (power / 2) * 2.0 ** (power / 2))
    top = torch.tensor([4.0, 8.0, 1.0, 2.0 ** -124, 2.0 ** -126], device="cuda")
    x = torch.zeros((15, 32), device="cuda")
    x[:, 31] = torch.stack((top, torch.nextafter(top, top * 2), torch.nextafter(top, top * 0)), 1).view(-1)
    x[:, 0] = x[:, 31] / 3
    check_quantized(x)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_quantize_not_finite(dtype, bad):
    """A block with a NaN or an infinity reads back as NaN, its neighbours do not notice."""
    x = torch.randn((4, 128), device="cuda").to(dtype)
    y = x.clone()
    y[2, 70] = bad
    q, s = B.quantize_mxfp4(y)
    want_q, want_s = B.quantize_mxfp4(x)
    want_s[2, 2] = 255
    want_q[2, 32:48] = 0
    assert torch.equal(q, want_q) and torch.equal(s, want_s)
    back = B.dequantize_mxfp4(q, s)
    assert torch.isnan(back[2, 64:96]).all() and int(torch.isnan(back).sum()) == 32


def test_dequantize_every_code_and_scale():
    codes = torch.arange(256, device="cuda", dtype=torch.int32).to(torch.uint8).view(1, 16, 16).repeat(256, 1, 1)
    scales = torch.arange(256, device="cuda", dtype=torch.int32).to(torch.uint8)[:, None, None].repeat(1, 16, 1)
    for dtype in (torch.bfloat16, torch.float32):
        y = B.dequantize_mxfp4(codes, scales.contiguous(), dtype)
        want = mx.values(codes, scales).to(dtype)
        assert torch.equal(torch.isnan(y), torch.isnan(want))
        keep = ~torch.isnan(want)
        assert torch.equal(y[keep], want[keep])
        assert torch.equal(torch.signbit(y[keep]), torch.signbit(want[keep]))


def test_quantize_leaves_the_rest_alone():
    x = torch.randn((5, 96), device="cuda")
    q = torch.full((6, 48), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((6, 3), 0x55, dtype=torch.uint8, device="cuda")
    B.moe_quantize_mxfp4(x, 5, 96, q, s)
    assert (q[5:] == 0x55).all() and (s[5:] == 0x55).all()
    out = torch.full((6, 96), 7.0, device="cuda")
    B.moe_dequantize_mxfp4(q, s, 5, 96, out)
    assert (out[5:] == 7.0).all()
    B.moe_quantize_mxfp4(x[:0], 0, 96, q, s)
    B.moe_dequantize_mxfp4(q, s, 0, 96, out[:0])
    assert B.quantize_mxfp4(x[:0])[0].shape == (0, 48)


# ---------------------------------------------------------------------------
# dispatch
# ---------------------------------------------------------------------------
def routing(T, E, k, empty, seed, dup=False):
    g = torch.Generator().manual_seed(seed)
    idx = torch.rand((T, E), generator=g).topk(k, 1).indices
    idx[torch.rand((T, k), generator=g) < empty] = -1
    if dup and T:
        idx[0, -1] = idx[0, 0]
    return idx.to(torch.int32).cuda(), torch.rand((T, k), generator=g).cuda()


@pytest.mark.parametrize("sync_free", [False, True])
@pytest.mark.parametrize("T,E,k,lb,EL,P,H", [
    (1, 8, 2, 0, 8, 1, 256), (5, 16, 4, 3, 6, 8, 768), (300, 32, 4, 0, 32, 16, 2048), (77, 128, 8, 5, 99, 1, 4096),
    (0, 8, 2, 0, 8, 4, 512), (40, 4, 4, 0, 4, 128, 1280), (1500, 16, 2, 8, 8, 1, 2304)])
def test_dispatch(T, E, k, lb, EL, P, H, sync_free):
    idx, w = routing(T, E, k, 0.15, T + H, dup=True)
    d = B.make_desc(T, k, E, lb, EL, P)
    if sync_free:
        d = B.make_desc(T, k, E, lb, EL, P, B.MOE_SYNC_FREE, False, B.moe_capacity_min(d) + 13)
    h, _ = B.route(d, idx)
    x = (torch.randn((T, H), device="cuda") * torch.exp(torch.randn(H, device="cuda"))).to(torch.bfloat16)
    rows, row_w, rt, re = B.dispatch(d, h, x, w)
    R = B.rows_for(d, h)
    q = torch.full((R + 2, H // 2), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((R + 2, H // 32), 0x55, dtype=torch.uint8, device="cuda")
    m = [torch.full((R,), -7, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
    B.moe_dispatch_mxfp4(d, h, x, H, R, q, s, w, *m)
    want_q, want_s = mx.make(rows)
    pad = rt < 0
    want_s[pad] = 0
    assert torch.equal(q[:R], want_q) and torch.equal(s[:R], want_s)
    assert (q[R:] == 0x55).all() and (s[R:] == 0x55).all()
    assert torch.equal(m[0], row_w) and torch.equal(m[1], rt) and torch.equal(m[2], re)
    q2, s2, *_ = B.dispatch_mxfp4(d, h, x, meta=False)
    assert torch.equal(q2, want_q) and torch.equal(s2, want_s)


def test_dispatch_large_tail():
    """A worst-case row array past 32 MiB: the tail is zeroed by its own launch."""
    T, E, k, H = 4096, 64, 8, 4096
    idx, w = routing(T, E, k, 0.0, 3)
    d = B.make_desc(T, k, E, 0, 8, 1)
    d = B.make_desc(T, k, E, 0, 8, 1, B.MOE_SYNC_FREE, False, B.moe_capacity_min(d))
    h, _ = B.route(d, idx)
    x = torch.randn((T, H), device="cuda").to(torch.bfloat16)
    q = torch.full((d.capacity, H // 2), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((d.capacity, H // 32), 0x55, dtype=torch.uint8, device="cuda")
    rt = torch.empty(d.capacity, dtype=torch.int32, device="cuda")
    B.moe_dispatch_mxfp4(d, h, x, H, d.capacity, q, s, None, None, rt)
    want_q, want_s = B.quantize_mxfp4(x)
    data = rt >= 0
    assert torch.equal(q[data], want_q[rt[data].long()]) and torch.equal(s[data], want_s[rt[data].long()])
    assert not q[~data].any() and not s[~data].any()


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
class Layer:
    """A routed layer whose expert e has counts[e] tokens (top-1), or random top-k routing."""

    def __init__(self, K, counts=None, T=0, E=0, k=1, lb=0, EL=None, P=1, sync_free=False, seed=0,
                 empty=0.0, extra=0):
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        if counts is not None:
            E = len(counts)
            idx = torch.repeat_interleave(torch.arange(E), torch.tensor(counts))
            T, k = len(idx), 1
            idx = idx[torch.randperm(T, generator=torch.Generator().manual_seed(seed))].view(T, 1)
            idx = idx.to(torch.int32).cuda()
        else:
            idx, _ = routing(T, E, k, empty, seed)
        EL = E if EL is None else EL
        d = B.make_desc(T, k, E, lb, EL, P)
        if sync_free:
            d = B.make_desc(T, k, E, lb, EL, P, B.MOE_SYNC_FREE, False, B.moe_capacity_min(d) + extra)
        self.d, self.K, self.EL = d, K, EL
        self.h, _ = B.route(d, idx)
        self.off = self.h.padded_offsets.tolist()
        self.total = self.off[-1]
        self.R = B.rows_for(d, self.h)
        # rows of random codes and scales; those past the total hold NaN scales, which nothing may read
        # into a result; pad rows are zero
        codes = torch.randint(0, 256, (self.R, K // 2), generator=g, device="cuda", dtype=torch.int32)
        power = torch.randint(120, 128, (self.R, K // 32), generator=g, device="cuda", dtype=torch.int32)
        self.rows_q, self.row_scale = codes.to(torch.uint8), power.to(torch.uint8)
        self.row_scale[self.total:] = 255
        tpe = self.h.tokens_per_expert.tolist()
        for e in range(EL):
            self.rows_q[self.off[e] + tpe[e]:self.off[e + 1]] = 0
            self.row_scale[self.off[e] + tpe[e]:self.off[e + 1]] = 0

    def exact(self, w_q, w_scale):
        return mx.product(self.rows_q, self.row_scale, w_q, w_scale, self.off)


def fill(shape, dtype):
    """A buffer of a value no result has, to see what a call leaves."""
    return torch.full(shape, 0x55 if dtype == torch.uint8 else -12345.0, dtype=dtype, device="cuda")


def untouched(t, r):
    return torch.equal(t[r:], fill(t[r:].shape, t.dtype))


def check_gemm(L, w_q, w_scale, what):
    N = w_q.shape[1]
    out = fill((L.R + 3, N), torch.bfloat16)
    B.moe_expert_gemm_mxfp4(L.d, L.h, L.rows_q, L.row_scale, L.K, L.R, w_q, w_scale, N, out)
    torch.cuda.synchronize()
    ref.check_bf16(out[:L.total], *L.exact(w_q, w_scale), what)
    assert untouched(out, L.total), what


def check_swiglu(L, w_q, w_scale, packed, what):
    I = w_q.shape[1] // 2
    out = fill((L.R + 3, I // 2), torch.uint8) if packed else fill((L.R + 3, I), torch.bfloat16)
    sc = fill((L.R + 3, I // 32), torch.uint8) if packed else None
    B.moe_expert_swiglu_mxfp4(L.d, L.h, L.rows_q, L.row_scale, L.K, L.R, w_q, w_scale, I, out, sc)
    torch.cuda.synchronize()
    h, err = mx.swiglu(*L.exact(w_q, w_scale))
    if packed:
        mx.check_codes(out[:L.total], sc[:L.total], h, err, what)
        assert untouched(sc, L.total), what
    else:
        ref.check_bf16(out[:L.total], h, err, what)
    assert untouched(out, L.total), what
    return out, sc


# group sizes around 16, 32, 64, 128 and 256 rows, with few and with many rows per expert on average
EDGES = [0, 1, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 0, 300]
LAYERS = {
    "edges": dict(counts=EDGES),
    "edges_padded": dict(counts=EDGES, P=16),
    "edges_few_per_expert": dict(counts=EDGES + [0] * 110),
    "edges_middle": dict(counts=EDGES + [0] * 22, P=3),
    "large_groups": dict(counts=[511, 0, 513, 700, 1]),
    "one_group": dict(counts=[1000]),
    "one_token": dict(T=1, E=128, k=8, sync_free=True, extra=5),
    "two_tokens": dict(T=2, E=4, k=4),
    "few_tokens": dict(counts=[0, 20, 1, 11]),
    "few_tokens_padded": dict(counts=[17, 0, 3, 7], P=8, sync_free=True, extra=9),
    "few_of_many": dict(T=3, E=200, k=5),
    "two_large": dict(counts=[1000, 900, 40]),
    "decode": dict(T=77, E=32, k=4, sync_free=True, P=8, empty=0.2),
    "share": dict(T=700, E=32, k=8, lb=5, EL=7, sync_free=True, extra=100),
    "single_local": dict(T=90, E=16, k=3, lb=15, EL=1),
    "many_experts": dict(T=300, E=1024, k=6, lb=1, EL=1000, P=2),
}
# depths of one and more steps of 128 and 256 columns, odd numbers of 128 among them; many column tiles
# (tall tiles of rows, as fewer would leave most of the chip idle)
SHAPES = [(128, 8), (256, 136), (384, 512), (768, 200), (2048, 264), (256, 2312), (384, 2312), (640, 2560),
          (1024, 2560), (2176, 2312)]


@pytest.mark.parametrize("K,N", SHAPES)
@pytest.mark.parametrize("name", LAYERS)
def test_gemm(name, K, N):
    if name == "many_experts" and K * N > 200_000:
        K, N = 256, 136
    L = Layer(K, seed=K + N, **LAYERS[name])
    check_gemm(L, *mx.make_weights(L.EL, N, K, L.g), f"{name} {K} {N}")


@pytest.mark.parametrize("K,I", [(128, 128), (640, 256), (2048, 384), (256, 1280), (640, 1280), (1152, 1280)])
@pytest.mark.parametrize("name", LAYERS)
def test_swiglu(name, K, I):
    if name == "many_experts":
        K, I = min(K, 256), min(I, 128)
    L = Layer(K, seed=K + I, **LAYERS[name])
    w = mx.make_weights(L.EL, 2 * I, K, L.g)
    check_swiglu(L, *w, True, f"{name} {K} {I} codes")
    check_swiglu(L, *w, False, f"{name} {K} {I} bf16")


@pytest.mark.parametrize("sync_free", [False, True])
@pytest.mark.parametrize("T,P", [(3, 128), (40, 128), (300, 32)])
def test_mostly_pad_rows(T, P, sync_free):
    """Groups of a few tokens padded to many rows."""
    L = Layer(384, T=T, E=16, k=4, P=P, sync_free=sync_free, seed=T)
    w = mx.make_weights(16, 2560, 384, L.g)
    check_gemm(L, *w, f"{T} padded to {P}")
    check_swiglu(L, *w, True, f"{T} padded to {P} codes")
    check_swiglu(L, *w, False, f"{T} padded to {P} bf16")


def test_swiglu_saturated_gates_and_zero_blocks():
    """Gates far on both sides: silu(g) -> g and -> 0; blocks whose h is 0 get scale byte 0."""
    L = Layer(256, counts=[40, 3, 300])
    w_q, w_s = mx.make_weights(3, 256, 256, L.g)
    w_s[0] += 5
    w_q[1, 128:] = 0
    w_q[2, 128 + 32:128 + 64] = 0
    out, sc = check_swiglu(L, w_q, w_s, True, "saturated")
    assert not sc[40:43].any() and not (out[40:43] & 0x77).any()
    assert not sc[43:343, 1].any() and sc[43:343, 0].all()
    check_swiglu(L, w_q, w_s, False, "saturated bf16")


def test_products_at_the_ends_of_the_scale():
    """Scale bytes of 0 and of 252 against each other: products of ordinary size."""
    for counts in ([3], [700, 40]):
        L = Layer(384, counts=counts)
        w_q, w_s = mx.make_weights(L.EL, 2560, 384, L.g)
        L.row_scale[:] = 0
        w_s[:] = 252
        check_gemm(L, w_q, w_s, "small rows, large weights")
        L.row_scale[:] = 252
        w_s[:] = 0
        check_gemm(L, w_q, w_s, "large rows, small weights")


@pytest.mark.parametrize("counts,N", [([5, 9, 0], 256), ([200, 300, 0], 256), ([1200, 600], 5120)])
@pytest.mark.parametrize("K", [256, 384])
def test_nan_row_and_weight_row_stay_alone(counts, N, K):
    L = Layer(K, counts=counts)
    w_q, w_s = mx.make_weights(L.EL, N, K, L.g)
    args = (L.d, L.h, L.rows_q, L.row_scale)
    clean = B.expert_gemm_mxfp4(*args, w_q, w_s)
    h_clean, _ = B.expert_swiglu_mxfp4(*args, w_q, w_s, torch.bfloat16)
    scale = L.row_scale.clone()
    scale[3, K // 32 - 1] = 255
    scale[counts[0] + 1, 1] = 255
    L.rows_q[3, -16:] = 0  # codes of 0 under a NaN scale
    bad_w = w_s.clone()
    bad_w[1, 7, K // 32 - 2] = 255
    y = B.expert_gemm_mxfp4(L.d, L.h, L.rows_q, scale, w_q, bad_w)
    h, _ = B.expert_swiglu_mxfp4(L.d, L.h, L.rows_q, scale, w_q, bad_w, torch.bfloat16)
    q, qs = B.expert_swiglu_mxfp4(L.d, L.h, L.rows_q, scale, w_q, bad_w)
    back = B.dequantize_mxfp4(q, qs)
    for r in (3, counts[0] + 1):
        assert torch.isnan(y[r]).all() and torch.isnan(h[r]).all() and torch.isnan(back[r]).all()
    first, second = torch.arange(L.total) < counts[0], torch.arange(L.total) >= counts[0]
    first[3], second[counts[0] + 1] = False, False
    assert torch.equal(y[first], clean[first]) and torch.equal(h[first], h_clean[first])
    cols = torch.arange(N) != 7
    assert torch.isnan(y[second][:, 7]).all() and torch.equal(y[second][:, cols], clean[second][:, cols])
    cols = torch.arange(N // 2) != 7
    assert torch.isnan(h[second][:, 7]).all() and torch.equal(h[second][:, cols], h_clean[second][:, cols])
    assert torch.isnan(back[second][:, :32]).all() and not torch.isnan(back[second][:, 32:]).any()


def test_repeats_and_prepared_give_equal_bits():
    L = Layer(768, T=1500, E=16, k=2, P=16)
    w = mx.make_weights(16, 512, 768, L.g)
    a = B.expert_gemm_mxfp4(L.d, L.h, L.rows_q, L.row_scale, *w)
    out = torch.empty_like(a)
    call = B.PreparedExpertGemmMxfp4(L.d, L.h, L.rows_q, L.row_scale, 768, *w, 512, out)
    for _ in range(3):
        out.fill_(7.0)
        call(L.R)
        assert torch.equal(out, a)
    q, s = B.expert_swiglu_mxfp4(L.d, L.h, L.rows_q, L.row_scale, *w)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    B.PreparedExpertSwigluMxfp4(L.d, L.h, L.rows_q, L.row_scale, 768, *w, 256, q2, s2)(L.R)
    assert torch.equal(q2, q) and torch.equal(s2, s)


def test_eager_fewer_rows_than_routed():
    """R below the device's total: only rows [0, R) are computed and the mismatch is flagged."""
    L = Layer(256, counts=[30, 50, 20])
    w = mx.make_weights(3, 128, 256, L.g)
    out = fill((L.R, 128), torch.bfloat16)
    R = 61
    B.moe_expert_gemm_mxfp4(L.d, L.h, L.rows_q, L.row_scale, 256, R, *w, 128, out)
    y, bound = L.exact(*w)
    ref.check_bf16(out[:R], y[:R], bound[:R], "short")
    assert untouched(out, R)
    assert int(L.h.status[1]) & B.MOE_FLAG_ROWS_MISMATCH


def test_past_32_bits():
    """Values, codes, rows, weights and outputs of more than 2^32 bytes."""
    n, K = (1 << 18) + 5, 1 << 15  # 8.6e9 values
    last = slice(n - 9, n)
    x = torch.empty((n, K), dtype=torch.bfloat16, device="cuda").normal_()
    q, s = B.quantize_mxfp4(x)
    assert q.nbytes > 1 << 32
    for r in (slice(0, 3), last):
        want_q, want_s = mx.make(x[r])
        assert torch.equal(q[r], want_q) and torch.equal(s[r], want_s)
    # dispatch: the token's codes, at its row
    idx = torch.arange(n, dtype=torch.int32, device="cuda").view(n, 1) % 4
    d = B.make_desc(n, 1, 4)
    h, _ = B.route(d, idx)
    rows_q, row_scale, _, rt, _ = B.dispatch_mxfp4(d, h, x)
    for r in (slice(0, 3), last):
        t = rt[r].long()
        assert torch.equal(rows_q[r], q[t]) and torch.equal(row_scale[r], s[t])
    y = B.dequantize_mxfp4(q, s)
    assert torch.equal(y[last].double(), mx.values(q[last], s[last]))
    del x, q, s, y
    # rows past 2^32 bytes, then outputs
    g = torch.Generator(device="cuda").manual_seed(1)
    off = h.padded_offsets.tolist()
    w, ws = mx.make_weights(4, 16, K, g)
    out = B.expert_gemm_mxfp4(d, h, rows_q, row_scale, w, ws)
    r = slice(off[-1] - 9, off[-1])
    want = mx.product(rows_q[r], row_scale[r], w[3:], ws[3:], [0, 9])
    ref.check_bf16(out[r], *want, "rows")
    a, sa = rows_q[:, :64].contiguous(), row_scale[:, :4].contiguous()
    del rows_q, row_scale, out
    w, ws = mx.make_weights(4, 2 * 8320, 128, g)
    out = B.expert_gemm_mxfp4(d, h, a, sa, w, ws)
    assert out.nbytes > 1 << 33
    ref.check_bf16(out[r], *mx.product(a[r], sa[r], w[3:], ws[3:], [0, 9]), "outputs")
    out, _ = B.expert_swiglu_mxfp4(d, h, a, sa, w, ws, torch.bfloat16)
    assert out.nbytes > 1 << 32
    ref.check_bf16(out[r], *mx.swiglu(*mx.product(a[r], sa[r], w[3:], ws[3:], [0, 9])), "gated")


@pytest.mark.parametrize("rows", [1, 30, 700])
def test_weights_past_32_bits(rows):
    """The last expert of weights of more than 2^32 bytes, in each of the kernels."""
    E, N, K = 260, 8192, 4096
    L = Layer(K, counts=[rows] + [0] * (E - 2) + [rows], seed=rows)
    few, few_s = mx.make_weights(2, N, K, L.g)
    w = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    ws = torch.zeros((E, N, K // 32), dtype=torch.uint8, device="cuda")
    w[0], w[-1], ws[0], ws[-1] = few[0], few[1], few_s[0], few_s[1]
    assert w.nbytes > 1 << 32
    where = [0, rows, 2 * rows]
    y, bound = mx.product(L.rows_q, L.row_scale, few, few_s, where)
    out = B.expert_gemm_mxfp4(L.d, L.h, L.rows_q, L.row_scale, w, ws)
    ref.check_bf16(out, y, bound, "plain")
    out, _ = B.expert_swiglu_mxfp4(L.d, L.h, L.rows_q, L.row_scale, w, ws, torch.bfloat16)
    ref.check_bf16(out, *mx.swiglu(y, bound), "gated")


def test_no_tokens():
    d = B.make_desc(0, 2, 4)
    h, _ = B.route(d, torch.empty((0, 2), dtype=torch.int32, device="cuda"))
    w_q, w_s = mx.make_weights(4, 256, 256, torch.Generator(device="cuda"))
    q = torch.empty((0, 128), dtype=torch.uint8, device="cuda")
    s = torch.empty((0, 8), dtype=torch.uint8, device="cuda")
    assert B.expert_gemm_mxfp4(d, h, q, s, w_q, w_s).shape == (0, 256)
    assert B.expert_swiglu_mxfp4(d, h, q, s, w_q, w_s)[0].shape == (0, 64)


def test_typed_codes():
    """torch's own types of packed codes and scales, where it has them."""
    if not hasattr(torch, "float4_e2m1fn_x2"):
        pytest.skip("no float4_e2m1fn_x2")
    L = Layer(256, counts=[3, 4])
    w_q, w_s = mx.make_weights(2, 64, 256, L.g)
    a = B.expert_gemm_mxfp4(L.d, L.h, L.rows_q, L.row_scale, w_q, w_s)
    t, e = torch.float4_e2m1fn_x2, torch.float8_e8m0fnu
    assert torch.equal(a, B.expert_gemm_mxfp4(L.d, L.h, L.rows_q.view(t), L.row_scale.view(e), w_q.view(t),
                                              w_s.view(e)))


# ---------------------------------------------------------------------------
# the layer made of them, streams and graphs
# ---------------------------------------------------------------------------
def layer_by_steps(idx, w, x, E, lb, P, w1, s1, w2, s2):
    """The layer from the binding's calls, eager."""
    d = B.make_desc(*idx.shape, E, lb, w1.shape[0], P)
    h, _ = B.route(d, idx)
    q, s, *_ = B.dispatch_mxfp4(d, h, x, meta=False)
    hq, hs = B.expert_swiglu_mxfp4(d, h, q, s, w1, s1)
    return B.combine_weighted(d, h, B.expert_gemm_mxfp4(d, h, hq, hs, w2, s2), w)


def test_layer_against_64_bits():
    """Every step of the layer from the one before it, in 64 bits."""
    T, E, k, H, I, lb, EL = 150, 16, 4, 512, 384, 4, 8
    idx, w = routing(T, E, k, 0.1, 5)
    g = torch.Generator(device="cuda").manual_seed(1)
    w1, s1 = mx.make_weights(EL, 2 * I, H, g)
    w2, s2 = mx.make_weights(EL, H, I, g)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    d = B.make_desc(T, k, E, lb, EL, 8)
    h, _ = B.route(d, idx)
    off = h.padded_offsets.tolist()
    q, s, *_ = B.dispatch_mxfp4(d, h, x, meta=False)
    hq, hs = B.expert_swiglu_mxfp4(d, h, q, s, w1, s1)
    mx.check_codes(hq, hs, *mx.swiglu(*mx.product(q, s, w1, s1, off)), "gated")
    Y = B.expert_gemm_mxfp4(d, h, hq, hs, w2, s2)
    ref.check_bf16(Y, *mx.product(hq, hs, w2, s2, off), "down")
    out = B.combine_weighted(d, h, Y, w)
    ros = h.row_of_slot.long()
    want = (Y[ros.clamp_min(0)].double() * torch.where(ros >= 0, w, 0.0).double()[:, :, None]).sum(1)
    mag = (Y[ros.clamp_min(0)].double().abs() * torch.where(ros >= 0, w, 0.0).double()[:, :, None]).sum(1)
    ref.check_bf16(out, want, (k + 1) * ref.U * mag, "combine")
    for capacity in (0, B.moe_capacity_min(d) + 3):
        got = ops.moe_layer_mxfp4(x, idx, w, w1, s1, w2, s2, E, lb, 8, capacity)
        assert torch.equal(got, out)


def test_side_stream():
    L = Layer(512, counts=[40, 0, 7])
    w = mx.make_weights(3, 256, 512, L.g)
    want = B.expert_gemm_mxfp4(L.d, L.h, L.rows_q, L.row_scale, *w)
    x = torch.randn((300, 512), device="cuda")
    q, s = B.quantize_mxfp4(x)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = B.expert_gemm_mxfp4(L.d, L.h, L.rows_q, L.row_scale, *w)
        q2, s2 = B.quantize_mxfp4(x)
        y2 = B.dequantize_mxfp4(q2, s2)
    st.synchronize()
    assert torch.equal(got, want) and torch.equal(q, q2) and torch.equal(s, s2)
    assert torch.equal(y2, B.dequantize_mxfp4(q, s))


@pytest.mark.parametrize("T", [1, 40, 600])
def test_layer_in_a_graph(T):
    """Two layers captured in one graph, replayed with new tokens and routes between eager calls."""
    E, k, H, I, P = 16, 4, 512, 256, 8
    g = torch.Generator(device="cuda").manual_seed(2)
    w1, s1 = mx.make_weights(E, 2 * I, H, g)
    w2, s2 = mx.make_weights(E, H, I, g)
    idx, w = routing(T, E, k, 0.1, 0)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    cap = T * k + E * (P - 1)

    def two(x, idx, w):
        y = ops.moe_layer_mxfp4(x, idx, w, w1, s1, w2, s2, E, 0, P, cap)
        return y, ops.moe_layer_mxfp4(y, idx, w, w1, s1, w2, s2, E, 0, P, cap)

    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        two(x, idx, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = two(x, idx, w)
    for step in range(3):
        i2, wt = routing(T, E, k, 0.1, 10 + step)
        idx.copy_(i2)
        w.copy_(wt)
        x.copy_(torch.randn((T, H), device="cuda"))
        graph.replay()
        first = layer_by_steps(idx, w, x, E, 0, P, w1, s1, w2, s2)
        assert torch.equal(out[0], first)
        assert torch.equal(out[1], layer_by_steps(idx, w, first, E, 0, P, w1, s1, w2, s2))


def test_times_of_a_call():
    L = Layer(512, counts=[40, 7])
    w = mx.make_weights(2, 256, 512, L.g)
    x = torch.randn((64, 512), device="cuda")
    q, s = B.quantize_mxfp4(x)
    t = B.KernelTimer()
    for call in (lambda: B.expert_gemm_mxfp4(L.d, L.h, L.rows_q, L.row_scale, *w),
                 lambda: B.expert_swiglu_mxfp4(L.d, L.h, L.rows_q, L.row_scale, *w),
                 lambda: B.quantize_mxfp4(x), lambda: B.dequantize_mxfp4(q, s)):
        t.arm()
        call()
        torch.cuda.synchronize()
        assert 0 < t.elapsed_ms() < 50
