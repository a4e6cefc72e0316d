"""Cases for timing and comparing the 4-bit expert path of a MoE layer and the layer of a few tokens.

Microscaled 4-bit floating point (MXFP4): blocks of 32 consecutive values share a power of two, held as
an E8M0 byte, and each value is an E2M1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives).

  quantize   values -> codes and block powers -> the values that they stand for.
  dispatch   rows grouped by local expert, each the token's row quantized.
  gemm       Y[r, n] = sum_k A[r, k] W[e(r), n, k], rows and weights in MXFP4.
  swiglu     the same product with the gate and up halves of W (2I rows), then h = silu(gate) * up, as
             bf16 or again in MXFP4.
  layer      out[t] = sum_j w[t, j] W2[e] (silu(W1g[e] x[t]) * (W1u[e] x[t])), e the expert of slot j,
             for a few tokens, with weights in bf16, in E4M3 (one fp32 scale per 128 x 128 block) or in
             MXFP4.

With `own` false, `run` computes them from elementary torch operations in fp32; with `own` true it
calls the library.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
AMAX_FLOOR = 1e-4
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _case(name, op, T=0, k=1, E=1, EL=1, lb=0, P=1, sync_free=False, K=0, N=0, H=0, I=0, out="bf16",
          fmt="mxfp4", src="bf16", skew=0.0, empty=0.0):
    c = {"op": op, "T": T, "k": k, "E": E, "EL": EL, "lb": lb, "P": P, "sync_free": sync_free, "K": K,
         "N": N, "H": H, "I": I, "out": out, "fmt": fmt, "src": src, "skew": skew, "empty": empty}
    if name:
        c = {"name": name, **c}
    return c


def listed():
    return [
        # the rows of a small decode batch
        _case("quantize_rows_8", "quantize", T=8, K=2048),
        # a layer's weights at load time: 16 experts' fp32 weights of 2048 x 4096
        _case("quantize_weights_32768", "quantize", T=32768, K=4096, src="f32"),
        # serving, one token of a Qwen3-30B-A3B-shaped layer: eight rows
        _case("dispatch_token_1", "dispatch", 1, 8, 128, 128, sync_free=True, H=2048),
        # a large batch of an H = 4096 layer, all experts local
        _case("dispatch_tokens_16384", "dispatch", 16384, 8, 128, 128, P=16, H=4096),
        # one token's down projection: eight rows in eight experts
        _case("gemm_token_1", "gemm", 1, 8, 128, 128, sync_free=True, K=768, N=2048),
        # the large batch, about 1024 rows per expert
        _case("gemm_tokens_16384", "gemm", 16384, 8, 128, 128, P=16, K=2048, N=4096),
        # the gate and up projection of an odd decode batch on a quarter of the experts, requantized
        _case("swiglu_tokens_333", "swiglu", 333, 8, 128, 32, sync_free=True, K=2048, N=768,
              out="mxfp4"),
        # a prefill chunk, about 256 rows per expert, requantized for the down projection
        _case("swiglu_tokens_4096", "swiglu", 4096, 8, 128, 128, P=16, K=2048, N=768, out="mxfp4"),
        # the whole layer for one token with E4M3 weights
        _case("layer_fp8_token_1", "layer", 1, 8, 128, 128, H=2048, I=768, fmt="fp8"),
        # one token of a wider layer with MXFP4 weights
        _case("layer_mxfp4_token_1", "layer", 1, 8, 128, 128, H=4096, I=1024),
        # a decode batch of 32 tokens, MXFP4 weights, most experts in use
        _case("layer_mxfp4_tokens_32", "layer", 32, 8, 128, 128, H=2048, I=768),
        # an odd few tokens on one rank's share of the experts, bf16 weights, some slots empty
        _case("layer_bf16_tokens_5", "layer", 5, 6, 64, 32, 16, H=2048, I=768, fmt="bf16", empty=0.1),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    top = {}
    for c in listed():
        w = work(c)
        b, f = top.get(c["op"], (0, 0))
        top[c["op"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    while True:
        op = rng.choice(("quantize", "dispatch", "gemm", "swiglu", "layer"))
        E = rng.choice((4, 8, 16, 32, 60, 64, 128, 160))
        k = min(E, rng.choice((1, 2, 3, 4, 6, 8)))
        EL = max(1, E // rng.choice((1, 1, 2, 4, 8)))
        lb = rng.randrange(0, E - EL + 1)
        T, P = log(1, 16384), rng.choice((1, 1, 8, 16, 128))
        route = dict(sync_free=rng.random() < 0.5, skew=rng.choice((0.0, 0.0, 0.4)),
                     empty=rng.choice((0.0, 0.0, 0.1, 0.3)))
        if op == "quantize":
            c = _case(None, op, T=log(1, 32768), K=32 * log(1, 256), src=rng.choice(("bf16", "f32")))
        elif op == "dispatch":
            c = _case(None, op, T, k, E, EL, lb, P, H=256 * log(1, 16), **route)
        elif op == "gemm":
            c = _case(None, op, T, k, E, EL, lb, P, K=128 * log(1, 32), N=8 * log(8, 512), **route)
        elif op == "swiglu":
            c = _case(None, op, T, k, E, EL, lb, P, K=128 * log(1, 32), N=128 * log(1, 16),
                      out=rng.choice(("bf16", "mxfp4")), **route)
        else:
            route["sync_free"] = False
            c = _case(None, op, log(1, 1024 // k), k, E, EL, lb, H=256 * log(1, 16), I=128 * log(1, 16),
                      fmt=rng.choice(("bf16", "fp8", "mxfp4")), **route)
        w = work(c)
        if w["bytes"] <= top[op][0] and w["flops"] <= top[op][1]:
            return c


def _capacity(c):
    return c["T"] * min(c["k"], c["EL"]) + c["EL"] * (c["P"] - 1)


def _weight_bytes(fmt, n, K):
    if fmt == "bf16":
        return 2.0 * n * K
    if fmt == "fp8":
        return n * K + 4.0 * -(-n // 128) * -(-K // 128)
    return n * K * (0.5 + 1.0 / 32)


def work(case):
    c = case
    T, k, E, EL, K, N, H, I = (c[x] for x in ("T", "k", "E", "EL", "K", "N", "H", "I"))
    mx = 0.5 + 1.0 / 32  # bytes of a value in MXFP4
    if c["op"] == "quantize":  # values read, codes and the values they stand for written
        return {"bytes": T * K * ({"bf16": 2.0, "f32": 4.0}[c["src"]] + mx + 2.0), "flops": 2.0 * T * K}
    rows = max(1.0, T * k * (1.0 - c["empty"]) * EL / E)  # routed rows
    touched = EL * (1.0 - (1.0 - k * (1.0 - c["empty"]) / E) ** T)  # experts with a row
    if c["op"] == "dispatch":
        written = _capacity(c) if c["sync_free"] else rows
        return {"bytes": T * 2.0 * H + written * (H * (mx + 2.0) + 12.0), "flops": 2.0 * T * H}
    if c["op"] == "layer":
        wbytes = _weight_bytes(c["fmt"], 2 * I, H) + _weight_bytes(c["fmt"], H, I)
        return {"bytes": T * 4.0 * H + T * k * 8.0 + touched * wbytes, "flops": 6.0 * rows * H * I}
    n = N if c["op"] == "gemm" else 2 * N
    out = (2.0 if c["out"] == "bf16" else mx + 2.0) * N
    return {"bytes": rows * K * mx + touched * _weight_bytes("mxfp4", n, K) + rows * out,
            "flops": 2.0 * rows * n * K}


# ---------------------------------------------------------------------------
# MXFP4 from elementary operations
# ---------------------------------------------------------------------------
def _pow2(e):
    """2^e as fp32, e in [-126, 127], from its bits (exp2 and ldexp round on some devices)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _shift(v, e):
    """v * 2^e, e in [-252, 254], exact while the result is a normal number."""
    half = torch.div(e, 2, rounding_mode="floor")
    return v * _pow2(half) * _pow2(e - half)


def _mx_quant(v):
    """fp32 [..., K] -> E2M1 code values [..., K / 32, 32] and the blocks' exponents: the largest
    magnitude's power of two over 4, at least 2^-127; nearest codes, ties to even, up to 6."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    e = (torch.frexp(b.abs().amax(-1)).exponent - 3).clamp_min(-127)
    e = torch.where(b.abs().amax(-1) > 0, e, torch.full_like(e, -127))
    a = _shift(b, -e[..., None]).abs().clamp_max(6.0)
    unit = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.round(a / unit) * unit, b), e


def _mx_values(q, e, shape):
    """bf16 values of codes and exponents (exact: two significant bits)."""
    return _shift(q, e[..., None]).reshape(shape).to(torch.bfloat16)


def _mx_pack(q, e, shape):
    """Code values and exponents -> bytes of two codes, the first in the low half, and E8M0 bytes."""
    a = q.abs()
    u = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    u = (u | (torch.signbit(q).to(torch.uint8) << 3)).reshape(*shape[:-1], -1, 2)
    return u[..., 0] | (u[..., 1] << 4), (e + 127).to(torch.uint8)


def _mx_unpack(codes, scales):
    """Packed codes [..., K / 2] and E8M0 bytes [..., K / 32] -> fp32 [..., K]."""
    table = torch.tensor([*E2M1, *(-x for x in E2M1)], device=codes.device)
    q = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1, 32)
    e = scales.to(torch.int32)[..., None] - 127
    return _shift(table[q.int()], e).reshape(*codes.shape[:-1], -1)


def _mx_make(v):
    """Packed MXFP4 of fp32 values, some rows at a time."""
    flat = v.reshape(-1, v.shape[-1])
    parts = [_mx_pack(*_mx_quant(p), p.shape) for p in flat.split(max(1, (1 << 27) // v.shape[-1]))]
    return (torch.cat([p[0] for p in parts]).reshape(*v.shape[:-1], -1),
            torch.cat([p[1] for p in parts]).reshape(*v.shape[:-1], -1))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _weights(fmt, EL, n, K, g, dev):
    """Normal weights [EL, n, K] in the format and their scales, one expert after the other."""
    qs, ss = [], []
    nb, kb = -(-n // 128), K // 128
    for _ in range(EL):
        w = torch.randn((n, K), generator=g, device=dev) * K ** -0.5
        if fmt == "bf16":
            qs.append(w.to(torch.bfloat16))
        elif fmt == "fp8":
            p = torch.zeros((nb * 128, K), device=dev)
            p[:n] = w
            b = p.view(nb, 128, kb, 128)
            a = b.abs().amax((1, 3), keepdim=True).clamp_min(AMAX_FLOOR)
            q = (b * (E4M3_MAX / a)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            qs.append(q.view(nb * 128, K)[:n].contiguous().view(torch.uint8))
            ss.append((a / E4M3_MAX).view(nb, kb))
        else:
            q, s = _mx_make(w)
            qs.append(q)
            ss.append(s)
    q = torch.stack(qs)
    return (q.view(torch.float8_e4m3fn) if fmt == "fp8" else q), (torch.stack(ss) if ss else None)


def prepare(case, seed):
    c, dev = case, _device()
    g = torch.Generator(device=dev).manual_seed(seed * 7919 + 31)
    T, k, E, EL, lb, P = (c[x] for x in ("T", "k", "E", "EL", "lb", "P"))
    s = {"case": c}
    if c["op"] == "quantize":
        # rows (or weights) whose columns differ in size, a few rows of zeros among them
        x = torch.randn((T, c["K"]), generator=g, device=dev)
        x *= torch.exp(0.5 * torch.randn(c["K"], generator=g, device=dev))
        x[torch.rand(T, generator=g, device=dev) < 0.001] = 0.0
        s["x"] = x.to(torch.bfloat16) if c["src"] == "bf16" else x
        if own:
            s["q"] = torch.zeros((T, c["K"] // 2), dtype=torch.uint8, device=dev)
            s["qs"] = torch.zeros((T, c["K"] // 32), dtype=torch.uint8, device=dev)
            s["y"] = torch.zeros((T, c["K"]), dtype=torch.bfloat16, device=dev)
        return s
    # the router's answer: distinct experts, renormalised softmax weights, -1 in empty slots
    u = torch.rand((T, E), generator=g, device=dev).clamp(1e-7, 1 - 1e-7)
    score = -torch.log(-torch.log(u))
    score = score - c["skew"] * torch.log(torch.arange(1, E + 1, device=dev, dtype=torch.float32))
    top, idx = score.topk(k, dim=1)
    w = torch.softmax(top, dim=1)
    if c["empty"] > 0:
        gone = torch.rand((T, k), generator=g, device=dev) < c["empty"]
        gone |= torch.rand((T, 1), generator=g, device=dev) < 0.1 * c["empty"]
        idx = torch.where(gone, torch.full_like(idx, -1), idx)
    s["idx"], s["w"] = idx.to(torch.int32).contiguous(), w.contiguous()
    # rows: grouped by local expert, ascending token, each group padded to a multiple of P
    flat = idx.reshape(-1).long() - lb
    flat = torch.where((idx.reshape(-1) >= 0) & (flat >= 0) & (flat < EL), flat, torch.full_like(flat, EL))
    order = torch.argsort(flat, stable=True)
    tpe = torch.bincount(flat, minlength=EL + 1)[:EL]
    padded = (tpe + P - 1) // P * P
    off = torch.zeros(EL + 1, dtype=torch.int64, device=dev)
    off[1:] = padded.cumsum(0)
    start = tpe.cumsum(0) - tpe
    ndata = int(tpe.sum())
    slot = order[:ndata]
    e = flat[slot]
    row = off[e] + torch.arange(ndata, device=dev) - start[e]
    total = int(off[-1])
    cap = max(1, _capacity(c))
    R = cap if c["sync_free"] else total
    s.update(cap=cap, R=R, total=total)
    s["slot_of_row"] = torch.full((cap,), -1, dtype=torch.int64, device=dev)
    s["slot_of_row"][row] = slot
    s["row_of_slot"] = torch.full((T * k,), -1, dtype=torch.int64, device=dev)
    s["row_of_slot"][slot] = row
    s["off"] = off
    # the plain form's plan: the rows of every expert that has some, side by side
    s["used"] = (padded > 0).nonzero().view(-1)
    m = max(1, int(padded.max()))
    s["rows_of_group"] = (off[s["used"], None] + torch.arange(m, device=dev)).clamp_max(cap - 1)
    r = torch.arange(total, device=dev)
    er = torch.searchsorted(off[1:].contiguous(), r, right=True)
    s["place_of_row"] = torch.searchsorted(s["used"], er) * m + r - off[er]
    data = (s["slot_of_row"] >= 0)[:, None]
    token = s["slot_of_row"].clamp_min(0) // k
    s["expert_of_row"] = torch.full((cap,), EL, dtype=torch.int32, device=dev)
    s["expert_of_row"][:total] = er.to(torch.int32)
    # token rows with a few large columns, as hidden states have
    width = c["K"] or c["H"]
    x = torch.randn((T, width), generator=g, device=dev)
    x *= torch.exp(0.5 * torch.randn(width, generator=g, device=dev))
    n = {"dispatch": 0, "gemm": c["N"], "swiglu": 2 * c["N"], "layer": 0}[c["op"]]
    bf16, u8 = torch.bfloat16, torch.uint8
    if c["op"] in ("dispatch", "layer"):
        s["x"] = x.to(bf16)
    if c["op"] == "dispatch":
        s["y"] = torch.zeros((cap, width), dtype=bf16, device=dev)
        s["row_w"] = torch.zeros(cap, device=dev)
        s["row_token"] = torch.full((cap,), -1, dtype=torch.int32, device=dev)
        s["row_expert"] = torch.full((cap,), EL, dtype=torch.int32, device=dev)
        if own:
            s["q"] = torch.zeros((cap, width // 2), dtype=u8, device=dev)
            s["qs"] = torch.zeros((cap, width // 32), dtype=u8, device=dev)
    elif c["op"] == "layer":
        s["w1"], s["s1"] = _weights(c["fmt"], EL, 2 * c["I"], width, g, dev)
        s["w2"], s["s2"] = _weights(c["fmt"], EL, width, c["I"], g, dev)
        s["out"] = torch.zeros((T, width), dtype=bf16, device=dev)
    else:
        q, sc = _mx_make(x)
        zero = torch.zeros((), dtype=u8, device=dev)
        s["a"] = torch.where(data, q[token], zero).contiguous()
        s["sa"] = torch.where(data, sc[token], zero).contiguous()
        s["wq"], s["sw"] = _weights("mxfp4", EL, n, width, g, dev)
        s["y"] = torch.zeros((cap, c["N"]), dtype=bf16, device=dev)
        if own and c["out"] == "mxfp4":
            s["q"] = torch.zeros((cap, c["N"] // 2), dtype=u8, device=dev)
            s["qs"] = torch.zeros((cap, c["N"] // 32), dtype=u8, device=dev)
    if own:
        # what a user's program keeps: the handle of this step's route and, over its reused buffers,
        # the prepared call
        from combine_topk_idx_multihot_amd import binding as B

        mode = B.MOE_SYNC_FREE if c["sync_free"] else B.MOE_EAGER
        s["d"] = d = B.make_desc(T, k, E, lb, EL, P, mode, False, R if c["sync_free"] else 0)
        if c["op"] == "layer":
            s["call"] = B.PreparedLayerTokens(d, s["idx"], s["w"], s["x"], s["w1"], s["w2"], s["out"],
                                              s["s1"], s["s2"])
            return s
        s["h"], _ = B.route(d, s["idx"])
        if c["op"] == "gemm":
            s["call"] = B.PreparedExpertGemmMxfp4(d, s["h"], s["a"], s["sa"], c["K"], s["wq"], s["sw"], c["N"],
                                                  s["y"])
        elif c["op"] == "swiglu":
            s["call"] = B.PreparedExpertSwigluMxfp4(d, s["h"], s["a"], s["sa"], c["K"], s["wq"], s["sw"],
                                                    c["N"], s.get("q", s["y"]), s.get("qs"))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _dequant(fmt, q, sc):
    """fp32 weights [n experts, n, K]."""
    if fmt == "bf16":
        return q.float()
    if fmt == "mxfp4":
        return _mx_unpack(q, sc)
    sc = sc.repeat_interleave(128, 1)[:, :q.shape[1]]
    return (q.float().view(*q.shape[:2], -1, 128) * sc[..., None]).view(q.shape)


def _grouped(s, a, fmt, q, sc):
    """fp32 [total, n]: rows `a` [cap, K] times their experts' weights."""
    w = _dequant(fmt, q[s["used"]], None if sc is None else sc[s["used"]])
    y = torch.bmm(a[s["rows_of_group"]], w.transpose(1, 2).contiguous())
    return y.view(-1, y.shape[2])[s["place_of_row"]]


def _gated(y):
    gate, up = y.chunk(2, dim=1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain(s):
    c = s["case"]
    op, total = c["op"], s.get("total")
    if op == "quantize":
        x = s["x"].float()
        s["y"] = _mx_values(*_mx_quant(x), x.shape)
        return
    k = c["k"]
    data = s["slot_of_row"] >= 0
    slot = s["slot_of_row"].clamp_min(0)
    if op == "dispatch":
        x = s["x"].float()
        v = _mx_values(*_mx_quant(x), x.shape)
        s["y"].copy_(torch.where(data[:, None], v[slot // k], torch.zeros((), dtype=v.dtype, device=v.device)))
        s["row_w"].copy_(torch.where(data, s["w"].view(-1)[slot], torch.zeros((), device=x.device)))
        s["row_token"].copy_(torch.where(data, slot // k, torch.full_like(slot, -1)))
        s["row_expert"].copy_(s["expert_of_row"])
    elif op == "layer":
        out = torch.zeros((c["T"], c["H"]), device=s["x"].device)
        if total:
            h = _gated(_grouped(s, s["x"].float()[slot // k], c["fmt"], s["w1"], s["s1"]))
            rows = torch.zeros((s["cap"], c["I"]), device=h.device)
            rows[:total] = h
            y = _grouped(s, rows, c["fmt"], s["w2"], s["s2"])
            ros = s["row_of_slot"].view(c["T"], k)
            w = torch.where(ros >= 0, s["w"], torch.zeros_like(s["w"]))
            out = (y[ros.clamp_min(0)] * w[:, :, None]).sum(1)
        s["out"].copy_(out)
    elif total:
        y = _grouped(s, _mx_unpack(s["a"], s["sa"]), "mxfp4", s["wq"], s["sw"])
        if op == "swiglu":
            y = _gated(y)
            if c["out"] == "mxfp4":
                y = _mx_values(*_mx_quant(y), y.shape)
        s["y"][:total] = y.to(torch.bfloat16)


def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if not own:
        _plain(s)
    else:
        from combine_topk_idx_multihot_amd import binding as B

        if op == "quantize":
            B.moe_quantize_mxfp4(s["x"], c["T"], c["K"], s["q"], s["qs"])
            B.moe_dequantize_mxfp4(s["q"], s["qs"], c["T"], c["K"], s["y"])
        elif op == "dispatch":
            B.moe_dispatch_mxfp4(s["d"], s["h"], s["x"], c["H"], s["R"], s["q"], s["qs"], s["w"], s["row_w"],
                                 s["row_token"], s["row_expert"])
            B.moe_dequantize_mxfp4(s["q"], s["qs"], s["cap"], c["H"], s["y"])
        elif op == "layer":
            s["call"]()
        else:
            s["call"](s["R"])
            if "q" in s:
                B.moe_dequantize_mxfp4(s["q"], s["qs"], s["cap"], c["N"], s["y"])
    if op == "dispatch":
        return {"rows": s["y"], "row_w": s["row_w"], "row_token": s["row_token"], "row_expert": s["row_expert"]}
    return {"out": s["out"]} if op == "layer" else {"y": s["y"]}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_pow2(e):
    """2^e in fp64, e whole, from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_mx(v):
    """Values that the MXFP4 codes of v [..., K] stand for: the nearest of the code values, the even
    one of two as near."""
    v = v.double()
    grid = torch.tensor(E2M1, dtype=torch.float64, device=v.device)
    out = torch.empty_like(v)
    for lo in range(0, v.shape[-1], 32):
        b = v[..., lo:lo + 32]
        top = b.abs().amax(-1, keepdim=True)
        power = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
        # log2 may round up to a whole number just below a power of two
        power = torch.where(_exact_pow2(power) > top, power - 1, power)
        s = _exact_pow2((power - 2).clamp_min(-127.0))
        a = (b.abs() / s).clamp_max(6.0)
        above = torch.searchsorted(grid, a.contiguous()).clamp(1, 7)
        under = above - 1
        d = (a - grid[under]) - (grid[above] - a)
        pick = torch.where((d > 0) | ((d == 0) & (above % 2 == 0)), above, under)
        out[..., lo:lo + 32] = torch.sign(b) * grid[pick] * s
    return out


def _exact_weight(fmt, q, sc, e):
    """fp64 weights [n, K] of expert e."""
    if fmt == "bf16":
        return q[e].double()
    if fmt == "mxfp4":
        return _exact_unpack(q[e], sc[e])
    n, K = q[e].shape
    kb = torch.arange(K, device=q.device) // 128
    nb = torch.arange(n, device=q.device) // 128
    return q[e].to(torch.float64) * sc[e].double()[nb][:, kb]


def _exact_unpack(codes, scales):
    b = torch.empty((codes.shape[0], codes.shape[1] * 2), dtype=torch.long, device=codes.device)
    b[:, 0::2], b[:, 1::2] = codes.long() % 16, codes.long() // 16
    mag = b % 8
    v = torch.where(mag < 2, mag / 2.0, (1 + 0.5 * (mag % 2)) * _exact_pow2(mag // 2 - 1))
    v = torch.where(b >= 8, -v.double(), v.double())
    kb = torch.arange(v.shape[1], device=codes.device) // 32
    return v * _exact_pow2(scales.long() - 127)[:, kb]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c = case
    op = c["op"]
    if op == "quantize":
        return {"y": _exact_mx(s["x"])}
    T, k = c["T"], c["k"]
    dev = s["off"].device
    off = s["off"].tolist()
    slots = s["slot_of_row"]
    filled = (slots >= 0).nonzero().view(-1)
    if op == "dispatch":
        rows = torch.zeros((s["cap"], c["H"]), dtype=torch.float64, device=dev)
        rows[filled] = _exact_mx(s["x"])[slots[filled] // k]
        row_w = torch.zeros(s["cap"], dtype=torch.float64, device=dev)
        row_w[filled] = s["w"].double().view(-1)[slots[filled]]
        row_token = torch.full((s["cap"],), -1, dtype=torch.int32, device=dev)
        row_token[filled] = (slots[filled] // k).to(torch.int32)
        row_expert = torch.full((s["cap"],), c["EL"], dtype=torch.int32, device=dev)
        for e in range(c["EL"]):
            row_expert[off[e]:off[e + 1]] = e
        return {"rows": rows, "row_w": row_w, "row_token": row_token, "row_expert": row_expert}
    if op == "layer":
        out = torch.zeros((T, c["H"]), dtype=torch.float64, device=dev)
        for e in range(c["EL"]):
            for_e = slots[off[e]:off[e + 1]]
            if not len(for_e):
                continue
            y = s["x"][for_e // k].double() @ _exact_weight(c["fmt"], s["w1"], s["s1"], e).T
            gate, up = y[:, :c["I"]], y[:, c["I"]:]
            y = (gate * torch.sigmoid(gate) * up) @ _exact_weight(c["fmt"], s["w2"], s["s2"], e).T
            out.index_add_(0, for_e // k, y * s["w"].double().view(-1)[for_e, None])
        return {"out": out}
    y = torch.zeros((s["cap"], c["N"]), dtype=torch.float64, device=dev)
    for e in range(c["EL"]):
        if off[e + 1] > off[e]:
            r = slice(off[e], off[e + 1])
            v = _exact_unpack(s["a"][r], s["sa"][r]) @ _exact_unpack(s["wq"][e], s["sw"][e]).T
            if op == "swiglu":
                gate, up = v[:, :c["N"]], v[:, c["N"]:]
                v = gate * torch.sigmoid(gate) * up
                v = _exact_mx(v) if c["out"] == "mxfp4" else v
            y[r] = v
    return {"y": y}
