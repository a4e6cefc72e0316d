"""Cases for timing and comparing the expert-side operators of a MoE layer in the expanded layout.

Four operators work on rows grouped by local expert, group e being rows [off[e], off[e+1]):

  gemm          Y[r, n] = sum_k A[r, k] W[e(r), n, k] with A and W in 8-bit floating point (E4M3):
                A has one fp32 scale per row and 128 columns, W one per 128 x 128 block.
  swiglu        the same product with the gate and up halves of W (2I rows), then
                h = silu(gate) * up, as bf16 or again as E4M3 with one scale per 128 columns.
  combine       out[t] = sum over the token's rows r of w[t, r] Y[r].
  combine_bwd   grad_rows[r] = w[t, r] grad_out[t] and dw[t, j] = dot(grad_out[t], Y[row of slot j]).

With `own` false, `run` computes them from elementary torch operations in fp32; with `own` true it
calls the library.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
AMAX_FLOOR = 1e-4


def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _case(name, op, T, k, E, EL, P, sync_free, K=0, N=0, H=0, out="bf16", skew=0.0, empty=0.0):
    c = {"op": op, "T": T, "k": k, "E": E, "EL": EL, "P": P, "sync_free": sync_free, "K": K,
         "N": N, "H": H, "out": out, "skew": skew, "empty": empty}
    if name:
        c = {"name": name, **c}
    return c


def listed():
    return [
        # serving, one token: the down projection of a Qwen3-30B-A3B-shaped layer, eight rows in
        # eight experts, bound by latency and by reading eight experts' weights
        _case("gemm_token_1", "gemm", 1, 8, 128, 128, 1, True, K=768, N=2048),
        # a decode batch of 256 tokens: about 16 rows in every expert, all weights read once
        _case("gemm_tokens_256", "gemm", 256, 8, 128, 128, 1, True, K=768, N=2048),
        # a prefill chunk of that layer, about 256 rows per expert
        _case("gemm_tokens_4096", "gemm", 4096, 8, 128, 128, 16, False, K=768, N=2048),
        # a large batch of an H = 4096 layer, all experts local, about 1024 rows per expert
        _case("gemm_tokens_16384", "gemm", 16384, 8, 128, 128, 16, False, K=2048, N=4096),
        # the gate and up projection with its activation, one token
        _case("swiglu_token_1", "swiglu", 1, 8, 128, 128, 1, True, K=2048, N=768, out="fp8"),
        # an odd decode batch on a quarter of the experts
        _case("swiglu_tokens_333", "swiglu", 333, 8, 128, 32, 1, True, K=2048, N=768, out="fp8"),
        # the prefill chunk, requantized for the second product
        _case("swiglu_tokens_4096", "swiglu", 4096, 8, 128, 128, 16, False, K=2048, N=768,
              out="fp8"),
        # one rank's share (16 of 128 experts) of a large batch, rows sized for the worst case,
        # bf16 activations
        _case("swiglu_share_16384", "swiglu", 16384, 8, 128, 16, 1, True, K=4096, N=1024),
        # one token's eight rows back to token order
        _case("combine_token_1", "combine", 1, 8, 128, 128, 1, True, H=2048),
        # the large batch back to token order
        _case("combine_tokens_16384", "combine", 16384, 8, 128, 128, 16, False, H=4096),
        # training step with uneven experts, empty slots and an odd number of tokens
        _case("combine_bwd_skewed_8191", "combine_bwd", 8191, 8, 128, 128, 128, False, H=2048,
              skew=1.2, empty=0.1),
        # training step on the large batch
        _case("combine_bwd_tokens_16384", "combine_bwd", 16384, 8, 128, 128, 16, False, H=4096),
    ]


def draw(rng):
    top = {}
    for c in listed():
        w = work(c)
        b, f = top.get(c["op"], (0, 0))
        top[c["op"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    while True:
        op = rng.choice(("gemm", "swiglu", "combine", "combine_bwd"))
        E = rng.choice((4, 8, 16, 32, 60, 64, 128, 160))
        k = min(E, rng.choice((1, 2, 3, 4, 6, 8)))
        EL = max(1, E // rng.choice((1, 1, 2, 4, 8)))
        T = int(round(math.exp(rng.uniform(0, math.log(16384)))))
        P = rng.choice((1, 1, 8, 16, 128))
        sync_free = rng.random() < 0.5
        skew = rng.choice((0.0, 0.0, 0.4))
        empty = rng.choice((0.0, 0.0, 0.1, 0.3))
        if op in ("combine", "combine_bwd"):
            H = 256 * int(round(math.exp(rng.uniform(0, math.log(16)))))
            c = _case(None, op, T, k, E, EL, P, sync_free, H=H,
                      out=rng.choice(("bf16", "f32")) if op == "combine" else "bf16", skew=skew,
                      empty=empty)
        else:
            K = 128 * int(round(math.exp(rng.uniform(math.log(2), math.log(32)))))
            if op == "gemm":
                N = 8 * int(round(math.exp(rng.uniform(math.log(8), math.log(512)))))
                out = "bf16"
            else:
                N = 128 * int(round(math.exp(rng.uniform(0, math.log(16)))))
                out = rng.choice(("bf16", "fp8"))
            c = _case(None, op, T, k, E, EL, P, sync_free, K=K, N=N, out=out, skew=skew,
                      empty=empty)
        w = work(c)
        if w["bytes"] <= top[op][0] and w["flops"] <= top[op][1]:
            return c


def _capacity(c):
    return c["T"] * min(c["k"], c["EL"]) + c["EL"] * (c["P"] - 1)


def work(case):
    c = case
    T, k, E, EL, K, N, H = (c[x] for x in ("T", "k", "E", "EL", "K", "N", "H"))
    share = (1.0 - c["empty"]) * EL / E
    rows = max(1.0, T * k * share)  # routed rows
    if c["op"] in ("gemm", "swiglu"):
        touched = EL * (1.0 - (1.0 - k * (1.0 - c["empty"]) / E) ** T)  # experts with a row
        n = N if c["op"] == "gemm" else 2 * N
        out = {"bf16": 2.0, "f32": 4.0, "fp8": 1.0 + 4.0 / 128}[c["out"]] * N
        wbytes = n * K + 4.0 * -(-n // 128) * (K // 128)
        flops = 2.0 * rows * n * K
        return {"bytes": rows * (K + 4.0 * (K // 128)) + touched * wbytes + rows * out,
                "flops": flops}
    if c["op"] == "combine":
        return {"bytes": rows * 2.0 * H + T * H * (4.0 if c["out"] == "f32" else 2.0) + T * k * 8.0,
                "flops": 2.0 * rows * H}
    written = _capacity(c) if c["sync_free"] else rows
    return {"bytes": T * 2.0 * H + rows * 2.0 * H + written * 2.0 * H + T * k * 12.0,
            "flops": 3.0 * rows * H}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _quant_rows(v):
    """fp32 [..., n], n a multiple of 128 -> E4M3 codes and one scale per 128 columns."""
    b = v.reshape(*v.shape[:-1], -1, 128)
    a = b.abs().amax(-1, keepdim=True).clamp_min(AMAX_FLOOR)
    q = (b * (E4M3_MAX / a)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.reshape(v.shape), (a / E4M3_MAX).squeeze(-1).contiguous()


def _weights(EL, n, K, g, dev):
    """E4M3 [EL, n, K] and fp32 scales [EL, ceil(n / 128), K / 128] of normal weights."""
    nb = -(-n // 128)
    w = torch.zeros((EL, nb * 128, K), dtype=torch.float32, device=dev)
    w[:, :n] = torch.randn((EL, n, K), generator=g, device=dev) * K ** -0.5
    b = w.view(EL, nb, 128, K // 128, 128)
    a = b.abs().amax((2, 4), keepdim=True).clamp_min(AMAX_FLOOR)
    q = (b * (E4M3_MAX / a)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    q = q.view(EL, nb * 128, K)[:, :n].contiguous()
    return q, (a / E4M3_MAX).reshape(EL, nb, K // 128).contiguous()


def prepare(case, seed):
    c, dev = case, _device()
    T, k, E, EL, P = (c[x] for x in ("T", "k", "E", "EL", "P"))
    g = torch.Generator(device=dev).manual_seed(seed * 7919 + 13)
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
    idx = idx.to(torch.int32).contiguous()
    # rows: grouped by local expert, ascending token, each group padded to a multiple of P
    flat = idx.reshape(-1).long()
    local = (flat >= 0) & (flat < EL)
    key = torch.where(local, flat, torch.full_like(flat, EL))
    order = torch.argsort(key, stable=True)
    tpe = torch.bincount(key, minlength=EL + 1)[:EL]
    padded = (tpe + P - 1) // P * P
    off = torch.zeros(EL + 1, dtype=torch.int64, device=dev)
    off[1:] = padded.cumsum(0)
    start = tpe.cumsum(0) - tpe
    ndata = int(tpe.sum())
    slot = order[:ndata]
    e = key[slot]
    row = off[e] + torch.arange(ndata, device=dev) - start[e]
    row_of_slot = torch.full((T * k,), -1, dtype=torch.int64, device=dev)
    row_of_slot[slot] = row
    total = int(off[-1])
    # row buffers hold the worst case, as in a loop that keeps them; eager calls get the step's rows
    cap = _capacity(c)
    R = cap if c["sync_free"] else total
    token_of_row = torch.full((cap,), -1, dtype=torch.int64, device=dev)
    token_of_row[row] = slot // k
    s = {"case": c, "cap": cap, "R": R, "total": total, "w": w.contiguous(),
         "row_of_slot": row_of_slot.view(T, k)}
    # the plain form's plan: every group's rows side by side, groups of equal length
    m = max(1, int(padded.max()))
    s["rows_of_group"] = (off[:-1, None] + torch.arange(m, device=dev)).clamp_max(cap - 1)
    r = torch.arange(total, device=dev)
    eg = torch.searchsorted(off[1:].contiguous(), r, right=True)
    s["place_of_row"] = eg * m + r - off[eg]
    s["slot_of_row"] = torch.zeros(cap, dtype=torch.int64, device=dev)
    s["slot_of_row"][row] = slot
    s["data_row"] = token_of_row >= 0
    data = s["data_row"][:, None]
    if c["op"] in ("gemm", "swiglu"):
        K, n = c["K"], c["N"] * (1 if c["op"] == "gemm" else 2)
        # token rows with a few large columns, as hidden states have
        x = torch.randn((T, K), generator=g, device=dev)
        x = x * torch.exp(0.5 * torch.randn(K, generator=g, device=dev))
        q, sc = _quant_rows(x)
        pick = token_of_row.clamp_min(0)
        s["a"] = torch.where(data, q.view(torch.uint8)[pick], torch.zeros((), dtype=torch.uint8, device=dev))
        s["a"] = s["a"].view(torch.float8_e4m3fn).contiguous()
        s["sa"] = torch.where(data, sc[pick], torch.zeros((), device=dev)).contiguous()
        s["wq"], s["sw"] = _weights(EL, n, K, g, dev)
        kind = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}[c["out"]]
        s["y"] = torch.zeros((cap, c["N"]), dtype=torch.uint8 if c["out"] == "fp8" else kind, device=dev).view(kind)
        s["ys"] = torch.zeros((cap, c["N"] // 128), dtype=torch.float32, device=dev) if c["out"] == "fp8" else None
    else:
        H = c["H"]
        y = torch.randn((cap, H), generator=g, device=dev, dtype=torch.bfloat16)
        s["y"] = torch.where(data, y, torch.zeros((), dtype=torch.bfloat16, device=dev))
        del y
        if c["op"] == "combine":
            s["out"] = torch.zeros((T, H), dtype=torch.float32 if c["out"] == "f32" else torch.bfloat16, device=dev)
        else:
            s["g"] = torch.randn((T, H), generator=g, device=dev, dtype=torch.bfloat16)
            s["grad_rows"] = torch.zeros((cap, H), dtype=torch.bfloat16, device=dev)
            s["dw"] = torch.zeros((T, k), dtype=torch.float32, device=dev)
    if own:
        # what a user's program keeps: the handle of this step's route and, over its reused
        # buffers, the prepared call
        from combine_topk_idx_multihot_amd import binding as B

        mode = B.MOE_SYNC_FREE if c["sync_free"] else B.MOE_EAGER
        d = B.make_desc(T, k, E, 0, EL, P, mode, False, R if c["sync_free"] else 0)
        h, _ = B.route(d, idx)
        if c["op"] == "gemm":
            s["call"] = B.PreparedExpertGemmFp8(d, h, s["a"], s["sa"], c["K"], s["wq"], s["sw"], c["N"], s["y"])
        elif c["op"] == "swiglu":
            s["call"] = B.PreparedExpertSwigluFp8(d, h, s["a"], s["sa"], c["K"], s["wq"], s["sw"], c["N"], s["y"], s["ys"])
        elif c["op"] == "combine":
            s["call"] = B.PreparedCombineWeighted(d, h, s["y"], c["H"], s["w"], s["out"])
        else:
            s["call"] = B.PreparedCombineWeightedBwd(d, h, s["g"], s["y"], c["H"], s["w"], s["grad_rows"], s["dw"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _values(q, sc):
    """The values that E4M3 codes with a scale per 128 columns stand for; bf16 keeps 16 times the
    codes' own precision."""
    v = q.view(q.shape[0], -1, 128).to(torch.bfloat16) * sc.to(torch.bfloat16)[:, :, None]
    return v.view(q.shape)


def _product(s):
    """fp32 rows [total, n] of the grouped product."""
    a = (s["a"].float().view(s["cap"], -1, 128) * s["sa"][:, :, None]).view(s["cap"], -1)
    EL, n, K = s["wq"].shape
    sw = s["sw"].repeat_interleave(128, 1)[:, :n]
    w = (s["wq"].float().view(EL, n, -1, 128) * sw[..., None]).view(EL, n, K)
    y = torch.bmm(a[s["rows_of_group"]], w.transpose(1, 2).contiguous())
    return y.view(-1, n)[s["place_of_row"]]


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        s["call"](s["R"])
    elif op == "gemm":
        if s["total"]:
            s["y"][:s["total"]] = _product(s).to(s["y"].dtype)
    elif op == "swiglu":
        if s["total"]:
            gate, up = _product(s).chunk(2, dim=1)
            h = gate / (1.0 + torch.exp(-gate)) * up
            if s["ys"] is None:
                s["y"][:s["total"]] = h.to(s["y"].dtype)
            else:
                q, sc = _quant_rows(h)
                s["y"].view(torch.uint8)[:s["total"]] = q.view(torch.uint8)
                s["ys"][:s["total"]] = sc
    elif op == "combine":
        ros = s["row_of_slot"]
        w = torch.where(ros >= 0, s["w"], torch.zeros_like(s["w"]))
        rows = s["y"][ros.clamp_min(0)].float()
        s["out"].copy_((rows * w[:, :, None]).sum(1))
    else:
        ros, g = s["row_of_slot"], s["g"].float()
        slot = s["slot_of_row"]
        wr = torch.where(s["data_row"], s["w"].view(-1)[slot], torch.zeros((), device=g.device))
        s["grad_rows"].copy_(g[slot // ros.shape[1]] * wr[:, None])
        dots = (s["y"][ros.clamp_min(0)].float() * g[:, None]).sum(2)
        s["dw"].copy_(torch.where(ros >= 0, dots, torch.zeros_like(dots)))
    if op == "gemm":
        return {"y": s["y"]}
    if op == "swiglu":
        return {"h": s["y"] if s["ys"] is None else _values(s["y"], s["ys"])}
    if op == "combine":
        return {"out": s["out"]}
    return {"grad_rows": s["grad_rows"], "dw": s["dw"]}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_product(s):
    """fp64 rows [cap, n], one expert's block of rows after the other."""
    EL, n, K = s["wq"].shape
    kb = torch.arange(K, device=s["a"].device) // 128
    nb = torch.arange(n, device=s["a"].device) // 128
    y = torch.zeros((s["cap"], n), dtype=torch.float64, device=s["a"].device)
    groups = torch.bincount(s["place_of_row"] // s["rows_of_group"].shape[1], minlength=EL).tolist()
    r0 = 0
    for e in range(EL):
        r1 = r0 + groups[e]
        if r1 > r0:
            a = s["a"][r0:r1].to(torch.float64) * s["sa"][r0:r1].double()[:, kb]
            w = s["wq"][e].to(torch.float64) * s["sw"][e].double()[nb][:, kb]
            y[r0:r1] = a @ w.T
        r0 = r1
    return y


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "gemm":
        return {"y": _exact_product(s)}
    if op == "swiglu":
        y = _exact_product(s)
        I = case["N"]
        h = y[:, :I] * torch.sigmoid(y[:, :I]) * y[:, I:]
        if s["ys"] is None:
            return {"h": h}
        amax = torch.stack([b.abs().amax(1) for b in h.split(128, 1)], 1).clamp_min(AMAX_FLOOR)
        step = (amax / E4M3_MAX).repeat_interleave(128, 1)
        v = (h / step).clamp(-E4M3_MAX, E4M3_MAX)
        # nearest E4M3 value, ties to even: three bits below the leading one, 2^-9 at the least
        unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
        return {"h": torch.round(v / unit) * unit * step}
    ros, k = s["row_of_slot"], s["row_of_slot"].shape[1]
    if op == "combine":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=ros.device)
        for j in range(k):
            here = (ros[:, j] >= 0).nonzero().view(-1)
            out[here] += s["y"][ros[here, j]].double() * s["w"][here, j].double()[:, None]
        return {"out": out}
    gr = torch.zeros(s["grad_rows"].shape, dtype=torch.float64, device=ros.device)
    dw = torch.zeros(s["dw"].shape, dtype=torch.float64, device=ros.device)
    for j in range(k):
        here = (ros[:, j] >= 0).nonzero().view(-1)
        g = s["g"][here].double()
        gr[ros[here, j]] = g * s["w"][here, j].double()[:, None]
        dw[here, j] = (g * s["y"][ros[here, j]].double()).sum(1)
    return {"grad_rows": gr, "dw": dw}
