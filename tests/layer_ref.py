"""Inputs of the layer for a few tokens whose gate and up sums are exact in fp32 in any order, and the
64-bit layer with the bound on an fp32 evaluation that holds h to a given precision.  Used by
test_layer_h_host.py and test_gpu_layer_h.py.

Tokens are integers of at most 4, rows of w1 integers of at most 8 (MXFP4: E2M1 values, halves up to 6)
times powers of two that differ by at most 2: sums of up to 2048 such products are whole multiples of half the
smallest power and less than 2^18 of them, so no addition rounds.  What is left (u = 2^-24, half a step):

h      (|g| + 8) u |h|, as in expert_ref.swiglu with exact products; then `h_step` |h|: 0 where h stays in
       fp32, 2^-16 where it is two bf16 terms (each off by half a step, 2^-8, of what it stands for: the
       second one of at most 2^-8 |h|).
z      sums of I products: (1.1 I + 8) 2u S, as in test_gpu_layer_tokens.py, twice the terms of one rounding each
       where h has two of them: (2.2 I + 8) 2u S covers both.
out    k products added, (k + 1) u of their magnitudes, then rounded to bf16 (2^-8).
"""
import math

import torch

import expert_ref as ref
import mx_ref as mx


def _ints(shape, top, g):
    return torch.randint(-top, top + 1, shape, generator=g).double()


def weights_exact(fmt, EL, n, K, g):
    """(w, scales, fp64 values) of w1."""
    p = -round(math.log2(12.7 * K ** 0.5 / 1.5))  # gate and up of about 1.5
    if fmt == "bf16":
        v = _ints((EL, n, K), 8, g) * 2.0 ** p
        return v.to(torch.bfloat16), None, v
    if fmt == "fp8":
        q = _ints((EL, n, K), 8, g)
        s = torch.exp2(p + torch.randint(0, 2, (EL, n // 128, K // 128), generator=g).double())
        return (q.to(torch.float8_e4m3fn), s.float(),
                q * s.repeat_interleave(128, 1).repeat_interleave(128, 2))
    q = torch.randint(0, 256, (EL, n, K // 2), generator=g, dtype=torch.int32).to(torch.uint8)
    s = (torch.randint(0, 2, (EL, n, K // 32), generator=g, dtype=torch.int32) + (127 + p)).to(torch.uint8)
    return q, s, mx.values(q, s)


def weights_any(fmt, EL, n, K, g):
    """The same of w2: rounded normal values."""
    v = torch.randn((EL, n, K), generator=g) * K ** -0.5
    if fmt == "bf16":
        q = v.to(torch.bfloat16)
        return q, None, q.double()
    if fmt == "fp8":
        s = torch.exp(torch.randn((EL, n // 128, K // 128), generator=g)) / (64 * K ** 0.5)
        q = (torch.randn((EL, n, K), generator=g) * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
        return q, s, q.double() * s.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
    q, s = mx.make(v)
    return q, s, mx.values(q, s)


def make(fmt, T, k, E, lb, EL, H, I, seed):
    """idx, topk_w, x, (w1, s1, its values), (w2, s2, its values), on the CPU."""
    g = torch.Generator().manual_seed(seed)
    idx = torch.rand((T, E), generator=g).topk(k, 1).indices.int()
    x = _ints((T, H), 4, g).to(torch.bfloat16)
    w = torch.rand((T, k), generator=g) - 0.3
    return idx, w, x, weights_exact(fmt, EL, 2 * I, H, g), weights_any(fmt, EL, H, I, g)


def layer(idx, w, x, w1, w2, lb, h_step, hold=lambda h: h):
    """fp64 (out, bound) of the layer with values w1 [EL,2I,H], w2 [EL,H,I]; `hold` is what becomes of h on its
    way from one product to the other."""
    out = torch.zeros(x.shape, dtype=torch.float64)
    bound, mag = torch.zeros_like(out), torch.zeros_like(out)
    k, I = idx.shape[1], w2.shape[2]
    for e in range(w1.shape[0]):
        t, j = (idx == lb + e).nonzero(as_tuple=True)
        if not len(t):
            continue
        h, eh = ref.swiglu(x[t].double() @ w1[e].T, torch.zeros((len(t), 2 * I), dtype=torch.float64))
        eh = eh + h_step * (h.abs() + eh)
        z = hold(h) @ w2[e].T
        ez = eh @ w2[e].abs().T + (2.2 * I + 8) * 2 * ref.U * ((h.abs() + eh) @ w2[e].abs().T)
        wt = w[t, j].double()[:, None]
        out.index_add_(0, t, z * wt)
        bound.index_add_(0, t, ez * wt.abs())
        mag.index_add_(0, t, (z.abs() + ez) * wt.abs())
    return out, bound + (k + 1) * ref.U * mag + ref.TINY
