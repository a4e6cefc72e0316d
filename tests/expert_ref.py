"""Plain 64-bit references of the experts' products and of the weighted combine, with the bounds
that the GPU results are held to.  Used by test_gpu_experts.py and test_gpu_weighted.py.

Bounds (u = 2^-24, half a step of fp32; bf16 half step 2^-8, E4M3 half step 2^-4 of a normal value
and 2^-10 below the normal range):

product   y = sum over blocks b of s_b p_b.  The 8-bit matrix instructions form p_b from exact
          products in groups of 8 consecutive columns: relative to the group's largest exponent
          sum E (exponent of a plus exponent of w, at most the two maxima's), bits below
          2^(E - 13) are cut off each product, the largest one keeping all of its own: within
          7 * 2^(E - 13).  The 16 group sums are added in fp32 in some order (off by up to one
          step each, cut or rounded): 16 * 2u * S_b, S_b the sum of magnitudes.  s_b is one rounded
          product (u), each fma into the accumulator rounds once (u per block).  With S = sum of
          s_b S_b and G = sum of s_b 2^E over the groups:
          |y - exact| <= 7 * 2^-13 G + (32 + 1 + KB) u S.
silu      exp(-g) to a relative (|g| + 4) u (the argument's rounding is scaled by |g|), then an
          addition, a division and a product: silu(g) * u within (|g| + 8) u |h|.
          The product's errors eg, eu enter h with |silu'| <= 1.1:  1.1 eg (|u| + eu) + |silu| eu.
"""
import torch

U = 2.0 ** -24
E4M3_MAX = 448.0
TINY = 1e-30  # far below every tested value: results that underflow in fp32


def quant_rows(v):
    """fp32 [n, K] -> E4M3 codes and one scale per 128 columns."""
    b = v.reshape(v.shape[0], -1, 128)
    a = b.abs().amax(2, keepdim=True).clamp_min(1e-4)
    q = (b * (E4M3_MAX / a)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.reshape(v.shape), (a / E4M3_MAX)[:, :, 0].contiguous()


def make_weights(EL, n, K, g):
    """E4M3 [EL, n, K] with scales per 128 x 128 block that differ from block to block."""
    nb = -(-n // 128)
    q = (torch.randn((EL, n, K), generator=g, device="cuda") * 64).clamp(-E4M3_MAX, E4M3_MAX)
    s = torch.exp(torch.randn((EL, nb, K // 128), generator=g, device="cuda")) / (64 * K ** 0.5)
    return q.to(torch.float8_e4m3fn), s


def group_power(v):
    """The power of two of the largest magnitude in each group of 8 columns (E4M3's smallest normal
    exponent at the least; 0 for a group of zeros)."""
    m = v.abs().view(*v.shape[:-1], v.shape[-1] // 8, 8).amax(-1)
    return torch.where(m > 0, torch.exp2(torch.floor(torch.log2(m.clamp_min(2.0 ** -6)))), m)


def product(rows_q, row_scale, w_q, w_scale, off):
    """fp64 (y, bound) [total, n] of the groups [off[e], off[e+1])."""
    K = rows_q.shape[1]
    kb = torch.arange(K, device="cuda") // 128
    gb = torch.arange(K // 8, device="cuda") // 16
    nb = torch.arange(w_q.shape[1], device="cuda") // 128
    y, bound = [], []
    for e in range(len(off) - 1):
        r = slice(off[e], off[e + 1])
        qa, sa = rows_q[r].double(), row_scale[r].double()
        qw, sw = w_q[e].double(), w_scale[e].double()[nb]
        a, w = qa * sa[:, kb], qw * sw[:, kb]
        y.append(a @ w.T)
        G = (group_power(qa) * sa[:, gb]) @ (group_power(qw) * sw[:, gb]).T
        bound.append(7 * 2.0 ** -13 * G + (33 + K // 128) * U * (a.abs() @ w.abs().T) + TINY)
    return torch.cat(y), torch.cat(bound)


def swiglu(y, bound):
    """fp64 h and the bound on an fp32 evaluation of it."""
    I = y.shape[1] // 2
    g, u = y[:, :I], y[:, I:]
    eg, eu = bound.split(I, dim=1)
    silu = g * torch.sigmoid(g)
    h = silu * u
    err = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + (g.abs() + 8) * U * h.abs()
    return h, err + TINY * (1 + u.abs())


def e4m3(v):
    """Nearest E4M3 value (ties to even) of fp64 v, saturating at +-448."""
    v = v.clamp(-E4M3_MAX, E4M3_MAX)
    unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / unit) * unit


def check_close(got, want, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() - bound
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} values off, worst by {over.max()}"


def check_bf16(got, want, bound, what):
    """An fp32 value within `bound`, rounded once to bf16."""
    check_close(got, want, bound + 2.0 ** -8 * (want.abs() + bound), what)
    # the bound above is the worst case; in norm the rounding alone stays under 2^-8 and the rest
    # is far smaller, so a wrong scale or a missed block of columns shows here
    off = (got.double() - want).norm()
    assert off <= 2.0 ** -8 * want.norm() + TINY, f"{what}: {off / want.norm()} in norm"


def check_fp8(q, scale, h, err, what):
    """Codes and scales of h, itself only known within err: every code lies between those of the
    two ends of its interval."""
    n, I = h.shape
    hb, eb = h.view(n, I // 128, 128), err.view(n, I // 128, 128)
    a = hb.abs().amax(2, keepdim=True)
    da = eb.amax(2, keepdim=True)
    lo, hi = (a - da).clamp_min(1e-4), (a + da).clamp_min(1e-4)
    s = scale.double()[:, :, None]
    assert (s >= lo / E4M3_MAX * (1 - 2 * U)).all() and (s <= hi / E4M3_MAX * (1 + 2 * U)).all(), what
    # y = h * (448 / a'), a' in [lo, hi]; 448 / a' and the product round once each
    big = (hb.abs() + eb) * (E4M3_MAX / lo) * (1 + 3 * U)
    small = (hb.abs() - eb).clamp_min(0) * (E4M3_MAX / hi) * (1 - 3 * U)
    v = q.double().view(n, I // 128, 128)
    same = (hb.abs() <= eb) | (v == 0) | (torch.sign(v) == torch.sign(hb))
    ok = (v.abs() <= e4m3(big)) & (v.abs() >= e4m3(small)) & same
    assert ok.all(), f"{what}: {int((~ok).sum())} codes off"
