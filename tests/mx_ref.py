"""Plain 64-bit references of the MXFP4 operators and the bounds that the GPU results are held to.
Used by test_gpu_mxfp4.py and test_gpu_layer_tokens.py.

Bounds (u = 2^-24, half a step of fp32; bf16 half step 2^-8):

product   y = sum over K columns.  A 4-bit matrix instruction (64 or 128 columns) gives the sum of its
          products and its accumulator within 2^-22 of the sum of their magnitudes (two steps of fp32,
          wherever in the sum the bits are lost).  K / 64 instructions and up to 3 additions of
          partial sums, each within that of S, the sum of all magnitudes:
          |y - exact| <= (K / 64 + 3) 2^-22 S.
silu      as in expert_ref.swiglu, from the bounds of the two products, but with a reciprocal (within one
          step, 2u) and a product (u) where that has a division (u): 2u |h| more.
codes     of a value known within err: every code lies between those of the two ends of its interval, the
          block's power between those of the ends of the largest magnitude's.
"""
import torch

import expert_ref as ref

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def pow2(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def floor_log2(v):
    """Exponent of positive fp64 values, from their bits."""
    return (v.view(torch.int64) >> 52 & 0x7FF) - 1023


def e2m1(v):
    """Nearest E2M1 value (ties to even) of fp64 v, saturating at +-6."""
    a = v.abs().clamp_max(6.0)
    unit = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    return torch.copysign(torch.round(a / unit) * unit, v)


def scale_byte(amax):
    """E8M0 byte of blocks with largest magnitudes `amax` (fp64, finite)."""
    e = floor_log2(amax.clamp_min(2.0 ** -300))
    return (e - 2 + 127).clamp_min(0)


def quant(v):
    """fp64 [..., K] -> (code values [..., K/32, 32], bytes [..., K/32])."""
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    byte = scale_byte(b.abs().amax(-1))
    return e2m1(b / pow2(byte - 127)[..., None]), byte


def pack(q, byte):
    a = q.abs()
    u = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    u = (u | (torch.signbit(q).to(torch.uint8) << 3)).reshape(*q.shape[:-2], 16 * q.shape[-2], 2)
    return u[..., 0] | (u[..., 1] << 4), byte.to(torch.uint8)


def code_values(codes):
    """fp64 code values [..., K] of packed codes [..., K/2]."""
    t = torch.tensor([*GRID, *(-x for x in GRID)], dtype=torch.float64, device=codes.device)
    return t[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]


def values(codes, scales):
    """fp64 [..., K] that packed codes and scale bytes stand for."""
    v = code_values(codes).reshape(*codes.shape[:-1], codes.shape[-1] // 16, 32)
    s = pow2(scales.long() - 127)
    s = torch.where(scales == 255, torch.full_like(s, float("nan")), s)
    return (v * s[..., None]).flatten(-2)


def make(v):
    return pack(*quant(v.double()))


def make_weights(EL, n, K, g):
    """MXFP4 [EL, n, K/2] and scales that differ from block to block."""
    codes = torch.randint(0, 256, (EL, n, K // 2), generator=g, device="cuda", dtype=torch.int32)
    power = torch.randint(-3, 3, (EL, n, K // 32), generator=g, device="cuda", dtype=torch.int32)
    base = -int(torch.tensor(3.0 * K ** 0.5).log2().round())
    return codes.to(torch.uint8), (power + (127 + base)).to(torch.uint8)


def product(rows_q, row_scale, w_q, w_scale, off):
    """fp64 (y, bound) [total, n] of the groups [off[e], off[e+1])."""
    K = rows_q.shape[1] * 2
    y, bound = [], []
    for e in range(len(off) - 1):
        r = slice(off[e], off[e + 1])
        a, w = values(rows_q[r], row_scale[r]), values(w_q[e], w_scale[e])
        y.append(a @ w.T)
        bound.append((K / 64 + 3) * 2.0 ** -22 * (a.abs() @ w.abs().T) + ref.TINY)
    return torch.cat(y), torch.cat(bound)


def swiglu(y, bound):
    """fp64 h and the bound on an fp32 evaluation of it."""
    h, err = ref.swiglu(y, bound)
    return h, err + 2 * ref.U * h.abs()


def check_codes(codes, scales, h, err, what):
    """Packed codes and scale bytes of h, itself only known within err."""
    n, I = h.shape
    hb, eb = h.view(n, I // 32, 32), err.view(n, I // 32, 32)
    lo = (hb.abs() - eb).clamp_min(0).amax(2)
    hi = (hb.abs() + eb).amax(2)
    s = scales.long()
    assert ((s >= scale_byte(lo)) & (s <= scale_byte(hi))).all(), f"{what}: scales"
    unit = pow2(s - 127)[:, :, None]
    v = code_values(codes).view(n, I // 32, 32)
    big, small = e2m1((hb.abs() + eb) / unit), e2m1((hb.abs() - eb).clamp_min(0) / unit)
    same = (hb.abs() <= eb) | (v == 0) | (torch.sign(v) == torch.sign(hb))
    ok = (v.abs() <= big) & (v.abs() >= small) & same
    assert ok.all(), f"{what}: {int((~ok).sum())} codes off"
