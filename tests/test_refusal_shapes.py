"""CPU: a product's refusal of a pointer says the shape and the type that its own format wants.  Every call fails
validation before any HIP call."""
import ctypes

import pytest

from combine_topk_idx_multihot_amd import binding as B

FAKE = 0x100000  # 16-byte aligned, never dereferenced by validation

WANTS = {
    ("gemm", "fp8"): {"a": "[R,K] byte", "sa": "[R,K/128] fp32", "w": "[EL,N,K] byte",
                      "sw": "[EL,ceil(N/128),K/128] fp32", "out": "[R,N] bf16"},
    ("swiglu", "fp8"): {"a": "[R,K] byte", "sa": "[R,K/128] fp32", "w": "[EL,N,K] byte",
                        "sw": "[EL,ceil(N/128),K/128] fp32", "out": "[R,I] byte", "os": "[R,I/128] fp32"},
    ("gemm", "mxfp4"): {"a": "[R,K/2] byte", "sa": "[R,K/32] byte", "w": "[EL,N,K/2] byte",
                        "sw": "[EL,N,K/32] byte", "out": "[R,N] bf16"},
    ("swiglu", "mxfp4"): {"a": "[R,K/2] byte", "sa": "[R,K/32] byte", "w": "[EL,N,K/2] byte",
                          "sw": "[EL,N,K/32] byte", "out": "[R,I/2] byte", "os": "[R,I/32] byte"},
}


def call(op, fmt, a=FAKE, sa=FAKE, w=FAKE, sw=FAKE, out=FAKE, os=FAKE):
    d = B.make_desc(100, 8, 128, 0, 128, 16)
    h = B._Handle(routing_map=FAKE, tokens_per_expert=FAKE, padded_offsets=FAKE, row_of_slot=FAKE, status=FAKE,
                  workspace=FAKE, workspace_bytes=1 << 30)
    args = [ctypes.byref(d), ctypes.byref(h), a, sa, 512, 10, w, sw, 256, out, *([os] if op == "swiglu" else []), None]
    return getattr(B.lib(), f"moe_expert_{op}_{fmt}")(*args)


@pytest.mark.parametrize("op,fmt", WANTS)
def test_shapes(op, fmt):
    for name, shape in WANTS[op, fmt].items():
        for bad in (None, FAKE + 8) if name != "os" else (FAKE + 8,):
            assert call(op, fmt, **{name: bad}) == B.MOE_ERR_ARG, name
            assert shape in B.last_error() and "16-byte aligned" in B.last_error(), (name, B.last_error())
    if op == "swiglu":
        assert call(op, fmt, out=None, os=None) == B.MOE_ERR_ARG and "[R,I] bf16" in B.last_error()
