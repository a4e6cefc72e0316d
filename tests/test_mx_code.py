"""CPU: which kernel a product on MXFP4 rows takes (csrc/expert_choice.h, compiled with the host compiler),
how many items the plan of a layer of a few tokens can hold (csrc/moe_internal.h's formula), and what the
kernels take for granted of the compiled code, read from the library's own gfx950 code object."""
import os
import random
import re
import shutil
import subprocess

import pytest

from combine_topk_idx_multihot_amd import binding as B
from combine_topk_idx_multihot_amd import build

MAIN = r"""
#include "expert_choice.h"
#include <cstdio>
int main()
{
    long long T, k, E, EL, P, worst, R;
    int eager, N, gated;
    while (std::scanf("%lld %lld %lld %lld %lld %lld %lld %d %d %d", &T, &k, &E, &EL, &P, &worst, &R, &eager, &N,
                      &gated) == 10)
        std::printf("%d\n", static_cast<int>(moe::choose_mx_kernel(
                                moe::expert_load(T, k, E, EL, P, worst, R, eager != 0), N, gated != 0)));
}
"""
KERNELS = ("rows", "ring", "tile")


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    at = tmp_path_factory.mktemp("choice")
    (at / "main.cpp").write_text(MAIN)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-I" + build.CSRC, "-o", at / "main",
                    at / "main.cpp"], check=True)

    def ask(T, k, E, P, N, R=None, EL=None, gated=False):
        """R: the rows of an eager call, None for a sync-free one."""
        EL = E if EL is None else EL
        worst = T * min(k, EL) + EL * (P - 1)
        line = " ".join(map(str, (T, k, E, EL, P, worst, worst if R is None else R, int(R is not None), N,
                                  int(gated))))
        return KERNELS[int(subprocess.run([os.path.join(at, "main")], input=line, check=True, text=True,
                                          capture_output=True).stdout)]

    return ask


def test_choices(rule):
    assert rule(1, 8, 128, 1, 2048) == "rows" and rule(1, 8, 128, 1, 768, gated=True) == "rows"
    assert rule(8, 8, 128, 1, 2048) == "ring" and rule(256, 8, 128, 1, 2048) == "ring"
    assert rule(1, 8, 128, 32, 2048) == "ring"  # 32 rows in a group, pad rows among them
    assert rule(4096, 8, 128, 16, 768, R=32768, gated=True) == "tile"
    assert rule(1024, 8, 128, 1, 2048) == "tile" and rule(16384, 8, 128, 16, 4096, R=131072) == "tile"
    assert rule(512, 1, 1, 1, 4096) == "ring"  # one expert: too few tall tiles for the chip


def test_few_rows_take_one_pass(rule):
    """The kernel for few rows is made for groups of up to 16."""
    rng = random.Random(5)
    for _ in range(200):
        T, k, E, P = rng.randint(1, 64), rng.randint(1, 8), rng.randint(8, 64), rng.choice((1, 2, 16, 32))
        if -(-T // P) * P > 16:
            assert rule(T, k, E, P, 8 * rng.randint(1, 300)) != "rows"


def test_items_of_a_plan():
    """groups + (slots - groups) / 16 items hold every way of dealing slots to experts."""
    rng = random.Random(3)
    for _ in range(3000):
        slots, EL = rng.randint(1, 1024), rng.randint(1, 1024)
        used = rng.randint(1, min(slots, EL))
        counts = [1] * used
        for _ in range(slots - used if rng.random() < 0.7 else rng.randint(0, slots - used)):
            counts[min(int(rng.random() ** rng.choice((1, 3, 20)) * used), used - 1)] += 1
        groups = min(slots, EL)
        assert sum(-(-c // 16) for c in counts) <= groups + (slots - groups) // 16 <= 1024


LLVM = "/opt/rocm/llvm/bin"


def test_lds_by_address_has_no_static_neighbour(tmp_path):
    """The ring and the tile kernel address their dynamic LDS from 0, so they may have no static LDS before
    it; the kernel for few rows has some, which the same reading finds."""
    if not os.path.exists(os.path.join(LLVM, "llvm-objdump")):
        pytest.skip("no llvm-objdump")
    B.lib()
    lib = shutil.copy(B.LIB_PATH, tmp_path)

    def tool(name, *args):
        return subprocess.run([os.path.join(LLVM, name), *args], cwd=tmp_path, check=True, text=True,
                              capture_output=True).stdout

    tool("llvm-objdump", "--offloading", os.path.basename(lib))
    code = [f for f in sorted(tmp_path.iterdir()) if "gfx950" in f.name and b"16k_expert_mx_tile" in f.read_bytes()]
    sizes = re.findall(r"\.group_segment_fixed_size: (\d+).*?\.name: +(\S+)",
                       tool("llvm-readelf", "--notes", str(code[0])), re.S)
    by_address = {name: int(size) for size, name in sizes if re.search("16k_expert_mx_(ring|tile)", name)}
    assert len(by_address) == 6 and not any(by_address.values()), by_address
    assert all(int(size) > 0 for size, name in sizes if "16k_expert_mx_rows" in name)


def test_layer_ring_has_no_static_lds(tmp_path):
    """The layer's ring kernels address their dynamic LDS from 0, too."""
    if not os.path.exists(os.path.join(LLVM, "llvm-objdump")):
        pytest.skip("no llvm-objdump")
    B.lib()
    lib = shutil.copy(B.LIB_PATH, tmp_path)
    run = dict(cwd=tmp_path, check=True, text=True, capture_output=True)
    subprocess.run([os.path.join(LLVM, "llvm-objdump"), "--offloading", os.path.basename(lib)], **run)
    code = [f for f in sorted(tmp_path.iterdir()) if "gfx950" in f.name and b"12k_layer_ring" in f.read_bytes()]
    notes = subprocess.run([os.path.join(LLVM, "llvm-readelf"), "--notes", str(code[0])], **run).stdout
    sizes = [int(size) for size, name in re.findall(r"\.group_segment_fixed_size: (\d+).*?\.name: +(\S+)", notes, re.S)
             if "12k_layer_ring" in name]
    assert len(sizes) == 6 and not any(sizes), sizes
