"""CPU: the waits of the MXFP4 tile kernel count on every output store of a whole tile as one vector memory
access, newer than the loads of the next tile's first step.  Read from the library's own gfx950 code object: a
compiler that merged two neighbouring stores would have to use a wider one than any that the kernel writes,
and one that moved a store ahead of those loads would show it before them."""
import os
import shutil

import pytest

from combine_topk_idx_multihot_amd import binding as B
from test_experts_code import LLVM, kernels, stores_ahead_of_loads, tool

TILE = "16k_expert_mx_tile"
# (gated, MXFP4 out): the widths that the source stores
WIDTHS = {"ILb0ELb0E": {"dwordx4"}, "ILb1ELb0E": {"dwordx4"}, "ILb1ELb1E": {"dwordx2", "byte"}}


def stores(lines):
    """Stores by width."""
    n = {}
    for line in lines:
        if line.split(" ")[0].startswith(("global_store_", "flat_store_", "buffer_store_", "scratch_store_")):
            kind = line.split(" ")[0].split("_store_")
            n[kind[0], kind[1]] = n.get((kind[0], kind[1]), 0) + 1
    return n


def fits(lines, widths, per_block):
    """Only global stores of those widths, and as many as tiles of 1 to 4 blocks of 64 rows make; equal ends of
    the four may be one piece of code (a store less for each of the three others, and each width)."""
    found = stores(lines)
    whole = per_block * (1 + 2 + 3 + 4)
    return (set(found) <= {("global", w) for w in widths} and
            whole - 3 * len(widths) <= sum(found.values()) <= whole and
            all(n >= whole // len(widths) - 3 for n in found.values()))


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    if not os.path.exists(os.path.join(LLVM, "llvm-objdump")):
        pytest.skip("no llvm-objdump")
    B.lib()
    at = tmp_path_factory.mktemp("mx")
    lib = shutil.copy(B.LIB_PATH, at)
    tool("llvm-objdump", "--offloading", os.path.basename(lib), cwd=at)
    files = [f for f in sorted(at.iterdir()) if "gfx950" in f.name and TILE.encode() in f.read_bytes()]
    return kernels(str(files[0]), TILE)


def test_every_store_is_its_own_and_behind_the_loads(code):
    assert len(code) == 3
    for name, lines in code.items():
        widths = next(w for key, w in WIDTHS.items() if key in name)
        per_block = 4 if "ILb1" in name else 8  # what mx_tile_run returns for a block of 64 rows
        assert fits(lines, widths, per_block), (name, stores(lines))
        assert stores_ahead_of_loads(lines) == 0, name
        assert not any(line.startswith(("scratch_", "buffer_")) for line in lines), name


def test_merged_and_missing_stores_are_seen(code):
    lines = next(lines for name, lines in code.items() if "ILb1ELb1E" in name)
    widths = WIDTHS["ILb1ELb1E"]
    byte = [i for i, line in enumerate(lines) if line.startswith("global_store_byte")]
    pair = [i for i, line in enumerate(lines) if line.startswith("global_store_dwordx2")]
    merged = [line.replace("_byte", "_short") if i == byte[0] else line for i, line in enumerate(lines)
              if i != byte[1]]
    wide = [line.replace("dwordx2", "dwordx4") if i == pair[0] else line for i, line in enumerate(lines)
            if i != pair[1]]
    fewer = [line for i, line in enumerate(lines) if i not in byte[:4]]
    for bad in (merged, wide, fewer):
        assert not fits(bad, widths, 4)
    assert fits(lines, widths, 4)
