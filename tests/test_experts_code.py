"""CPU: what the expert kernels' schedule takes for granted of the compiled code, read from the library's
own gfx950 code object (no GPU needed)."""
import os
import re
import shutil
import subprocess

import pytest

from combine_topk_idx_multihot_amd import binding as B

LLVM = "/opt/rocm/llvm/bin"
TILE = "13k_expert_tile"
RING = "13k_expert_ring"


def tool(name, *args, cwd=None):
    return subprocess.run([os.path.join(LLVM, name), *args], cwd=cwd, check=True, text=True,
                          capture_output=True).stdout


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    """The code object of experts.hip out of the built library."""
    if not os.path.exists(os.path.join(LLVM, "llvm-objdump")):
        pytest.skip("no llvm-objdump")
    B.lib()
    at = tmp_path_factory.mktemp("code")
    lib = shutil.copy(B.LIB_PATH, at)
    tool("llvm-objdump", "--offloading", os.path.basename(lib), cwd=at)
    for f in sorted(at.iterdir()):
        if "gfx950" in f.name and TILE.encode() in f.read_bytes():
            return str(f)
    raise AssertionError("no code object holds the tile kernel")


def kernels(code, name):
    """Disassembly of every kernel whose symbol holds `name`."""
    found, lines = {}, None
    for line in tool("llvm-objdump", "-d", "--no-show-raw-insn", code).splitlines():
        m = re.match(r"[0-9a-f]+ <(\S+)>:", line)
        if m:
            lines = found.setdefault(m[1], []) if name in m[1] else None
        elif lines is not None:
            lines.append(line.split("//")[0].strip())
    return found


def stores_ahead_of_loads(lines):
    """Output stores that a load to LDS follows before the next wait for loads (a wait with vmcnt and a
    barrier behind it: the start of a tile or of a step)."""
    bad, stores, last = 0, 0, ""
    for line in lines:
        if line.startswith("s_barrier") and "vmcnt" in last:
            stores = 0
        elif line.startswith("global_store"):
            stores += 1
        elif line.startswith("global_load_lds_dwordx4"):
            bad, stores = bad + stores, 0
        last = line
    return bad


def test_order_check_sees_a_store_moved_ahead():
    load, store = "global_load_lds_dwordx4 v[0:1], off", "global_store_dwordx4 v[0:1], v[2:5], off"
    start, barrier = ["s_waitcnt vmcnt(8) lgkmcnt(0)", "s_barrier"], ["s_waitcnt lgkmcnt(0)", "s_barrier"]
    assert stores_ahead_of_loads([*barrier, load, load, *barrier, store, store, *start, load]) == 0
    assert stores_ahead_of_loads([*barrier, load, store, load, store, *start, load]) == 1
    assert stores_ahead_of_loads([store, store, *barrier, load, *start]) == 2


def test_tile_stores_come_after_the_next_tiles_loads(code):
    """The waits at a tile's start count the last tile's stores as newer than the eight loads of its
    second step: a store ahead of those loads would leave one of them unwaited for."""
    found = kernels(code, TILE)
    assert len(found) == 3
    for name, lines in found.items():
        assert sum(line.startswith("global_load_lds_dwordx4") for line in lines) >= 4 * 8, name
        assert sum(line.startswith("global_store") for line in lines) >= 4, name
        assert stores_ahead_of_loads(lines) == 0, name


def test_lds_by_address_has_no_static_neighbour(code):
    """Both kernels address their dynamic LDS from 0, so they may have no static LDS before it."""
    notes = tool("llvm-readelf", "--notes", code)
    sizes = re.findall(r"\.group_segment_fixed_size: (\d+).*?\.name: +(\S+)", notes, re.S)
    mine = {name: int(size) for size, name in sizes if TILE in name or RING in name}
    assert len(mine) == 6 and not any(mine.values()), mine


def test_notes_of_a_kernel_with_static_lds_are_seen(code):
    """The reading above finds static LDS where there is some: the kernel for a few tokens has 6 KiB."""
    notes = tool("llvm-readelf", "--notes", code)
    sizes = re.findall(r"\.group_segment_fixed_size: (\d+).*?\.name: +(\S+)", notes, re.S)
    assert [int(size) for size, name in sizes if "13k_expert_rows" in name] == [6144]
