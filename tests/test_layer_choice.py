"""CPU: which form a layer for a few tokens takes, its bound on the work list and its workspace
(csrc/layer_choice.h, compiled with the host compiler)."""
import os
import random
import subprocess

import pytest

from combine_topk_idx_multihot_amd import binding as B
from combine_topk_idx_multihot_amd import build

MAIN = r"""
#include "layer_choice.h"
#include <cstdio>
int main()
{
    long long slots, E, EL, H, I;
    while (std::scanf("%lld %lld %lld %lld %lld", &slots, &E, &EL, &H, &I) == 5)
        std::printf("%d %d %d %lld %zu\n", moe::layer_singles(slots, E, moe::kLayerBf16),
                    moe::layer_singles(slots, E, moe::kLayerFp8), moe::layer_singles(slots, E, moe::kLayerMxfp4),
                    (long long)moe::layer_items(slots, EL), moe::layer_ws_bytes(slots, E, H, I));
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    """(bf16, fp8, mxfp4 on its own, items, workspace bytes) of each (slots, E, EL, H, I)."""
    at = tmp_path_factory.mktemp("layer")
    (at / "main.cpp").write_text(MAIN)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-I" + build.CSRC, "-o", at / "main",
                    at / "main.cpp"], check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([os.path.join(at, "main")], input=text, check=True, text=True,
                             capture_output=True).stdout
        got = [tuple(map(int, line.split())) for line in out.splitlines()]
        assert len(got) == len(cases)
        return got

    return run


def test_both_sides_of_every_border(ask):
    for fmt, eighths in enumerate((7, 5, 4)):
        for E in (32, 64, 128, 256, 1000):
            at = eighths * E // 8
            below, above = ask([(at, E, E, 256, 128), (at + 1, E, E, 256, 128)])
            assert below[fmt] == 1 and above[fmt] == (at + 1 <= 16), (fmt, E)
    for E in (1, 2, 8, 18):
        below, above = ask([(16, E, E, 256, 128), (17, E, E, 256, 128)])
        assert below[:3] == (1, 1, 1) and above[:3] == (0, 0, 0), E


def test_the_workspace_holds_what_any_format_needs(ask):
    """The size does not depend on the format: it has the slots' outputs wherever one format's kernels write
    them, which only those that let slots share experts do."""
    cases = [(s, E, E, 512, 256) for s in range(0, 1025, 1) for E in (1, 3, 8, 37, 64, 128, 512, 1024)]
    for (slots, E, *_), (*own, _, size) in zip(cases, ask(cases)):
        assert size == 16 + slots * 256 * 4 + (0 if all(own) else slots * 512 * 4), (slots, E)
        assert own[0] >= own[1] >= own[2]


def test_the_library_asks_for_that_size(ask):
    rng = random.Random(11)
    cases = []
    for _ in range(300):
        k = rng.randint(1, 16)
        E = rng.choice((max(k, 8), 64, 128, 300))
        cases.append((rng.randint(0, 1024 // k), k, E, 256 * rng.randint(1, 16), 128 * rng.randint(1, 16)))
    want = ask([(T * k, E, E, H, I) for T, k, E, H, I in cases])
    for (T, k, E, H, I), w in zip(cases, want):
        assert B.moe_layer_tokens_workspace_size(B.make_desc(T, k, E), H, I) == w[4]


def test_items_hold_every_way_of_dealing_slots(ask):
    rng = random.Random(3)
    dealt, cases = [], []
    for _ in range(3000):
        slots, EL = rng.randint(1, 1024), rng.randint(1, 1024)
        used = rng.randint(1, min(slots, EL))
        counts = [1] * used
        for _ in range(slots - used if rng.random() < 0.7 else rng.randint(0, slots - used)):
            counts[min(int(rng.random() ** rng.choice((1, 3, 20)) * used), used - 1)] += 1
        dealt.append(sum(-(-c // 16) for c in counts))
        cases.append((slots, EL, EL, 256, 128))
    # and the worst ones: every group one slot past a whole number of items
    for EL in (1, 2, 7, 60):
        for n in (1, 17, 33):
            if n * EL <= 1024:
                dealt.append(EL * -(-n // 16))
                cases.append((n * EL, EL, EL, 256, 128))
    got = ask(cases)
    assert all(d <= g[3] <= 1024 for d, g in zip(dealt, got))
    assert [g[3] for g in got[-12:] if g[3]] and any(d == g[3] for d, g in zip(dealt[-12:], got[-12:]))
