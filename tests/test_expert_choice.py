"""CPU: which kernel an experts' product takes (csrc/expert_choice.h), compiled with the host compiler."""
import os
import random
import subprocess

import pytest

from combine_topk_idx_multihot_amd import build

MAIN = r"""
#include "expert_choice.h"
#include <cstdio>
int main()
{
    long long T, k, E, EL, P, worst, R;
    int eager, K, N, gated;
    while (std::scanf("%lld %lld %lld %lld %lld %lld %lld %d %d %d %d", &T, &k, &E, &EL, &P, &worst, &R, &eager,
                      &K, &N, &gated) == 11) {
        const moe::ExpertLoad l = moe::expert_load(T, k, E, EL, P, worst, R, eager != 0);
        std::printf("%lld %lld %lld %lld %lld %d\n", (long long)l.rows_max, (long long)l.group_max,
                    (long long)l.slots, (long long)l.groups, (long long)l.rows_mean, static_cast<int>(moe::choose_expert_kernel(l, K, N, gated != 0)));
    }
}
"""
KERNELS = ("rows", "ring", "tile")


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    at = tmp_path_factory.mktemp("choice")
    (at / "main.cpp").write_text(MAIN)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-I" + build.CSRC, "-o", at / "main",
                    at / "main.cpp"], check=True)

    def ask(T, k, E, P, K, N, R=None, EL=None, gated=False):
        """R: the rows of an eager call, None for a sync-free one."""
        EL = E if EL is None else EL
        worst = T * min(k, EL) + EL * (P - 1)
        line = " ".join(map(str, (T, k, E, EL, P, worst, worst if R is None else R, int(R is not None), K, N,
                                  int(gated))))
        out = subprocess.run([os.path.join(at, "main")], input=line, check=True, text=True,
                             capture_output=True).stdout.split()
        return dict(zip(("rows_max", "group_max", "slots", "groups", "rows_mean"), map(int, out))), KERNELS[int(out[5])]

    return ask


def test_pad_rows_count(rule):
    """Pad rows are computed like any other: 64 rows of data in groups of 128 are 128 rows."""
    load, kernel = rule(1024, 8, 128, 128, 2048, 4096)
    assert load["rows_mean"] == 128 and kernel == "tile"
    load, kernel = rule(1024, 8, 128, 128, 2048, 4096, R=128 * 128)
    assert load["rows_mean"] == 128 and kernel == "tile"
    load, kernel = rule(256, 8, 128, 128, 768, 2048)
    assert load["rows_mean"] == 128 and kernel == "tile"
    # without padding the same tokens stay with the kernel for few rows
    assert rule(1024, 8, 128, 1, 2048, 4096)[1] == rule(256, 8, 128, 16, 768, 2048)[1] == "ring"


def test_rows_of_an_eager_call_count(rule):
    """Eager calls know their rows: a share that the router favours is not taken for the mean."""
    load, kernel = rule(2048, 8, 128, 1, 2048, 4096, R=16 * 1000, EL=16)
    assert load["rows_mean"] == 1000 and kernel == "tile"
    load, kernel = rule(2048, 8, 128, 1, 2048, 4096, R=16 * 3, EL=16)
    assert load["rows_mean"] == 3 and kernel == "ring"
    # groups that cannot all have rows
    load, _ = rule(1, 8, 128, 16, 768, 2048, R=8 * 16)
    assert load["groups"] == 8 and load["rows_mean"] == 16


def test_bounds(rule):
    for T, k, E, EL, P in ((0, 2, 4, 4, 1), (0, 2, 4, 4, 8), (1, 1, 1, 1, 1), (5, 8, 64, 3, 7), (900, 4, 16, 16, 16)):
        worst = T * min(k, EL) + EL * (P - 1)
        for R in (None, 0, worst, worst + 100):
            load, _ = rule(T, k, E, P, 512, 256, R=R, EL=EL)
            assert load["rows_max"] == (worst if R is None else min(R, worst))
            assert load["group_max"] <= load["rows_max"] and 1 <= load["groups"] <= EL
            assert load["rows_mean"] * load["groups"] >= load["rows_max"] or R is None


def test_no_routing_makes_more_groups(rule):
    """The kernel for few rows launches one slot per group: `slots` is a bound for every routing, also
    where R cuts the rows off or the description of the product names another padding than the route's;
    `groups` is one for the route's padding."""
    rng = random.Random(5)
    for _ in range(400):
        E, P, T = rng.choice((1, 3, 8, 40)), rng.choice((1, 2, 5, 16)), rng.randrange(0, 12)
        k, lb = rng.randint(1, 9), rng.randrange(E)
        EL = rng.randint(1, E - lb)
        rows = [0] * EL
        for _ in range(T):
            for e in {rng.randrange(-1, E) for _ in range(k)}:
                if lb <= e < lb + EL:
                    rows[e - lb] += 1
        off = [0]
        for n in rows:
            off.append(off[-1] + -(-n // P) * P)
        for R in {None, off[-1], rng.randrange(off[-1] + 1), off[-1] + 7}:
            cut = [min(o, off[-1] if R is None else R) for o in off]
            load, _ = rule(T, k, E, P, 512, 256, R=R, EL=EL)
            n = sum(b > a for a, b in zip(cut, cut[1:]))
            assert n <= load["groups"] <= load["slots"] <= EL
            if R is not None:
                assert n <= rule(T, k, E, P + 3, 512, 256, R=R, EL=EL)[0]["slots"]
            assert max((b - a for a, b in zip(cut, cut[1:]))) <= load["group_max"]


@pytest.mark.parametrize("T,k,E,EL,P,R,K,N,gated,kernel", [
    (1, 8, 128, 128, 1, None, 768, 2048, False, "rows"),
    (1, 8, 128, 128, 16, None, 768, 2048, False, "rows"),
    (256, 8, 128, 128, 1, None, 768, 2048, False, "ring"),
    (4096, 8, 128, 128, 16, 33700, 768, 2048, False, "tile"),
    (4096, 8, 128, 128, 16, 33700, 128, 2048, False, "ring"),  # one step: the tile kernel sends two ahead
    (1, 8, 128, 128, 1, None, 2048, 768, True, "ring"),
    (333, 8, 128, 32, 1, None, 2048, 768, True, "ring"),
    (4096, 8, 128, 128, 16, 33700, 2048, 768, True, "tile"),
    (16384, 8, 128, 16, 1, None, 4096, 1024, True, "tile")])
def test_choice(rule, T, k, E, EL, P, R, K, N, gated, kernel):
    assert rule(T, k, E, P, K, N, R=R, EL=EL, gated=gated)[1] == kernel


def test_deep_gpu_cases_take_the_tall_tiles(rule):
    """The cases of test_gpu_experts.test_deep_products reach the kernel that they are for."""
    import test_gpu_experts as gpu

    for name in ("edges", "edges_padded", "large_groups"):
        counts, P = gpu.LAYERS[name]["counts"], gpu.LAYERS[name].get("P", 1)
        R = sum(-(-n // P) * P for n in counts)
        for K in gpu.DEEP:
            for N, gated in ((2560, False), (1280, True)):
                assert rule(sum(counts), 1, len(counts), P, K, N, R=R, gated=gated)[1] == "tile", (name, K)
