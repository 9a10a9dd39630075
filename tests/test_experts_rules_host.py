"""CPU tests of what the experts' step decides on the host (csrc/experts_rules.hpp), compiled as plain C++."""
import os
import random
import subprocess

import pytest

import _experts_forms as F

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "combine_moe_route_count_amd", "csrc")

LISTS = r"""
#include <cstdio>
#include "experts_rules.hpp"
int main() {   // reads N, E and a block's 16-bit words, prints what they are used as
    int N, E;
    while (std::scanf("%d %d", &N, &E) == 2) {
        const moe::ListLayout l{N};
        std::printf("%d %d %d %d", l.expert(), l.first(), l.ent(), l.words32());
        for (int i = 0; i < 2 * l.words32(); ++i) {
            unsigned v;
            if (std::scanf("%u", &v) != 1) return 1;
            std::printf(" %u", l.bounded(i, v, E));
        }
        std::puts("");
    }
}
"""


def _compile(tmp_path, source):
    (tmp_path / "p.cpp").write_text(source)
    exe = str(tmp_path / "p")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(tmp_path / "p.cpp"), "-o", exe],
                   check=True)
    return lambda text: subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout


def _size(N):
    return 2 * ((4 + 3 * N + 1) // 2)


@pytest.fixture(scope="module")
def lists(tmp_path_factory):
    run = _compile(tmp_path_factory.mktemp("lists"), LISTS)

    def call(N, E, words):
        out = [int(v) for v in run(" ".join(map(str, [N, E] + words))).split()]
        return out[:4], out[4:]
    return call


@pytest.mark.parametrize("N,E", [(1, 1), (2, 7), (3, 1024), (64, 8), (1023, 1024), (1024, 3)])
def test_lists_of_any_content_stay_inside(lists, N, E):
    """A block that another call has overwritten: every index taken from it is within its array."""
    rng = random.Random(N)
    for fill in (lambda: 0xffff, lambda: rng.randrange(1 << 16), lambda: rng.choice([0, N, N + 1, E, 0xffff])):
        (expert, first, ent, words), got = lists(N, E, [fill() for _ in range(_size(N))])
        assert (expert, first, ent, 2 * words) == (2, 2 + N, 4 + 2 * N, _size(N))
        slots = got[0]
        assert slots <= N
        for s in range(slots):
            assert got[expert + s] < E and expert + s < first
            lo, hi = got[first + s], got[first + s + 1]
            assert first + s + 1 < ent
            for at in range(lo, hi):             # entries that are worked on; without any, ent[0] is read
                assert at < N and got[ent + at] < N
        assert got[ent] < N


@pytest.mark.parametrize("N,E", [(1, 1), (5, 3), (1024, 1024)])
def test_lists_in_order_are_kept(lists, N, E):
    """Blocks as they are written come through as they are."""
    rng = random.Random(E)
    cuts = sorted(rng.sample(range(1, N), min(N - 1, 4)))
    first = [0] + cuts + [N]
    words = [len(first) - 1, 0]
    words += [rng.randrange(E) for _ in range(N)]
    words += first + [0] * (N + 2 - len(first))
    words += rng.sample(range(N), N)
    words += [0] * (_size(N) - len(words))
    _, got = lists(N, E, words)
    assert got == words


RULES = r"""
#include <cstdio>
#include "experts_rules.hpp"
int main() {   // "p rows E N"
    char what;
    while (std::scanf(" %c", &what) == 1) {
        long a, b;
        int d;
        if (std::scanf("%ld %d %ld", &a, &d, &b) != 3) return 1;
        std::printf("%d\n", moe::ProductSize{a, b, d}.tile_rows());
    }
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    run = _compile(tmp_path_factory.mktemp("rules"), RULES)
    return lambda lines: [[int(v) for v in l.split()] for l in run("\n".join(lines)).splitlines()]


def test_tested_products_reach_their_tiles(rules):
    for height, sizes in F.PRODUCT.items():
        assert rules(["p %d %d %d" % s for s in sizes]) == [[height]] * len(sizes), height
