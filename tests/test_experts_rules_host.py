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
static void show(moe::StreamForm f) { std::printf(" %d %d %d %d %d", f.width, f.stage, f.waves, f.split, f.pack); }
int main() {   // "p rows E N" or "d T H I E K mx parts"
    char what;
    while (std::scanf(" %c", &what) == 1) {
        long a, b, c;
        int d, e, mx, parts;
        if (what == 'p') {
            if (std::scanf("%ld %d %ld", &a, &d, &b) != 3) return 1;
            std::printf("%d", moe::ProductSize{a, b, d}.tile_rows());
        } else {
            if (std::scanf("%ld %ld %ld %d %d %d %d", &a, &b, &c, &e, &d, &mx, &parts) != 7) return 1;
            const moe::DecodeSize s{a, b, c, d, e, mx != 0, parts};
            show(s.up());
            show(s.down());
        }
        std::puts("");
    }
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    run = _compile(tmp_path_factory.mktemp("rules"), RULES)
    return lambda lines: [[int(v) for v in l.split()] for l in run("\n".join(lines)).splitlines()]


def _decode_forms(rules, sizes, mx, parts):
    got = rules(["d %d %d %d %d %d" % s + f" {int(mx)} {parts}" for s in sizes])
    as_form = lambda v: (v[0], v[1], v[2], bool(v[3]), bool(v[4]))
    return [(as_form(g[:5]), as_form(g[5:])) for g in got]


def test_tested_products_reach_their_tiles(rules):
    for height, sizes in F.PRODUCT.items():
        assert rules(["p %d %d %d" % s for s in sizes]) == [[height]] * len(sizes), height


@pytest.mark.parametrize("mx", [False, True])
def test_tested_decode_steps_reach_their_kernels(rules, mx):
    table = F.MXFP4 if mx else F.BF16
    assert _decode_forms(rules, table, mx, 2) == list(table.values())
    wider = [(up, (5,) + down[1:] if down[4] else down) for up, down in table.values()]
    assert _decode_forms(rules, table, mx, 3) == wider


@pytest.mark.parametrize("mx", [False, True])
def test_no_form_is_out_of_the_tests(rules, mx):
    """Every form that a size can have is that of a tested one."""
    rng = random.Random(mx)
    step = 32 if mx else 8
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))
    sizes = []
    for _ in range(6000):
        K = rng.randint(1, 16)
        sizes.append((log(1, 1024 // K), step * log(1, 16384 // step), step * log(1, 16384 // step), log(1, 1024), K))
    table = F.MXFP4 if mx else F.BF16
    seen = _decode_forms(rules, sizes, mx, 2)
    assert {u for u, _ in seen} == {u for u, _ in table.values()}
    assert {d for _, d in seen} == {d for _, d in table.values()}
