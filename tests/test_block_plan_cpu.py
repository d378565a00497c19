"""How the products of a gated layer are run (paired_plan in
ops_csrc/plan.h), checked on the host."""
import os
import random
import subprocess

import pytest

from test_ops_plan_cpu import CSRC, SHAPE

BIG, MID, SMALL, FEW, ROWS = range(5)
GATED, SUMMED, APART = range(3)
TOP = 1 << 27

SOURCE = r"""
#include <stdio.h>
#include "plan.h"
using namespace mmaops;
int main() {
  long long M, N, K, lda, ldb, lda2, ldb2, at_a, at_b, at_a2, at_b2;
  int kind, la, lb, saves;
  while (scanf("%d %lld %lld %lld %d %d %lld %lld %lld %lld %lld %lld %lld %lld %d", &kind, &M, &N,
               &K, &la, &lb, &lda, &ldb, &at_a, &at_b, &lda2, &ldb2, &at_a2, &at_b2,
               &saves) == 15) {
    const Paired p{kind, Product{M, N, K, la, lb, (const void*)at_a, (const void*)at_b, lda, ldb},
                   (const void*)at_a2, (const void*)at_b2, lda2, ldb2};
    const Plan q = paired_plan(p, saves != 0);
    printf("%d %d %d %d %d %d %d %lld\n", q.tile, q.splits, q.direct, q.partial, q.copy_a,
           q.copy_b, q.guard, (long long)paired_bytes(p, q));
  }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    d = tmp_path_factory.mktemp("paired")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror",
                    "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", CSRC,
                    str(d / "plan.cpp"), "-o", str(d / "plan")], check=True)

    def ask(cases, **env):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([str(d / "plan")], input=text, capture_output=True, text=True,
                             check=True, env=dict(os.environ, **env)).stdout.split("\n")
        names = "tile splits direct partial copy_a copy_b guard bytes".split()
        return [dict(zip(names, map(int, line.split()))) for line in out if line]
    return ask


def stored(layout, size, k):
    """(rows, row length) of an operand as it is in memory."""
    return (size, k) if layout == 0 else (k, size)


def up(v, to):
    return -(-v // to) * to


def check(case, plan):
    (kind, m, n, k, la, lb, lda, ldb, at_a, at_b, lda2, ldb2, at_a2, at_b2, saves) = case
    want = 0
    if plan["partial"]:
        want += up(m * n * plan["splits"] * 4 * (1 if kind == SUMMED else 2), 256)
    sides = (("a", la, m, lda, at_a, lda2, at_a2), ("b", lb, n, ldb, at_b, ldb2, at_b2))
    for which, layout, size, ld, at, ld2, at2 in sides:
        rows, row = stored(layout, size, k)
        copied = plan["copy_" + which]
        if copied:
            want += up(rows * up(row, 8) * 2, 256) * (2 if at2 else 1)
            ld = up(row, 8)
        else:  # one leading dimension serves both
            assert not at2 or ld2 == ld, (case, plan)
        if not plan["direct"]:
            continue
        if not copied:
            assert at % 16 == 0 and ld % 8 == 0 and at2 % 16 == 0, (case, plan)
        if plan["tile"] == ROWS and which == "a":
            continue  # X through registers, whole 16-byte pieces
        bm, bn, bk = SHAPE[plan["tile"]]
        most = bm if which == "a" else bn
        if which == "b" and kind == GATED:
            most = 64 if plan["tile"] == FEW else 32 if plan["tile"] == ROWS else bn // 2
        reach = ((min(most, size) - 1) * ld + bk if layout == 0 else (bk - 1) * ld + most) * 2
        assert reach < 1 << 32, (case, plan)
        # past a row's end there is another row, but behind the last
        if layout == 1 and size % 8 and not copied and plan["tile"] != ROWS:
            assert plan["guard"], (case, plan)
    if plan["tile"] == ROWS:
        assert kind == GATED and m <= 16 and k % 64 == 0 and plan["splits"] == 1
        assert lb == 0 or n % 8 == 0
    assert plan["bytes"] == want, (case, plan)
    assert plan["splits"] >= 1
    # a wave of the gated small tiles has half a checkpoint block
    if saves and plan["tile"] in (SMALL, FEW):
        assert plan["partial"]


def random_case(rng, big):
    kind = rng.choice([GATED, SUMMED, APART])
    size = lambda top: max(1, int(2 ** rng.uniform(0, top)))  # noqa: E731
    m, n, k = ((size(27), size(10), size(10)) if big == 0 else (size(9), size(27), size(9))
               if big == 1 else (size(9), size(9), size(27)) if big == 2 else
               (size(13), size(13), size(13)))
    la, lb = {GATED: (0, rng.choice([0, 1])), SUMMED: (0, rng.choice([0, 1])),
              APART: (1, 1)}[kind]

    def side(layout, s):
        _, row = stored(layout, s, k)
        ld = row + rng.choice([0, 0, 0, 1, 3, 8, 64])
        if rng.random() < 0.5:
            ld = up(ld, 8)
        return ld, rng.choice([1 << 40, (1 << 40) + 2, (1 << 40) + 16])

    lda, at_a = side(la, m)
    ldb, at_b = side(lb, n)
    lda2, at_a2 = (lda, at_a + (1 << 44)) if rng.random() < 0.7 else side(la, m)
    ldb2, at_b2 = (ldb, at_b + (1 << 44)) if rng.random() < 0.7 else side(lb, n)
    if kind == GATED:
        lda2, at_a2 = 0, 0
    if kind == APART:  # one of the pair is the same operand
        if rng.random() < 0.5:
            lda2, at_a2 = 0, 0
        else:
            ldb2, at_b2 = 0, 0
    return (kind, m, n, k, la, lb, lda, ldb, at_a, at_b, lda2, ldb2, at_a2, at_b2,
            int(kind == GATED and rng.random() < 0.5))


@pytest.mark.parametrize("big", [0, 1, 2, 3])
def test_plans(plans, big):
    rng = random.Random(big)
    cases = [random_case(rng, big) for _ in range(1500)]
    for case, plan in zip(cases, plans(cases)):
        check(case, plan)


@pytest.mark.parametrize("tile", range(6))
def test_forced_plans(plans, tile):
    rng = random.Random(100 + tile)
    cases = [random_case(rng, 3) for _ in range(400)]
    for splits in (None, "3"):
        env = {"MMAOPS_LINEAR_TILE": str(tile)}
        if splits:
            env["MMAOPS_LINEAR_SPLITS"] = splits
        for case, plan in zip(cases, plans(cases, **env)):
            check(case, plan)


def test_what_is_saved_does_not_choose_the_kernel(plans):
    rng = random.Random(7)
    cases = [c for c in (random_case(rng, 3) for _ in range(900)) if c[0] == GATED]
    with_, without = ([(*c[:-1], s) for c in cases] for s in (1, 0))
    for a, b in zip(plans(with_), plans(without)):
        for name in ("tile", "splits", "direct", "copy_a", "copy_b", "guard"):
            assert a[name] == b[name]


def test_the_planner_takes_the_measured_sides(plans):
    """The choices that plan.h's comments name, with their sizes."""
    def gated(m, n, k, lb):
        return (GATED, m, n, k, 0, lb, k, n if lb else k, 1 << 40, 2 << 40, 0, n if lb else k, 0,
                3 << 40, 0)

    tiles = [p["tile"] for p in plans([gated(1, 4096, 4096, 0), gated(16, 4096, 1024, 1),
                                       gated(4096, 4096, 4096, 1), gated(1, 4096, 4096, 1)])]
    assert tiles == [ROWS, ROWS, BIG, FEW]
