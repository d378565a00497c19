"""How the products are run (ops_csrc/plan.h), checked on the host: the
header is compiled by itself and asked for its plans."""
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_exact_matrix_amd", "ops_csrc")
BIG, MID, SMALL, FEW, ROWS, VEC = range(6)
# rows of A, columns of B (the most that a workgroup takes), inner step
SHAPE = {BIG: (256, 256, 64), MID: (128, 128, 64), SMALL: (64, 64, 64), FEW: (16, 64, 128),
         ROWS: (16, 32, 64), VEC: (2, 64, 8)}
TOP = 1 << 27  # the longest row and the largest size that a product takes

SOURCE = r"""
#include <stdio.h>
#include "plan.h"
using namespace mmaops;
int main() {
  long long M, N, K, lda, ldb, at_a, at_b;
  int la, lb, saves;
  while (scanf("%lld %lld %lld %d %d %lld %lld %lld %lld %d", &M, &N, &K, &la, &lb, &lda, &ldb,
               &at_a, &at_b, &saves) == 10) {
    const Product p{M, N, K, la, lb, (const void*)at_a, (const void*)at_b, lda, ldb};
    const Plan q = linear_plan(p, saves != 0);
    printf("%d %d %d %d %d %d %lld\n", q.tile, q.splits, q.direct, q.copy_a, q.copy_b, q.guard,
           (long long)product_bytes(p, q));
  }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """(M, N, K, la, lb, lda, ldb, address of A, of B, saves) -> the plan."""
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror",
                    "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", CSRC,
                    str(d / "plan.cpp"), "-o", str(d / "plan")], check=True)

    def ask(cases, **env):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([str(d / "plan")], input=text, capture_output=True, text=True,
                             check=True, env=dict(os.environ, **env)).stdout.split("\n")
        names = "tile splits direct copy_a copy_b guard bytes".split()
        return [dict(zip(names, map(int, line.split()))) for line in out if line]
    return ask


def length(layout, len_, k):
    """Row length of an operand as it is stored."""
    return k if layout == 0 else len_


def reach(plan, which, case):
    """The largest byte offset of a direct load from its tile's first
    element, in a 64-bit integer, as the loads take it: a 16-byte piece of
    each of the tile's rows (of the inner step's, with the rows running
    fastest); rows past the matrix are not read."""
    m, n, k, la, lb, lda, ldb = case[:7]
    layout, size, ld = (la, m, lda) if which == "a" else (lb, n, ldb)
    most, bk = SHAPE[plan["tile"]][0 if which == "a" else 1], SHAPE[plan["tile"]][2]
    if plan["copy_" + which]:
        ld = (length(layout, size, k) + 7) // 8 * 8
    rows, row = (min(most, size), bk) if layout == 0 else (bk, most)
    return ((rows - 1) * ld + row) * 2


def check(case, plan):
    if plan["tile"] in (VEC,) or not plan["direct"]:
        return  # offsets of 64 bits
    for which in "ab":
        if plan["tile"] == ROWS and which == "a":
            continue  # X through registers, as above
        assert reach(plan, which, case) < 1 << 32, (case, plan)
    # direct loads are of rows that start on 16 bytes
    for which, at, ld in (("a", case[7], case[5]), ("b", case[8], case[6])):
        assert plan["copy_" + which] or (at % 16 == 0 and ld % 8 == 0), (case, plan)


# long rows of X, of W stored N x K and K x N, of both operands of X^T dz
LONG = [(1024, 1024, 10_000_000, 0, 1), (1024, 512, 9_000_000, 0, 1), (512, 256, 20_000_000, 0, 0),
        (16, 64, 100_000_000, 0, 0), (16, 64, 40_000_000, 0, 0), (64, 50_000_000, 64, 0, 1),
        (128, 40_000_000, 64, 0, 1), (1024, 1024, 9_000_000, 0, 0), (9_000_000, 64, 256, 1, 1),
        (64, 60_000_000, 4096, 1, 1), (TOP, 16, 200, 1, 1), (1, TOP, 64, 0, 1), (2, 300, TOP, 0, 0),
        (300, 16, TOP, 0, 1), (2000, 2000, TOP, 0, 0), (16, 30_000_001, 129, 0, 1)]


@pytest.mark.parametrize("tile", [None, "0", "1", "2", "3", "4", "5"])
def test_offsets_of_long_rows(plans, tile):
    """Direct loads take 32-bit offsets within a tile: no plan passes them,
    the copies of unaligned operands and strides larger than the row among
    them, whichever tile is asked for."""
    cases = []
    for m, n, k, la, lb in LONG:
        for pad, off in ((0, 0), (1, 0), (0, 2), (8, 0), (1 << 24, 0)):
            lda, ldb = length(la, m, k) + pad, length(lb, n, k) + pad
            for saves in (0, 1):
                cases.append((m, n, k, la, lb, lda, ldb, 4096 + off, 8192 + off, saves))
    env = {} if tile is None else {"MMAOPS_LINEAR_TILE": tile}
    for case, plan in zip(cases, plans(cases, **env), strict=True):
        check(case, plan)


def test_offsets_of_any_size(plans):
    rng = random.Random(1)

    def size(top):
        return max(1, min(top, int(2 ** rng.uniform(0, 27.1))))

    cases = []
    for _ in range(20000):
        m, n, k = size(TOP), size(TOP), size(TOP)
        while max(-(-m // 16) * -(-n // 16), -(-m // 16) * -(-k // 16),
                  -(-n // 16) * -(-k // 16)) >= 1 << 31:
            m, n, k = size(TOP), size(TOP), size(TOP)
        la, lb = rng.choice([(0, 0), (0, 1), (1, 1)])
        pad = [rng.choice([0, 0, 3, 8, size(1 << 30)]) for _ in range(2)]
        cases.append((m, n, k, la, lb, length(la, m, k) + pad[0], length(lb, n, k) + pad[1],
                      4096 + rng.choice([0, 0, 2]), 8192 + rng.choice([0, 0, 2]),
                      rng.randrange(2)))
    for case, plan in zip(cases, plans(cases), strict=True):
        check(case, plan)


def test_a_long_stride_alone_is_no_reason_to_copy(plans):
    """Rows that start on 16 bytes are read where they are while the tile's
    offsets hold them."""
    for ld in (1 << 22, (1 << 22) + 8, 1 << 23):
        case = (64, 64, 4096, 0, 0, ld, ld, 4096, 8192, 0)
        plan, = plans([case])
        assert plan["direct"] and not plan["copy_a"] and not plan["copy_b"], (ld, plan)
    # beyond them, a copy of a shorter row helps
    case = (4096, 4096, 4096, 0, 0, 1 << 30, 4096, 4096, 8192, 0)
    plan, = plans([case])
    assert plan["direct"] and plan["copy_a"] and not plan["copy_b"]
