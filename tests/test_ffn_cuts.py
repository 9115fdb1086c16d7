"""Which kernels the feed-forward block's GPU tests reach: csrc/ffn_plan.hpp, host code of sizes
alone, compiled into a small program that answers for every size of theirs.  A change of the
costs that leaves a kernel untested fails here."""

import random
import subprocess

import pytest

import test_gpu_ffn
import test_gpu_ffn_plans
import test_gpu_ffn_sizes
from dispatch_grouped_gemm_amd import _build

PROGRAM = r"""
#include "ffn_plan.hpp"
#include <stdio.h>
using namespace moe;
static const char *names[] = {"256x256", "128x256", "128x128", "64x128", "64x64", "32x64",
                              "192x256", "192x128"};
static void say(long T, long N, long K, bool pairs, bool forward)
{
    const Cut c = product_cut(T, N, K, pairs);
    if (forward && few_rows_pay(T, N, K, c)) {
        printf("%d rows;", 16 * few_blocks(T));
        return;
    }
    const int rest = c.kind == kHuge
                         ? huge_rest(tiles_down(kHuge, T) * tiles_across(kHuge, N)) : 0;
    printf("%s%s%s;", names[c.kind], c.splits > 1 ? " parts" : "",
           rest == 4 ? " quarters" : rest == 2 ? " halves" : "");
}
int main()
{
    long T, H, I;
    while (scanf("%ld %ld %ld", &T, &H, &I) == 3) {
        say(T, 2 * I, H, true, true);
        say(T, H, I, false, true);
        say(T, I, H, false, false);
        const Sides s[] = {{T, H, 2 * I}, {2 * I, H, T}, {H, I, T}};
        TileKind kind[3];
        choose_tiles(s, 3, 1, kind);
        printf("%s;%s;%s\n", names[kind[0]], names[kind[1]], names[kind[2]]);
    }
}
"""


@pytest.fixture(scope="module")
def cuts(tmp_path_factory):
    at = tmp_path_factory.mktemp("cuts")
    (at / "cuts.cpp").write_text(PROGRAM)
    subprocess.run([_build.CXX, "-std=c++17", "-O1", "-Wall", "-I", _build.CSRC,
                    str(at / "cuts.cpp"), "-o", str(at / "cuts")], check=True)

    def ask(sizes):
        text = "".join("%d %d %d\n" % s for s in sizes)
        r = subprocess.run([str(at / "cuts")], input=text, capture_output=True, text=True,
                           check=True)
        return [tuple(line.split(";")) for line in r.stdout.splitlines()]
    return ask


# every kernel that a launch can take, for the first product, the second, dh; dx, dW13, dW2
WHOLE = {"256x256", "256x256 halves", "256x256 quarters", "192x256", "128x256", "192x128",
         "128x128", "64x128"}
PARTS = {"128x128 parts", "64x128 parts", "64x64 parts", "32x64 parts"}
ROWS = {"16 rows", "32 rows", "64 rows"}
DOWN = {"256x256", "128x256", "128x128"}
EVERY = [WHOLE | PARTS | ROWS, WHOLE | PARTS | ROWS | {"64x64", "32x64"},
         WHOLE | PARTS | {"64x64", "32x64"}, DOWN | {"192x256", "64x128"}, DOWN, DOWN]


def test_every_kernel_is_reached(cuts):
    sizes = test_gpu_ffn.SIZES + test_gpu_ffn_sizes.SIZES + test_gpu_ffn_plans.SIZES
    answers = cuts(sizes)
    for i, every in enumerate(EVERY):
        assert {a[i] for a in answers} == every, i


def test_no_other_kernel_is_chosen(cuts):
    """Over sizes drawn from the whole range, as over the tests'."""
    r = random.Random(11)

    def one(low, high):
        return int(2 ** r.uniform(low, high))

    sizes = [(one(0, 18), 32 * one(0, 9), 32 * one(0, 9)) for _ in range(20000)]
    for s, a in zip(sizes, cuts(sizes)):
        assert all(k in every for k, every in zip(a, EVERY)), (s, a)


def test_cuts(cuts):
    """The first, the second product and dh of test_gpu_ffn_sizes.py's sizes, in their order."""
    want = ["192x128, 192x128, 128x128", "192x256, 64x128, 192x256", "256x256, 192x256, 256x256",
            "128x128, 128x128, 64x128", "128x128 parts, 32x64, 64x128 parts",
            "64x128 parts, 64x64, 64x128 parts", "128x256, 128x128 parts, 128x128",
            "64x128, 64x128 parts, 64x64", "64x128, 32x64 parts, 32x64",
            "64x64 parts, 128x128, 64x64 parts", "32x64 parts, 64x64, 32x64 parts",
            "192x256, 64x64, 192x128", "256x256, 192x256, 192x256",
            "128x128 parts, 64x128, 128x128 parts", "128x128, 128x128, 64x128",
            "32x64 parts, 16 rows, 32x64 parts", "64 rows, 64 rows, 32x64",
            "64 rows, 64 rows, 32x64 parts", "64 rows, 64 rows, 64x64 parts"]
    assert [", ".join(a[:3]) for a in cuts(test_gpu_ffn_sizes.SIZES)] == want
