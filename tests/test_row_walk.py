"""The walk of the convolution's kernels over a run of rows, run on the CPU: every
row once and in order, each read before it is computed and none beyond the
whole fetches (a row more would store a gradient that the next run stores)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "scan_canonical_reduce_amd", "csrc")

MAIN = """
#include <cstdio>
#include "row_walk.hpp"

template <int ROWS, int U>
void walk()
{
    int held[2][U];
    auto fetch = [&](int b, int r0) {
        std::printf(" f%d", r0);
        for (int u = 0; u < U; ++u) held[b][u] = r0 + u;
    };
    std::printf("%d %d", ROWS, U);
    fetch(0, 0);
    canon::seq::walk_rows<ROWS, U>(fetch, [&](int b, int u, int r) {
        std::printf(" %d:%d", r, held[b][u]);
    });
    std::printf("\\n");
}

int main()
{
    walk<8, 4>();
    walk<32, 4>(), walk<33, 4>(), walk<34, 4>(), walk<35, 4>();
    walk<36, 4>(), walk<37, 4>(), walk<38, 4>(), walk<39, 4>();
    walk<1, 4>(), walk<5, 2>(), walk<40, 8>();
}
"""


@pytest.fixture(scope="module")
def walks(tmp_path_factory):
    from scan_canonical_reduce_amd.build import _hipcc
    d = tmp_path_factory.mktemp("row_walk")
    src, exe = d / "main.hip", d / "main"
    src.write_text(MAIN)
    subprocess.run([_hipcc(), "--cuda-host-only", "-std=c++17", "-I", CSRC, str(src), "-o",
                    str(exe)], check=True, capture_output=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    return [line.split() for line in out.splitlines()]


def test_each_row_once_in_order(walks):
    assert len(walks) == 12
    for rows, _, *steps in walks:
        done = [s for s in steps if s[0] != "f"]
        assert done == [f"{r}:{r}" for r in range(int(rows))], rows


def test_reads_end_with_the_last_whole_fetch(walks):
    for rows, unroll, *steps in walks:
        rows, unroll = int(rows), int(unroll)
        reads = [int(s[1:]) for s in steps if s[0] == "f"]
        assert reads == list(range(0, rows, unroll)), (rows, unroll)
