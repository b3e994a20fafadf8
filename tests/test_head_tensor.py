"""Where the attention kernels' tile loads read, for tensors of one token and of several: every
16 bytes that the buffer's size lets through belong to the sequence's own rows, whatever
the strides.  The addressing is the library's (head_tensor.hpp), built for the CPU."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "head_tensor.hpp"
using namespace fp8k;

// argv: tokens heads head_dim token_stride head_stride; a line for every load that is let
// through but is no row of the sequence, or lies outside the tensor
int main(int, char** argv)
{
    HeadLayout h;
    h.tokens = atoll(argv[1]), h.heads = atoll(argv[2]), h.d = atoll(argv[3]);
    h.head = h.heads == 1 ? 0 : atoll(argv[5]);
    h.row = kernel_row(h.tokens, h.d, atoll(argv[4]));
    const int64_t row_bytes = h.row * 2;
    long bad = 0, whole = 0;
    for (int64_t row0 = 0; row0 < h.tokens; row0 += 32)
        for (int r = 0; r < 256; ++r)                    // the longest tile's rows
            for (int c = 0; c < 16; ++c) {
                const int64_t at = stream_offset(r, c, row_bytes, (int)h.d);
                const bool read = at + 16 <= stream_bytes(h.tokens - row0, row_bytes);
                const bool ours = row0 + r < h.tokens && c * 8 < h.d;
                const int64_t end = (h.heads - 1) * h.head * 2 + row0 * row_bytes + at + 16;   // of the last head
                whole += read && ours;
                if (read != ours || (read && (end > 2 * h.span() || at != r * row_bytes + c * 16))) {
                    if (bad++ < 4) printf("row0 %lld row %d chunk %d: offset %lld\n", (long long)row0, r, c, (long long)at);
                }
            }
    printf("%ld let through, %ld wrong\n", whole, bad);
    return bad != 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    where = tmp_path_factory.mktemp("head_tensor")
    src, exe = where / "loads.cpp", where / "loads"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", os.path.join(ROOT, "fp8_precision_amd", "csrc"), str(src), "-o",
                    str(exe)], check=True)
    return exe


# tokens, heads, head_dim, token stride, head stride
CASES = [(1, 1, 64, 64, 64), (1, 8, 128, 1024, 128), (33, 8, 128, 1024, 128), (300, 4, 80, 3 * 320, 80),
         (1, 8, 128, 128, 131072 * 128),      # one token of a head-major cache of 131072
         (1, 32, 128, 128, 4096 * 128), (1, 32, 128, 128, 32768 * 128), (1, 32, 128, 128, 65536 * 128),
         (1, 2, 64, 0, 1 << 40), (1, 4, 64, 64, 0), (1, 1, 128, 1 << 50, 1 << 50),
         (5, 32, 128, 128, 65536 * 128), (5, 2, 128, (1 << 22) - 8, 128), (600, 2, 72, (1 << 22) - 8, 1 << 40)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_loads_stay_inside_the_sequence(program, case):
    out = subprocess.run([str(program), *map(str, case)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout
