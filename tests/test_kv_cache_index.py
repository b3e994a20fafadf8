"""Which places of a paged cache the write and read kernels touch (kv_cache.hpp, built for the
CPU): every token with a place exactly once, at that place, and nothing outside the table's
row, the page or the call's tokens, whatever bounds and lengths say."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <vector>
#include "kv_cache.hpp"
using namespace fp8k;

// argv: seed, wild (bounds and lengths of any value)
int main(int, char** argv)
{
    std::mt19937 rng(atoi(argv[1]));
    const bool wild = atoi(argv[2]);
    auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
    long bad = 0, seen = 0;
    for (int round = 0; round < 300; ++round) {
        const int shift = pick(4, 7), page = 1 << shift, batch = pick(1, 70), blocks = pick(1, 6);
        const bool even = pick(0, 3) == 0;
        std::vector<int> cu(batch + 1), len(batch);
        const int each = pick(1, 3 * page);
        for (int b = 0; b < batch; ++b) cu[b + 1] = cu[b] + (even ? each : pick(0, 2) ? pick(0, 5) : pick(0, 3 * page));
        int tokens = cu[batch] + (even ? 0 : pick(0, 3));
        if (tokens < 1) tokens = 1;
        for (int b = 0; b < batch; ++b) len[b] = pick(0, blocks * page + (pick(0, 3) ? 0 : 40));
        if (wild && !even)
            for (int b = 0; b <= batch; ++b) {
                if (pick(0, 3) == 0) cu[b] = pick(-1000, tokens + 1000);
                if (b < batch && pick(0, 3) == 0) len[b] = pick(0, 1) ? 2000000000 : -2000000000;
            }
        auto held_in = [&](int v) { return v < 0 ? 0 : v > tokens ? tokens : v; };
        std::map<std::pair<int, int>, int> hits;           // (sequence, position) -> times
        const int64_t items = even ? batch * pieces_of(each, shift) : piece_bound(tokens, batch, shift);
        for (int64_t item = 0; item < items + 3; ++item) {
            int b = -1, count, from;
            int64_t local;
            if (even) {
                b = (int)(item / pieces_of(each, shift));
                local = item % pieces_of(each, shift);
                count = each;
                from = b * each;
                if (b >= batch) continue;
            } else {
                for (int c = 0; c < batch; ++c)
                    if (piece_base(held_in(cu[c]), c, shift) <= item) b = c;
                if (b < 0) continue;
                from = held_in(cu[b]);
                count = held_in(cu[b + 1]) - from;
                if (count < 0) count = 0;
                local = item - piece_base(from, b, shift);
            }
            const int first = first_position(len[b], count, blocks, shift), length = len[b] < 0 ? 0 : len[b];
            const CachePiece p = cache_piece(count, first, local, shift);
            if (p.count <= 0) continue;
            bad += p.slot < 0 || p.slot + p.count > page || p.skip < 0 || p.skip + p.count > count;
            // a token has a place where its position lies in the row, and there alone
            bad += (p.block >= 0 && p.block < blocks) != (length - count + p.skip >= 0 && length - count + p.skip < blocks * page);
            bad += from + p.skip + p.count > tokens;
            for (int i = 0; i < p.count; ++i) {
                const int64_t pos = p.block * page + p.slot + i;
                if (p.block >= 0 && p.block < blocks) bad += pos != (int64_t)length - count + p.skip + i;
                bad += hits[{b, (int)pos}]++ != 0;
                ++seen;
            }
        }
        if (!wild || even)                                 // nothing is missed
            for (int b = 0; b < batch; ++b) {
                const int n = cu[b + 1] - cu[b];
                for (int pos = len[b] - n; pos < len[b] && pos < blocks * page; ++pos) bad += hits[{b, pos}] != 1;
            }
    }
    printf("%ld tokens placed, %ld wrong\n", seen, bad);
    return bad != 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    where = tmp_path_factory.mktemp("kv_cache_index")
    src, exe = where / "pieces.cpp", where / "pieces"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", os.path.join(ROOT, "fp8_precision_amd", "csrc"), str(src), "-o",
                    str(exe)], check=True)
    return exe


@pytest.mark.parametrize("wild", [0, 1])
@pytest.mark.parametrize("seed", range(3))
def test_every_token_has_its_place(program, seed, wild):
    out = subprocess.run([str(program), str(seed), str(wild)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout
    assert int(out.stdout.split()[0]) > 10000
