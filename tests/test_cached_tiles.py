"""Which workgroup of a cached attention takes which part of which tile of rows (cached_tiles.hpp,
built for the CPU): every unit once, whole or in all of its parts, and what the parts leave to be
joined within the workspace and the launch."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "cached_tiles.hpp"
using namespace fp8k;

// argv: workers, least and most heads, most units
int main(int, char** argv)
{
    const int workers = atoi(argv[1]), heads0 = atoi(argv[2]), heads1 = atoi(argv[3]), most = atoi(argv[4]);
    long bad = 0, seen = 0, inside = 0;
    for (int heads = heads0; heads <= heads1; ++heads)
        for (int tiles = 1; tiles * heads <= most; ++tiles)
            for (int average : {0, 3, 47, 48, 112, 1 << 20}) {
                const int units = tiles * heads;
                const TileSplit how = tile_split(units, workers, average);
                std::vector<int> taken(units), parts_of(units);
                const long before = bad;
                bad += how.whole < 0 || how.whole > units || how.splits < 1 || (how.splits == 1 && how.whole != units);
                for (int64_t block = 0; block < tile_blocks(how, units); ++block) {
                    const TilePart p = tile_part((int)block, units, heads, how);
                    if (p.unit < 0 || p.unit >= units || p.split < 0 || p.split >= p.parts) {
                        ++bad;
                        continue;
                    }
                    bad += p.parts != (p.unit < how.whole ? 1 : how.splits) || (taken[p.unit] && parts_of[p.unit] != p.parts);
                    taken[p.unit] += 1;
                    parts_of[p.unit] = p.parts;
                    ++seen;
                }
                // every unit is taken as often as it has parts, each part once: as many in all
                for (int u = 0; u < units; ++u) bad += taken[u] != (u < how.whole ? 1 : how.splits);
                std::vector<char> once(units * (size_t)how.splits);
                for (int64_t block = 0; block < tile_blocks(how, units); ++block) {
                    const TilePart p = tile_part((int)block, units, heads, how);
                    if (p.unit >= 0 && p.unit < units && p.split >= 0 && p.split < how.splits) bad += once[(size_t)p.unit * how.splits + p.split]++;
                }
                // parts are read by somebody: entries, sums and workgroups as many as there is room for
                bad += how.splits > 1 && (4 * (units - how.whole) > 3 * workers || 2 * (units - how.whole) * how.splits > 3 * workers);
                bad += tile_blocks(how, units) > (units > workers ? units + workers : workers * 3 / 2);
                inside += how.splits > 1 && how.whole % heads != 0;
                if (bad != before && before < 4) printf("heads %d tiles %d average %d\n", heads, tiles, average);
            }
    printf("%ld parts, %ld launches whose whole units end inside a tile, %ld wrong\n", seen, inside, bad);
    return bad != 0;
}
"""


def build(where, source):
    src, exe = where / "tiles.cpp", where / "tiles"
    src.write_text(source)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", os.path.join(ROOT, "fp8_precision_amd", "csrc"), str(src), "-o",
                    str(exe)], check=True)
    return exe


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    return build(tmp_path_factory.mktemp("cached_tiles"), PROGRAM)


@pytest.mark.parametrize("workers", [512, 608, 64])
@pytest.mark.parametrize("heads", [(1, 40), (41, 80), (81, 128)])
def test_every_part_is_taken_once(program, workers, heads):
    out = subprocess.run([str(program), str(workers), str(heads[0]), str(heads[1]), str(4 * workers + 200)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout
    assert int(out.stdout.split()[0]) > 10000 and int(out.stdout.split()[2]) > 0
