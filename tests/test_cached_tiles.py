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
                // parts are read by somebody: entries, sums and workgroups as many as there is room for, and a join where needed
                bad += how.splits > 1 && (units - how.whole > joined_units(workers) || !may_split(units, workers, average));
                std::vector<char> slot((size_t)split_parts(workers) * kTileSlots);
                for (int u = how.whole; how.splits > 1 && u < units; ++u)
                    for (int i = 0; i < how.splits; ++i)
                        for (int j = 0; j < kTileSlots; ++j) {
                            const int64_t at = tile_slot0(workers, u - how.whole, how.splits) + i * kTileSlots + j - 2 * workers;
                            bad += at < 0 || at >= (int64_t)slot.size() || slot[at]++;
                        }
                bad += tile_blocks(how, units) > row_blocks(units, workers);
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


FEW = r"""
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
#include "cached_tiles.hpp"
using namespace fp8k;

// argv: workers, seed.  Few tiles of sequences of any length, as the workgroups count them.
int main(int, char** argv)
{
    const int workers = atoi(argv[1]);
    std::mt19937 rng(atoi(argv[2]));
    auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
    long bad = 0, seen = 0, launches = 0, split = 0;
    while (launches < 4000) {
        const int heads = pick(0, 2) ? pick(1, 16) : pick(1, workers / 2), batch = pick(1, 12);
        std::vector<int> tiles(batch), steps(batch);
        int total = 0, longest = 0;
        int64_t all_steps = 0;
        for (int b = 0; b < batch; ++b) {
            tiles[b] = pick(0, 1) ? 0 : pick(0, 4) ? pick(1, 8) : pick(1, 256);
            steps[b] = pick(0, 3) ? pick(0, 70) : pick(0, 3) ? pick(0, 2000) : pick(0, 1 << 24);
            if (total + tiles[b] > workers / 2 / heads) tiles[b] = 0;
            total += tiles[b];
            all_steps += (int64_t)tiles[b] * (steps[b] - pick(0, steps[b] / 4));
            if (tiles[b] && steps[b] > longest) longest = steps[b];
        }
        const int units = total * heads, marks = step_marks(longest);
        if (!few_split(units, total, workers, marks)) continue;
        ++launches;
        const int share = few_share(all_steps * heads, workers);
        uint64_t parts = 0;
        for (int b = 0; b < batch; ++b)
            for (int k = 0; tiles[b] && k < kFewChoices; ++k) parts += (uint64_t)(tiles[b] * few_parts(steps[b], share, k, marks)) << 16 * k;
        const int k = few_choice(parts, heads, workers), pieces = few_parts_of_all(parts, k);
        int count = 0;
        for (int b = 0; b < batch; ++b) count += tiles[b] ? tiles[b] * few_parts(steps[b], share, k, marks) : 0;
        const long before = bad;
        bad += count != pieces || pieces * heads > workers || pieces * heads > row_blocks(units, workers);
        std::vector<std::vector<char>> taken(units);
        std::vector<char> entries(workers), slot((size_t)split_parts(workers) * kTileSlots);
        for (int64_t block = 0; block < row_blocks(units, workers); ++block) {
            if (block < workers && block >= units) bad += entries[block]++;
            if (block >= pieces * heads) continue;
            const int at = pieces - 1 - (int)(block / heads), head = (int)(block % heads);
            int left = at, tile = 0, b = 0, each = 0;
            for (;; ++b) {
                if (!tiles[b]) continue;
                each = few_parts(steps[b], share, k, marks);
                if (left < tiles[b] * each) break;
                left -= tiles[b] * each;
                tile += tiles[b];
            }
            const int unit = (tile + left / each) * heads + head, part = left % each;
            if (unit < 0 || unit >= units || each < 1) { ++bad; continue; }
            taken[unit].resize(each);
            bad += taken[unit][part]++;
            ++seen;
            bad += each > 1 && !may_split(units, workers, longest);
            bad += each > 1 && unit >= joined_units(workers);
            if (part == 0) bad += entries[unit]++;
            const int64_t first = few_slot0(workers, at, part, heads, head);
            for (int j = 0; each > 1 && j < kTileSlots; ++j) {
                const int64_t to = first + (int64_t)part * few_step(heads) + j - 2 * workers;
                bad += to < 0 || to >= (int64_t)slot.size() || slot[to]++;
            }
            // the join takes a tile's parts from the first one's slot on
            bad += first != few_slot0(workers, at - part, 0, heads, head);
            split += each > 1;
        }
        for (auto& t : taken) {
            bad += t.empty();
            for (char c : t) bad += c != 1;
        }
        for (char c : entries) bad += c != 1;              // each entry is written or cleared, once
        if (bad != before && before < 4) printf("heads %d units %d longest %d\n", heads, units, longest);
    }
    printf("%ld parts, %ld of split tiles, %ld wrong\n", seen, split, bad);
    return bad != 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    return build(tmp_path_factory.mktemp("cached_tiles"), PROGRAM)


@pytest.mark.parametrize("workers", [512, 608, 64])
@pytest.mark.parametrize("heads", [(1, 40), (41, 80), (81, 128)])
def test_every_part_is_taken_once(program, workers, heads):
    out = subprocess.run([str(program), str(workers), str(heads[0]), str(heads[1]), str(4 * workers + 200)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout
    assert int(out.stdout.split()[0]) > 10000 and int(out.stdout.split()[2]) > 0


@pytest.fixture(scope="module")
def few(tmp_path_factory):
    return build(tmp_path_factory.mktemp("few_tiles"), FEW)


@pytest.mark.parametrize("workers", [512, 608, 64])
@pytest.mark.parametrize("seed", range(3))
def test_few_tiles_are_taken_once(few, workers, seed):
    out = subprocess.run([str(few), str(workers), str(seed)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout
    assert int(out.stdout.split()[0]) > 10000 and int(out.stdout.split()[2]) > 1000
