// cached_tiles.hpp -- which workgroup of a call of attention_cached.hip takes which part of which
// tile of rows, and where it leaves what is to be joined: what the kernel's workgroups, the join's and
// the host's sizes have to agree on, in plain C++ (constexpr functions are the device's too).
//
// A unit is a tile of one head; units are numbered a tile's heads after another.  Few units are
// all split into parts of one size (the few_ functions).  Otherwise the first `whole` units are
// taken by a workgroup each, the others in `splits` parts of their keys.
#pragma once
#include <stdint.h>

namespace fp8k {

constexpr int kTileSlots = 8;              // 16 rows each, for the sums of a tile's part
constexpr int kLeastSplit = 4;             // steps of a part of a tile's keys
constexpr int kFewTiles = 256;             // that can be split as few are: 16 bits count 255 parts of each

// Where at most half of the workgroups have a tile: steps of the longest from which on all tiles'
// keys are split into parts of the same size, into two only from twice as many on; the fewer
// tiles, the sooner: the sums of the parts are less.  MI355X, not split / split: 5 queries on 8005 keys
// (40 and 8 heads) 158 / 21 us; 1425 of 1425, 38 on 2035 and 122 on 158 (one head) 50 / 20; 1024
// causal ones of 8 heads 31 / 26, of 32 (in two, of 8 steps) 32 / 38; 64 on 704, 16 heads (16
// tiles of 11 steps) 21.7 / 18.0; 500 on 700, 32 and 8 (128 of 11) 24 / 32.
constexpr int kSplitFrom = 16, kSplitFewFrom = 10;
constexpr bool few_tiles(int64_t units, int workers) { return 8 * units <= workers; }

// The longest tile's steps as the workgroups tell one another of them.
constexpr int step_marks(int longest)
{
    return (longest >= kSplitFewFrom ? 1 : 0) | (longest >= kSplitFrom ? 2 : 0) | (longest >= 2 * kSplitFrom ? 4 : 0);
}

constexpr bool few_split(int units, int tiles, int workers, int marks)
{
    return units > 0 && 2 * (int64_t)units <= workers && tiles <= kFewTiles && (marks & (few_tiles(units, workers) ? 1 : 2));
}

// What a workgroup would have of all units' steps.
constexpr int few_share(int64_t steps, int workers)
{
    const int64_t share = (steps + workers - 1) / workers;
    return share < 1 << 24 ? (int)share : 1 << 24;
}

// Parts of a tile of so many steps under choice k: of 2, 3 or 4 halves of a share (255 parts at most),
// or, the last, two.
constexpr int kFewChoices = 4;
constexpr int few_parts(int steps, int share, int k, int marks)
{
    const int half = share * (2 + k) / 2, size = half > kLeastSplit ? half : kLeastSplit, n = (steps + size - 1) / size;
    const int parts = k == kFewChoices - 1 ? (steps < 2 ? steps : 2) : n < 255 ? n : 255;
    return parts < 2 || (parts == 2 && !(marks & 4)) ? 1 : parts;
}

// The first choice with which there are no more parts than workgroups; `parts`: of each choice, in 16
// bits, a head's of all tiles.
constexpr int few_parts_of_all(uint64_t parts, int k) { return (int)(parts >> 16 * k & 0xFFFF); }
constexpr int few_choice(uint64_t parts, int heads, int workers)
{
    int k = 0;
    while (k < kFewChoices - 1 && few_parts_of_all(parts, k) * heads > workers) ++k;
    return k;
}

// A part's first slot, of part `at` (of a head's, in order) that is the split-th of its tile; the next part's
// lie few_step further.
constexpr int few_slot0(int workers, int at, int split, int heads, int head)
{
    return 2 * workers + ((at - split) * heads + head) * kTileSlots;
}
constexpr int few_step(int heads) { return heads * kTileSlots; }

// With more tiles than few, steps on average: in two where there are more tiles than CUs, but not three for
// two; and of many, those behind the last whole round of the workgroups.  MI355X, not split / split, in us:
// 320 tiles: 1280 queries on 8192 keys without a mask, 32 heads (128 steps) 267 / 226, 1200 on 3700, 32 heads (49)
// 107.5 / 101, 1000 on 2500 among 31 single ones, 40 and 8 (32) 77.5 / 80, on 1500 (16) 47.5 / 63; 640: 2048 on
// 8192, 40 and 8 (112) 355 / 328; 552: 1100 on 8100, 64 and 8 (118) 369 / 286; 1280: 4096 of 4096, 40 and 8 (32) 189 / 198.
constexpr int kHalveFrom = 48, kTailFrom = 48;

struct TileSplit {
    int whole, splits;
};

// `average`: steps of a tile.
constexpr TileSplit tile_split(int units, int workers, int average)
{
    int splits = 1;
    if (units < workers) {
        if (4 * (int64_t)units <= 3 * (int64_t)workers && average >= kHalveFrom) splits = 2;
        return {splits > 1 ? 0 : units, splits};
    }
    const int rest = units % workers;
    if (units > workers && average >= kTailFrom && rest > 0 && 2 * rest <= workers) {
        const int most = workers / rest, of = average / kLeastSplit;
        splits = most < of ? most : of;
    }
    return {splits > 1 ? units - rest : units, splits};
}

// Workgroups that have a part.
constexpr int64_t tile_blocks(TileSplit s, int units) { return s.whole + (int64_t)(units - s.whole) * s.splits; }

struct TilePart {
    int unit, split, parts;
};

// Workgroup `block`'s, block < tile_blocks: a tile after another, each head's parts side by side.
// Workgroups are dealt round-robin to the 8 XCDs: where a tile's heads and parts divide so, each XCD
// gets whole heads of it.  That exchanges the places of one tile's workgroups, so the tile has to be
// complete: `whole` can end inside one, whose workgroups keep their order.
constexpr TilePart tile_part(int block, int units, int heads, TileSplit s)
{
    const bool part = block >= s.whole;
    const int parts = part ? s.splits : 1, first = part ? s.whole : 0, index = block - first, wide = heads * parts;
    const int count = part ? (units - s.whole) * parts : s.whole;
    if (wide % 8 == 0 && first % heads == 0 && index < count / wide * wide) {
        const int at = index % 8 * (wide / 8) + index / 8 % (wide / 8);
        return {first + index / wide * heads + at / parts, at % parts, parts};
    }
    return {first + index / parts, index % parts, parts};
}

// The first slot of a unit that is split; the next part's lie kTileSlots further.
constexpr int tile_slot0(int workers, int entry, int parts) { return 2 * workers + entry * parts * kTileSlots; }

// What the host makes room for: units that are joined, parts of units that are split (behind two
// slots of each workgroup's share), and workgroups, all or as many as can share the tiles.
constexpr int joined_units(int workers) { return workers * 3 / 4; }
constexpr int split_parts(int workers) { return workers * 3 / 2; }
constexpr int64_t row_blocks(int64_t units, int workers) { return units > workers ? units + workers : split_parts(workers); }

// Whether the device may split any of exactly `units` tiles of at most `steps` steps.
constexpr bool may_split(int64_t units, int workers, int64_t steps)
{
    const int64_t rest = units % workers;
    return units > workers ? rest > 0 && 2 * rest <= workers && steps >= kTailFrom
                           : 4 * units <= 3 * (int64_t)workers && steps >= (few_tiles(units, workers) ? kSplitFewFrom : kSplitFrom);
}

}  // namespace fp8k
