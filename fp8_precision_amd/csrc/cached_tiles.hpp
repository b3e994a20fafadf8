// cached_tiles.hpp -- which workgroup of a call of attention_cached.hip takes which part of which
// tile of rows: what the kernel's workgroups have to agree on, in plain C++ (constexpr functions
// are the device's too).
//
// A unit is a tile of one head; units are numbered a tile's heads after another.  The first
// `whole` units are taken by a workgroup each, the others in `splits` parts of their keys.
#pragma once
#include <stdint.h>

namespace fp8k {

// With more tiles than few, steps on average: in two where there are more tiles than CUs, but not three for
// two; and of many, those behind the last whole round of the workgroups: 1280 on 8192, no mask (32
// heads: 320 tiles) 262 / 231, 1000 on 1500 among 31 single ones (320) 65 / 75; 2048 on 8192 (40
// and 8: 640) 370 / 347, 1100 on 8100 (64 and 8: 552) 383 / 306, 4096 of 4096 (40 and 8: 1280) 211 / 217.
constexpr int kHalveFrom = 48, kTailFrom = 48;
constexpr int kLeastSplit = 4;             // steps of a part of a tile's keys

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

}  // namespace fp8k
