// kv_cache.hpp -- which places of a paged cache a call touches: what the launches' sizes and
// the kernels' addressing have to agree on, in plain C++ (constexpr functions are the
// device's too).
//
// The call's `count` tokens of a sequence are the last ones of its length: they stand at the
// positions first .. first + count - 1.  Those below 0 or past the sequence's row of the table
// have no place.  They are worked on a block of one page at a time: piece `local` of a
// sequence is its block floor(first / page) + local.  So that a workgroup finds its sequence
// without a sum over those before it, the pieces of sequence b begin at (start / page) + 2 b,
// with start the sequence's first token in the call: n tokens touch at most n / page + 2 pages.
#pragma once
#include <stdint.h>

namespace fp8k {

constexpr int64_t piece_base(int64_t start, int64_t b, int shift) { return (start >> shift) + 2 * b; }
constexpr int64_t piece_bound(int64_t tokens, int64_t batch, int shift) { return piece_base(tokens, batch, shift); }

// Pages that n tokens touch at most, wherever they begin.
constexpr int64_t pieces_of(int64_t n, int shift) { return ((n + (1 << shift) - 2) >> shift) + 1; }

// Tokens that a row of the table has places for (2^30 at most).
constexpr int row_capacity(int blocks, int shift) { return blocks << shift; }

// Of a sequence's tokens, those that can have a place, whatever `length` says.
constexpr int held_tokens(int length, int blocks, int shift)
{
    const int most = row_capacity(blocks, shift);
    return length < 0 ? 0 : length > most ? most : length;
}

// The position of the first of its `count` tokens in the call; from the end of the row on all
// are alike, and are counted as there.
constexpr int first_position(int length, int count, int blocks, int shift)
{
    const int most = row_capacity(blocks, shift), first = (length < 0 ? 0 : length) - count;
    return first > most ? most : first;
}

struct CachePiece {
    int64_t block;      // of the sequence's row of the table; below 0: no place in the cache
    int slot;           // the first token's place in the page
    int count;          // tokens, none if <= 0
    int skip;           // the first token's number among the call's tokens of this sequence
};

// Every token of the call has a piece, those without a place too: their block lies outside the row.
constexpr CachePiece cache_piece(int count, int first, int64_t local, int shift)
{
    const int64_t block = ((int64_t)first >> shift) + local, a = block << shift, b = a + (1 << shift);
    const int64_t end = (int64_t)first + count, lo = first > a ? first : a, hi = end < b ? end : b;
    if (count <= 0 || lo >= hi) return {block, 0, 0, 0};
    return {block, (int)(lo - a), (int)(hi - lo), (int)(lo - first)};
}

}  // namespace fp8k
