// kv_cache.hpp -- which places of a paged cache a call touches: what the launches' sizes and
// the kernels' addressing have to agree on, in plain C++ (constexpr functions are the
// device's too).
//
// A sequence holds `held` tokens; a call's `count` tokens of it are the last ones, at the
// positions held - count .. held - 1 (those below 0 have no place).  They are worked on a
// block of one page at a time: piece `local` of a sequence is its block floor(first / page)
// + local.  So that a workgroup finds its sequence without a sum over those before it, the
// pieces of sequence b begin at (start / page) + 2 b, with start the sequence's first token
// in the call: n tokens touch at most n / page + 2 pages.
#pragma once
#include <stdint.h>

namespace fp8k {

constexpr int64_t piece_base(int64_t start, int64_t b, int shift) { return (start >> shift) + 2 * b; }
constexpr int64_t piece_bound(int64_t tokens, int64_t batch, int shift) { return piece_base(tokens, batch, shift); }

// Pages that n tokens touch at most, wherever they begin.
constexpr int64_t pieces_of(int64_t n, int shift) { return ((n + (1 << shift) - 2) >> shift) + 1; }

// Tokens that a sequence holds, whatever `length` says: none, to what its row of the table can.
constexpr int held_tokens(int length, int blocks, int shift)
{
    const int64_t most = (int64_t)blocks << shift;
    return length < 0 ? 0 : length > most ? (int)most : length;
}

struct CachePiece {
    int64_t block;      // of the sequence's row of the table; below 0: no place in the cache
    int slot;           // the first token's place in the page
    int count;          // tokens, none if <= 0
    int skip;           // the first token's number among the call's tokens of this sequence
};

constexpr CachePiece cache_piece(int count, int held, int64_t local, int shift)
{
    const int64_t first = (int64_t)held - count, block = (first >> shift) + local;
    const int64_t a = block << shift, b = a + (1 << shift);
    const int64_t lo = first > a ? first : a, hi = held < b ? held : b;
    if (count <= 0 || lo >= hi) return {block, 0, 0, 0};
    return {block, (int)(lo - a), (int)(hi - lo), (int)(lo - first)};
}

}  // namespace fp8k
