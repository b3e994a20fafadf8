// head_tensor.hpp -- how a [tokens, heads, head_dim] bf16 tensor of an attention call lies
// in memory, and where the kernels' tile loads of it read: what host checks and device
// addressing have to agree on, in plain C++ (constexpr functions are the device's too).
#pragma once
#include <stdint.h>

namespace fp8k {

// Strides and sizes in elements.
struct HeadLayout {
    int64_t tokens = 0, heads = 0, d = 0, row = 0, head = 0;
    int64_t row_span() const { return (heads - 1) * head + d; }       // of one token's heads
    int64_t span() const { return (tokens - 1) * row + row_span(); }
    // each element has a place of its own
    bool distinct() const
    {
        return (head >= d || heads == 1) && row >= row_span() ? true : row >= d && head >= (tokens - 1) * row + d;
    }
};

// Two tensors of one head dimension share an element, b's first lying `off` elements after
// a's.  Exact where both strides agree (slices of one tensor, in whatever order its axes
// lie); with other strides between heads a token's heads count as one block, and with
// other strides between tokens the whole tensor does.
inline bool share_element(const HeadLayout& a, const HeadLayout& b, int64_t off)
{
    if (off >= a.span() || -off >= b.span()) return false;
    // the stride of a single token or head leads nowhere: it is whatever the other's is
    const int64_t row = a.tokens > 1 ? a.row : b.row, head = a.heads > 1 ? a.head : b.head;
    if (a.tokens > 1 && b.tokens > 1 && a.row != b.row) return true;
    if (a.heads > 1 && b.heads > 1 && a.head != b.head) {
        if (a.row_span() > row || b.row_span() > row) return true;
        const int64_t m = (off % row + row) % row;
        return m < a.row_span() || m + b.row_span() > row;
    }
    // a head of b, y heads and x tokens after one of a's: x the least that is not too far before it
    for (int64_t y = 1 - a.heads; y < b.heads; ++y) {
        const int64_t at = off + y * head, need = 1 - b.d - at;        // x row >= need
        int64_t x = need > 0 ? (need + row - 1) / row : -(-need / row);
        if (x < 1 - a.tokens) x = 1 - a.tokens;
        if (x < b.tokens && at + x * row < a.d) return true;
    }
    return false;
}

// The stride between tokens that the kernels are given.  A single token's own may be
// anything (its heads may lie gigabytes apart) and leads nowhere; a tile's rows past the
// only one need no more than to lie past the buffer's end.  Of several tokens it is below
// kMaxRow, so that a tile's 256 rows stay below kPastBuffer.
constexpr int64_t kMaxRow = (int64_t)1 << 22;
constexpr int64_t kernel_row(int64_t tokens, int64_t d, int64_t token_stride) { return tokens == 1 ? d : token_stride; }

// A tile's rows are read through a buffer that begins at its first row and ends with the
// sequence: 16-byte chunk c of row r lies at stream_offset, and reads as zero where that is
// not below stream_bytes -- rows past the sequence's end, and chunks past the head dimension.
constexpr uint32_t kPastBuffer = 0x80000000u;

constexpr uint32_t stream_offset(int r, int c, int64_t row_bytes, int d)
{
    return c * 8 < d ? (uint32_t)(r * row_bytes) + (uint32_t)c * 16u : kPastBuffer;
}

constexpr int64_t stream_bytes(int64_t rows_left, int64_t row_bytes)
{
    const int64_t n = rows_left * row_bytes;
    return n < 0 ? 0 : n > 0x7FFFFFFF ? 0x7FFFFFFF : n;
}

}  // namespace fp8k
