// attention_cached.hip -- softmax attention over a paged cache of E4M3 keys and values
// (kv_cache.hip), for gfx950.
//
// Query i of a sequence's n stands at position length - n + i and sees the keys at positions
// up to its own (causal) or all that are held:
//   s = scale q . k,  p = exp(s - lse),  lse = log sum exp(s),  out = sum p v
// with k and v the codes times the power of two of their page and head.  Codes become bf16
// exactly on their way into the matrix instructions (the conversion takes the scale), so the
// only roundings are p's to bf16 (of few rows to twice its precision) and out's.
//
// A sequence's rows are its queries of the heads that share a key head (row r: query
// r / group, head r % group of them).  Sequences of up to 16 rows, the single tokens of a
// step of generation, are bound by reading the cache: their steps are dealt to the
// workgroups in equal shares whatever the lengths, and each wave works from registers.
// Sequences of more rows are bound by the matrix units: tiles of 128 rows, with the keys and
// values as bf16 tiles in LDS.  Both kinds can be in one launch.
#include <algorithm>
#include <type_traits>

#include "attention_tile.hpp"
#include "cached_tiles.hpp"
#include "fp8_device.hpp"
#include "fp8_internal.hpp"
#include "kv_cache.hpp"

namespace fp8k {

namespace {

typedef unsigned int au32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kFew = 16;                   // rows of a sequence that is read in shares, or twice as many (a.few)
constexpr int kOwn = 128;                  // rows of a tile: 32 per wave
static_assert(kOwn == 16 * kTileSlots, "a tile's slots");
constexpr int kLeastSteps = kWaves;        // of a share
constexpr int kPiece = 4;                  // what a head of a sequence costs besides its steps, in steps
constexpr int kMostTiles = (1 << 23) - 1;   // that a thread counts: no call has more in all
// Keys that a row of the table holds at most, up to which a head is not shared out; as many times more as the heads of
// all sequences fill two workgroups a CU, up to four.  MI355X, 32 and 8 heads, a chain of calls, whole / shared out:
// 100 keys of one sequence 5.6 / 7.8 us, 1000 10.3 / 9.9, of 64 23.4 / 25.5; of rows for 2048, 128 sequences of
// 2048 82 / 88, of 1 to 2048 59 / 56, one of 2048 and the others 256 22 / 28, but 64 like these 20.6 / 18.5; of
// rows for 4096, 64 sequences of 32 heads, 4096 315 / 331, 1 to 4096 193 / 192, one 4096 and the others 512
// 54 / 65, but 32 like these 41 / 40 and 64 of 8 38 / 24.
constexpr int kWholeKeys = 1024, kMostWhole = 4;
constexpr int kJoinThreads = 512;
// Of a buffer load's cache policy: no call reads the keys and values of few rows twice, and
// before the next call on them a model reads more than the caches hold.  MI355X, without /
// with: 64 sequences of 4096 keys (0.54 GB) 104 / 94 us, of 16384 394 / 366; but 19.6 / 22.4 for
// 500 (67 MB), where the last-level cache still has them from the call before.
constexpr int kNonTemporal = 2;
constexpr uint32_t kNowhere = 0x7FFFFFF0u; // an offset outside every buffer

__device__ __forceinline__ af32x4 mma16(const Frag& a, const Frag& b, const af32x4& c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.b, b.b, c, 0, 0, 0);
}

// Of the four lanes that share lane % 16: a register swapped with itself, by rows of 16 lanes and
// by halves, gives both sides in every lane.
__device__ __forceinline__ float max4(float v)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    const auto t = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(t[0]), __uint_as_float(t[1]));
}

__device__ __forceinline__ float sum4(float v)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    const auto t = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(t[0]) + __uint_as_float(t[1]);
}

// A sequence's queries and keys.
struct Sequence {
    int from, queries, held;
    int first;                             // the first query's position
};

__device__ __forceinline__ Sequence sequence(const CacheArgs& a, int b)
{
    Sequence s;
    const int length = a.lengths[b];
    if (a.cu) {
        const int from = a.cu[b], to = a.cu[b + 1];
        s.from = min(max(from, 0), (int)a.tokens);
        s.queries = max(min(max(to, 0), (int)a.tokens) - s.from, 0);
    } else {
        s.queries = a.each;
        s.from = b * s.queries;
    }
    s.held = held_tokens(length, a.blocks, a.shift);
    s.first = first_position(length, s.queries, a.blocks, a.shift);
    return s;
}

// Keys that its query i sees.
__device__ __forceinline__ int seen(const CachedAttentionArgs& a, int held, int first, int i)
{
    return a.causal ? (int)min((int64_t)held, (int64_t)first + i + 1) : held;
}

__device__ __forceinline__ bool few(const CachedAttentionArgs& a, const Sequence& s) { return s.queries * a.group <= a.few; }

// Steps of one head of a sequence of few rows: kPiece, in which nothing is done, and its keys';
// one of these at least, for the rows that see nothing.
__device__ __forceinline__ int share_steps(const CachedAttentionArgs& a, const Sequence& s)
{
    return s.queries == 0 || !few(a, s) ? 0 : kPiece + max(1, (s.held + kKeys - 1) / kKeys);
}

__device__ __forceinline__ int row_tiles(const CachedAttentionArgs& a, const Sequence& s)
{
    return few(a, s) ? 0 : (s.queries * a.group + kOwn - 1) / kOwn;
}

// Steps of the keys that query i of a sequence sees.
__device__ __forceinline__ int tile_steps(const CachedAttentionArgs& a, const Sequence& s, int i)
{
    return (max(seen(a, s.held, s.first, i), 0) + kKeys - 1) / kKeys;
}

// The sums of every thread's (x, y): all threads' in total, the x of those before it in before; and
// which bits of the waves' `marks` are set in any.
struct Sums {
    int before, total;
    int64_t total_y;
    int marks;
};

__device__ __forceinline__ Sums block_sums(int x, int64_t y, int (*lds)[4], int marks = 0)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int upto = x;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(upto, off, 64);
        if (lane >= off) upto += o;
    }
    if (__any(y != 0)) {
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) y += __shfl_xor(y, off, 64);
    }
    if (lane == 63) {
        lds[wave][0] = upto;
        lds[wave][1] = marks;
        lds[wave][2] = (int)y;
        lds[wave][3] = (int)(y >> 32);
    }
    __syncthreads();
    Sums s{upto - x, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) s.before += lds[w][0];
        s.total += lds[w][0];
        s.marks |= lds[w][1];
        s.total_y += (int64_t)lds[w][3] << 32 | (uint32_t)lds[w][2];
    }
    s.total = __builtin_amdgcn_readfirstlane(s.total);
    s.marks = __builtin_amdgcn_readfirstlane(s.marks);
    return s;
}

// The sum of the threads' before this one, and of all.
__device__ __forceinline__ void block_scan(uint64_t x, int (*lds)[4], uint64_t& before, uint64_t& total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint64_t upto = x;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint64_t o = __shfl_up(upto, off, 64);
        if (lane >= off) upto += o;
    }
    if (lane == 63) {
        lds[wave][0] = (int)upto;
        lds[wave][1] = (int)(upto >> 32);
    }
    __syncthreads();
    before = upto - x;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const uint64_t y = (uint64_t)(uint32_t)lds[w][1] << 32 | (uint32_t)lds[w][0];
        if (w < wave) before += y;
        total += y;
    }
}

// Where 16 keys of one head lie: their bytes in the pool and how many are held.
struct Keys16 {
    int64_t byte;
    int rows;
};

// A sequence's pages and their scales of one head, 64 blocks in the lanes of a wave at a
// time: this window, the next (its scales on their way) and the one after (its pages).
struct Pages {
    const int* table;
    const uint8_t *k_scale, *v_scale;
    int64_t pages;
    int heads, head, held, shift, d;
    int first;                             // the window's first block
    int page[3];
    int k_byte[2], v_byte[2];              // their scales

    __device__ __forceinline__ int entry(int window) const
    {
        const int at = first + 64 * window + (int)(threadIdx.x & 63);
        return (int64_t)at << shift < held ? table[at] : -1;
    }
    __device__ __forceinline__ void scales(int window)
    {
        const int p = page[window];
        k_byte[window] = v_byte[window] = 127;
        if (p >= 0 && p < pages) {
            const int64_t at = (int64_t)p * heads + head;
            k_byte[window] = k_scale[at];
            v_byte[window] = v_scale[at];
        }
    }
    __device__ __forceinline__ void init(const CacheArgs& a, int b, int head_, int held_, int key)
    {
        table = a.table + (int64_t)b * a.blocks;
        k_scale = a.k_scale;
        v_scale = a.v_scale;
        pages = a.pages;
        heads = a.heads;
        head = head_;
        held = held_;
        shift = a.shift;
        d = a.d;
        first = key >> shift;
#pragma unroll
        for (int w = 0; w < 3; ++w) page[w] = entry(w);
    }
    // the first scales: they need the pages
    __device__ __forceinline__ void start()
    {
#pragma unroll
        for (int w = 0; w < 2; ++w) scales(w);
    }
    // the window holds the blocks of the 64 keys from key on (a multiple of 64, as the first was; never falling)
    __device__ __forceinline__ void advance(int key)
    {
        while ((key >> shift) - first >= 64) {
            first += 64;
            page[0] = page[1];
            page[1] = page[2];
            k_byte[0] = k_byte[1];
            v_byte[0] = v_byte[1];
            scales(1);
            page[2] = entry(2);
        }
    }
    // the keys key .. key + 15 within the window (key: the same in all lanes, a multiple of 16), below `limit`
    __device__ __forceinline__ Keys16 at(int key, int limit) const
    {
        const int block = (key >> shift) - first;
        const int p = __builtin_amdgcn_readlane(page[0], block);
        const bool none = key >= limit || p < 0 || p >= pages;
        Keys16 x;
        x.byte = ((((int64_t)(none ? 0 : p) * heads + head) << shift) + (key & ((1 << shift) - 1))) * d;
        x.rows = none ? 0 : min(limit - key, 16);
        return x;
    }
    // their scales (asked for when the codes are here, so that the codes do not wait for them)
    __device__ __forceinline__ float scale_k(int key) const { return lane_scale(k_byte[0], key); }
    __device__ __forceinline__ float scale_v(int key) const { return lane_scale(v_byte[0], key); }
    __device__ __forceinline__ float lane_scale(int byte, int key) const
    {
        return cache_scale((uint8_t)__builtin_amdgcn_readlane(byte, (key >> shift) - first));
    }
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const uint8_t* pool, const Keys16& x, int d)
{
    return __builtin_amdgcn_make_buffer_rsrc((void*)(pool + x.byte), 0, x.rows * d, 0x00020000);
}

// What is to be joined: rows of a sequence whose sums are left in parts, 16 rows to a slot.
struct Join {
    int from, head, row, rows;             // the sequence's first query; rows row .. rows - 1 of it
    int count;                             // parts; nothing to do below 2
    int first, second, step;               // their slots: first, second, second + step, ...
};

template <int DT> constexpr int share_lds() { return kWaves * kFew * (DT + 4 + 2) * 4; }
template <int DT> constexpr int tile_lds() { return 4 * kKeys * DT * 2; }

// What a row's sums are multiplied with: 0 for one that sees nothing; a NaN sum stays NaN.
__device__ __forceinline__ float inverse(float l) { return l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l); }

// The larger of `top` and the magnitudes (fp32 bits) of two bf16.
__device__ __forceinline__ uint32_t top_of(uint32_t w, uint32_t top)
{
    return max(max(top, w & 0x7FFF0000u), w << 16 & 0x7FFFFFFFu);
}

// A share of the steps of all sequences of few rows.  The steps are counted in order (sequence,
// head, 64 keys) and dealt in equal shares, so that one long sequence among short ones is
// spread like any other; pieces of a share that are no whole head of a sequence are left as
// partial sums and joined.  The four waves take a piece's steps in turn.  Nothing of a step
// goes through LDS: 16 keys are the rows of a 16x16x32 product with the queries as its
// columns, in which a lane has 4 keys' scores of one query, and these are the second operand
// of the product with the values, whose rows are the head dimension: its first operand is 4 +
// 4 codes of one column, taken from 8 rows by byte permutations.  A step's keys are loaded
// into the registers of the last one's as soon as its scores are there, the values after
// its output.  R blocks of 16 rows.
// Bound by reading: MI355X, one query each of 64 sequences, 40 and 8 heads of 128, 4096 keys 94
// us (5.7 TB/s), 16384 365 (5.9, a large copy's rate); one on 16384 keys of 32 heads 26 and
// a join of 4; one of 65536 keys among 31 of 500 34 and 5.  8 waves to a CU and 4 read at the same
// rate, 12 slower.
template <int DT, bool FULL, int R>
__device__ __forceinline__ uint32_t attend_share(const CachedAttentionArgs& a, int worker, uint8_t* lds, int (*sums)[4], int* found)
{
    constexpr int kPer = DT / 16;          // values' elements of a lane, and the product's tiles
    constexpr int kRow = DT + 4;
    float* const s_out = reinterpret_cast<float*>(lds);               // [wave][row][kRow]
    float* const s_top = s_out + kWaves * kFew * kRow;                // [wave][row]
    float* const s_sum = s_top + kWaves * kFew;
    const CacheArgs& c = a.c;
    const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint32_t top_out = 0;

    Join* const joins = reinterpret_cast<Join*>(a.joins);
    int b, head, done, at, end, share = 1, steps;           // done: of the head's steps, by other shares
    Sequence s;
    if (a.whole) {
        b = worker / c.heads;
        head = worker % c.heads;
        done = at = 0;
        s = sequence(c, b);
        end = steps = __builtin_amdgcn_readfirstlane(share_steps(a, s));
        if (end == 0) return 0;
    } else if (c.batch <= 64) {
        // the share: every lane counts a sequence's steps
        const Sequence own = sequence(c, min(lane, c.batch - 1));
        const int one = lane < c.batch ? share_steps(a, own) : 0, mine = one * c.heads;
        int sum = mine;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int o = __shfl_up(sum, off, 64);
            if (lane >= off) sum += o;
        }
        const int total = __builtin_amdgcn_readlane(sum, 63);
        share = max((total + a.workers - 1) / a.workers, kLeastSteps);
        if (threadIdx.x == 0) joins[worker].count = 0;
        if (total == 0 || worker > (total - 1) / share) return 0;
        at = worker * share;
        end = min(at + share, total);
        b = __ffsll((unsigned long long)__ballot(sum > at)) - 1;
        const int left = at - __builtin_amdgcn_readlane(sum - mine, b);
        steps = __builtin_amdgcn_readlane(one, b);
        s = Sequence{__builtin_amdgcn_readlane(own.from, b), __builtin_amdgcn_readlane(own.queries, b),
                     __builtin_amdgcn_readlane(own.held, b), __builtin_amdgcn_readlane(own.first, b)};
        head = __builtin_amdgcn_readfirstlane(left / steps);
        done = __builtin_amdgcn_readfirstlane(left - head * steps);
    } else {
        // more sequences: every thread counts some, in order
        const int per = (c.batch + kThreads - 1) / kThreads, b0 = threadIdx.x * per, b1 = min(b0 + per, c.batch);
        int mine = 0;
        for (int b = b0; b < b1; ++b) mine += share_steps(a, sequence(c, b)) * c.heads;
        const Sums all = block_sums(mine, 0, sums);
        share = max((all.total + a.workers - 1) / a.workers, kLeastSteps);
        if (threadIdx.x == 0) joins[worker].count = 0;
        if (worker > (all.total - 1) / share || all.total == 0) return 0;
        at = worker * share;
        end = min(at + share, all.total);
        if (all.before <= at && at < all.before + mine) {
            int left = at - all.before, b = b0;
            for (;; ++b) {
                const int n = share_steps(a, sequence(c, b)) * c.heads;
                if (left < n) break;
                left -= n;
            }
            found[0] = b;
            found[1] = left;
        }
        __syncthreads();
        b = __builtin_amdgcn_readfirstlane(found[0]);
        s = sequence(c, b);
        steps = __builtin_amdgcn_readfirstlane(share_steps(a, s));
        head = __builtin_amdgcn_readfirstlane(found[1] / steps);
        done = __builtin_amdgcn_readfirstlane(found[1] - head * steps);
    }
    const float scale2 = a.scale * kLog2e;
    const float far = fminf(8.0f / scale2, 1e38f);         // scores may pass the running maximum by 2^8 before a rescale

    while (true) {
        const int from = __builtin_amdgcn_readfirstlane(s.from), queries = __builtin_amdgcn_readfirstlane(s.queries);
        const int held = __builtin_amdgcn_readfirstlane(s.held), first = __builtin_amdgcn_readfirstlane(s.first);
        const int upto = __builtin_amdgcn_readfirstlane(min(steps, done + end - at));
        // the piece: the keys' steps step0 .. last - 1 of all
        const int step0 = max(done - kPiece, 0), last = max(upto - kPiece, 0), all_steps = steps - kPiece;
        if (last > step0) {
            const int rows = queries * a.group, see_first = seen(a, held, first, 0);

            // the queries' operands: lane's column m, elements of chunk g as the keys' lanes have them
            Frag q[R][DT / 32];
            int see[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = 16 * r + m, qi = row / a.group, hq = head * a.group + row - qi * a.group;
                see[r] = seen(a, held, first, qi);
#pragma unroll
                for (int i = 0; i < DT / 32; ++i) {
                    q[r][i].u = au32x4{0, 0, 0, 0};
                    const int e = 64 * (i / 2) + 16 * g + 8 * (i % 2);
                    if (row < rows && (FULL || e < c.d))
                        q[r][i].u = *reinterpret_cast<const au32x4*>(a.q + (int64_t)(from + qi) * a.q_row + (int64_t)hq * a.q_head + e);
                }
            }
            Pages pages;
            if (step0 + wave < last) pages.init(c, b, head, held, (step0 + wave) * kKeys);
            // waited for here, with the pages: at its first use, in the loop, the wait would be one for every load in flight
            af32x4 o[R][kPer];
            float top[R], sum[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int i = 0; i < DT / 32; ++i) asm volatile("" : "+v"(q[r][i].u));
#pragma unroll
                for (int t = 0; t < kPer; ++t) o[r][t] = af32x4{0, 0, 0, 0};
                top[r] = -kInf;
                sum[r] = 0.0f;
            }

            // Codes of 64 keys, as loaded.  Of each block of 16 keys a lane has DT / 4 codes of key
            // m (16 of each 64, chunk g), and DT / 16 codes (chunk m) of each of the values 4 g + i.
            uint32_t ck[4][DT / 16], cv[4][4][DT / 64];
            Keys16 x[4];
            const int limit = min(held, last * kKeys);
            auto load_k = [&](int key) __attribute__((always_inline)) {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    x[n] = pages.at(key + 16 * n, limit);
                    const auto src = rows_of(c.k, x[n], FULL ? DT : c.d);
                    if constexpr (FULL) {
#pragma unroll
                        for (int i = 0; i < DT / 64; ++i) {
                            const au32x4 w = __builtin_amdgcn_raw_buffer_load_b128(src, m * DT + 64 * i + 16 * g, 0, kNonTemporal);
#pragma unroll
                            for (int j = 0; j < 4; ++j) ck[n][4 * i + j] = w[j];
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < DT / 32; ++i) {
                            const int e = 64 * (i / 2) + 16 * g + 8 * (i % 2);
                            const au32x2 w = __builtin_amdgcn_raw_buffer_load_b64(src, e < c.d ? m * c.d + e : kNowhere, 0, kNonTemporal);
                            ck[n][2 * i] = w[0];
                            ck[n][2 * i + 1] = w[1];
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            };
            auto load_v = [&]() __attribute__((always_inline)) {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int d = FULL ? DT : c.d, e = kPer * m;
                    const auto src = rows_of(c.v, x[n], d);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t off = FULL || e < d ? (uint32_t)((4 * g + i) * d + e) : kNowhere;
                        if constexpr (DT == 128) {
                            const au32x2 w = __builtin_amdgcn_raw_buffer_load_b64(src, off, 0, kNonTemporal);
                            cv[n][i][0] = w[0];
                            cv[n][i][1] = w[1];
                        } else {
                            cv[n][i][0] = __builtin_amdgcn_raw_buffer_load_b32(src, off, 0, kNonTemporal);
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            };

            if (step0 + wave < last) {
                pages.start();
                load_k((step0 + wave) * kKeys);
                load_v();
            }
            for (int t = step0 + wave; t < last; t += kWaves) {
                const int j0 = t * kKeys;
                float k_scale[4], v_scale[4];              // before the window moves on to the next step
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    k_scale[n] = pages.scale_k(j0 + 16 * n);
                    v_scale[n] = pages.scale_v(j0 + 16 * n);
                }
                af32x4 p[R][4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
#pragma unroll
                    for (int r = 0; r < R; ++r) p[r][n] = af32x4{0, 0, 0, 0};
#pragma unroll
                    for (int i = 0; i < DT / 32; ++i) {
                        Frag k;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            k.w[2 * j] = values2<false>(ck[n][2 * i + j], k_scale[n]);
                            k.w[2 * j + 1] = values2<true>(ck[n][2 * i + j], k_scale[n]);
                        }
#pragma unroll
                        for (int r = 0; r < R; ++r) p[r][n] = mma16(k, q[r][i], p[r][n]);
                    }
                }
                // (past the last step from buffers of no rows: with loads that some path leaves out, the
                // compiler would wait for the values together with the next keys)
                __builtin_amdgcn_sched_barrier(0);
                pages.advance(j0 + kWaves * kKeys);
                load_k(j0 + kWaves * kKeys);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (j0 + kKeys > see_first) {
#pragma unroll
                        for (int n = 0; n < 4; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (j0 + 16 * n + 4 * g + i >= see[r]) p[r][n][i] = -kInf;
                    }
                    float up = fmaxf(fmaxf(p[r][0][0], p[r][0][1]), fmaxf(p[r][0][2], p[r][0][3]));
#pragma unroll
                    for (int n = 1; n < 4; ++n) up = fmaxf(up, fmaxf(fmaxf(p[r][n][0], p[r][n][1]), fmaxf(p[r][n][2], p[r][n][3])));
                    up = max4(up);
                    if (__any(up > top[r] + far)) {            // top = -inf: any key seen
                        up = fmaxf(up, top[r]);
                        const float by = up == -kInf ? 1.0f : __builtin_amdgcn_exp2f((top[r] - up) * scale2);
                        sum[r] *= by;
#pragma unroll
                        for (int i = 0; i < kPer; ++i)
#pragma unroll
                            for (int j = 0; j < 4; ++j) o[r][i][j] *= by;
                        top[r] = up;
                    }
                    const float use = top[r] == -kInf ? 0.0f : top[r] * scale2;
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            p[r][n][i] = __builtin_amdgcn_exp2f(fmaf(p[r][n][i], scale2, -use));
                            sum[r] += p[r][n][i];
                        }
                }
#pragma unroll
                for (int n = 0; n < 4; n += 2) {
                    // p as two bf16, the second what the first's rounding left off: the matrix units have the time
                    Frag f[R], f2[R];
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float y = p[r][n + i / 2][2 * (i % 2)], z = p[r][n + i / 2][2 * (i % 2) + 1];
                            f[r].w[i] = bf16_pair(y, z);
                            f2[r].w[i] = bf16_pair(y - bf16_lo(f[r].w[i]), z - bf16_hi(f[r].w[i]));
                        }
#pragma unroll
                    for (int w = 0; w < DT / 64; ++w) {
                        uint32_t lo[4], hi[4];
                        transpose4x4(cv[n][0][w], cv[n][1][w], cv[n][2][w], cv[n][3][w], lo[0], lo[1], lo[2], lo[3]);
                        transpose4x4(cv[n + 1][0][w], cv[n + 1][1][w], cv[n + 1][2][w], cv[n + 1][3][w], hi[0], hi[1], hi[2], hi[3]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            Frag v;
                            v.w[0] = values2<false>(lo[i], v_scale[n]);
                            v.w[1] = values2<true>(lo[i], v_scale[n]);
                            v.w[2] = values2<false>(hi[i], v_scale[n + 1]);
                            v.w[3] = values2<true>(hi[i], v_scale[n + 1]);
#pragma unroll
                            for (int r = 0; r < R; ++r) {
                                o[r][4 * w + i] = mma16(v, f[r], o[r][4 * w + i]);
                                o[r][4 * w + i] = mma16(v, f2[r], o[r][4 * w + i]);
                            }
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                load_v();
            }
            // the waves' sums together, 16 rows at a time: o[t][i] is element kPer (4 g + i) + t of row m
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (R > 1 && r > 0) __syncthreads();
                sum[r] = sum4(sum[r]);
                if (g == 0) {
                    s_top[wave * kFew + m] = top[r];
                    s_sum[wave * kFew + m] = sum[r];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int t = 0; t < kPer; t += 4)
                        *reinterpret_cast<af32x4*>(s_out + (wave * kFew + m) * kRow + kPer * (4 * g + i) + t) =
                            af32x4{o[r][t][i], o[r][t + 1][i], o[r][t + 2][i], o[r][t + 3][i]};
                __syncthreads();
                const int n = threadIdx.x / 16, e = threadIdx.x % 16 * kPer;
                if (16 * r + n < rows) {
                    const int q2 = (16 * r + n) / a.group, h2 = head * a.group + 16 * r + n - q2 * a.group;
                    float best = -kInf, l = 0.0f, y[kPer];
#pragma unroll
                    for (int w = 0; w < kWaves; ++w) best = fmaxf(best, s_top[w * kFew + n]);
                    const float base = best == -kInf ? 0.0f : best;
#pragma unroll
                    for (int i = 0; i < kPer; ++i) y[i] = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWaves; ++w) {
                        const float by = __builtin_amdgcn_exp2f((s_top[w * kFew + n] - base) * scale2);
                        l = fmaf(s_sum[w * kFew + n], by, l);
#pragma unroll
                        for (int i = 0; i < kPer; ++i) y[i] = fmaf(s_out[(w * kFew + n) * kRow + e + i], by, y[i]);
                    }
                    if (step0 == 0 && last == all_steps) {
                        const float by = inverse(l);
                        uint32_t w[kPer / 2];
                        if (FULL || e < c.d) {
#pragma unroll
                            for (int i = 0; i < kPer / 2; ++i) {
                                w[i] = bf16_pair(y[2 * i] * by, y[2 * i + 1] * by);
                                top_out = top_of(w[i], top_out);
                            }
                            uint16_t* to = a.out + (int64_t)(from + q2) * a.out_row + (int64_t)h2 * a.out_head + e;
                            if constexpr (kPer == 8) *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
                            else *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
                        }
                        if (e == 0)
                            a.lse[(int64_t)h2 * c.tokens + from + q2] =
                                l == 0.0f ? -kInf : (base * scale2 + __builtin_amdgcn_logf(l)) * kLn2;
                    } else {
                        const int64_t slot = (2 * (int64_t)worker + (step0 == 0 ? 1 : 0)) * R + r;
                        float* to = a.partial + (slot * 16 + n) * DT + e;
#pragma unroll
                        for (int i = 0; i < kPer; i += 4) *reinterpret_cast<af32x4*>(to + i) = af32x4{y[i], y[i + 1], y[i + 2], y[i + 3]};
                        if (e == 0) a.tops[slot * 16 + n] = make_float2(best == -kInf ? -kInf : best * scale2, l);
                    }
                }
            }
            if (threadIdx.x == 0 && step0 == 0 && last < all_steps)
                joins[worker] = Join{from, head, 0, rows, (at - done + steps - 1) / share - worker + 1, (2 * worker + 1) * R,
                                     (2 * worker + 2) * R, 2 * R};
        }
        at += upto - done;
        if (at >= end) break;
        __syncthreads();                                   // what is in LDS has been read
        done = 0;
        if (++head == c.heads) {
            head = 0;
            do {
                s = sequence(c, ++b);
                steps = __builtin_amdgcn_readfirstlane(share_steps(a, s));
            } while (steps == 0);
        }
    }
    return top_out;
}

// 128 rows of one head's sequence of more: attention.hip's forward, whose tiles of keys and
// values are here made of codes.  Each wave loads 16 of a tile's 64 rows a step ahead and
// writes them into LDS as bf16.  Where the tiles are few, up to two workgroups per CU share
// a tile's keys, and the parts are joined.
// Bound by the matrix units and the softmax: MI355X, heads of 128, 4096 causal queries of 32 heads
// 152 to 158 us (0.87 to 0.90 PFLOP/s; from bf16 keys 150), 4096 on 8192 without a mask 541 (1.02); 35% of the cycles
// are the matrix units', at 2.06 GHz.  A tile's conversion is 32 of a wave's 219 vector instructions a step.
// p is rounded to bf16 once: with what that leaves off as a second operand, as in a share, the error is
// out's own rounding (2.2e-3 -> 1.7e-3 of its norm), but the 4096 take 154 -> 197 us, 2048 on 8192 328 -> 423.
template <int DT, bool FULL>
__device__ __forceinline__ uint32_t attend_rows(const CachedAttentionArgs& a, int block, uint8_t* lds, int (*sums)[4], int* found)
{
    constexpr int kTile = kKeys * DT * 2, kCh = DT / 8, kCodes = DT / 16, kLoads = DT / 64;
    const CacheArgs& c = a.c;
    const int lane = threadIdx.x & 63, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

    // the tile: every thread counts some sequences', in order
    const int per = (c.batch + kThreads - 1) / kThreads, b0 = threadIdx.x * per, b1 = min(b0 + per, c.batch);
    // (held to what the launch has room for, should bounds overlap)
    int mine = 0, longest = 0;
    int64_t mine_steps = 0;
    for (int b = b0; b < b1 && mine < kMostTiles; ++b) {
        const Sequence s = sequence(c, b);
        const int n = min(row_tiles(a, s), kMostTiles - mine);
        mine += n;
        mine_steps += (int64_t)n * tile_steps(a, s, s.queries / 2);
        if (n > 0) longest = max(longest, tile_steps(a, s, s.queries - 1));
    }
    int marks = 0;
#pragma unroll
    for (int bit = 1; bit <= 4; bit <<= 1) marks |= __any(step_marks(longest) & bit) ? bit : 0;
    Sums all = block_sums(mine, mine_steps, sums, marks);
    const bool fits = all.total <= a.tiles;
    all.total = min(all.total, a.tiles);
    Join* const joins = reinterpret_cast<Join*>(a.joins) + a.workers;
    const int units = all.total * c.heads;
    int head, split, parts, entry, slot0, slot_step;                       // of the unit's parts: what to join, and their sums' slots
    if (fits && few_split(units, all.total, a.workers, all.marks)) {
        // few: all tiles in parts of so many steps, the least of three with which there are no more parts than
        // workgroups, or in two; counted for all of these at once
        const int share = few_share(all.total_y * c.heads, a.workers);
        auto parts_of = [&](const Sequence& s, int k) __attribute__((always_inline)) {
            return few_parts(tile_steps(a, s, s.queries - 1), share, k, all.marks);
        };
        uint64_t own = 0;
        for (int b = b0; b < b1; ++b) {
            const Sequence s = sequence(c, b);
            const int n = row_tiles(a, s);
            if (n > 0)
#pragma unroll
                for (int k = 0; k < kFewChoices; ++k) own += (uint64_t)(n * parts_of(s, k)) << 16 * k;
        }
        uint64_t before, total;
        block_scan(own, sums + kWaves, before, total);
        const int k = few_choice(total, c.heads, a.workers), pieces = __builtin_amdgcn_readfirstlane(few_parts_of_all(total, k));
        if (threadIdx.x == 0 && block < a.workers && block >= units) joins[block].count = 0;
        if (block >= pieces * c.heads) return 0;
        const int at = pieces - 1 - block / c.heads;                       // a sequence's last (longest) tiles first
        head = block % c.heads;                                            // (blocks are dealt round-robin to the 8 XCDs)
        int left = at - few_parts_of_all(before, k);
        if (0 <= left && left < few_parts_of_all(own, k)) {
            int tile = all.before, b = b0, each;
            for (;; ++b) {
                const Sequence s = sequence(c, b);
                const int n = row_tiles(a, s);
                if (n == 0) continue;
                each = parts_of(s, k);
                if (left < n * each) break;
                left -= n * each;
                tile += n;
            }
            found[0] = b;
            found[1] = left / each;
            found[2] = left % each;
            found[3] = each;
            found[4] = tile + left / each;
        }
        __syncthreads();
        split = __builtin_amdgcn_readfirstlane(found[2]);
        parts = __builtin_amdgcn_readfirstlane(found[3]);
        entry = __builtin_amdgcn_readfirstlane(found[4]) * c.heads + head;
        slot0 = few_slot0(a.workers, at, split, c.heads, head);
        slot_step = few_step(c.heads);
        if (parts == 1 && threadIdx.x == 0) joins[entry].count = 0;
    } else {
        const int average = units == 0 ? 0 : (int)(all.total_y / all.total);
        const TileSplit how = tile_split(units, a.workers, average);
        const int joined = how.splits > 1 ? units - how.whole : 0;
        // what is to be joined: an entry for each unit that is split (by its first part, below), no others
        if (threadIdx.x == 0 && block < a.workers && block >= joined) joins[block].count = 0;
        if (block >= tile_blocks(how, units)) return 0;
        const TilePart taken = tile_part(block, units, c.heads, how);
        split = taken.split;
        parts = taken.parts;
        head = taken.unit % c.heads;
        const int t = all.total - 1 - taken.unit / c.heads;                // a sequence's last (longest) tiles first
        if (all.before <= t && t < all.before + mine) {
            int left = t - all.before, b = b0;
            for (;; ++b) {
                const int n = row_tiles(a, sequence(c, b));
                if (left < n) break;
                left -= n;
            }
            found[0] = b;
            found[1] = left;
        }
        __syncthreads();
        entry = taken.unit - how.whole;
        slot0 = tile_slot0(a.workers, entry, parts);
        slot_step = kTileSlots;
    }
    const int b = __builtin_amdgcn_readfirstlane(found[0]);
    const int row0 = __builtin_amdgcn_readfirstlane(found[1]) * kOwn;
    const Sequence s = sequence(c, b);
    const int from = __builtin_amdgcn_readfirstlane(s.from), queries = __builtin_amdgcn_readfirstlane(s.queries);
    const int held = __builtin_amdgcn_readfirstlane(s.held);
    const int rows = queries * a.group, r_wave = row0 + wave * 32, ri = r_wave + (lane & 31);
    const int q_wave = r_wave / a.group, q_last = (r_wave + 31) / a.group;
    const int qi = ri / a.group, hq = head * a.group + ri - qi * a.group;
    const bool valid = ri < rows;
    const int first = __builtin_amdgcn_readfirstlane(s.first);
    // keys seen: by this lane's query, by the wave's first and last, by the workgroup's last
    const int see = seen(a, held, first, qi);
    const int see_first = seen(a, held, first, q_wave);
    const int see_last = r_wave >= rows ? 0 : seen(a, held, first, q_last);
    const int end = seen(a, held, first, min((row0 + kOwn - 1) / a.group, queries - 1));
    const int steps = end > 0 ? (end + kKeys - 1) / kKeys : 0;
    const int s_begin = (int)((int64_t)steps * split / parts), s_end = (int)((int64_t)steps * (split + 1) / parts);

    Frag q[DT / 16];
    load_own<DT>(q, a.q + (int64_t)(from + qi) * a.q_row + (int64_t)hq * a.q_head, c.d, valid);

    const float c2 = a.scale * kLog2e;
    const float far = fminf(8.0f / c2, 1e38f);
    af32x16 o[DT / 32];
#pragma unroll
    for (int db = 0; db < DT / 32; ++db) o[db] = af32x16{0};
    float m = -kInf, mc = 0.0f, l = 0.0f;
    Tile<DT> tile;
    tile.init(lds0);

    // 16-code chunk i of a lane: row (lane + 64 i) / kCodes of the wave's 16, chunk % kCodes; in LDS two chunks of bf16
    uint32_t off[kLoads][2], put[kLoads][2];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int r = (lane + 64 * i) / kCodes, ch = (lane + 64 * i) % kCodes, row = 16 * wave + r;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int d = FULL ? DT : c.d, e = 16 * ch + 8 * j;
            off[i][j] = FULL || e < d ? (uint32_t)(r * d + e) : kNowhere;
            put[i][j] = lds0 + row * (DT * 2) + (((2 * ch + j) ^ spread<kCh>(row)) * 16);
        }
    }
    au32x4 ck[kLoads], cv[kLoads];
    Pages pages;
    auto fetch = [&](int key) __attribute__((always_inline)) {
        const Keys16 x = pages.at(key + 16 * wave, held);
        const auto k = rows_of(c.k, x, FULL ? DT : c.d), v = rows_of(c.v, x, FULL ? DT : c.d);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if constexpr (FULL) {
                ck[i] = __builtin_amdgcn_raw_buffer_load_b128(k, off[i][0], 0, 0);
                cv[i] = __builtin_amdgcn_raw_buffer_load_b128(v, off[i][0], 0, 0);
            } else {
                const au32x2 k0 = __builtin_amdgcn_raw_buffer_load_b64(k, off[i][0], 0, 0);
                const au32x2 k1 = __builtin_amdgcn_raw_buffer_load_b64(k, off[i][1], 0, 0);
                const au32x2 v0 = __builtin_amdgcn_raw_buffer_load_b64(v, off[i][0], 0, 0);
                const au32x2 v1 = __builtin_amdgcn_raw_buffer_load_b64(v, off[i][1], 0, 0);
                ck[i] = au32x4{k0[0], k0[1], k1[0], k1[1]};
                cv[i] = au32x4{v0[0], v0[1], v1[0], v1[1]};
            }
        }
    };
    auto values = [&](uint32_t a0, uint32_t a1, float by) __attribute__((always_inline)) {
        return au32x4{values2<false>(a0, by), values2<true>(a0, by), values2<false>(a1, by), values2<true>(a1, by)};
    };
    auto step = [&](auto stage, int st) __attribute__((always_inline)) {
        constexpr int at = stage.value * 2 * kTile;
        const float k_scale = pages.scale_k(st * kKeys + 16 * wave), v_scale = pages.scale_v(st * kKeys + 16 * wave);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                lds_u32x4* to = (lds_u32x4*)(uintptr_t)put[i][j];
                to[at / 16] = values(ck[i][2 * j], ck[i][2 * j + 1], k_scale);
                to[(at + kTile) / 16] = values(cv[i][2 * j], cv[i][2 * j + 1], v_scale);
            }
        if (st + 1 < s_end) {
            pages.advance((st + 1) * kKeys);
            fetch((st + 1) * kKeys);
        }
        // tile st is written by all; the other stage was last read in step st - 1, by the waves that are here
        __syncthreads();
        const int j0 = st * kKeys;
        if (j0 < see_last) attend_tile<DT, at>(tile, q, see - j0, j0 + kKeys > see_first, c2, far, o, m, mc, l);
    };
    if (s_begin < s_end) {
        pages.init(c, b, head, held, s_begin * kKeys);
        pages.start();
        fetch(s_begin * kKeys);
    }
    for (int st = s_begin; st < s_end; st += 2) {
        step(std::integral_constant<int, 0>{}, st);
        if (st + 1 < s_end) step(std::integral_constant<int, 1>{}, st + 1);
    }

    l += partner(l);
    if (parts > 1) {
        const int64_t row = (int64_t)(slot0 + split * slot_step) * 16 + wave * 32 + (lane & 31);
        store_partial<DT>(o, a.partial + row * DT, DT, valid);
        if (valid && h == 0) a.tops[row] = make_float2(m == -kInf ? -kInf : mc, l);
        if (split == 0 && threadIdx.x == 0) joins[entry] = Join{from, head, row0, rows, parts, slot0, slot0 + slot_step, slot_step};
        return 0;
    }
    const uint32_t top = store_own<DT>(o, inverse(l), a.out + (int64_t)(from + qi) * a.out_row + (int64_t)hq * a.out_head, c.d, valid);
    if (valid && h == 0)
        a.lse[(int64_t)hq * c.tokens + from + qi] = l == 0.0f ? -kInf : (mc + __builtin_amdgcn_logf(l)) * kLn2;
    return top;
}

}  // namespace

// KINDS 1: sequences of few rows alone; 2: of more alone; 3: both, the tiles' workgroups first, so
// that the shares run in what room they leave (1000 queries on 1500 keys among 31 single ones,
// 40 and 8 heads: 47.5 us, the tiles alone 45.5, the shares alone 18; with both in turn, 8 by 8, 70 where this order took 49).
template <int DT, bool FULL, int KINDS, int R>
__global__ void __launch_bounds__(kThreads, R == 1 ? 2 : 1) attention_cached_kernel(const CachedAttentionArgs a)
{
    constexpr int kBytes = KINDS == 1 ? share_lds<DT>() : std::max(share_lds<DT>(), tile_lds<DT>());
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kBytes];
    __shared__ int sums[2 * kWaves][4], found[5];
    const int shares = KINDS == 1 ? gridDim.x : KINDS == 2 ? 0 : a.workers, tiles = gridDim.x - shares;
    const bool share = (int)blockIdx.x >= tiles;
    const int block = share ? blockIdx.x - tiles : blockIdx.x;
    uint32_t top = 0;
    if (KINDS != 2 && share) top = attend_share<DT, FULL, R>(a, block, lds, sums, found);
    else if constexpr (KINDS != 1) top = attend_rows<DT, FULL>(a, block, lds, sums, found);
    if (a.absmax) block_max_to_global(top, a.absmax);
}

// out and lse of rows whose keys several workgroups shared: 16 rows to a workgroup, a row's
// parts dealt to several groups of DT / 8 threads, each with its own running maximum, which
// are then added in order.
template <int DT>
__global__ void __launch_bounds__(kJoinThreads) attention_cached_join_kernel(const CachedAttentionArgs a, int shares)
{
    constexpr int kPer = 8, kLanes = DT / kPer, kGroups = kJoinThreads / kLanes;
    __shared__ float s_sum[kGroups][2], s_out[kGroups][DT + 4];
    const CacheArgs& c = a.c;
    const int i = blockIdx.x;
    const int groups = i < shares ? a.few / 16 : kOwn / 16, j = i < shares ? i : i - shares;
    const int entry = (i < shares ? 0 : a.workers) + j / groups, group16 = j % groups;
    const Join job = reinterpret_cast<const Join*>(a.joins)[entry];
    if (job.count <= 1) return;
    const int rows = min(job.rows - job.row - 16 * group16, 16);
    if (rows <= 0) return;
    const int wide = rows > 8 ? 16 : rows > 4 ? 8 : rows > 2 ? 4 : rows;       // rows side by side
    const int k = threadIdx.x / kLanes, e = threadIdx.x % kLanes * kPer, n = k % wide, lead = k / wide;
    auto slot = [&](int p) __attribute__((always_inline)) {
        return (int64_t)((p == 0 ? job.first : job.second + (p - 1) * job.step) + group16) * 16 + n;
    };
    float m = -kInf, l = 0.0f, t[kPer] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (n < rows)
#pragma unroll 4
        for (int p = lead; p < job.count; p += kGroups / wide) {
            const float2 y = a.tops[slot(p)];
            const float4* from = reinterpret_cast<const float4*>(a.partial + slot(p) * DT + e);
            const float4 u = from[0], v = from[1];
            const float up = fmaxf(m, y.x), base = up == -kInf ? 0.0f : up;
            const float old = __builtin_amdgcn_exp2f(m - base), by = __builtin_amdgcn_exp2f(y.x - base);
            const float w[kPer] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
            l = fmaf(y.y, by, l * old);
#pragma unroll
            for (int j = 0; j < kPer; ++j) t[j] = fmaf(w[j], by, t[j] * old);
            m = up;
        }
    if (e == 0) {
        s_sum[k][0] = m;
        s_sum[k][1] = l;
    }
    *reinterpret_cast<float4*>(&s_out[k][e]) = make_float4(t[0], t[1], t[2], t[3]);
    *reinterpret_cast<float4*>(&s_out[k][e + 4]) = make_float4(t[4], t[5], t[6], t[7]);
    __syncthreads();
    uint32_t top = 0;
    if (lead == 0 && n < rows && e < c.d) {
        float all = -kInf, total = 0.0f;
        const int upto = min(kGroups, n + job.count * wide);            // groups that had a part
#pragma unroll 8
        for (int g = n; g < upto; g += wide) all = fmaxf(all, s_sum[g][0]);
        const float base = all == -kInf ? 0.0f : all;
#pragma unroll
        for (int j = 0; j < kPer; ++j) t[j] = 0.0f;
#pragma unroll 4
        for (int g = n; g < upto; g += wide) {
            const float by = __builtin_amdgcn_exp2f(s_sum[g][0] - base);
            total = fmaf(s_sum[g][1], by, total);
#pragma unroll
            for (int j = 0; j < kPer; ++j) t[j] = fmaf(s_out[g][e + j], by, t[j]);
        }
        const float by = inverse(total);
        const int row = job.row + 16 * group16 + n, qi = row / a.group, hq = job.head * a.group + row - qi * a.group;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = bf16_pair(t[2 * j] * by, t[2 * j + 1] * by);
            top = top_of(w[j], top);
        }
        *reinterpret_cast<uint4*>(a.out + (int64_t)(job.from + qi) * a.out_row + (int64_t)hq * a.out_head + e) =
            make_uint4(w[0], w[1], w[2], w[3]);
        if (e == 0) a.lse[(int64_t)hq * c.tokens + job.from + qi] = total == 0.0f ? -kInf : (base + __builtin_amdgcn_logf(total)) * kLn2;
    }
    if (a.absmax) block_max_to_global(top, a.absmax);
}

namespace {

// What a call's sequences can be, as far as the host knows.
struct Plan {
    int kinds, few, workers;
    bool whole;            // few rows of short contexts: a workgroup for each head of a sequence, nothing to join
    int64_t tiles;         // of rows, at most
};

Plan plan(int64_t tokens, int group, int heads, int batch, int64_t capacity, bool bounds)
{
    Plan p{};
    const int64_t rows = (bounds ? tokens : tokens / batch) * group;           // of a sequence, at most
    // (up to 32 in shares where no sequence has more, MI355X, shares / tiles: 4 queries of 64 heads on 4096 keys of 8, 64
    // sequences 107 / 108 us, 5 of 32 on 65535 among 31 times on 505 50 / 67, 5 of 10 on 1000 keys of 2, 8 times 16.6 / 17.9)
    p.few = rows <= kFew || rows > 2 * kFew ? kFew : 2 * kFew;
    p.kinds = rows <= p.few ? 1 : bounds ? 3 : 2;
    // two per CU (one where the rows take more than half of the registers), whole rounds of the XCDs
    const int cus = device_cu_count();
    p.workers = ((p.few == kFew ? 2 : 1) * cus + 7) / 8 * 8;
    const int64_t all = (int64_t)batch * heads, times = std::min<int64_t>(std::max<int64_t>(all / (2 * cus), 1), kMostWhole);
    p.whole = p.kinds == 1 && capacity <= kWholeKeys * times && all <= 1 << 20;
    if (p.kinds & 2) p.tiles = bounds ? tokens * group / kOwn + std::min<int64_t>(batch, tokens * group / (kFew + 1))
                                      : batch * ((tokens / batch * group + kOwn - 1) / kOwn);
    return p;
}

// Slots of 16 rows that hold parts: two to a share, and the tiles'.
int64_t slots(const Plan& p) { return p.whole ? 0 : p.workers * 2 * (p.few / 16) + (p.kinds & 2 ? split_parts(p.workers) * kTileSlots : 0); }

template <int DT, bool FULL>
void (*kernel_of(const Plan& p))(CachedAttentionArgs)
{
    if (p.kinds == 1)
        return p.few == kFew ? attention_cached_kernel<DT, FULL, 1, 1> : attention_cached_kernel<DT, FULL, 1, 2>;
    return p.kinds == 2 ? attention_cached_kernel<DT, FULL, 2, 1> : attention_cached_kernel<DT, FULL, 3, 1>;
}

}  // namespace

bool attention_cached_grid_ok(int64_t tokens, int group, int heads, int batch, int blocks, int shift)
{
    // the steps of all sequences of few rows are counted in 32 bits, and so are a launch's threads
    const int64_t steps = (((int64_t)blocks << shift) + kKeys - 1) / kKeys + kPiece + 1;
    return batch * steps <= ((int64_t)0x7FFFFFFF - (1 << 20)) / heads && tokens * group / kOwn + batch <= 0xFFFFFFFFll / kThreads / 2 / heads;
}

static int64_t capacity(int blocks, int shift) { return (int64_t)blocks << shift; }

int64_t attention_cached_workspace(int64_t tokens, int group, int heads, int d, int batch, int blocks, int shift, bool bounds)
{
    const Plan p = plan(tokens, group, heads, batch, capacity(blocks, shift), bounds);
    return p.whole ? 0 : 2 * p.workers * (int64_t)sizeof(Join) + slots(p) * 16 * (8 + 4 * (d <= 64 ? 64 : 128));
}

hipError_t launch_attention_cached(const CachedAttentionArgs& args, void* workspace, hipStream_t stream)
{
    CachedAttentionArgs a = args;
    const int d = a.c.d, heads = a.c.heads;
    const Plan p = plan(a.c.tokens, a.group, heads, a.c.batch, capacity(a.c.blocks, a.c.shift), a.c.cu != nullptr);
    a.workers = p.workers;
    a.whole = p.whole;
    a.few = p.few;
    a.tiles = (int)p.tiles;
    a.joins = workspace;
    a.tops = reinterpret_cast<float2*>(static_cast<Join*>(workspace) + 2 * p.workers);
    a.partial = reinterpret_cast<float*>(a.tops + slots(p) * 16);
    const int64_t blocks = p.whole ? (int64_t)a.c.batch * heads
                                   : (p.kinds & 1 ? p.workers : 0) + (p.kinds & 2 ? row_blocks(p.tiles * heads, p.workers) : 0);
    const hipError_t e = launch(d == 64 ? kernel_of<64, true>(p) : d == 128 ? kernel_of<128, true>(p)
                                : d < 64 ? kernel_of<64, false>(p) : kernel_of<128, false>(p),
                                dim3((unsigned)blocks), dim3(kThreads), stream, a);
    // without bounds the tiles are known, and whether they can be split
    const int64_t steps = (capacity(a.c.blocks, a.c.shift) + kKeys - 1) / kKeys;
    const bool split = p.kinds != 2 || may_split(p.tiles * heads, p.workers, steps);
    if (e != hipSuccess || p.whole || !split) return e;
    const int shares = p.kinds & 1 ? p.workers * (p.few / 16) : 0, joins = shares + (p.kinds & 2 ? joined_units(p.workers) * kTileSlots : 0);
    return launch(d <= 64 ? attention_cached_join_kernel<64> : attention_cached_join_kernel<128>, dim3(joins), dim3(kJoinThreads),
                  stream, a, shares);
}

}  // namespace fp8k
