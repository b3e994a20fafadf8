// attention.hip -- softmax attention over packed sequences, forward and backward,
// for gfx950.
//
// For one sequence of nq queries and nk keys and one query head, with the key head
// it shares, s = scale q k^T, and a key j seen by query i if j < nk and, causal,
// j <= i + nk - nq (the last query sees every key):
//   p = exp(s - lse) over the keys seen, lse = log sum exp(s),   out = p v
// and backward, which takes p from q, k and lse again instead of keeping it,
//   delta = rowsum(dout out)          dv = p^T dout
//   dp = dout v^T                     ds = p (dp - delta)
//   dq = scale ds k                   dk = scale ds^T q
// (dk and dv summed over the query heads that share the key head).  A query that
// sees nothing has out = 0, lse = -inf, and gives no gradient.
//
// Bound by the matrix units and, next to them, by the exponentials: 4 d
// multiply-adds per score against one exponential, a handful of fp32 operations
// and two roundings.
//
// Layout.  Every product runs on v_mfma_f32_32x32x16_bf16, and scores are always
// computed so that what the workgroup keeps (32 queries per wave in the forward
// and the dq kernel, 32 keys per wave in the dk/dv kernel) is the product's
// column: a lane then owns one of them, holds 16 of a block's 32 scores for it,
// and its partner 32 lanes away the other 16.  So
//  - a query's maximum and sum are sums over the lane's registers and one swap
//    with the partner lane;
//  - the lane's 8 scores of registers 8 c .. 8 c + 7, rounded to bf16, are exactly
//    the second operand of the next product for 16 of the streamed rows, in the
//    order 16 c + 8 (e / 4) + 4 (lane / 32) + e % 4: p and ds never leave the
//    registers;
//  - the first operand of that product is the streamed tile's transpose in the same
//    order, which ds_read_b64_tr_b16 delivers from the row-major tile in LDS.
// Streamed tiles (k and v, or q and dout) go global -> LDS with 16-byte
// direct-to-LDS buffer loads, two stages (four in the dk/dv kernel); the buffer's size
// is set to what is left of the sequence, so that rows past its end read as zero, and
// lanes past the head dimension are given an offset outside it.  16-byte chunk c of tile row r lies at
// chunk c ^ f(r): with f's low row bits in the high chunk bits, the 4-row pieces
// of the transposing reads and the 16-row columns of the plain reads both spread
// over all banks.
#include <algorithm>

#include "fp8_device.hpp"
#include "fp8_internal.hpp"
#include "head_tensor.hpp"

namespace fp8k {

namespace {

typedef __bf16 ab16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 ab16x2 __attribute__((ext_vector_type(2)));
typedef float af32x2 __attribute__((ext_vector_type(2)));
typedef float af32x16 __attribute__((ext_vector_type(16)));
typedef short as16x4 __attribute__((ext_vector_type(4)));
typedef unsigned int au32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) as16x4 lds_s16x4;
typedef __attribute__((address_space(3))) au32x4 lds_u32x4;
typedef float af32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) af32x4 lds_f32x4;

constexpr int kAttThreads = 256;
constexpr int kAttWaves = 4;
constexpr int kOwn = 128;                 // queries a workgroup keeps: 32 per wave
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kInf = __builtin_inff();

union Frag {
    au32x4 u;
    ab16x8 b;
    struct { as16x4 lo, hi; } s;
    uint32_t w[4];
};

__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(af32x2{a, b}, ab16x2));
}

__device__ __forceinline__ af32x16 mma(const Frag& a, const Frag& b, const af32x16& c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.b, b.b, c, 0, 0, 0);
}

// The value of the lane 32 away.
__device__ __forceinline__ float partner(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// Chunk permutation of tile row r (rows of CH 16-byte chunks).
template <int CH>
__device__ __forceinline__ int spread(int r)
{
    return CH == 16 ? ((r & 3) << 2 | (r >> 2 & 3)) : ((r >> 1 & 1) << 2 | (r >> 2 & 3));
}

// One 16-byte direct-to-LDS load per lane through a buffer descriptor: lane L reads
// at base + voff[L] (zero past the descriptor's size) and writes LDS bytes
// lds + 16 L.  Inline assembly, so that the compiler does not put a wait for every
// load in flight in front of each LDS read; the kernels wait and synchronise.
__device__ __forceinline__ void buffer_to_lds(uint32_t voff, const au32x4& desc, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :
                 : "v"(voff), "s"(desc), "s"(lds)
                 : "memory", "m0");
}

// The same with 4 bytes per lane (LDS bytes lds + 4 L).
__device__ __forceinline__ void buffer4_to_lds(uint32_t voff, const au32x4& desc, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dword %0, %1, 0 offen lds"
                 :
                 : "v"(voff), "s"(desc), "s"(lds)
                 : "memory", "m0");
}

// s_waitcnt immediate: at most n vector memory operations in flight.
constexpr int wait_loads(int n) { return 0x0F70 | (n & 15) | (n >> 4) << 14; }

__device__ __forceinline__ au32x4 descriptor(const uint8_t* base, int64_t n)
{
    const uint64_t b = (uint64_t)base;
    au32x4 d;
    d[0] = __builtin_amdgcn_readfirstlane((uint32_t)b);
    d[1] = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32) & 0xFFFFu);
    d[2] = __builtin_amdgcn_readfirstlane((uint32_t)n);
    d[3] = 0x00020000u;                   // raw buffer, 32-bit elements
    return d;
}

// Streams ROWS-row tiles of one head's rows [0, n) of a packed tensor into LDS.
template <int DT, int ROWS, int WAVES = kAttWaves>
struct Stream {
    static constexpr int kRow = DT * 2;                        // bytes of a tile row
    static constexpr int kCh = DT / 8;                         // its 16-byte chunks
    static constexpr int kPer = 64 / kCh;                      // rows per wave and load
    static constexpr int kLoads = ROWS / (kPer * WAVES);       // loads per wave and tile
    static_assert(kLoads * kPer * WAVES == ROWS, "whole loads");
    const uint8_t* base;
    int64_t stride;                       // bytes between rows
    int n;
    uint32_t voff[kLoads];

    __device__ __forceinline__ void init(const uint16_t* p, int64_t row_stride, int rows, int d)
    {
        base = reinterpret_cast<const uint8_t*>(p);
        stride = row_stride * 2;
        n = rows;
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = (wave * kLoads + i) * kPer + lane / kCh;
            const int c = (lane % kCh) ^ spread<kCh>(r);
            voff[i] = stream_offset(r, c, stride, d);
        }
    }

    // rows row0 .. row0 + ROWS - 1 into the ROWS * kRow bytes at LDS address lds
    __device__ __forceinline__ void issue(int row0, uint32_t lds, int wave) const
    {
        const au32x4 desc = descriptor(base + (int64_t)row0 * stride, stream_bytes(n - row0, stride));
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            buffer_to_lds(voff[i], desc, __builtin_amdgcn_readfirstlane(lds + (uint32_t)((wave * kLoads + i) * 1024)));
    }
};

// Operand reads from tiles in LDS.  rows(): a tile's rows as the product's rows, the
// head dimension reduced (chunk c: elements 16 c ..).  cols(): its columns (32 of the
// head dimension, block db) as the product's rows, 16 of its rows reduced, in the
// order that the score registers have.  A lane keeps one address per c and per (db,
// half), relative to which every tile, stage and block is a constant: the tiles of a
// kernel lie within the 64 KB that an LDS instruction's offset reaches.
template <int DT>
struct Tile {
    static constexpr int kRow = DT * 2;
    static constexpr int kCh = DT / 8;
    uint32_t plain[DT / 16], trans[DT / 32][2];

    __device__ __forceinline__ void init(uint32_t lds)
    {
        const int lane = threadIdx.x & 63, h = lane >> 5;
        const int r = lane & 31;
#pragma unroll
        for (int c = 0; c < DT / 16; ++c) plain[c] = lds + r * kRow + (((2 * c + h) ^ spread<kCh>(r)) * 16);
        const int t = 4 * h + ((lane & 15) >> 2);
#pragma unroll
        for (int db = 0; db < DT / 32; ++db)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                trans[db][i] = lds + (t + 8 * i) * kRow +
                               (((4 * db + 2 * (lane >> 4 & 1) + (lane & 3) / 2) ^ spread<kCh>(t + 8 * i)) * 16) +
                               (lane & 1) * 8;
    }
    // at: the tile's constant offset
    __device__ __forceinline__ Frag rows(int at, int block, int c) const
    {
        Frag f;
        f.u = *((const lds_u32x4*)(uintptr_t)plain[c] + (at + block * 32 * kRow) / 16);
        return f;
    }
    __device__ __forceinline__ Frag cols(int at, int block, int c, int db) const
    {
        const int off = (at + (block * 32 + c * 16) * kRow) / 8;
        Frag f;
        f.s.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)trans[db][0] + off);
        f.s.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)trans[db][1] + off);
        return f;
    }
};

// 16 scores -> the two operands of 16 reduced rows each.
__device__ __forceinline__ void to_operands(const af32x16& p, Frag (&f)[2])
{
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) f[c].w[e] = bf16_pair(p[8 * c + 2 * e], p[8 * c + 2 * e + 1]);
}

// What their rounding left off, as further operands of the same rows.
__device__ __forceinline__ void to_residuals(const af32x16& p, const Frag (&f)[2], Frag (&l)[2])
{
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            l[c].w[e] = bf16_pair(p[8 * c + 2 * e] - bf16_lo(f[c].w[e]), p[8 * c + 2 * e + 1] - bf16_hi(f[c].w[e]));
}

// A lane's fixed operand: row `row` of a head, chunk c holding elements
// 16 c + 8 (lane / 32) ..; zero past the head dimension or where !valid.
template <int DT>
__device__ __forceinline__ void load_own(Frag (&f)[DT / 16], const uint16_t* row, int d, bool valid)
{
    const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int c = 0; c < DT / 16; ++c) {
        f[c].u = au32x4{0, 0, 0, 0};
        if (valid && 16 * c + 8 * h < d) f[c].u = *reinterpret_cast<const au32x4*>(row + 16 * c + 8 * h);
    }
    // Waited for here: at its first use, in the loop, the compiler's wait (it does not see
    // the direct-to-LDS loads) would be one for every tile in flight, in every step.
#pragma unroll
    for (int c = 0; c < DT / 16; ++c) asm volatile("" : "+v"(f[c].u));
}

// Store a lane's accumulated row (acc[db][i]: element 32 db + 8 (i / 4) + 4 (lane / 32)
// + i % 4), times `by`; returns the largest magnitude pattern stored.
template <int DT>
__device__ __forceinline__ uint32_t store_own(const af32x16 (&acc)[DT / 32], float by, uint16_t* row, int d, bool valid)
{
    const int h = (threadIdx.x & 63) >> 5;
    uint32_t top = 0;
    if (!valid) return 0;
#pragma unroll
    for (int db = 0; db < DT / 32; ++db)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int at = 32 * db + 8 * b + 4 * h;
            if (at < d) {
                uint2 o;
                o.x = bf16_pair(acc[db][4 * b] * by, acc[db][4 * b + 1] * by);
                o.y = bf16_pair(acc[db][4 * b + 2] * by, acc[db][4 * b + 3] * by);
                *reinterpret_cast<uint2*>(row + at) = o;
                top = max(max(max(top, o.x & 0x7FFF0000u), o.x << 16 & 0x7FFFFFFFu),
                          max(o.y & 0x7FFF0000u, o.y << 16 & 0x7FFFFFFFu));
            }
        }
    return top;
}

// The same row as fp32 partial sums.
template <int DT>
__device__ __forceinline__ void store_partial(const af32x16 (&acc)[DT / 32], float* row, int d, bool valid)
{
    const int h = (threadIdx.x & 63) >> 5;
    if (!valid) return;
#pragma unroll
    for (int db = 0; db < DT / 32; ++db)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int at = 32 * db + 8 * b + 4 * h;
            if (at < d)
                *reinterpret_cast<float4*>(row + at) =
                    make_float4(acc[db][4 * b], acc[db][4 * b + 1], acc[db][4 * b + 2], acc[db][4 * b + 3]);
        }
}

// Which rows a workgroup keeps: tile `t` of the tiles of all sequences, in order.
struct Place {
    int q0, nq, k0, nk;       // the sequence's queries and keys within the packed tensors
    int first;                // the tile's first row within the sequence
    bool any;
};

// The bounds of sequence i, held inside the tensor and in order whatever cu says.
__device__ __forceinline__ void bounds(const int* cu, int i, int total, int& from, int& count)
{
    if (!cu) {
        from = 0;
        count = total;
        return;
    }
    const int a = min(max(cu[i], 0), total), b = min(max(cu[i + 1], 0), total);
    from = a;
    count = max(b - a, 0);
}

// Every lane takes a sequence, 64 at a time; a prefix sum over the wave finds the one
// that holds tile t.  `own` is the side that is tiled (0: queries, 1: keys).
__device__ __forceinline__ Place find_tile(const AttentionArgs& a, int t, int own, int rows = kOwn, int group = 1)
{
    const int lane = threadIdx.x & 63;
    Place p{};
    int before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
        int from = 0, count = 0;
        if (b0 + lane < a.batch) bounds(own ? a.cu_k : a.cu_q, b0 + lane, own ? a.tk : a.tq, from, count);
        const int tiles = (int)(((int64_t)count * group + rows - 1) / rows);
        int upto = tiles;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int o = __shfl_up(upto, off, 64);
            if (lane >= off) upto += o;
        }
        const uint64_t past = __ballot(before + upto > t);
        if (past) {
            const int l = __ffsll((unsigned long long)past) - 1;
            const int seq = __builtin_amdgcn_readfirstlane(b0 + l);
            const int tile = t - before - __shfl(upto - tiles, l, 64);
            p.first = __builtin_amdgcn_readfirstlane(tile * rows);
            bounds(a.cu_q, seq, a.tq, p.q0, p.nq);
            bounds(a.cu_k, seq, a.tk, p.k0, p.nk);
            p.q0 = __builtin_amdgcn_readfirstlane(p.q0);
            p.nq = __builtin_amdgcn_readfirstlane(p.nq);
            p.k0 = __builtin_amdgcn_readfirstlane(p.k0);
            p.nk = __builtin_amdgcn_readfirstlane(p.nk);
            p.any = true;
            return p;
        }
        before += __shfl(upto, 63, 64);
    }
    return p;
}

// Workgroup -> (tile, head).  Workgroups are dealt round-robin to the 8 XCDs: with a
// multiple of 8 heads each XCD gets whole heads, so that a head's streamed tiles are
// shared in its L2.
__device__ __forceinline__ void deal(int b, int heads, int& tile, int& head)
{
    if (heads % 8 == 0) {
        const int per = heads / 8;
        head = (b % 8) * per + (b / 8) % per;
        tile = b / heads;
    } else {
        head = b % heads;
        tile = b / heads;
    }
}

constexpr int kKeys = 64;                 // keys per streamed tile, forward and dq

}  // namespace

// ---------------------------------------------------------------------- forward

// 32 rows per wave, a row being a query of one head, or, where the queries are few, of one of
// the `group` heads that share a key head, which then read its keys once; 64 keys a step,
// with one running maximum and sum per row.  Operands
// are read from LDS four instructions ahead of the matrix instruction that takes them.
// MI355X, causal, heads of 128: 4096 tokens, 32 heads 148 us (0.93 PFLOP/s); 8192 packed
// tokens, 40 query and 8 key heads 263 us (0.92).  Bound by the two products and the
// softmax between them, at the power limit (without a mask the clock falls to 1.83 GHz,
// where this is half of what the matrix units can do): 32 matrix instructions to 32
// exponentials and some 120 other vector instructions per step and wave.  Giving a wave
// its softmax to interleave with its own products measured no faster (151 us).
template <int DT>
__global__ void __launch_bounds__(kAttThreads, 2) attention_forward_kernel(const AttentionArgs a)
{
    constexpr int kTile = kKeys * DT * 2;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[4 * kTile];
    int t, unit;
    deal(blockIdx.x, a.hq / a.group * a.splits, t, unit);
    const int split = unit % a.splits, head0 = unit / a.splits * a.group;
    const Place pl = find_tile(a, a.tiles - 1 - a.tile0 - t, 0, kOwn, a.group);   // a sequence's last (longest) tiles first
    if (!pl.any) return;
    const int lane = threadIdx.x & 63, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
    const int khead = head0 / (a.hq / a.hk);

    // row r of the sequence: query r / group, head head0 + r % group
    const int rows = pl.nq * a.group, r_wave = pl.first + wave * 32, ri = r_wave + (lane & 31);
    const int q_wave = r_wave / a.group, q_last = (r_wave + 31) / a.group;
    const int qi = ri / a.group, head = head0 + ri - qi * a.group;
    const bool mine = ri < rows;
    const int shift = pl.nk - pl.nq;
    // keys seen: by this lane's query, by the wave's first and last, by the workgroup's last
    const int see = a.causal ? min(pl.nk, qi + shift + 1) : pl.nk;
    const int see_first = a.causal ? min(pl.nk, q_wave + shift + 1) : pl.nk;
    const int see_last = r_wave >= rows ? 0 : a.causal ? min(pl.nk, q_last + shift + 1) : pl.nk;
    const int end = a.causal ? min(pl.nk, min((pl.first + kOwn - 1) / a.group + 1, pl.nq) + shift) : pl.nk;
    const int all = end > 0 ? (end + kKeys - 1) / kKeys : 0;
    const int s_begin = (int)((int64_t)all * split / a.splits), s_end = (int)((int64_t)all * (split + 1) / a.splits);

    Frag q[DT / 16];
    load_own<DT>(q, a.q + (int64_t)(pl.q0 + qi) * a.q_row + (int64_t)head * a.q_head, a.d, mine);

    Stream<DT, kKeys> ks, vs;
    ks.init(a.k + (int64_t)pl.k0 * a.k_row + (int64_t)khead * a.k_head, a.k_row, pl.nk, a.d);
    vs.init(a.v + (int64_t)pl.k0 * a.v_row + (int64_t)khead * a.v_head, a.v_row, pl.nk, a.d);
    Tile<DT> tile;
    tile.init(lds0);

    const float c = a.scale * kLog2e;
    // scores may pass the running maximum by 2^8 before a rescale (any key seen passes the
    // first maximum, -inf: the step to it is finite however small the scale)
    const float far = fminf(8.0f / c, 1e38f);
    af32x16 o[DT / 32];
#pragma unroll
    for (int db = 0; db < DT / 32; ++db) o[db] = af32x16{0};
    float m = -kInf, mc = 0.0f, l = 0.0f;

    if (s_begin < s_end) {
        ks.issue(s_begin * kKeys, lds0, wave);
        vs.issue(s_begin * kKeys, lds0 + kTile, wave);
    }
    auto step = [&](auto stage, int s) {
        constexpr int at = stage.value * 2 * kTile, to = (2 - stage.value * 2) * kTile;
        __builtin_amdgcn_s_waitcnt(0x0F70);                // this wave's loads of tile s have landed
        __syncthreads();                                   // everyone's; tile s - 1 is read
        if (s + 1 < s_end) {
            ks.issue((s + 1) * kKeys, lds0 + to, wave);
            vs.issue((s + 1) * kKeys, lds0 + to + kTile, wave);
        }
        const int j0 = s * kKeys;
        if (j0 >= see_last) return;                        // nothing of this tile is seen by the wave
        // The tile's matrix instructions in order -- the scores' (two blocks of keys by the
        // chunks of the head dimension), then the values' -- each with its operand read
        // from LDS kAhead instructions before it; the first values are read before the
        // softmax.
        constexpr int kS = DT / 8, kAll = kS + DT / 8, kAhead = 4;
        Frag r[kAhead];
        auto fetch = [&](int t) __attribute__((always_inline)) {
            if (t < kS) r[t % kAhead] = tile.rows(at, t % 2, t / 2);
            else if (t < kAll) r[t % kAhead] = tile.cols(at + kTile, (t - kS) / (DT / 16), (t - kS) / (DT / 32) % 2, (t - kS) % (DT / 32));
        };
#pragma unroll
        for (int t = 0; t < kAhead; ++t) fetch(t);
        af32x16 p[2] = {af32x16{0}, af32x16{0}};
#pragma unroll
        for (int t = 0; t < kS; ++t) {
            p[t % 2] = mma(r[t % kAhead], q[t / 2], p[t % 2]);
            fetch(t + kAhead);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (j0 + kKeys > see_first) {
            const int see0 = see - j0 - 4 * h;             // register i: key 32 kb + 8 (i / 4) + i % 4 of what is left
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (32 * kb + 8 * (i / 4) + i % 4 >= see0) p[kb][i] = -kInf;
        }
        float tops[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            tops[x] = fmaxf(p[x / 2][8 * (x % 2)], p[x / 2][8 * (x % 2) + 1]);
#pragma unroll
            for (int i = 2; i < 8; i += 2)
                tops[x] = fmaxf(fmaxf(tops[x], p[x / 2][8 * (x % 2) + i]), p[x / 2][8 * (x % 2) + i + 1]);
        }
        float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        top = fmaxf(top, partner(top));
        if (__any(top > m + far)) {                        // m = -inf: any seen key
            const float up = fmaxf(m, top);
            const float use = up == -kInf ? 0.0f : up;
            const float by = __builtin_amdgcn_exp2f((m - use) * c);
            m = up;
            mc = use * c;
            l *= by;
#pragma unroll
            for (int db = 0; db < DT / 32; ++db)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[db][i] *= by;
        }
        float sums[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        Frag f[2][2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                p[kb][i] = __builtin_amdgcn_exp2f(fmaf(p[kb][i], c, -mc));
                sums[i % 4] += p[kb][i];
            }
            to_operands(p[kb], f[kb]);
#pragma unroll
            for (int t = kS + kb * (DT / 16); t < kS + (kb + 1) * (DT / 16); ++t) {
                const int db = (t - kS) % (DT / 32);
                o[db] = mma(r[t % kAhead], f[kb][(t - kS) / (DT / 32) % 2], o[db]);
                fetch(t + kAhead);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        l += (sums[0] + sums[1]) + (sums[2] + sums[3]);
    };
    for (int s = s_begin; s < s_end; s += 2) {
        step(std::integral_constant<int, 0>{}, s);
        if (s + 1 < s_end) step(std::integral_constant<int, 1>{}, s + 1);
    }

    l += partner(l);
    if (a.splits > 1) {
        const int64_t row = ((int64_t)split * a.hq + head) * a.tq + pl.q0 + qi;
        store_partial<DT>(o, a.partial + row * a.d, a.d, mine);
        if (mine && h == 0) a.tops[row] = make_float2(m == -kInf ? -kInf : mc, l);
        return;
    }
    const float by = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);   // a NaN sum stays NaN
    const uint32_t top = store_own<DT>(o, by, a.out + (int64_t)(pl.q0 + qi) * a.out_row + (int64_t)head * a.out_head,
                                       a.d, mine);
    if (mine && h == 0)
        a.lse[(int64_t)head * a.tq + pl.q0 + qi] = l == 0.0f ? -kInf : (mc + __builtin_amdgcn_logf(l)) * kLn2;
    if (a.absmax) block_max_to_global(top, a.absmax);
}

// out and lse of one (token, head) per workgroup, from its splits' unnormalised sums, their
// maxima (in powers of two) and totals: 8 elements per thread, the splits dealt over as
// many groups of d / 8 threads as there are, which are then added in order.  (With one
// group per row, whose threads walk all splits, one query of 40 heads on 16384 keys of 8
// took 51 us at 64 splits, longer than the work that is split; so, 21 us.)
__global__ void __launch_bounds__(256) attention_forward_join_kernel(const AttentionArgs a)
{
    __shared__ float4 part[256][2];
    const int64_t rows = (int64_t)a.tq * a.hq, row = blockIdx.x;
    const int head = (int)(row / a.tq), token = (int)(row % a.tq);
    if (a.cu_q && (token < a.cu_q[0] || token >= a.cu_q[a.batch])) return;   // of no sequence
    const int per = a.d / 8, groups = 256 / per, k = threadIdx.x / per, c = threadIdx.x % per * 8;
    float m = -kInf, l = 0.0f;
    for (int s = threadIdx.x & 63; s < a.splits; s += 64) m = fmaxf(m, a.tops[s * rows + row].x);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
    const float use = m == -kInf ? 0.0f : m;
    for (int s = threadIdx.x & 63; s < a.splits; s += 64) {
        const float2 x = a.tops[s * rows + row];
        l = fmaf(x.y, __builtin_amdgcn_exp2f(x.x - use), l);
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) l += __shfl_xor(l, off, 64);
    float t[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (k < groups)
#pragma unroll 4
        for (int s = k; s < a.splits; s += groups) {
            const float by = __builtin_amdgcn_exp2f(a.tops[s * rows + row].x - use);
            const float4* p = reinterpret_cast<const float4*>(a.partial + (s * rows + row) * a.d + c);
            const float4 u = p[0], v = p[1];
            const float e[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = fmaf(e[i], by, t[i]);
        }
    part[threadIdx.x][0] = make_float4(t[0], t[1], t[2], t[3]);
    part[threadIdx.x][1] = make_float4(t[4], t[5], t[6], t[7]);
    __syncthreads();
    uint32_t top = 0;
    if (k == 0) {
        for (int g = 1; g < groups; ++g) {
            const float4 u = part[g * per + threadIdx.x][0], v = part[g * per + threadIdx.x][1];
            const float e[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] += e[i];
        }
        const float by = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = bf16_pair(t[2 * i] * by, t[2 * i + 1] * by);
            top = max(max(top, w[i] & 0x7FFF0000u), w[i] << 16 & 0x7FFFFFFFu);
        }
        *reinterpret_cast<uint4*>(a.out + (int64_t)token * a.out_row + (int64_t)head * a.out_head + c) =
            make_uint4(w[0], w[1], w[2], w[3]);
        if (c == 0) a.lse[row] = l == 0.0f ? -kInf : (use + __builtin_amdgcn_logf(l)) * kLn2;
    }
    if (a.absmax) block_max_to_global(top, a.absmax);
}

// ---------------------------------------------------------------------- backward

// dq: 32 queries per wave, keys and values streamed.  A wave first takes its queries'
// delta and leaves it for the dk/dv kernel: stats[0][head][token] = lse in powers of two
// (+inf where the row is empty, so that every p of it is 0), stats[1][head][token] = delta.
// 4096 causal tokens, 32 heads of 128: 202 us in a kernel trace (three products: 1.02 PFLOP/s).
template <int DT>
__global__ void __launch_bounds__(kAttThreads, 2) attention_dq_kernel(const AttentionArgs a)
{
    constexpr int kTile = kKeys * DT * 2;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[4 * kTile];
    int t, unit;
    deal(blockIdx.x, a.hq * a.splits, t, unit);
    const int head = unit / a.splits, split = unit % a.splits;
    const Place pl = find_tile(a, a.tiles - 1 - a.tile0 - t, 0);
    if (!pl.any) return;
    const int lane = threadIdx.x & 63, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
    const int khead = head / (a.hq / a.hk);

    const int q_wave = pl.first + wave * 32, qi = q_wave + (lane & 31);
    const bool mine = qi < pl.nq;
    const int shift = pl.nk - pl.nq;
    const int see = a.causal ? min(pl.nk, qi + shift + 1) : pl.nk;
    const int see_first = a.causal ? min(pl.nk, q_wave + shift + 1) : pl.nk;
    const int see_last = a.causal ? min(pl.nk, q_wave + 31 + shift + 1) : pl.nk;
    const int end = a.causal ? min(pl.nk, min(pl.first + kOwn, pl.nq) + shift) : pl.nk;
    const int steps = end > 0 ? (end + kKeys - 1) / kKeys : 0;

    Frag q[DT / 16], g[DT / 16];
    load_own<DT>(q, a.q + (int64_t)(pl.q0 + qi) * a.q_row + (int64_t)head * a.q_head, a.d, mine);
    load_own<DT>(g, a.dout + (int64_t)(pl.q0 + qi) * a.dout_row + (int64_t)head * a.dout_head, a.d, mine);
    float lse = kInf, delta = 0.0f;
    {
        Frag o[DT / 16];
        load_own<DT>(o, a.out + (int64_t)(pl.q0 + qi) * a.out_row + (int64_t)head * a.out_head, a.d, mine);
#pragma unroll
        for (int ch = 0; ch < DT / 16; ++ch)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                delta = fmaf(bf16_lo(o[ch].w[i]), bf16_lo(g[ch].w[i]), fmaf(bf16_hi(o[ch].w[i]), bf16_hi(g[ch].w[i]), delta));
        delta += partner(delta);
        if (mine) {
            lse = a.lse[(int64_t)head * a.tq + pl.q0 + qi];
            lse = lse == -kInf ? kInf : lse * kLog2e;
        }
        asm volatile("" : "+v"(lse));
    }

    Stream<DT, kKeys> ks, vs;
    ks.init(a.k + (int64_t)pl.k0 * a.k_row + (int64_t)khead * a.k_head, a.k_row, pl.nk, a.d);
    vs.init(a.v + (int64_t)pl.k0 * a.v_row + (int64_t)khead * a.v_head, a.v_row, pl.nk, a.d);
    Tile<DT> tile;
    tile.init(lds0);
    const float c = a.scale * kLog2e;
    af32x16 dq[DT / 32];
#pragma unroll
    for (int db = 0; db < DT / 32; ++db) dq[db] = af32x16{0};

    // Where at most two tiles of keys are seen, delta is taken again as the sum of p dp:
    // out is rounded to bf16, which weighs most where it is the average of few values (in
    // a causal sequence's first rows, whose gradients are its largest).
    if (steps == 1 || steps == 2) {
        for (int s = 0; s < steps; ++s) {
            ks.issue(s * kKeys, lds0 + s * 2 * kTile, wave);
            vs.issue(s * kKeys, lds0 + s * 2 * kTile + kTile, wave);
        }
        __builtin_amdgcn_s_waitcnt(wait_loads(0));
        __syncthreads();
        float sum = 0.0f;
#pragma unroll 1
        for (int u = 0; u < 2 * steps && 32 * u < see_last; ++u) {
            const uint32_t at = (uint32_t)(u / 2 * 2 * kTile + u % 2 * 32 * DT * 2);
            af32x16 p = af32x16{0}, dp = af32x16{0};
#pragma unroll
            for (int ch = 0; ch < DT / 16; ++ch) {
                Frag x, y;
                x.u = *(const lds_u32x4*)(uintptr_t)(tile.plain[ch] + at);
                y.u = *(const lds_u32x4*)(uintptr_t)(tile.plain[ch] + at + kTile);
                p = mma(x, q[ch], p);
                dp = mma(y, g[ch], dp);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float x = __builtin_amdgcn_exp2f(fmaf(p[i], c, -lse)) * dp[i];
                sum += 32 * u + 8 * (i / 4) + 4 * h + i % 4 < see ? x : 0.0f;
            }
        }
        delta = sum + partner(sum);
    }
    if (mine && split == 0)
        a.stats[(h ? (int64_t)a.tq * a.hq : 0) + (int64_t)head * a.tq + pl.q0 + qi] = h ? delta : lse;

    const bool loaded = steps <= 2;       // with their tiles in LDS already, in place (no split then)
    const int s_begin = loaded ? 0 : (int)((int64_t)steps * split / a.splits);
    const int s_end = !loaded ? (int)((int64_t)steps * (split + 1) / a.splits) : split == 0 ? steps : 0;
    const int load_end = loaded ? 0 : s_end;
    if (s_begin < load_end) {
        ks.issue(s_begin * kKeys, lds0, wave);
        vs.issue(s_begin * kKeys, lds0 + kTile, wave);
    }
    auto step = [&](auto stage, auto fine, int s) {
        constexpr int at = stage.value * 2 * kTile, to = (2 - stage.value * 2) * kTile;
        __builtin_amdgcn_s_waitcnt(0x0F70);
        __syncthreads();
        if (s + 1 < load_end) {
            ks.issue((s + 1) * kKeys, lds0 + to, wave);
            vs.issue((s + 1) * kKeys, lds0 + to + kTile, wave);
        }
        const int j0 = s * kKeys;
        if (j0 >= see_last) return;
        const bool masked = j0 + kKeys > see_first;
        // as in the forward: per block of 32 keys the scores and dp (k and v rows in turn),
        // then dq (k columns)
        constexpr int kS = DT / 8, kB = kS + DT / 16, kAll = 2 * kB, kAhead = 4;
        Frag r[kAhead];
        auto fetch = [&](int t) __attribute__((always_inline)) {
            const int kb = t / kB, x = t % kB;
            if (t >= kAll) return;
            if (x < kS) r[t % kAhead] = tile.rows(at + x % 2 * kTile, kb, x / 2);
            else r[t % kAhead] = tile.cols(at, kb, (x - kS) / (DT / 32), (x - kS) % (DT / 32));
        };
#pragma unroll
        for (int t = 0; t < kAhead; ++t) fetch(t);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            af32x16 p = af32x16{0}, dp = af32x16{0};
#pragma unroll
            for (int x = 0; x < kS; ++x) {
                const int t = kb * kB + x;
                if (x % 2 == 0) p = mma(r[t % kAhead], q[x / 2], p);
                else dp = mma(r[t % kAhead], g[x / 2], dp);
                fetch(t + kAhead);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                p[i] = __builtin_amdgcn_exp2f(fmaf(p[i], c, -lse));
                dp[i] = p[i] * (dp[i] - delta);
            }
            if (masked) {
                const int see0 = see - j0 - 4 * h;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (32 * kb + 8 * (i / 4) + i % 4 >= see0) dp[i] = 0.0f;
            }
            Frag f[2], l[2];
            to_operands(dp, f);
            if (fine.value) to_residuals(dp, f, l);
#pragma unroll
            for (int x = kS; x < kB; ++x) {
                const int t = kb * kB + x, db = (x - kS) % (DT / 32);
                dq[db] = mma(r[t % kAhead], f[(x - kS) / (DT / 32)], dq[db]);
                if (fine.value) dq[db] = mma(r[t % kAhead], l[(x - kS) / (DT / 32)], dq[db]);
                fetch(t + kAhead);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    // Where few keys are seen, single ds make up the result, and their rounding adds as much
    // to its error as its own does (2.4e-3 of the gradients' norm instead of 1.7e-3): what
    // the rounding leaves off is then taken as a further operand.  Over more keys it would
    // cost a fifth of the kernel's products.
    if (loaded) {
        if (s_begin < s_end) step(std::integral_constant<int, 0>{}, std::true_type{}, s_begin);
        if (s_begin + 1 < s_end) step(std::integral_constant<int, 1>{}, std::true_type{}, s_begin + 1);
    } else {
        for (int s = s_begin; s < s_end; s += 2) {
            step(std::integral_constant<int, 0>{}, std::false_type{}, s);
            if (s + 1 < s_end) step(std::integral_constant<int, 1>{}, std::false_type{}, s + 1);
        }
    }
    if (a.splits > 1) {
        const int64_t row = ((int64_t)split * a.tq + pl.q0 + qi) * a.hq + head;
        store_partial<DT>(dq, a.partial + row * a.d, a.d, mine);
        return;
    }
    const uint32_t top = store_own<DT>(dq, a.scale, a.dq + (int64_t)(pl.q0 + qi) * a.dq_row + (int64_t)head * a.dq_head,
                                       a.d, mine);
    if (a.absmax) block_max_to_global(top, a.absmax);
}

constexpr int kQueries = 32;              // queries per streamed tile, dk/dv
constexpr int kRing = 4;                  // stages of them
constexpr int keys_waves(int dt) { return dt == 128 ? 8 : 4; }

// (The workgroups of sequences of at most 128 keys take, like dq's, what the rounding of p and
// ds leaves off; the loop for it is compiled apart, as the main one has no register to spare.)
// dk, dv: 32 keys per wave; the queries of every head that shares the key head are
// streamed, with their dout, lse and delta, three tiles ahead.  A wave's keys stay in
// registers; its values are read from a fixed tile in LDS (keeping them in registers too
// would leave the two accumulators no room at two waves per SIMD).  At head dimension 128
// a workgroup is 8 waves: they share each streamed tile, and the LDS of two workgroups of
// 4 makes room for the ring (with two stages of it, and a barrier to each 32 queries, the
// waves waited for their loads for half of the time).
// 4096 causal tokens, 32 heads of 128: 292 us in a kernel trace (four products: 0.94 PFLOP/s);
// this and dq's kernel untraced 466 (seven products: 1.03).
// chunks > 1: the steps are dealt over that many workgroups, each of which leaves fp32
// partial sums [chunk][dk, dv][token][head][d].
template <int DT>
__global__ void __launch_bounds__(64 * keys_waves(DT), DT == 64 ? 3 : 2) attention_dkv_kernel(const AttentionArgs a)
{
    constexpr int WAVES = keys_waves(DT), kMine = 32 * WAVES;
    constexpr int kTile = kQueries * DT * 2, kOwnTile = kMine * DT * 2, kStat = 512;
    using Q = Stream<DT, kQueries, WAVES>;
    constexpr int kLoads = 2 * Q::kLoads + 1;              // per wave and step
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kRing * 2 * kTile + kOwnTile + kRing * kStat];
    int t, unit;
    deal(blockIdx.x, a.hk * a.chunks, t, unit);
    const int khead = unit / a.chunks, chunk = unit % a.chunks;
    Place pl = find_tile(a, a.tile0 + t, 1, kMine);        // a sequence's first keys are seen by most
    if (!pl.any) return;
    // queries that see nothing come first; they are not read, as 0 times whatever they hold
    // need not be 0
    const int unseeing = a.causal ? max(0, pl.nq - pl.nk) : 0;
    pl.q0 += unseeing;
    pl.nq -= unseeing;
    const int lane = threadIdx.x & 63, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t lds0 = (uint32_t)(uintptr_t)lds, stat0 = lds0 + kRing * 2 * kTile + kOwnTile;
    const int group = a.hq / a.hk;

    const int k_wave = pl.first + wave * 32, ki = k_wave + (lane & 31);
    const bool mine = ki < pl.nk;
    const int shift = pl.nk - pl.nq;
    // the first query that sees this lane's key, the wave's first key, its last, the workgroup's first
    const int lane_from = (a.causal ? max(0, ki - shift) : 0) - 4 * h;   // (4 h: its first row of a block)
    const int from_first = a.causal ? max(0, k_wave - shift) : 0;
    const int from_last = a.causal ? max(0, k_wave + 31 - shift) : 0;
    const int begin = a.causal ? max(0, pl.first - shift) / kQueries : 0;
    const int last = (pl.nq + kQueries - 1) / kQueries;
    const int per = max(0, last - begin);
    const int64_t all = (int64_t)per * group;
    const int s_begin = (int)(all * chunk / a.chunks), s_end = (int)(all * (chunk + 1) / a.chunks);

    Frag k[DT / 16];
    load_own<DT>(k, a.k + (int64_t)(pl.k0 + ki) * a.k_row + (int64_t)khead * a.k_head, a.d, mine);
    Tile<DT> tile;
    tile.init(lds0);
    const uint32_t own = (uint32_t)(kRing * 2 * kTile + wave * 32 * DT * 2);   // the wave's values
    Q qs, gs;
    qs.init(a.q + (int64_t)pl.q0 * a.q_row, a.q_row, pl.nq, a.d);
    gs.init(a.dout + (int64_t)pl.q0 * a.dout_row, a.dout_row, pl.nq, a.d);
    const uint8_t* q_base = qs.base;
    const uint8_t* g_base = gs.base;
    const uint32_t stat_off = lane < 32 ? lane * 4u : kPastBuffer;
    // even waves bring the tile's lse, odd ones its delta (the same bytes each)
    const float* stat_base = a.stats + (wave & 1 ? (int64_t)a.tq * a.hq : 0) + pl.q0;

    af32x16 dk[DT / 32], dv[DT / 32];
#pragma unroll
    for (int db = 0; db < DT / 32; ++db) dk[db] = dv[db] = af32x16{0};
    const float c = a.scale * kLog2e;

    // step s: query tile begin + s % per of head khead * group + s / per.  Past the last step
    // its loads are repeated, into a stage that is read no more, so that the count of loads
    // in flight stays the same.
    auto issue = [&](int s, int stage) __attribute__((always_inline)) {
        s = min(s, s_end - 1);
        const int head = khead * group + s / per, row0 = (begin + s % per) * kQueries;
        const uint32_t to = lds0 + (uint32_t)stage * 2 * kTile;
        qs.base = q_base + (int64_t)head * a.q_head * 2;
        gs.base = g_base + (int64_t)head * a.dout_head * 2;
        qs.issue(row0, to, wave);
        gs.issue(row0, to + kTile, wave);
        const au32x4 desc = descriptor(reinterpret_cast<const uint8_t*>(stat_base + (int64_t)head * a.tq + row0),
                                       stream_bytes(pl.nq - row0, 4));
        buffer4_to_lds(stat_off, desc, __builtin_amdgcn_readfirstlane(stat0 + (uint32_t)(stage * kStat + (wave & 1) * 256)));
    };

    auto step = [&](auto stage, auto fine, int s) __attribute__((always_inline)) {
        constexpr int at = stage.value * 2 * kTile;
        __builtin_amdgcn_s_waitcnt(wait_loads((kRing - 2) * kLoads));     // this wave's loads of step s
        __syncthreads();                                   // everyone's; step s - 1 is read
        issue(s + kRing - 1, (stage.value + kRing - 1) % kRing);
        const int i0 = (begin + s % per) * kQueries;
        if (i0 + kQueries <= from_first || k_wave >= pl.nk) return;   // no query of the tile sees a key of the wave
        // as in the forward: the scores and dp (q and dout rows in turn), then dv and dk
        // (dout and q columns in turn)
        constexpr int kS = DT / 8, kAll = kS + DT / 8, kAhead = 2;   // 4 spill
        Frag r[kAhead], v[2];
        auto fetch = [&](int t) __attribute__((always_inline)) {
            if (t < kS) {
                r[t % kAhead] = tile.rows(at + t % 2 * kTile, 0, t / 2);
                if (t % 2) v[t / 2 % 2].u = *(const lds_u32x4*)(uintptr_t)(tile.plain[t / 2] + own);
            } else if (t < kAll) {
                const int x = t - kS;
                r[t % kAhead] = tile.cols(at + (1 - x % 2) * kTile, 0, x / 2 / (DT / 32), x / 2 % (DT / 32));
            }
        };
#pragma unroll
        for (int t = 0; t < kAhead; ++t) fetch(t);
        af32x16 p = af32x16{0}, dp = af32x16{0};
#pragma unroll
        for (int t = 0; t < kS; ++t) {
            if (t % 2 == 0) p = mma(r[t % kAhead], k[t / 2], p);
            else dp = mma(r[t % kAhead], v[t / 2 % 2], dp);
            fetch(t + kAhead);
            __builtin_amdgcn_sched_barrier(0);
        }
        // (keys past the sequence's end are columns of their own, which are not stored)
        const bool masked = i0 < from_last;
        const lds_f32x4* stat = (const lds_f32x4*)(uintptr_t)(stat0 + stage.value * kStat + 16 * h);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const af32x4 ls = stat[2 * b], de = stat[2 * b + 16];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 4 * b + e;
                p[i] = __builtin_amdgcn_exp2f(fmaf(p[i], c, -ls[e]));
                dp[i] = p[i] * (dp[i] - de[e]);
            }
        }
        if (masked) {
            const int from0 = lane_from - i0;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (8 * (i / 4) + i % 4 < from0) p[i] = dp[i] = 0.0f;
        }
        Frag f[2], e[2], fl[2], el[2];
        to_operands(p, f);
        to_operands(dp, e);
        if (fine.value) {
            to_residuals(p, f, fl);
            to_residuals(dp, e, el);
        }
#pragma unroll
        for (int t = kS; t < kAll; ++t) {
            const int x = t - kS, ch = x / 2 / (DT / 32), db = x / 2 % (DT / 32);
            if (x % 2 == 0) dv[db] = mma(r[t % kAhead], f[ch], dv[db]);
            else dk[db] = mma(r[t % kAhead], e[ch], dk[db]);
            if (fine.value) {
                if (x % 2 == 0) dv[db] = mma(r[t % kAhead], fl[ch], dv[db]);
                else dk[db] = mma(r[t % kAhead], el[ch], dk[db]);
            }
            fetch(t + kAhead);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    if (s_begin < s_end) {
        Stream<DT, kMine, WAVES> vs;
        vs.init(a.v + (int64_t)pl.k0 * a.v_row + (int64_t)khead * a.v_head, a.v_row, pl.nk, a.d);
        vs.issue(pl.first, lds0 + kRing * 2 * kTile, wave);
#pragma unroll
        for (int i = 0; i < kRing - 1; ++i) issue(s_begin + i, i);
        auto walk = [&](auto fine) __attribute__((always_inline)) {
            for (int s = s_begin; s < s_end; s += kRing) {
                step(std::integral_constant<int, 0>{}, fine, s);
                if (s + 1 < s_end) step(std::integral_constant<int, 1>{}, fine, s + 1);
                if (s + 2 < s_end) step(std::integral_constant<int, 2>{}, fine, s + 2);
                if (s + 3 < s_end) step(std::integral_constant<int, 3>{}, fine, s + 3);
            }
        };
        // as for dq: with few keys, what the rounding of p and ds leaves off is taken too
        if (pl.nk <= 2 * kKeys) walk(std::true_type{});
        else walk(std::false_type{});
        __builtin_amdgcn_s_waitcnt(wait_loads(0));         // no load outlives the workgroup's LDS
    }
    if (a.chunks > 1) {
        const int64_t row = ((int64_t)(pl.k0 + ki) * a.hk + khead) * a.d, whole = (int64_t)a.tk * a.hk * a.d;
        store_partial<DT>(dk, a.partial + (int64_t)(2 * chunk) * whole + row, a.d, mine);
        store_partial<DT>(dv, a.partial + (int64_t)(2 * chunk + 1) * whole + row, a.d, mine);
        return;
    }
    uint32_t top = store_own<DT>(dk, a.scale, a.dk + (int64_t)(pl.k0 + ki) * a.dk_row + (int64_t)khead * a.dk_head, a.d, mine);
    top = max(top, store_own<DT>(dv, 1.0f, a.dv + (int64_t)(pl.k0 + ki) * a.dv_row + (int64_t)khead * a.dv_head, a.d, mine));
    if (a.absmax) block_max_to_global(top, a.absmax);
}

// Gradients from their partial sums [part][which][token][head][d], added in order: 8
// elements per thread.  dq (one tensor, a.splits parts), or dk and dv (a.chunks parts).
__global__ void __launch_bounds__(256) attention_join_kernel(const AttentionArgs a, int queries)
{
    const int tokens = queries ? a.tq : a.tk, heads = queries ? a.hq : a.hk, parts = queries ? a.splits : a.chunks;
    const int per_row = a.d / 8, which = blockIdx.y, tensors = gridDim.y;
    const int64_t whole = (int64_t)tokens * heads * a.d, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = i / per_row;
    const int c = (int)(i % per_row) * 8, head = (int)(row % heads), token = (int)(row / heads);
    const int* cu = queries ? a.cu_q : a.cu_k;
    int from = 0, upto = tokens;          // the tokens that belong to a sequence
    if (cu) {
        from = min(max(cu[0], 0), tokens);
        upto = min(max(cu[a.batch], 0), tokens);
    }
    uint32_t top = 0;
    if (i < whole / 8 && token >= from && token < upto) {
        const float* p = a.partial + which * whole + row * a.d + c;
        float t[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
        for (int s = 0; s < parts; ++s, p += tensors * whole) {
            const float4 x = reinterpret_cast<const float4*>(p)[0], y = reinterpret_cast<const float4*>(p)[1];
            const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] += v[e];
        }
        const float by = which ? 1.0f : a.scale;          // dq and dk carry the scale
        uint16_t* out = queries ? a.dq + (int64_t)token * a.dq_row + (int64_t)head * a.dq_head
                        : which ? a.dv + (int64_t)token * a.dv_row + (int64_t)head * a.dv_head
                                : a.dk + (int64_t)token * a.dk_row + (int64_t)head * a.dk_head;
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = bf16_pair(t[2 * e] * by, t[2 * e + 1] * by);
            top = max(max(top, w[e] & 0x7FFF0000u), w[e] << 16 & 0x7FFFFFFFu);
        }
        *reinterpret_cast<uint4*>(out + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (a.absmax) block_max_to_global(top, a.absmax);
}

// ---------------------------------------------------------------------- launches

// At most this many tiles: each sequence adds less than one to total / rows.
static int64_t tile_bound(int64_t total, int batch, int rows) { return total / rows + batch; }

static int key_rows(int d) { return 32 * keys_waves(d <= 64 ? 64 : 128); }

bool attention_grid_ok(int64_t tokens, int batch, int heads)
{
    return tile_bound(tokens, batch, kOwn) * heads <= 0x7FFFFFFF / 8;
}

// Workgroups that share the steps of one tile of keys.  With less than two tiles per CU
// (few key heads, or short sequences of many queries) the causal mask leaves the first
// tiles' workgroups running alone: their steps are then split, at 8 or more to a chunk
// (8192 causal tokens, 40 query and 8 key heads of 128: 264 workgroups).  The backward at
// 32 or more to a chunk and at 8, MI355X, heads of 128: 1024 tokens of 8 query and 2 key
// heads 92 / 62 us, 512 of 16 and 4 84 / 58, 2048 of 8 and 8 121 / 118; at 4, 1024 tokens
// of 16 and 16 heads took 86 instead of 71.
static int key_chunks(int64_t tq, int64_t tk, int hq, int hk, int d, int batch)
{
    const int64_t tiles = tile_bound(tk, batch, key_rows(d)) * hk, want = 2 * (int64_t)device_cu_count();
    const int64_t steps = (tq / batch + kQueries - 1) / kQueries * (hq / hk);   // of a sequence of average length
    return (int)std::max<int64_t>(1, std::min<int64_t>({(want + tiles - 1) / tiles, steps / 8, 16}));
}

// Workgroups that share the keys of one tile of queries, in the forward and for dq: where
// there are fewer tiles than CUs and the keys are many, up to two workgroups per CU, at 4 or
// more streamed tiles (256 keys) each.  Unsplit / split, MI355X, heads of 128: 100 queries
// of 8 heads on 4000 keys, forward 72 / 19 us, backward 107 / 46; one query of 32 heads on
// 16384 keys 270 / 47 and 493 / 231; 512 queries of 4 heads on 4096 keys 73 / 28 and 124 / 63.
// The rule goes by averages, and is measured on even batches: one query on 131072 keys among
// 31 on 500 (32 and 8 heads) is not split and takes 2300 us, 32 queries on as many keys in
// all, 4577 each, 124.
static int query_splits(int64_t tq, int64_t tk, int hq, int batch, int group)
{
    const int64_t tiles = tile_bound(tq * group, batch, kOwn) * (hq / group), cus = device_cu_count();
    if (tiles > cus) return 1;
    const int64_t steps = tk / batch / kKeys;             // of a sequence of average length
    return (int)std::max<int64_t>(1, std::min<int64_t>({2 * cus / tiles, steps / 4, 128}));
}

// Query heads that share a tile of the forward: all that share a key head, where a
// sequence's queries are few (half a tile on average); else each has tiles of its own.
// MI355X, one query per sequence, heads of 128, apart / together: 64 sequences of 4096 keys,
// 32 and 8 heads 394 / 193 us (1.07 GB of keys and values, 5.6 TB/s); 8 of 8192, 40 and 8
// 157 / 61; one of 16384, 40 and 8 36 / 21.  By the average again: 63 single queries on 4096 keys
// each take 191 us (32 and 8 heads), a prompt of 8192 tokens 524, both packed together, where
// no head is shared, 874.
static int tile_group(int64_t tq, int hq, int hk, int batch)
{
    const int group = hq / hk;
    return tq / batch <= kOwn / 2 && tq * group < 0x7FFFFF00 ? group : 1;   // rows of a sequence are counted in int
}

static int64_t up4(int64_t n) { return (n + 3) / 4 * 4; }   // fp32 values, so that what follows is 16-byte aligned

int64_t attention_forward_workspace(int64_t tq, int64_t tk, int hq, int hk, int d, int batch)
{
    const int64_t splits = query_splits(tq, tk, hq, batch, tile_group(tq, hq, hk, batch));
    return splits > 1 ? 4 * splits * (up4(2 * tq * hq) + tq * hq * d) : 0;
}

int64_t attention_backward_workspace(int64_t tq, int64_t tk, int hq, int hk, int d, int batch)
{
    const int64_t chunks = key_chunks(tq, tk, hq, hk, d, batch), splits = query_splits(tq, tk, hq, batch, 1);
    // the partial sums of dq are joined before those of dk and dv are written
    return 4 * (up4(2 * tq * hq) + std::max(chunks > 1 ? 2 * chunks * tk * hk * d : 0, splits > 1 ? splits * tq * hq * d : 0));
}

// `units` workgroups of each of the a.tiles tiles, in as many launches as their threads take.
static hipError_t launch_tiles(void (*kernel)(AttentionArgs), AttentionArgs a, int64_t units, int threads, hipStream_t stream)
{
    const int64_t most = max_workgroups(threads) / units;
    for (int64_t first = 0; first < a.tiles; first += most) {
        a.tile0 = (int)first;
        const hipError_t e = launch(kernel, dim3((unsigned)(std::min(most, a.tiles - first) * units)), dim3(threads), stream, a);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_attention_forward(const AttentionArgs& args, void* workspace, hipStream_t stream)
{
    AttentionArgs a = args;
    a.group = tile_group(a.tq, a.hq, a.hk, a.batch);
    a.splits = query_splits(a.tq, a.tk, a.hq, a.batch, a.group);
    a.tops = static_cast<float2*>(workspace);
    a.partial = static_cast<float*>(workspace) + a.splits * up4(2 * (int64_t)a.tq * a.hq);
    a.tiles = (int)tile_bound((int64_t)a.tq * a.group, a.batch, kOwn);
    const hipError_t e = launch_tiles(a.d <= 64 ? attention_forward_kernel<64> : attention_forward_kernel<128>, a,
                                      (int64_t)(a.hq / a.group) * a.splits, kAttThreads, stream);
    if (e != hipSuccess || a.splits == 1) return e;
    return launch(attention_forward_join_kernel, dim3((unsigned)((int64_t)a.tq * a.hq)), dim3(256), stream, a);
}

hipError_t launch_attention_backward(const AttentionArgs& args, hipStream_t stream)
{
    AttentionArgs a = args;
    a.chunks = key_chunks(a.tq, a.tk, a.hq, a.hk, a.d, a.batch);
    a.splits = query_splits(a.tq, a.tk, a.hq, a.batch, 1);
    a.partial = a.stats + up4(2 * (int64_t)a.tq * a.hq);
    auto join = [&](int queries) {
        const int64_t units = (queries ? (int64_t)a.tq * a.hq : (int64_t)a.tk * a.hk) * a.d / 8;
        return launch(attention_join_kernel, dim3((unsigned)((units + 255) / 256), queries ? 1 : 2), dim3(256), stream,
                      a, queries);
    };
    a.tiles = (int)tile_bound(a.tq, a.batch, kOwn);
    hipError_t e = launch_tiles(a.d <= 64 ? attention_dq_kernel<64> : attention_dq_kernel<128>, a, (int64_t)a.hq * a.splits,
                                kAttThreads, stream);
    if (e == hipSuccess && a.splits > 1) e = join(1);
    if (e != hipSuccess) return e;
    a.tiles = (int)tile_bound(a.tk, a.batch, key_rows(a.d));
    e = a.d <= 64 ? launch_tiles(attention_dkv_kernel<64>, a, (int64_t)a.hk * a.chunks, 64 * keys_waves(64), stream)
                  : launch_tiles(attention_dkv_kernel<128>, a, (int64_t)a.hk * a.chunks, 64 * keys_waves(128), stream);
    if (e != hipSuccess || a.chunks == 1) return e;
    return join(0);
}

}  // namespace fp8k
