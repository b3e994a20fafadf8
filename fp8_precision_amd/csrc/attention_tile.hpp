// attention_tile.hpp -- what the attention kernels' tiles in LDS, and their operands and
// results in registers, look like: shared by attention.hip, which streams bf16 tiles, and
// attention_cached.hip, which makes them of 8-bit codes.  attention.hip explains the layout.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

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

constexpr int kKeys = 64;                 // keys per tile of the forward and dq

// One tile of 64 keys and their values (at LDS offsets AT and AT + a tile's bytes) against a
// wave's 32 rows q: the scores, the running maximum m (mc: in powers of two) and sum l of
// each row, and its output o.  `see` keys of the tile are seen by the lane's row, which
// matters where `masked`; c is the score's factor in powers of two.
template <int DT, int AT>
__device__ __forceinline__ void attend_tile(const Tile<DT>& tile, const Frag (&q)[DT / 16], int see, bool masked, float c,
                                            float far, af32x16 (&o)[DT / 32], float& m, float& mc, float& l)
{
    constexpr int kTile = kKeys * DT * 2, at = AT;
    const int h = (threadIdx.x & 63) >> 5;
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
    if (masked) {
        const int see0 = see - 4 * h;             // register i: key 32 kb + 8 (i / 4) + i % 4 of what is left
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

}  // namespace

}  // namespace fp8k
