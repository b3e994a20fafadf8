// kv_cache.hip -- keys and values in a paged cache of E4M3 codes, for gfx950: written with a
// scale per page and head, and read back.
//
// A page's tokens of one head share a scale 2^e: value = code 2^e, e the least with
// max |x| <= 448 2^e over the finite x, held to -100 .. 119 (every value is then a normal
// bf16 number, so reading is exact).  A power of two costs a floating-point code no
// precision, and it lets a page grow: when a later token needs a larger e, the older codes
// are multiplied by a power of two, exact except where they become subnormal and are rounded
// once more.  The scale stays a byte, e + 127, as the block-scaled formats have it.
//
// Bound by memory, 2 bytes read and 1 written per element (or the reverse): 8192 tokens of 8
// heads of 128 are written in 11.4 us (4.4 TB/s; the kernel begins with dependent reads: bounds
// and length, then table and tokens, then the page's scale), 32768 read in 34 (5.9).  For a
// single new token per sequence that chain and the launch are all: 3.4 us in a chain of calls.
#include <algorithm>

#include "fp8_device.hpp"
#include "fp8_internal.hpp"
#include "kv_cache.hpp"

namespace fp8k {

namespace {

typedef unsigned short ku16x2 __attribute__((ext_vector_type(2)));
typedef short ki16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 kb16x2 __attribute__((ext_vector_type(2)));
typedef unsigned int ku32x2 __attribute__((ext_vector_type(2)));

constexpr int kCacheThreads = 256;
// New tokens per sequence, on average, up to which a wave takes a piece; beyond, a workgroup does.
// 512 sequences, 8 heads of 128, in a chain of calls, a wave / a workgroup: written, 1 token each
// 5.2 / 13.0 us, 16 13.3 / 23.5, 32 25.0 / 24.5, 64 41.0 / 35.2; read 1 6.3 / 15.4, 32 26.5 / 41.1; of
// 64 sequences, 64 tokens each, 9.6 / 8.7.  Uneven ones are told by their average too, which a prompt's full pages among
// few single tokens pay for: written, 500 tokens among 31 single ones 12.7 / 4.8, 2000 among 127 13.2 / 7.7, 8000 among
// 511 23.9 / 25.3; read 4.6 / 4.0, 5.8 / 9.5, 18.2 / 35.7.
constexpr int kWriteWave = 16, kReadWave = 32;
constexpr int kHeld = 4;                   // 16-byte groups of a piece's keys, and of its values, that a thread keeps in registers

// The scale's exponent for a largest magnitude of these fp32 bits: 448 = 1.75 2^8.
__device__ __forceinline__ int exponent_for(uint32_t top)
{
    const int e = (int)(top >> 23) - 135 + ((top & 0x7FFFFFu) > 0x600000u);
    return min(max(e, kCacheLeastE), kCacheMostE);
}

struct Piece {
    CachePiece at;
    int b;
    int64_t token;      // the first token in the call's tensors
};

// Piece `item` of the call.  Every wave finds its own: 64 sequences are compared at a time,
// and the last comparison's lanes hold the sequence's bounds and length.
__device__ __forceinline__ Piece find_piece(const CacheArgs& a, int64_t item)
{
    const int lane = threadIdx.x & 63;
    Piece p{};
    int from, count, length;
    int64_t local;
    if (!a.cu) {
        count = a.each;
        const int64_t per = pieces_of(count, a.shift);
        p.b = (int)min(item / per, (int64_t)a.batch);
        if (p.b == a.batch) return p;
        local = item % per;
        from = p.b * count;
        length = a.lengths[p.b];
    } else {
        int first = 0, width = a.batch, lo = 0, hi = 0, n = 0, l = 0;
        while (true) {
            const int step = (width + 63) / 64, c = first + lane * step;
            const bool inside = c < first + width;
            if (inside) {
                lo = min(max(a.cu[c], 0), (int)a.tokens);
                hi = min(max(a.cu[c + 1], 0), (int)a.tokens);
                n = a.lengths[c];
            }
            const uint64_t all = __ballot(inside && piece_base(lo, c, a.shift) <= item);
            if (!all) return p;
            l = 63 - __clzll((long long)all);
            first += l * step;
            if (step == 1) break;
            width = min(step, width - l * step);
        }
        p.b = first;
        from = __builtin_amdgcn_readlane(lo, l);
        count = max(__builtin_amdgcn_readlane(hi, l) - from, 0);
        length = __builtin_amdgcn_readlane(n, l);
        local = item - piece_base(from, p.b, a.shift);
    }
    p.at = cache_piece(count, first_position(length, count, a.blocks, a.shift), local, a.shift);
    p.token = (int64_t)from + p.at.skip;
    return p;
}

// Its page in the pool; -1: none.
__device__ __forceinline__ int64_t page_of(const CacheArgs& a, const Piece& p)
{
    if (p.at.block < 0 || p.at.block >= a.blocks) return -1;
    const int at = a.table[(int64_t)p.b * a.blocks + p.at.block];
    return at >= 0 && at < a.pages ? at : -1;
}

// The larger of m's halves and the magnitudes of 8 bf16 (as 16-bit patterns, NaN above infinity).
__device__ __forceinline__ ku16x2 raw_top(const uint4& x, ku16x2 m)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(ku16x2, w[i] & 0x7FFF7FFFu));
    return m;
}

// The largest finite magnitude (fp32 bits) of 8 bf16.
__device__ __forceinline__ uint32_t finite_top(const uint4& x)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t hi = w[i] & 0x7FFF0000u, lo = w[i] << 16 & 0x7FFFFFFFu;
        top = max(top, hi >= 0x7F800000u ? 0u : hi);
        top = max(top, lo >= 0x7F800000u ? 0u : lo);
    }
    return top;
}

// The codes of 8 finite bf16 of at most 448 2^e, by = 2^e: the conversion divides by it.
__device__ __forceinline__ uint2 quant8_finite(const uint4& x, float by)
{
    ki16x2 a{0, 0}, b{0, 0};
    a = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(a, __builtin_bit_cast(kb16x2, x.x), by, false);
    a = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(a, __builtin_bit_cast(kb16x2, x.y), by, true);
    b = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(b, __builtin_bit_cast(kb16x2, x.z), by, false);
    b = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(b, __builtin_bit_cast(kb16x2, x.w), by, true);
    return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
}

// 4 codes times a power of two, rounded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float by)
{
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    return enc4<0>(lo[0] * by, lo[1] * by, hi[0] * by, hi[1] * by);
}

// T threads (a wave, or the workgroup) write one piece of one head's keys and values: the
// largest magnitudes, the page's new exponents, the codes; and where the page was begun
// before and an exponent grows, its older codes.  What is finite (one 16-bit maximum per two
// elements tells) takes one conversion per two elements; the rest is saturated first.
template <int T>
__global__ void __launch_bounds__(kCacheThreads) kv_cache_write_kernel(const CacheArgs a)
{
    constexpr int kUnits = kCacheThreads / T;
    __shared__ uint32_t part[2][kCacheThreads / 64];
    __shared__ int was_e[2];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t unit = a.unit0 + (int64_t)blockIdx.x * kUnits + (T == 64 ? wave : 0);
    const int tid = T == 64 ? threadIdx.x & 63 : threadIdx.x;
    const int head = (int)(unit % a.heads);
    const Piece p = find_piece(a, unit / a.heads);
    if (p.at.count <= 0) return;

    const int d = a.d, per = d / 8, groups = p.at.count * per;
    const uint32_t inverse = (65536 + per - 1) / per;      // i / per for i < 2^12
    const uint16_t* const x[2] = {a.xk + p.token * a.xk_row + head * a.xk_head, a.xv + p.token * a.xv_row + head * a.xv_head};
    const int64_t row[2] = {a.xk_row, a.xv_row};
    auto load = [&](int values, int i) __attribute__((always_inline)) {
        const int r = (int)(i * inverse >> 16);
        return *reinterpret_cast<const uint4*>(x[values] + r * row[values] + (i - r * per) * 8);
    };
    uint4 held[2][kHeld];
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
#pragma unroll
        for (int v = 0; v < 2; ++v)
            if (tid + h * T < groups) held[v][h] = load(v, tid + h * T);
    // (the page is looked up while the tokens are on their way)
    const int64_t page = page_of(a, p), place = max(page, (int64_t)0) * a.heads + head;
    if (page < 0) return;
    uint8_t* const codes[2] = {a.k + (place << a.shift) * d, a.v + (place << a.shift) * d};
    uint8_t* const scale[2] = {a.k_scale + place, a.v_scale + place};
    int was[2] = {kCacheLeastE, kCacheLeastE};
    if (p.at.slot > 0 && (T == 64 || threadIdx.x == 0))
#pragma unroll
        for (int v = 0; v < 2; ++v) was[v] = cache_exponent(*scale[v]);

    uint32_t top[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        ku16x2 raw{0, 0};
#pragma unroll
        for (int h = 0; h < kHeld; ++h)
            if (tid + h * T < groups) raw = raw_top(held[v][h], raw);
        for (int i = tid + kHeld * T; i < groups; i += T) raw = raw_top(load(v, i), raw);
        top[v] = (uint32_t)max(raw[0], raw[1]) << 16;
        top[v] = wave_max_u32(top[v]);
    }
    auto whole_max = [&]() __attribute__((always_inline)) {
        if (T == 64) return;
        if ((threadIdx.x & 63) == 0) part[0][wave] = top[0], part[1][wave] = top[1];
        __syncthreads();
#pragma unroll
        for (int v = 0; v < 2; ++v)
            for (int w = 0; w < kCacheThreads / 64; ++w) top[v] = max(top[v], part[v][w]);
    };
    if (T != 64 && threadIdx.x == 0) was_e[0] = was[0], was_e[1] = was[1];
    whole_max();
    if (T != 64) was[0] = was_e[0], was[1] = was_e[1];
    const bool finite = max(top[0], top[1]) < 0x7F800000u;
    if (!finite) {
        // the scales are those of the finite values
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            top[v] = 0;
            for (int i = tid; i < groups; i += T) top[v] = max(top[v], finite_top(load(v, i)));
            top[v] = wave_max_u32(top[v]);
        }
        if (T != 64) __syncthreads();                      // part has been read
        whole_max();
    }

#pragma unroll
    for (int v = 0; v < 2; ++v) {
        const int e = max(exponent_for(top[v]), was[v]);
        const float s = two_to(-e);
        uint2* to = reinterpret_cast<uint2*>(codes[v] + p.at.slot * d);
        if (finite && e < kCacheMostE) {
            const float by = two_to(e);
#pragma unroll
            for (int h = 0; h < kHeld; ++h)
                if (tid + h * T < groups) to[tid + h * T] = quant8_finite(held[v][h], by);
            for (int i = tid + kHeld * T; i < groups; i += T) to[i] = quant8_finite(load(v, i), by);
        } else {
            for (int i = tid; i < groups; i += T) to[i] = quant8<0>(load(v, i), s);
        }
        if (p.at.slot > 0 && e > was[v]) {
            // 2^-126 and less leave no code but 0
            const float by = two_to(max(was[v] - e, -126));
            uint2* old = reinterpret_cast<uint2*>(codes[v]);
            for (int i = tid; i < p.at.slot * per; i += T) {
                uint2 w = old[i];
                w.x = rescale4(w.x, by);
                w.y = rescale4(w.y, by);
                old[i] = w;
            }
        }
        // (a byte outside e's range that does not grow stays: it counts as was)
        if (tid == 0 && (p.at.slot == 0 || e > was[v])) *scale[v] = (uint8_t)(e + 127);
    }
}

__device__ __forceinline__ uint2 read_past(const uint2* p)
{
    const ku32x2 w = __builtin_nontemporal_load(reinterpret_cast<const ku32x2*>(p));
    return make_uint2(w[0], w[1]);
}

// T threads read one piece of one head's keys or values; tokens with no place read as zeros.  The
// codes are read past the caches, which are left to what is written: MI355X, 32768 tokens of 8
// heads of 128 (134 MB out) 34 us (5.9 TB/s) and 65 with attention of 8 queries over them after
// it, with ordinary loads 44 and 67, with ordinary loads and stores past the caches 32 and 74;
// 16384 tokens, whose codes the last-level cache still has from the call before, 21 (18).
template <int T>
__global__ void __launch_bounds__(kCacheThreads) kv_cache_read_kernel(const CacheArgs a)
{
    constexpr int kUnits = kCacheThreads / T;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t unit = a.unit0 + (int64_t)blockIdx.x * kUnits + (T == 64 ? wave : 0);
    const int tid = T == 64 ? threadIdx.x & 63 : threadIdx.x;
    const int head = (int)(unit % a.heads), values = (int)(unit / a.heads % 2);
    const Piece p = find_piece(a, unit / (2 * a.heads));
    if (p.at.count <= 0) return;

    const int d = a.d, per = d / 8, groups = p.at.count * per;
    const uint32_t inverse = (65536 + per - 1) / per;
    uint16_t* const x = (values ? a.xv : a.xk) + p.token * (values ? a.xv_row : a.xk_row) + head * (values ? a.xv_head : a.xk_head);
    const int64_t row = values ? a.xv_row : a.xk_row;
    const int64_t page = page_of(a, p), place = max(page, (int64_t)0) * a.heads + head;
    const uint2* codes = reinterpret_cast<const uint2*>((values ? a.v : a.k) + (place << a.shift) * d + p.at.slot * d);
    const float s = page < 0 ? 1.0f : cache_scale((values ? a.v_scale : a.k_scale)[place]);

    for (int i0 = tid; i0 < groups; i0 += 4 * T) {
        uint2 w[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            w[h] = make_uint2(0, 0);
            if (i0 + h * T < groups && page >= 0) w[h] = read_past(codes + i0 + h * T);
        }
#pragma unroll
        for (int h = 0; h < 4; ++h)
            if (i0 + h * T < groups) {
                const int i = i0 + h * T, r = (int)(i * inverse >> 16);
                *reinterpret_cast<uint4*>(x + r * row + (i - r * per) * 8) = values8(w[h], s);
            }
    }
}

}  // namespace

// One unit is a piece of one head's keys and values (written) or of one of them (read, which has
// more to write: `sides` 2).
template <typename K>
static hipError_t launch_pieces(K wave_kernel, K block_kernel, int wave_tokens, const CacheArgs& args, int sides,
                                hipStream_t stream)
{
    CacheArgs a = args;
    const bool wave = a.each <= wave_tokens;
    const int64_t pieces = a.cu ? piece_bound(a.tokens, a.batch, a.shift) : a.batch * pieces_of(a.each, a.shift);
    const int64_t units = pieces * a.heads * sides, per = wave ? kCacheThreads / 64 : 1;
    const int64_t most = max_workgroups(kCacheThreads) / 2 * per;
    for (a.unit0 = 0; a.unit0 < units; a.unit0 += most) {
        const int64_t blocks = (std::min(most, units - a.unit0) + per - 1) / per;
        const hipError_t e = launch(wave ? wave_kernel : block_kernel, dim3((unsigned)blocks), dim3(kCacheThreads), stream, a);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_kv_cache_write(const CacheArgs& args, hipStream_t stream)
{
    return launch_pieces(kv_cache_write_kernel<64>, kv_cache_write_kernel<256>, kWriteWave, args, 1, stream);
}

hipError_t launch_kv_cache_read(const CacheArgs& args, hipStream_t stream)
{
    return launch_pieces(kv_cache_read_kernel<64>, kv_cache_read_kernel<256>, kReadWave, args, 2, stream);
}

}  // namespace fp8k
