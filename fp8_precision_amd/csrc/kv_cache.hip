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
// Bound by memory, 2 bytes read and 1 written per element (or the reverse); for a single new
// token per sequence by the launch and three dependent reads (bounds, table, token).
#include <algorithm>

#include "fp8_device.hpp"
#include "fp8_internal.hpp"
#include "kv_cache.hpp"

namespace fp8k {

namespace {

constexpr int kCacheThreads = 256;
constexpr int kWaveTokens = 4;             // new tokens per sequence, on average, up to which a wave takes a piece
constexpr int kHeld = 8;                   // 16-byte groups of a piece that a thread keeps in registers

// The scale's exponent for a largest magnitude of these fp32 bits: 448 = 1.75 2^8.
__device__ __forceinline__ int exponent_for(uint32_t top)
{
    const int e = (int)(top >> 23) - 135 + ((top & 0x7FFFFFu) > 0x600000u);
    return min(max(e, kCacheLeastE), kCacheMostE);
}

struct Piece {
    CachePiece at;
    int64_t token;      // the first token in the call's tensors
    int64_t page;       // in the pool; -1: none
};

// Piece `item` of the call.  Every wave finds its own: 64 sequences are compared at a time.
__device__ __forceinline__ Piece find_piece(const CacheArgs& a, int64_t item)
{
    const int lane = threadIdx.x & 63;
    Piece p{};
    int b, from, count;
    int64_t local;
    if (!a.cu) {
        count = (int)(a.tokens / a.batch);
        const int64_t per = pieces_of(count, a.shift);
        b = (int)min(item / per, (int64_t)a.batch);
        local = item % per;
        from = (int)min((int64_t)b * count, a.tokens);
    } else {
        int first = 0, width = a.batch;
        do {
            const int step = (width + 63) / 64, c = first + lane * step;
            const bool before = c < first + width && piece_base(min(max(a.cu[c], 0), (int)a.tokens), c, a.shift) <= item;
            const uint64_t all = __ballot(before);
            if (!all) return p;
            const int l = 63 - __clzll((long long)all);
            width = min(step, width - l * step);
            first += l * step;
        } while (width > 1);
        b = __builtin_amdgcn_readfirstlane(first);
        from = min(max(a.cu[b], 0), (int)a.tokens);
        count = max(min(max(a.cu[b + 1], 0), (int)a.tokens) - from, 0);
        local = item - piece_base(from, b, a.shift);
    }
    if (b >= a.batch) return p;
    p.at = cache_piece(count, held_tokens(a.lengths[b], a.blocks, a.shift), local, a.shift);
    p.token = (int64_t)from + p.at.skip;
    p.page = -1;
    if (p.at.count > 0 && p.at.block >= 0) {
        const int at = a.table[(int64_t)b * a.blocks + p.at.block];
        if (at >= 0 && at < a.pages) p.page = at;
    }
    return p;
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

// 4 codes times a power of two, rounded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float by)
{
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    return enc4<0>(lo[0] * by, lo[1] * by, hi[0] * by, hi[1] * by);
}

// T threads (a wave, or the workgroup) write one piece of one head's keys or values: its
// largest magnitude, the page's new exponent, the codes; and where the page was begun
// before and its exponent grows, its older codes.
template <int T>
__global__ void __launch_bounds__(kCacheThreads) kv_cache_write_kernel(const CacheArgs a)
{
    constexpr int kUnits = kCacheThreads / T;
    __shared__ uint32_t part[kCacheThreads / 64];
    __shared__ int was_e;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t unit = a.unit0 + (int64_t)blockIdx.x * kUnits + (T == 64 ? wave : 0);
    const int tid = T == 64 ? threadIdx.x & 63 : threadIdx.x;
    const int head = (int)(unit % a.heads), values = (int)(unit / a.heads % 2);
    const Piece p = find_piece(a, unit / (2 * a.heads));
    if (p.at.count <= 0 || p.page < 0) return;

    const int d = a.d, per = d / 8, groups = p.at.count * per;
    const uint32_t inverse = (65536 + per - 1) / per;      // i / per for i < 2^12
    const uint16_t* x = (values ? a.xv : a.xk) + p.token * (values ? a.xv_row : a.xk_row) +
                        head * (values ? a.xv_head : a.xk_head);
    const int64_t row = values ? a.xv_row : a.xk_row;
    const int64_t place = p.page * a.heads + head;
    uint8_t* codes = (values ? a.v : a.k) + ((place << a.shift) * d);
    uint8_t* scale = (values ? a.v_scale : a.k_scale) + place;

    auto load = [&](int i) __attribute__((always_inline)) {
        const int r = (int)(i * inverse >> 16);
        return *reinterpret_cast<const uint4*>(x + r * row + (i - r * per) * 8);
    };
    uint4 held[kHeld];
    uint32_t top = 0;
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
        if (tid + h * T < groups) held[h] = load(tid + h * T);
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
        if (tid + h * T < groups) top = max(top, finite_top(held[h]));
    for (int i = tid + kHeld * T; i < groups; i += T) top = max(top, finite_top(load(i)));
    top = wave_max_u32(top);
    int was = kCacheLeastE;
    if (T == 64) {
        if (p.at.slot > 0) was = cache_exponent(*scale);
    } else {
        if ((threadIdx.x & 63) == 0) part[wave] = top;
        if (threadIdx.x == 0) was_e = p.at.slot > 0 ? cache_exponent(*scale) : kCacheLeastE;
        __syncthreads();
        for (int w = 0; w < kCacheThreads / 64; ++w) top = max(top, part[w]);
        was = was_e;
    }
    const int e = max(exponent_for(top), was);
    const float s = two_to(-e);

    uint2* to = reinterpret_cast<uint2*>(codes + p.at.slot * d);
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
        if (tid + h * T < groups) to[tid + h * T] = quant8<0>(held[h], s);
    for (int i = tid + kHeld * T; i < groups; i += T) to[i] = quant8<0>(load(i), s);
    if (p.at.slot > 0 && e > was) {
        // 2^-126 and less leave no code but 0
        const float by = two_to(max(was - e, -126));
        for (int i = tid; i < p.at.slot * per; i += T) {
            uint2 w = reinterpret_cast<uint2*>(codes)[i];
            w.x = rescale4(w.x, by);
            w.y = rescale4(w.y, by);
            reinterpret_cast<uint2*>(codes)[i] = w;
        }
    }
    if (tid == 0) *scale = (uint8_t)(e + 127);
}

// T threads read one piece of one head's keys or values; tokens with no place read as zeros.
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
    uint16_t* x = (values ? a.xv : a.xk) + p.token * (values ? a.xv_row : a.xk_row) + head * (values ? a.xv_head : a.xk_head);
    const int64_t row = values ? a.xv_row : a.xk_row;
    const int64_t place = max(p.page, (int64_t)0) * a.heads + head;
    const uint2* codes = reinterpret_cast<const uint2*>((values ? a.v : a.k) + (place << a.shift) * d + p.at.slot * d);
    const uint8_t byte = p.page < 0 ? 0 : (values ? a.v_scale : a.k_scale)[place];
    const float s = cache_scale(byte);

    for (int i0 = tid; i0 < groups; i0 += 4 * T) {
        uint2 w[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            w[h] = make_uint2(0, 0);
            if (i0 + h * T < groups && p.page >= 0) w[h] = codes[i0 + h * T];
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

// One unit is a piece of one head's keys, or of its values: a wave where the pieces are short
// (T = 64), a workgroup otherwise.
template <typename K>
static hipError_t launch_pieces(K wave_kernel, K block_kernel, const CacheArgs& args, hipStream_t stream)
{
    CacheArgs a = args;
    const int64_t n = a.tokens / a.batch;
    const bool wave = n <= kWaveTokens;
    const int64_t pieces = a.cu ? piece_bound(a.tokens, a.batch, a.shift) : a.batch * pieces_of(n, a.shift);
    const int64_t units = pieces * 2 * a.heads, per = wave ? kCacheThreads / 64 : 1;
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
    return launch_pieces(kv_cache_write_kernel<64>, kv_cache_write_kernel<256>, args, stream);
}

hipError_t launch_kv_cache_read(const CacheArgs& args, hipStream_t stream)
{
    return launch_pieces(kv_cache_read_kernel<64>, kv_cache_read_kernel<256>, args, stream);
}

}  // namespace fp8k
