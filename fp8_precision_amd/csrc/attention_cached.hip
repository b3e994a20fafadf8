// attention_cached.hip -- softmax attention over a paged cache of E4M3 keys and values
// (kv_cache.hip), for gfx950.
//
// Query i of a sequence's n stands at position held - n + i and sees the keys at positions
// up to its own (causal) or all that are held:
//   s = scale q . k,  p = exp(s - lse),  lse = log sum exp(s),  out = sum p v
// with k and v the codes times the power of two of their page and head.  Codes become bf16
// exactly on their way into the matrix instructions (the conversion takes the scale), so the
// only roundings are p's to bf16 and out's.
#include <algorithm>

#include "fp8_device.hpp"
#include "fp8_internal.hpp"
#include "kv_cache.hpp"

namespace fp8k {

namespace {

typedef __bf16 cb16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 cb16x2 __attribute__((ext_vector_type(2)));
typedef float cf32x2 __attribute__((ext_vector_type(2)));
typedef float cf32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int cu32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int cu32x2 __attribute__((ext_vector_type(2)));
typedef const __attribute__((address_space(4))) int const_int;

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kRows = 16;                  // rows of a unit: a query of one head each
constexpr int kStep = 64;                  // keys a wave takes at a time
constexpr int kLeastSteps = kWaves;        // a workgroup's share of the work, at least
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kInf = __builtin_inff();

union Operand {
    cu32x4 u;
    cb16x8 b;
    uint32_t w[4];
};

__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(cf32x2{a, b}, cb16x2));
}

__device__ __forceinline__ cf32x4 mma(const Operand& a, const Operand& b, const cf32x4& c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.b, b.b, c, 0, 0, 0);
}

// Of the four lanes that share lane % 16.
__device__ __forceinline__ float max4(float v)
{
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    return fmaxf(v, __shfl_xor(v, 32, 64));
}

__device__ __forceinline__ float sum4(float v)
{
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

// A sequence's queries and keys.
struct Sequence {
    int from, queries, held;
};

__device__ __forceinline__ Sequence sequence(const CacheArgs& a, int b)
{
    Sequence s;
    if (a.cu) {
        s.from = min(max(a.cu[b], 0), (int)a.tokens);
        s.queries = max(min(max(a.cu[b + 1], 0), (int)a.tokens) - s.from, 0);
    } else {
        s.queries = (int)(a.tokens / a.batch);
        s.from = b * s.queries;
    }
    s.held = held_tokens(a.lengths[b], a.blocks, a.shift);
    return s;
}

// Steps of unit `u` of one head of a sequence (rows kRows u ..): one at least, for the rows that see nothing.
__device__ __forceinline__ int unit_steps(const CachedAttentionArgs& a, const Sequence& s, int u)
{
    const int last = min((kRows * u + kRows - 1) / a.group, s.queries - 1);
    const int see = a.causal ? min(s.held, s.held - s.queries + last + 1) : s.held;
    return max(1, (see + kStep - 1) / kStep);
}

__device__ __forceinline__ int units_of(const CachedAttentionArgs& a, const Sequence& s)
{
    return (s.queries * a.group + kRows - 1) / kRows;
}

__device__ __forceinline__ int64_t head_steps(const CachedAttentionArgs& a, const Sequence& s)
{
    const int units = units_of(a, s);
    int64_t n = 0;
    for (int u = 0; u < units; ++u) n += unit_steps(a, s, u);
    return n;
}

// A wave's codes of 64 keys, as loaded.  Of each block of 16 keys a lane has DT / 4 codes of
// key lane % 16 (chunk lane / 16), and DT / 16 codes of each of the values 4 (lane / 16) + r.
template <int DT>
struct Codes {
    uint32_t k[4][DT / 16];
    uint32_t v[4][4][DT / 64];
    float k_scale[4], v_scale[4];
};

// Where the keys 16 x .. of a step lie: the page and head's place in the pool, -1 for none.
struct Block {
    int64_t place;
    int at, rows;        // first row in the page, rows held
};

}  // namespace

// Rows of one key head (its query heads' queries, 16 to a unit) against its keys.  The steps
// of all units, in order, are dealt to the workgroups in equal shares, so that one long
// sequence among short ones is spread like any other; a share's pieces of units that it does
// not hold whole are left as partial sums and joined.  The four waves take a piece's steps in
// turn.  Nothing of a step goes through LDS: 16 keys are the rows of a 16x16x32 product with
// the queries as its columns, in which a lane has 4 keys' scores of one query, and these are
// the second operand of the product with the values, whose rows are the head dimension: its
// first operand is 4 + 4 codes of one column, taken from 8 rows by byte permutations.
template <int DT, bool FULL>
__global__ void __launch_bounds__(kThreads, 2) attention_cached_kernel(const CachedAttentionArgs a)
{
    constexpr int kPer = DT / 16;          // values' elements of a lane, and the product's tiles
    __shared__ float s_out[kWaves][kRows][DT + 4];
    __shared__ float s_top[kWaves][kRows], s_sum[kWaves][kRows];
    __shared__ int64_t s_total[kWaves];
    __shared__ int64_t s_found[2];
    const CacheArgs& c = a.c;
    const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int worker = blockIdx.x;

    // the share: every thread sums some sequences' steps, in order
    const int per = (c.batch + kThreads - 1) / kThreads, b0 = threadIdx.x * per, b1 = min(b0 + per, c.batch);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += head_steps(a, sequence(c, b)) * c.heads;
    int64_t upto = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int64_t o = __shfl_up(upto, off, 64);
        if (lane >= off) upto += o;
    }
    if (lane == 63) s_total[wave] = upto;
    __syncthreads();
    int64_t total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before += s_total[w];
        total += s_total[w];
    }
    const int64_t share = max((total + a.workers - 1) / a.workers, (int64_t)kLeastSteps);
    int64_t at = worker * share;
    const int64_t end = min(at + share, total);
    if (threadIdx.x == 0) a.joins[worker] = make_int4(0, 0, 0, 0);
    if (at >= end) return;
    before += upto - mine;
    if (before <= at && at < before + mine) {
        int64_t left = at - before;
        int b = b0;
        for (;; ++b) {
            const int64_t n = head_steps(a, sequence(c, b)) * c.heads;
            if (left < n) break;
            left -= n;
        }
        s_found[0] = b;
        s_found[1] = left;
    }
    __syncthreads();
    int b = __builtin_amdgcn_readfirstlane((int)s_found[0]);
    int64_t left = s_found[1];
    Sequence s = sequence(c, b);
    int64_t per_head = head_steps(a, s);
    int head = __builtin_amdgcn_readfirstlane((int)(left / per_head));
    left -= head * per_head;
    int u = 0, steps;
    for (;; ++u) {
        steps = unit_steps(a, s, u);
        if (left < steps) break;
        left -= steps;
    }
    int step0 = __builtin_amdgcn_readfirstlane((int)left);
    const float scale2 = a.scale * kLog2e;
    uint32_t top_out = 0;

    while (true) {
        b = __builtin_amdgcn_readfirstlane(b);
        u = __builtin_amdgcn_readfirstlane(u);
        steps = __builtin_amdgcn_readfirstlane(steps);
        const int from = __builtin_amdgcn_readfirstlane(s.from), queries = __builtin_amdgcn_readfirstlane(s.queries);
        const int held = __builtin_amdgcn_readfirstlane(s.held);
        const int take = __builtin_amdgcn_readfirstlane((int)min((int64_t)(steps - step0), end - at));
        const int rows = queries * a.group, row = kRows * u + m;
        const int qi = row / a.group, hq = head * a.group + row - qi * a.group;
        const bool valid = row < rows;
        const int shift = held - queries;
        const int see = a.causal ? min(held, qi + shift + 1) : held;
        const int see_first = a.causal ? min(held, kRows * u / a.group + shift + 1) : held;

        // the queries' operand: lane's column m, elements of chunk g as the keys' lanes have them
        Operand q[DT / 32];
#pragma unroll
        for (int i = 0; i < DT / 32; ++i) {
            q[i].u = cu32x4{0, 0, 0, 0};
            const int e = DT / 4 * g + 8 * i;
            if (valid && (FULL || e < c.d))
                q[i].u = *reinterpret_cast<const cu32x4*>(a.q + (int64_t)(from + qi) * a.q_row + (int64_t)hq * a.q_head + e);
        }
        cf32x4 o[kPer];
#pragma unroll
        for (int t = 0; t < kPer; ++t) o[t] = cf32x4{0, 0, 0, 0};
        float top = -kInf, sum = 0.0f;

        const const_int* table = (const const_int*)(uintptr_t)(c.table + (int64_t)b * c.blocks);
        auto block = [&](int key) __attribute__((always_inline)) {
            Block x;
            const int page = key < held ? table[key >> c.shift] : -1;
            const bool none = page < 0 || page >= c.pages;
            x.place = none ? -1 : (int64_t)page * c.heads + head;
            x.at = key & ((1 << c.shift) - 1);
            x.rows = none ? 0 : min(held - key, 16);
            return x;
        };
        Codes<DT> r;
        Block bl[4];
        auto resource = [&](const uint8_t* pool, const Block& x) __attribute__((always_inline)) {
            const uint8_t* p = pool + (((max(x.place, (int64_t)0) << c.shift) + x.at) * c.d);
            return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, x.rows * c.d, 0x00020000);
        };
        auto load_k = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const auto src = resource(c.k, bl[x]);
                if constexpr (FULL) {
#pragma unroll
                    for (int i = 0; i < DT / 64; ++i) {
                        const cu32x4 w = __builtin_amdgcn_raw_buffer_load_b128(src, m * DT + DT / 4 * g + 16 * i, 0, 0);
#pragma unroll
                        for (int j = 0; j < 4; ++j) r.k[x][4 * i + j] = w[j];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < DT / 32; ++i) {
                        const int e = DT / 4 * g + 8 * i;
                        const cu32x2 w = __builtin_amdgcn_raw_buffer_load_b64(src, e < c.d ? m * c.d + e : 0x7FFFFFF0, 0, 0);
                        r.k[x][2 * i] = w[0];
                        r.k[x][2 * i + 1] = w[1];
                    }
                }
                r.k_scale[x] = cache_scale(c.k_scale[max(bl[x].place, (int64_t)0)]);
            }
        };
        auto load_v = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const auto src = resource(c.v, bl[x]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int d = FULL ? DT : c.d, e = kPer * m;
                    const int off = FULL || e < d ? (4 * g + i) * d + e : 0x7FFFFFF0;
                    if constexpr (DT == 128) {
                        const cu32x2 w = __builtin_amdgcn_raw_buffer_load_b64(src, off, 0, 0);
                        r.v[x][i][0] = w[0];
                        r.v[x][i][1] = w[1];
                    } else {
                        r.v[x][i][0] = __builtin_amdgcn_raw_buffer_load_b32(src, off, 0, 0);
                    }
                }
                r.v_scale[x] = cache_scale(c.v_scale[max(bl[x].place, (int64_t)0)]);
            }
        };

        const int last = step0 + take;
        for (int t = step0 + wave; t < last; t += kWaves) {
            const int j0 = t * kStep;
#pragma unroll
            for (int x = 0; x < 4; ++x) bl[x] = block(j0 + 16 * x);
            load_k();
            load_v();
            cf32x4 p[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                p[x] = cf32x4{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < DT / 32; ++i) {
                    Operand k;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        k.w[2 * j] = values2<false>(r.k[x][2 * i + j], r.k_scale[x]);
                        k.w[2 * j + 1] = values2<true>(r.k[x][2 * i + j], r.k_scale[x]);
                    }
                    p[x] = mma(k, q[i], p[x]);
                }
            }
            if (j0 + kStep > see_first) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (j0 + 16 * x + 4 * g + i >= see) p[x][i] = -kInf;
            }
            float up = top;
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) up = fmaxf(up, p[x][i]);
            up = max4(up);
            if (__any(up > top)) {
                const float by = up == -kInf ? 1.0f : __builtin_amdgcn_exp2f((top - up) * scale2);
                sum *= by;
#pragma unroll
                for (int i = 0; i < kPer; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[i][j] *= by;
                top = up;
            }
            const float use = top == -kInf ? 0.0f : top * scale2;
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p[x][i] = __builtin_amdgcn_exp2f(fmaf(p[x][i], scale2, -use));
                    sum += p[x][i];
                }
#pragma unroll
            for (int x = 0; x < 4; x += 2) {
                Operand f;
                f.w[0] = bf16_pair(p[x][0], p[x][1]);
                f.w[1] = bf16_pair(p[x][2], p[x][3]);
                f.w[2] = bf16_pair(p[x + 1][0], p[x + 1][1]);
                f.w[3] = bf16_pair(p[x + 1][2], p[x + 1][3]);
#pragma unroll
                for (int w = 0; w < DT / 64; ++w) {
                    uint32_t lo[4], hi[4];
                    transpose4x4(r.v[x][0][w], r.v[x][1][w], r.v[x][2][w], r.v[x][3][w], lo[0], lo[1], lo[2], lo[3]);
                    transpose4x4(r.v[x + 1][0][w], r.v[x + 1][1][w], r.v[x + 1][2][w], r.v[x + 1][3][w], hi[0], hi[1], hi[2], hi[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        Operand v;
                        v.w[0] = values2<false>(lo[i], r.v_scale[x]);
                        v.w[1] = values2<true>(lo[i], r.v_scale[x]);
                        v.w[2] = values2<false>(hi[i], r.v_scale[x + 1]);
                        v.w[3] = values2<true>(hi[i], r.v_scale[x + 1]);
                        o[4 * w + i] = mma(v, f, o[4 * w + i]);
                    }
                }
            }
        }
        sum = sum4(sum);

        // the waves' sums together: o[t][r] is element kPer (4 g + r) + t of row m
        if (g == 0) {
            s_top[wave][m] = top;
            s_sum[wave][m] = sum;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int t = 0; t < kPer; t += 4)
                *reinterpret_cast<cf32x4*>(&s_out[wave][m][kPer * (4 * g + i) + t]) =
                    cf32x4{o[t][i], o[t + 1][i], o[t + 2][i], o[t + 3][i]};
        __syncthreads();
        {
            const int n = threadIdx.x / 16, e = threadIdx.x % 16 * kPer, r2 = kRows * u + n;
            const int q2 = r2 / a.group, h2 = head * a.group + r2 - q2 * a.group;
            float best = -kInf, all = 0.0f, x[kPer];
#pragma unroll
            for (int w = 0; w < kWaves; ++w) best = fmaxf(best, s_top[w][n]);
            const float use = best == -kInf ? 0.0f : best;
#pragma unroll
            for (int i = 0; i < kPer; ++i) x[i] = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float by = __builtin_amdgcn_exp2f((s_top[w][n] - use) * scale2);
                all = fmaf(s_sum[w][n], by, all);
#pragma unroll
                for (int i = 0; i < kPer; ++i) x[i] = fmaf(s_out[w][n][e + i], by, x[i]);
            }
            if (r2 < rows) {
                if (take == steps) {
                    const float by = all > 0.0f ? 1.0f / all : (all == 0.0f ? 0.0f : all);    // a NaN sum stays NaN
                    uint32_t w[kPer / 2];
#pragma unroll
                    for (int i = 0; i < kPer / 2; ++i) {
                        w[i] = bf16_pair(x[2 * i] * by, x[2 * i + 1] * by);
                        if (FULL || e < c.d) top_out = max(max(top_out, w[i] & 0x7FFF0000u), w[i] << 16 & 0x7FFFFFFFu);
                    }
                    uint16_t* to = a.out + (int64_t)(from + q2) * a.out_row + (int64_t)h2 * a.out_head + e;
                    if (FULL || e < c.d) {
                        if constexpr (kPer == 8) *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
                        else *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
                    }
                    if (e == 0)
                        a.lse[(int64_t)h2 * c.tokens + from + q2] =
                            all == 0.0f ? -kInf : (use * scale2 + __builtin_amdgcn_logf(all)) * kLn2;
                } else {
                    const int64_t slot = 2 * (int64_t)worker + (step0 == 0 ? 1 : 0);
                    float* to = a.partial + (slot * kRows + n) * DT + e;
#pragma unroll
                    for (int i = 0; i < kPer; i += 4) *reinterpret_cast<cf32x4*>(to + i) = cf32x4{x[i], x[i + 1], x[i + 2], x[i + 3]};
                    if (e == 0) a.tops[slot * kRows + n] = make_float2(best == -kInf ? -kInf : best * scale2, all);
                }
            }
        }
        if (threadIdx.x == 0 && step0 == 0 && take < steps)
            a.joins[worker] = make_int4(b, head, u, (int)((at + steps - 1) / share) - worker + 1);
        __syncthreads();

        at += take;
        if (at >= end) break;
        step0 = 0;
        if (++u == units_of(a, s)) {
            u = 0;
            if (++head == c.heads) {
                head = 0;
                do s = sequence(c, ++b);
                while (s.queries == 0);
            }
        }
        steps = unit_steps(a, s, u);
    }
    if (a.absmax) block_max_to_global(top_out, a.absmax);
}

// out and lse of one row of a unit whose steps several workgroups shared: the first's last
// piece and the following ones' first, in order.
template <int DT>
__global__ void __launch_bounds__(256) attention_cached_join_kernel(const CachedAttentionArgs a)
{
    __shared__ float part[256][kRows / 2 + 1];
    const CacheArgs& c = a.c;
    const int worker = blockIdx.x, n = blockIdx.y;
    const int4 job = a.joins[worker];
    if (job.w <= 1) return;
    const Sequence s = sequence(c, job.x);
    const int row = kRows * job.z + n;
    if (row >= s.queries * a.group) return;
    constexpr int kPer = 8, kLanes = DT / kPer, kGroups = 256 / kLanes;
    const int k = threadIdx.x / kLanes, e = threadIdx.x % kLanes * kPer;
    auto slot = [&](int i) __attribute__((always_inline)) { return (2 * (int64_t)(worker + i) + (i == 0)) * kRows + n; };
    float m = -kInf, l = 0.0f;
    for (int i = threadIdx.x & 63; i < job.w; i += 64) m = fmaxf(m, a.tops[slot(i)].x);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
    const float use = m == -kInf ? 0.0f : m;
    for (int i = threadIdx.x & 63; i < job.w; i += 64) {
        const float2 x = a.tops[slot(i)];
        l = fmaf(x.y, __builtin_amdgcn_exp2f(x.x - use), l);
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) l += __shfl_xor(l, off, 64);
    float t[kPer] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
    for (int i = k; i < job.w; i += kGroups) {
        const float by = __builtin_amdgcn_exp2f(a.tops[slot(i)].x - use);
        const float4* p = reinterpret_cast<const float4*>(a.partial + slot(i) * DT + e);
        const float4 u = p[0], v = p[1];
        const float w[kPer] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < kPer; ++j) t[j] = fmaf(w[j], by, t[j]);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) part[threadIdx.x][j] = t[j];
    __syncthreads();
    uint32_t top = 0;
    if (k == 0 && e < c.d) {
        for (int i = 1; i < kGroups; ++i)
#pragma unroll
            for (int j = 0; j < kPer; ++j) t[j] += part[i * kLanes + threadIdx.x][j];
        const float by = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
        const int qi = row / a.group, hq = job.y * a.group + row - qi * a.group;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = bf16_pair(t[2 * j] * by, t[2 * j + 1] * by);
            top = max(max(top, w[j] & 0x7FFF0000u), w[j] << 16 & 0x7FFFFFFFu);
        }
        *reinterpret_cast<uint4*>(a.out + (int64_t)(s.from + qi) * a.out_row + (int64_t)hq * a.out_head + e) =
            make_uint4(w[0], w[1], w[2], w[3]);
        if (e == 0) a.lse[(int64_t)hq * c.tokens + s.from + qi] = l == 0.0f ? -kInf : (use + __builtin_amdgcn_logf(l)) * kLn2;
    }
    if (a.absmax) block_max_to_global(top, a.absmax);
}

// Two workgroups per CU share the work.
static int worker_count() { return 2 * device_cu_count(); }

int64_t attention_cached_workspace(int64_t, int, int, int d, int, int, int)
{
    const int64_t workers = worker_count();
    return workers * (16 + 2 * kRows * (8 + 4 * (d <= 64 ? 64 : 128)));
}

hipError_t launch_attention_cached(const CachedAttentionArgs& args, void* workspace, hipStream_t stream)
{
    CachedAttentionArgs a = args;
    a.workers = worker_count();
    a.joins = static_cast<int4*>(workspace);
    a.tops = reinterpret_cast<float2*>(a.joins + a.workers);
    a.partial = reinterpret_cast<float*>(a.tops + 2 * a.workers * kRows);
    void (*kernel)(CachedAttentionArgs) =
        a.c.d == 64 ? attention_cached_kernel<64, true> : a.c.d == 128 ? attention_cached_kernel<128, true>
        : a.c.d < 64 ? attention_cached_kernel<64, false> : attention_cached_kernel<128, false>;
    const hipError_t e = launch(kernel, dim3(a.workers), dim3(kThreads), stream, a);
    if (e != hipSuccess) return e;
    const unsigned rows = (unsigned)std::min<int64_t>(kRows, a.c.tokens * a.group);
    return launch(a.c.d <= 64 ? attention_cached_join_kernel<64> : attention_cached_join_kernel<128>, dim3(a.workers, rows), dim3(256),
                  stream, a);
}

}  // namespace fp8k
