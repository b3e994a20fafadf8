// norm.hip -- root-mean-square and layer norm of the rows of a residual stream,
// forward (with the residual sum in front and the statistic of the output that
// the FP8 quantisation takes next) and backward (with the gradients of the
// weight and the bias), for gfx950.
//
//   s = x + a                      (a: the previous block's output; or s = x)
//   m = mean(s) (layer) or 0 (rms),  r = 1 / sqrt(mean((s - m)^2) + eps)
//   h = (s - m) r,   y = h w + b
// and backward, with g = dy w per element and means over the row,
//   dx = r (g - h mean(g h) - mean(g) [layer only]) + ds
//   dw = sum over rows of dy h,   db = sum over rows of dy
// ds is the gradient that reaches s by the residual path around the norm.
//
// Everything between a load and a store is held in fp32: the mean, the sum of
// squared deviations (taken in a second sweep over the registers, so no
// difference of large sums is formed), the gradient sums; y, s and dx are
// rounded once, to their own type.
//
// Bound by memory: forward reads and writes each element once (the row stays in
// registers between the sweeps), backward too.  A row is one workgroup of
// W = ceil(cols / (512 NV)) waves, a lane holding NV groups of 8 consecutive
// elements; a row's sums are a butterfly in each wave and, for W > 1, one exchange
// through LDS.  Narrow rows share a workgroup.  Backward workgroups walk rows with the next row's loads issued
// before the current row's exchange, so that the exchange does not leave the
// memory idle, and keep the weight gradient of their rows in registers; they
// write one partial row each, which a second launch adds up in a fixed order
// (no atomics: the same bytes every time).
#include "fp8_device.hpp"
#include "fp8_internal.hpp"

namespace fp8k {

namespace {

typedef __bf16 nb16x2 __attribute__((ext_vector_type(2)));
typedef float nf32x2 __attribute__((ext_vector_type(2)));

constexpr int kNormMaxWaves = 16;
constexpr int kNarrow = 256;              // threads of a workgroup that takes several rows

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(nf32x2{a, b}, nb16x2));
}

// Eight consecutive elements as loaded: 16 bytes of bf16 or 32 of fp32.
template <bool F32> struct Raw8;
template <> struct Raw8<false> { uint4 a; };
template <> struct Raw8<true> { uint4 a, b; };

// What follows from these bits is computed from here on, not kept from before.
__device__ __forceinline__ void opaque(uint4& v)
{
    asm volatile("" : "+v"(v.x), "+v"(v.y), "+v"(v.z), "+v"(v.w));
}

// 16 bytes at an address that is only a multiple of an element's size: one instruction
// too, as the hardware takes global accesses of any alignment.  Rows that are no multiple
// of 8 elements (2048 x 9001 bf16, backward) took 99 us element by element, 57 so.
typedef uint32_t Loose16 __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ uint4 strict(const Loose16& v) { return make_uint4(v.x, v.y, v.z, v.w); }

// Load the 8 elements from column c of a row of `cols`; those past the row's end
// are zero.  VEC: cols is a multiple of 8, so every group is whole and 16-byte
// aligned; otherwise a row's last group is read element by element.
template <bool F32, bool VEC>
__device__ __forceinline__ Raw8<F32> load8(const void* row, int c, int cols)
{
    Raw8<F32> r{};
    if (VEC) {
        if (c < cols) {
            if constexpr (F32) {
                const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(row) + c);
                r.a = p[0];
                r.b = p[1];
            } else {
                r.a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + c);
            }
        }
    } else if (c + 8 <= cols) {
        if constexpr (F32) {
            const Loose16* p = reinterpret_cast<const Loose16*>(static_cast<const float*>(row) + c);
            r.a = strict(p[0]);
            r.b = strict(p[1]);
        } else {
            r.a = strict(*reinterpret_cast<const Loose16*>(static_cast<const uint16_t*>(row) + c));
        }
    } else if (c < cols) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[e] = 0;
            if (c + e < cols) {
                if constexpr (F32)
                    w[e] = __float_as_uint(static_cast<const float*>(row)[c + e]);
                else
                    w[e] = static_cast<const uint16_t*>(row)[c + e];
            }
        }
        if constexpr (F32) {
            r.a = make_uint4(w[0], w[1], w[2], w[3]);
            r.b = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
            r.a = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
        }
    }
    return r;
}

template <bool F32>
__device__ __forceinline__ void widen(const Raw8<F32>& r, float (&f)[8])
{
    if constexpr (F32) {
        const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(w[e]);
    } else {
        const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[2 * e] = bf16_lo(w[e]);
            f[2 * e + 1] = bf16_hi(w[e]);
        }
    }
}

template <bool F32, bool VEC>
__device__ __forceinline__ void store8(void* row, int c, int cols, const float (&f)[8])
{
    if (c >= cols) return;
    constexpr int kWords = F32 ? 8 : 4, kSize = F32 ? 4 : 2;
    uint8_t* p = static_cast<uint8_t*>(row) + (size_t)c * kSize;
    uint32_t w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = F32 ? __float_as_uint(f[i]) : pack2(f[2 * i & 7], f[(2 * i + 1) & 7]);
    if (VEC || c + 8 <= cols) {
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
            if (VEC)
                *reinterpret_cast<uint4*>(p + 4 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
            else
                *reinterpret_cast<Loose16*>(p + 4 * i) = Loose16{w[i], w[i + 1], w[i + 2], w[i + 3]};
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (c + e >= cols) continue;
        if (F32)
            reinterpret_cast<uint32_t*>(p)[e] = w[e & (kWords - 1)];
        else
            reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    }
}

// Sum over the `lanes` (a power of two) neighbouring lanes of a row.
template <int lanes>
__device__ __forceinline__ float lane_sum(float v)
{
#pragma unroll
    for (int off = lanes / 2; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

// Sum over the workgroup's waves of a value already summed in each wave; `part`
// is an LDS row that no other exchange in flight uses.
__device__ __forceinline__ float2 block_sum2(float2 v, float2* part, int wave, int waves)
{
    if (waves == 1) return v;
    if ((threadIdx.x & 63) == 0) part[wave] = v;
    __syncthreads();
    float2 t = part[0];
    for (int w = 1; w < waves; ++w) {
        t.x += part[w].x;
        t.y += part[w].y;
    }
    return t;
}

}  // namespace

// Forward.  L = 0: a row per workgroup; else L lanes per row, several rows per workgroup.
// 4096 x 4096 bf16 with the residual sum (134 MB): 23.6 us, 5.7 TB/s (a large copy on the
// same chip: 5.8); a single row is bound by the call.
template <bool F32, bool VEC, int NV, int L, bool RMS>
__global__ void __launch_bounds__(L ? kNarrow : kNormMaxWaves * 64)
norm_forward_kernel(const void* __restrict__ x, const uint16_t* __restrict__ add, const uint16_t* __restrict__ weight,
                    const uint16_t* __restrict__ bias, float eps, uint32_t rows, int cols, uint16_t* __restrict__ y,
                    void* __restrict__ sum, float* __restrict__ mean, float* __restrict__ rstd,
                    uint32_t* __restrict__ absmax)
{
    __shared__ float2 part[2][kNormMaxWaves];
    constexpr int kLanes = L ? L : 64;
    const uint32_t row = L ? blockIdx.x * (kNarrow / kLanes) + threadIdx.x / kLanes : blockIdx.x;   // rows < 2^31
    const bool have = !L || row < rows;
    const size_t at = have ? (size_t)row * (size_t)cols : 0;
    const int wave = threadIdx.x >> 6, waves = L ? 1 : blockDim.x >> 6;
    const int lane = L ? threadIdx.x % kLanes : threadIdx.x;
    const int col0 = have ? lane * 8 : cols, step = L ? 0 : blockDim.x * 8;
    const uint8_t* xr = static_cast<const uint8_t*>(x) + at * (F32 ? 4 : 2);

    Raw8<F32> xv[NV];
    Raw8<false> av[NV], wv[NV], bv[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) xv[v] = load8<F32, VEC>(xr, col0 + v * step, cols);
    if (add) {
#pragma unroll
        for (int v = 0; v < NV; ++v) av[v] = load8<false, VEC>(add + at, col0 + v * step, cols);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) wv[v] = load8<false, VEC>(weight, col0 + v * step, cols);
    if (bias) {
#pragma unroll
        for (int v = 0; v < NV; ++v) bv[v] = load8<false, VEC>(bias, col0 + v * step, cols);
    }

    float s[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        widen<F32>(xv[v], s[v]);
        if (add) {
            float a[8];
            widen<false>(av[v], a);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[v][e] += a[e];
        }
    }
    if (sum) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            store8<F32, VEC>(static_cast<uint8_t*>(sum) + at * (F32 ? 4 : 2), col0 + v * step, cols, s[v]);
    }

    const float inv_n = 1.0f / (float)cols;
    float m = 0.0f;
    if (!RMS) {
        float t = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) t += s[v][e];      // places past the row's end hold zero
        m = block_sum2(make_float2(lane_sum<kLanes>(t), 0.0f), part[0], wave, waves).x * inv_n;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s[v][e] = col0 + v * step + e < cols ? s[v][e] - m : 0.0f;
    }
    float q = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) q = fmaf(s[v][e], s[v][e], q);
    const float var = block_sum2(make_float2(lane_sum<kLanes>(q), 0.0f), part[1], wave, waves).x * inv_n;
    const float r = 1.0f / sqrtf(var + eps);
    if (lane == 0 && have) {
        rstd[row] = r;
        if (!RMS) mean[row] = m;
    }

    uint32_t top = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        float w[8], o[8];
        widen<false>(wv[v], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = s[v][e] * r * w[e];
        if (bias) {
            float b[8];
            widen<false>(bv[v], b);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] += b[e];
        }
        store8<false, VEC>(y + at, col0 + v * step, cols, o);
        if (absmax) {                                       // of the bf16 values as stored
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const uint32_t p = pack2(o[e], o[e + 1]);
                const int c = col0 + v * step + e;
                if (c < cols) top = max(top, p << 16 & 0x7FFFFFFFu);
                if (c + 1 < cols) top = max(top, p & 0x7FFF0000u);
            }
        }
    }
    if (absmax) block_max_to_global(top, absmax);
}

// Backward over every gridDim.x-th row (L = 0) or set of rows; partial[2][grid][cols]
// gets the workgroup's sums of dy h and, if asked for, of dy.
// 8192 x 5120 bf16 with dres (336 MB): 64 us, 5.2 TB/s, the sums' launch (4 us) included.
template <bool F32, bool VEC, int NV, int L, bool RMS>
__global__ void __launch_bounds__(L ? kNarrow : kNormMaxWaves * 64)
norm_backward_kernel(const uint16_t* __restrict__ dy, const void* __restrict__ x, const uint16_t* __restrict__ weight,
                     const float* __restrict__ mean, const float* __restrict__ rstd, const void* __restrict__ dres,
                     uint32_t rows, int cols, void* __restrict__ dx, float* __restrict__ partial, int want_db)
{
    __shared__ float2 part[2][kNormMaxWaves];
    constexpr size_t kX = F32 ? 4 : 2;
    constexpr int kLanes = L ? L : 64, kRows = L ? kNarrow / kLanes : 1;
    const int wave = threadIdx.x >> 6, waves = L ? 1 : blockDim.x >> 6;
    const int col0 = (L ? threadIdx.x % kLanes : threadIdx.x) * 8, step = L ? 0 : blockDim.x * 8;
    const float inv_n = 1.0f / (float)cols;
    const uint8_t* xb = static_cast<const uint8_t*>(x);
    const uint8_t* rb = static_cast<const uint8_t*>(dres);

    // Two groups per lane leave the registers no room for the weight's and the bias's sums,
    // which then lie in LDS (each lane its own), nor for what the second sweep needs in fp32,
    // which is formed again from the row as loaded; an fp32 dres is loaded in between.
    constexpr bool kAgain = NV > 1, kLate = NV > 1 && F32;
    constexpr int kSums = RMS ? 1 : 2;
    __shared__ float4 sums[kAgain ? kSums * NV * 2 : 1][kAgain ? kNormMaxWaves * 64 : 1];
    Raw8<false> wv[NV];
    float dw[NV][8], db[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        wv[v] = load8<false, VEC>(weight, col0 + v * step, cols);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[v][e] = db[v][e] = 0.0f;
    }
    if (kAgain)
        for (int i = 0; i < kSums * NV * 2; ++i) sums[i][threadIdx.x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    Raw8<false> yv[NV], yn[NV];
    Raw8<F32> xv[NV], xn[NV], rv[NV], rn[NV];
    float m = 0.0f, r = 0.0f, mn = 0.0f, rstd_n = 0.0f;
    auto fetch = [&](uint32_t row) __attribute__((always_inline)) {
        const size_t at = (size_t)row * (size_t)cols;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            yn[v] = load8<false, VEC>(dy + at, col0 + v * step, cols);
            xn[v] = load8<F32, VEC>(xb + at * kX, col0 + v * step, cols);
            if (!kLate && dres) rn[v] = load8<F32, VEC>(rb + at * kX, col0 + v * step, cols);
        }
        rstd_n = rstd[row];
        if (!RMS) mn = mean[row];
    };

    uint32_t row = L ? blockIdx.x * kRows + threadIdx.x / kLanes : blockIdx.x;
    if (row < rows) fetch(row);
    for (int turn = 0; row < rows; turn ^= 1) {
        float g[NV][8], h[NV][8], keep[NV][8];
        // h and g of group v; past the row's end dy and w are zero, so whatever h is there
        // adds nothing (the mean and the reciprocal deviation of a finite row are finite)
        auto form = [&](int v, float (&d)[8]) __attribute__((always_inline)) {
            float xs[8], w[8];
            widen<false>(yv[v], d);
            widen<F32>(xv[v], xs);
            widen<false>(wv[v], w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[v][e] = (xs[e] - m) * r;
                g[v][e] = d[e] * w[e];
            }
        };
        float2 t = make_float2(0.0f, 0.0f);
        m = mn;
        r = rstd_n;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            yv[v] = yn[v];
            xv[v] = xn[v];
            if (!kLate) rv[v] = rn[v];
            if (kAgain) __builtin_amdgcn_sched_barrier(0);   // one group's values at a time
            float d[8];
            form(v, d);
            if (!kAgain && dres) widen<F32>(rv[v], keep[v]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                t.x = fmaf(g[v][e], h[v][e], t.x);
                t.y += g[v][e];
            }
            if (kAgain) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float4* p = &sums[2 * v + k][threadIdx.x];
                    float4 a = *p;
                    a.x = fmaf(d[4 * k], h[v][4 * k], a.x);
                    a.y = fmaf(d[4 * k + 1], h[v][4 * k + 1], a.y);
                    a.z = fmaf(d[4 * k + 2], h[v][4 * k + 2], a.z);
                    a.w = fmaf(d[4 * k + 3], h[v][4 * k + 3], a.w);
                    *p = a;
                    if (!RMS) {
                        p = &sums[2 * (NV + v) + k][threadIdx.x];
                        a = *p;
                        a.x += d[4 * k];
                        a.y += d[4 * k + 1];
                        a.z += d[4 * k + 2];
                        a.w += d[4 * k + 3];
                        *p = a;
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dw[v][e] = fmaf(d[e], h[v][e], dw[v][e]);
                    db[v][e] += d[e];
                }
            }
        }
        const size_t at = (size_t)row * (size_t)cols;
        if (kLate && dres) {
#pragma unroll
            for (int v = 0; v < NV; ++v) rv[v] = load8<F32, VEC>(rb + at * kX, col0 + v * step, cols);
        }
        row += gridDim.x * kRows;
        if (row < rows) fetch(row);
        t.x = lane_sum<kLanes>(t.x);
        if (!RMS) t.y = lane_sum<kLanes>(t.y);
        t = block_sum2(t, part[turn], wave, waves);
        const float along = t.x * inv_n, flat = RMS ? 0.0f : t.y * inv_n;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float o[8], d[8];
            if (kAgain) {
                __builtin_amdgcn_sched_barrier(0);
                opaque(yv[v].a);
                opaque(xv[v].a);
                if constexpr (F32) opaque(xv[v].b);
                opaque(wv[v].a);
                if (dres) opaque(rv[v].a);
                form(v, d);
                if (dres) widen<F32>(rv[v], keep[v]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                o[e] = r * (g[v][e] - flat - h[v][e] * along);
                if (dres) o[e] += keep[v][e];
            }
            store8<F32, VEC>(static_cast<uint8_t*>(dx) + at * kX, col0 + v * step, cols, o);
        }
    }

    if (L) {                                                 // the workgroup's rows, in order
        __shared__ float join[L ? kNarrow / 64 : 1][2][L ? kLanes * 8 : 1];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
            for (int off = kLanes; off < 64; off <<= 1) {
                dw[0][e] += __shfl_xor(dw[0][e], off, 64);
                if (!RMS) db[0][e] += __shfl_xor(db[0][e], off, 64);
            }
            if ((int)(threadIdx.x & 63) < kLanes) {
                join[wave][0][col0 + e] = dw[0][e];
                if (!RMS) join[wave][1][col0 + e] = db[0][e];
            }
        }
        __syncthreads();
        if ((int)threadIdx.x >= kLanes) return;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            for (int k = 1; k < kNarrow / 64; ++k) {
                dw[0][e] += join[k][0][col0 + e];
                if (!RMS) db[0][e] += join[k][1][col0 + e];
            }
    }
    float* pw = partial + (size_t)blockIdx.x * (size_t)cols;
    float* pb = pw + (size_t)gridDim.x * (size_t)cols;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if (kAgain) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float4 a = sums[2 * v + k][threadIdx.x], b = sums[RMS ? 0 : 2 * (NV + v) + k][threadIdx.x];
                dw[v][4 * k] = a.x, dw[v][4 * k + 1] = a.y, dw[v][4 * k + 2] = a.z, dw[v][4 * k + 3] = a.w;
                db[v][4 * k] = b.x, db[v][4 * k + 1] = b.y, db[v][4 * k + 2] = b.z, db[v][4 * k + 3] = b.w;
            }
        }
        store8<true, VEC>(pw, col0 + v * step, cols, dw[v]);
        if (!RMS && want_db) store8<true, VEC>(pb, col0 + v * step, cols, db[v]);
    }
}

// out[c] = sum over i < parts of partial[i][c], 32 columns per workgroup: 32 lanes of
// consecutive columns by 32 slices of the parts, the slices joined in LDS in order.
// blockIdx.y picks the weight's or the bias's sums.
__global__ void __launch_bounds__(1024)
norm_join_kernel(const float* __restrict__ partial, int parts, int cols, float* __restrict__ dw, float* __restrict__ db)
{
    __shared__ float slice[32][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
    const float* p = partial + (size_t)blockIdx.y * (size_t)parts * (size_t)cols;
    float t = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int i = k; i < parts; i += 32) t += p[(size_t)i * (size_t)cols + c];
    }
    slice[k][threadIdx.x & 31] = t;
    __syncthreads();
    if (k == 0 && c < cols) {
        t = slice[0][threadIdx.x];
        for (int i = 1; i < 32; ++i) t += slice[i][threadIdx.x];
        (blockIdx.y ? db : dw)[c] = t;
    }
}

// How a row is laid over lanes.  Up to 512 columns: the fewest of 16, 32 or 64 lanes that
// hold it 8 elements each, 256 threads taking several rows: 131072 rows of 128 bf16 (one
// norm per head), forward 39.7 us with a wave per row and 24.2 so, backward 54 and 29.6;
// 327680 of 64: 86 and 31, 109 and 38; 32768 of 512: 23.4 and 24.1, 36 and 30.  Above, a
// workgroup of as many waves as it takes, up to 8192 columns; two groups per lane above that.
struct NormLayout {
    int lanes, groups, threads, rows;     // lanes 0: the workgroup's; rows of a workgroup
};

static NormLayout norm_layout(int64_t cols)
{
    if (cols <= 512) {
        const int lanes = cols <= 128 ? 16 : cols <= 256 ? 32 : 64;
        return {lanes, 1, kNarrow, kNarrow / lanes};
    }
    const int groups = cols <= 512 * kNormMaxWaves ? 1 : 2;
    return {0, groups, 64 * (int)((cols + 512 * groups - 1) / (512 * groups)), 1};
}

// Workgroups of the backward launch: enough to fill the chip (16 waves per CU when rows
// allow), but beyond one per CU only with four or more of its rows (or sets of rows) for
// each: every one costs a partial row to write and to add.  With a row or more, four or
// more, eight or more, bf16: 4096 x 1024 17.7 / 14.3 / 15.2 us, 2048 x 2048 15.5 / 13.0 / 14.9;
// 1537 x 1000 fp32 with a bias 17.6 / 13.0 / 15.0; 300 x 640 is fastest spread out, 5.9 / 7.9 / 10.9.
static int norm_backward_grid(int64_t rows, int64_t cols)
{
    const NormLayout l = norm_layout(cols);
    const int64_t cus = device_cu_count(), fill = cus * std::max(1, 1024 / l.threads), sets = (rows + l.rows - 1) / l.rows;
    return (int)std::min<int64_t>(fill, std::max<int64_t>((sets + 3) / 4, std::min<int64_t>(sets, cus)));
}

int64_t norm_backward_workspace(int64_t rows, int64_t cols)
{
    return (int64_t)norm_backward_grid(rows, cols) * cols * 4 * 2;
}

namespace {

template <typename Fn>
hipError_t norm_variant(bool f32, bool vec, const NormLayout& l, bool rms, Fn&& fn)
{
    auto pick_rms = [&](auto f, auto v, auto n, auto lanes) {
        return rms ? fn(f, v, n, lanes, std::true_type{}) : fn(f, v, n, lanes, std::false_type{});
    };
    auto pick_layout = [&](auto f, auto v) {
        using One = std::integral_constant<int, 1>;
        if (l.groups == 2) return pick_rms(f, v, std::integral_constant<int, 2>{}, std::integral_constant<int, 0>{});
        switch (l.lanes) {
        case 16: return pick_rms(f, v, One{}, std::integral_constant<int, 16>{});
        case 32: return pick_rms(f, v, One{}, std::integral_constant<int, 32>{});
        case 64: return pick_rms(f, v, One{}, std::integral_constant<int, 64>{});
        default: return pick_rms(f, v, One{}, std::integral_constant<int, 0>{});
        }
    };
    auto pick_vec = [&](auto f) {
        return vec ? pick_layout(f, std::true_type{}) : pick_layout(f, std::false_type{});
    };
    return f32 ? pick_vec(std::true_type{}) : pick_vec(std::false_type{});
}

}  // namespace

hipError_t launch_norm_forward(const void* x, bool f32, const void* add, const void* weight, const void* bias,
                               float eps, bool rms, int64_t rows, int64_t cols, void* y, void* sum, float* mean,
                               float* rstd, float* absmax, hipStream_t stream)
{
    const NormLayout l = norm_layout(cols);
    const int64_t most = max_workgroups(l.threads) * l.rows, size = f32 ? 4 : 2;   // rows of one launch; bytes
    auto after = [](auto* p, int64_t n) { return p ? p + n : p; };
    for (int64_t from = 0; from < rows; from += most) {
        const int64_t part = std::min(most, rows - from), at = from * cols;
        const hipError_t e = norm_variant(f32, cols % 8 == 0, l, rms, [&](auto f, auto v, auto n, auto lanes, auto ms) {
            return launch(norm_forward_kernel<f.value, v.value, n.value, lanes.value, ms.value>,
                          dim3((unsigned)((part + l.rows - 1) / l.rows)), dim3(l.threads), stream,
                          static_cast<const void*>(static_cast<const uint8_t*>(x) + at * size),
                          after(static_cast<const uint16_t*>(add), at), static_cast<const uint16_t*>(weight),
                          static_cast<const uint16_t*>(bias), eps, (uint32_t)part, (int)cols,
                          static_cast<uint16_t*>(y) + at, static_cast<void*>(after(static_cast<uint8_t*>(sum), at * size)),
                          after(mean, from), rstd + from, reinterpret_cast<uint32_t*>(absmax));
        });
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_norm_backward(const void* dy, const void* x, bool f32, const void* weight, const float* mean,
                                const float* rstd, const void* dres, bool rms, int64_t rows, int64_t cols, void* dx,
                                float* dw, float* db, float* partial, hipStream_t stream)
{
    const NormLayout l = norm_layout(cols);
    const int grid = norm_backward_grid(rows, cols);
    const hipError_t e = norm_variant(f32, cols % 8 == 0, l, rms, [&](auto f, auto v, auto n, auto lanes, auto ms) {
        return launch(norm_backward_kernel<f.value, v.value, n.value, lanes.value, ms.value>, dim3(grid),
                      dim3(l.threads), stream, static_cast<const uint16_t*>(dy), x,
                      static_cast<const uint16_t*>(weight), mean, rstd, dres, (uint32_t)rows, (int)cols, dx, partial,
                      db ? 1 : 0);
    });
    if (e != hipSuccess) return e;
    return launch(norm_join_kernel, dim3((unsigned)((cols + 31) / 32), db ? 2 : 1), dim3(1024), stream,
                  static_cast<const float*>(partial), grid, (int)cols, dw, db);
}

}  // namespace fp8k
