// api.cpp -- the C ABI of the FP8 hot path: argument checks, then launches.
//
// Every entry point validates its arguments on the host before enqueuing
// anything; see include/fp8_precision.h for the contract of each call.
#include "fp8_precision.h"

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <mutex>
#include <string>
#include <vector>

#include "fp8_internal.hpp"
#include "head_tensor.hpp"

namespace {

thread_local std::string t_last_error;

fp8_status fail(fp8_status st, const char* what)
{
    t_last_error = what;
    return st;
}

fp8_status fail(fp8_status st, const std::string& what)
{
    t_last_error = what;
    return st;
}

fp8_status fail_hip(const char* call, hipError_t e)
{
    char buf[256];
    std::snprintf(buf, sizeof(buf), "%s: HIP error %d (%s)", call, (int)e, hipGetErrorString(e));
    t_last_error = buf;
    return FP8_ERR_HIP;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Byte ranges [p, p + n) and [q, q + m) overlap.
bool overlap(const void* p, int64_t n, const void* q, int64_t m)
{
    if (!p || !q || n <= 0 || m <= 0) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + (uintptr_t)m && b < a + (uintptr_t)n;
}

struct Range {
    const void* p;
    int64_t n;
};

// True if any two of the ranges overlap.
template <int N>
bool any_overlap(const Range (&r)[N])
{
    for (int i = 0; i < N; ++i)
        for (int j = i + 1; j < N; ++j)
            if (overlap(r[i].p, r[i].n, r[j].p, r[j].n)) return true;
    return false;
}

bool mul_ok(int64_t a, int64_t b, int64_t limit) { return a > 0 && b > 0 && a <= limit / b; }

constexpr int64_t kMaxElems = (int64_t)1 << 40;

}  // namespace

namespace fp8k {

int device_cu_count()
{
    static std::mutex mu;
    static int cache[64] = {};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    std::lock_guard<std::mutex> lk(mu);
    if (cache[dev] == 0) {
        int cu = 0;
        if (hipDeviceGetAttribute(&cu, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cu <= 0)
            cu = 256;
        cache[dev] = cu;
    }
    return cache[dev];
}

}  // namespace fp8k

extern "C" {

const char* fp8_status_string(fp8_status s)
{
    switch (s) {
    case FP8_OK: return "ok";
    case FP8_ERR_INVALID: return "invalid argument";
    case FP8_ERR_UNSUPPORTED: return "unsupported argument (alignment or shape constraint)";
    case FP8_ERR_HIP: return "HIP runtime error";
    }
    return "unknown status";
}

const char* fp8_last_error(void) { return t_last_error.c_str(); }

static fp8_status absmax_common(const char* name, const void* x, int64_t n, float* absmax, bool accumulate,
                                hipStream_t stream)
{
    t_last_error.clear();
    const std::string f(name);
    if (!x || !absmax) return fail(FP8_ERR_INVALID, f + ": null pointer");
    if (n <= 0 || n > kMaxElems) return fail(FP8_ERR_INVALID, f + ": n must be in [1, 2^40]");
    if (overlap(x, 2 * n, absmax, 4)) return fail(FP8_ERR_INVALID, f + ": absmax overlaps x");
    if (!aligned(x, 16) || !aligned(absmax, 4))
        return fail(FP8_ERR_UNSUPPORTED, f + ": x must be 16-byte and absmax 4-byte aligned");
    hipError_t e = fp8k::launch_absmax_bf16(x, n, absmax, accumulate, stream);
    if (e != hipSuccess) return fail_hip(name, e);
    return FP8_OK;
}

fp8_status fp8_absmax(const void* x, int64_t n, float* absmax, hipStream_t stream)
{
    return absmax_common("fp8_absmax", x, n, absmax, false, stream);
}

fp8_status fp8_absmax_accumulate(const void* x, int64_t n, float* absmax, hipStream_t stream)
{
    return absmax_common("fp8_absmax_accumulate", x, n, absmax, true, stream);
}

fp8_status fp8_absmax_accumulate_many(int count, const void* const* x, const int64_t* n, float* const* absmax,
                                      hipStream_t stream)
{
    t_last_error.clear();
    const char* name = "fp8_absmax_accumulate_many";
    if (!x || !n || !absmax) return fail(FP8_ERR_INVALID, "fp8_absmax_accumulate_many: null array");
    if (count < 1 || count > fp8k::kMaxAbsTensors)
        return fail(FP8_ERR_INVALID, "fp8_absmax_accumulate_many: count must be in [1, 8]");
    for (int i = 0; i < count; ++i) {
        if (!x[i] || !absmax[i]) return fail(FP8_ERR_INVALID, "fp8_absmax_accumulate_many: null pointer");
        if (n[i] <= 0 || n[i] > kMaxElems)
            return fail(FP8_ERR_INVALID, "fp8_absmax_accumulate_many: every n must be in [1, 2^40]");
        if (!aligned(x[i], 16) || !aligned(absmax[i], 4))
            return fail(FP8_ERR_UNSUPPORTED, "fp8_absmax_accumulate_many: x 16-byte and absmax 4-byte aligned");
    }
    // an accumulator may be shared (the max is order-free), but none may lie inside an input
    for (int i = 0; i < count; ++i)
        for (int j = 0; j < count; ++j)
            if (overlap(x[j], 2 * n[j], absmax[i], 4))
                return fail(FP8_ERR_INVALID, "fp8_absmax_accumulate_many: an absmax overlaps an input");
    hipError_t e = fp8k::launch_absmax_many(count, x, n, absmax, stream);
    if (e != hipSuccess) return fail_hip(name, e);
    return FP8_OK;
}

fp8_status fp8_absmax_clear(float* absmax, int64_t count, hipStream_t stream)
{
    t_last_error.clear();
    if (!absmax) return fail(FP8_ERR_INVALID, "fp8_absmax_clear: null pointer");
    if (count < 1 || count > ((int64_t)1 << 20)) return fail(FP8_ERR_INVALID, "fp8_absmax_clear: count must be in [1, 2^20]");
    if (!aligned(absmax, 4)) return fail(FP8_ERR_UNSUPPORTED, "fp8_absmax_clear: absmax must be 4-byte aligned");
    hipError_t e = fp8k::launch_absmax_clear(absmax, count, stream);
    if (e != hipSuccess) return fail_hip("fp8_absmax_clear", e);
    return FP8_OK;
}

fp8_status fp8_quantize(const void* x, int64_t rows, int64_t cols, fp8_fmt fmt, const float* absmax,
                        uint8_t* q, uint8_t* qt, float* scale, float* inv_scale, hipStream_t stream)
{
    t_last_error.clear();
    if (!x || !absmax) return fail(FP8_ERR_INVALID, "fp8_quantize: null x or absmax");
    if (!q && !qt) return fail(FP8_ERR_INVALID, "fp8_quantize: at least one of q, qt is required");
    if (fmt != FP8_E4M3 && fmt != FP8_E5M2) return fail(FP8_ERR_INVALID, "fp8_quantize: bad format");
    if (!mul_ok(rows, cols, kMaxElems)) return fail(FP8_ERR_INVALID, "fp8_quantize: bad shape");
    const int64_t n = rows * cols;
    const Range r[] = {{x, 2 * n}, {absmax, 4}, {q, q ? n : 0}, {qt, qt ? n : 0},
                       {scale, scale ? 4 : 0}, {inv_scale, inv_scale ? 4 : 0}};
    if (any_overlap(r)) return fail(FP8_ERR_INVALID, "fp8_quantize: overlapping buffers");
    if (cols % 16) return fail(FP8_ERR_UNSUPPORTED, "fp8_quantize: cols must be a multiple of 16");
    if (qt && rows % 16) return fail(FP8_ERR_UNSUPPORTED, "fp8_quantize: rows must be a multiple of 16 with qt");
    if (qt && (rows + 127) / 128 > 65535) return fail(FP8_ERR_UNSUPPORTED, "fp8_quantize: too many rows for qt");
    if (!aligned(x, 16) || (q && !aligned(q, 16)) || (qt && !aligned(qt, 16)) || !aligned(absmax, 4) ||
        (scale && !aligned(scale, 4)) || (inv_scale && !aligned(inv_scale, 4)))
        return fail(FP8_ERR_UNSUPPORTED, "fp8_quantize: misaligned pointer");
    hipError_t e = fp8k::launch_quantize(x, rows, cols, (int)fmt, absmax, q, qt, scale, inv_scale, stream);
    if (e != hipSuccess) return fail_hip("fp8_quantize", e);
    return FP8_OK;
}

fp8_status fp8_quantize_many(int count, const void* const* x, const int64_t* rows, const int64_t* cols,
                             const fp8_fmt* fmt, const float* const* absmax, uint8_t* const* q, uint8_t* const* qt,
                             float* const* scale, float* const* inv_scale, const int* qt_later, hipStream_t stream)
{
    t_last_error.clear();
    const std::string f("fp8_quantize_many");
    if (!x || !rows || !cols || !fmt || !absmax || !q || !qt || !scale || !inv_scale)
        return fail(FP8_ERR_INVALID, f + ": null array");
    if (count < 1 || count > fp8k::kMaxQuantTensors) return fail(FP8_ERR_INVALID, f + ": count must be in [1, 8]");
    std::vector<Range> in, out;
    int64_t tiles = 0;
    int fm[fp8k::kMaxQuantTensors];
    for (int i = 0; i < count; ++i) {
        const std::string t = f + ": tensor " + std::to_string(i);
        if (!x[i] || !absmax[i]) return fail(FP8_ERR_INVALID, t + ": null x or absmax");
        if (!q[i] && !qt[i]) return fail(FP8_ERR_INVALID, t + ": at least one of q, qt is required");
        if (fmt[i] != FP8_E4M3 && fmt[i] != FP8_E5M2) return fail(FP8_ERR_INVALID, t + ": bad format");
        if (!mul_ok(rows[i], cols[i], kMaxElems)) return fail(FP8_ERR_INVALID, t + ": bad shape");
        if (rows[i] % 16 || cols[i] % 16)
            return fail(FP8_ERR_UNSUPPORTED, t + ": rows and cols must be multiples of 16");
        if (!aligned(x[i], 16) || (q[i] && !aligned(q[i], 16)) || (qt[i] && !aligned(qt[i], 16)) ||
            !aligned(absmax[i], 4) || (scale[i] && !aligned(scale[i], 4)) || (inv_scale[i] && !aligned(inv_scale[i], 4)))
            return fail(FP8_ERR_UNSUPPORTED, t + ": misaligned pointer");
        const int64_t n = rows[i] * cols[i];
        tiles += ((rows[i] + 127) / 128) * ((cols[i] + 127) / 128);
        in.push_back({x[i], 2 * n});
        in.push_back({absmax[i], 4});
        out.push_back({q[i], q[i] ? n : 0});
        out.push_back({qt[i], qt[i] ? n : 0});
        out.push_back({scale[i], scale[i] ? 4 : 0});
        out.push_back({inv_scale[i], inv_scale[i] ? 4 : 0});
        fm[i] = (int)fmt[i];
    }
    if (tiles > 0x7FFFFFFF) return fail(FP8_ERR_UNSUPPORTED, f + ": too many tiles for one launch");
    // inputs may be shared (they are only read); no output may overlap an input or another output
    for (size_t a = 0; a < out.size(); ++a) {
        for (size_t b = a + 1; b < out.size(); ++b)
            if (overlap(out[a].p, out[a].n, out[b].p, out[b].n)) return fail(FP8_ERR_INVALID, f + ": overlapping outputs");
        for (const Range& r : in)
            if (overlap(out[a].p, out[a].n, r.p, r.n)) return fail(FP8_ERR_INVALID, f + ": an output overlaps an input");
    }
    hipError_t e = fp8k::launch_quantize_many(count, x, rows, cols, fm, absmax, q, qt, scale, inv_scale, qt_later,
                                              stream);
    if (e != hipSuccess) return fail_hip("fp8_quantize_many", e);
    return FP8_OK;
}

fp8_status fp8_swiglu_requant(const void* gu, int64_t M, int64_t F, float* absmax_h, int compute_absmax,
                              uint8_t* hq, uint8_t* hqt, float* inv_scale_h, hipStream_t stream)
{
    t_last_error.clear();
    if (!gu || !absmax_h) return fail(FP8_ERR_INVALID, "fp8_swiglu_requant: null gu or absmax_h");
    if (!hq && !hqt) return fail(FP8_ERR_INVALID, "fp8_swiglu_requant: at least one of hq, hqt is required");
    if (compute_absmax < 0 || compute_absmax > 2)
        return fail(FP8_ERR_INVALID, "fp8_swiglu_requant: compute_absmax must be 0, 1 or 2");
    if (F <= 0 || F > kMaxElems || !mul_ok(M, 2 * F, kMaxElems))
        return fail(FP8_ERR_INVALID, "fp8_swiglu_requant: bad shape");
    const int64_t n = M * F;
    const Range r[] = {{gu, 4 * n}, {absmax_h, 4}, {hq, hq ? n : 0}, {hqt, hqt ? n : 0},
                       {inv_scale_h, inv_scale_h ? 4 : 0}};
    if (any_overlap(r)) return fail(FP8_ERR_INVALID, "fp8_swiglu_requant: overlapping buffers");
    if (F % 16) return fail(FP8_ERR_UNSUPPORTED, "fp8_swiglu_requant: F must be a multiple of 16");
    if (hqt && M % 16) return fail(FP8_ERR_UNSUPPORTED, "fp8_swiglu_requant: M must be a multiple of 16 with hqt");
    if (!aligned(gu, 16) || (hq && !aligned(hq, 16)) || (hqt && !aligned(hqt, 16)) || !aligned(absmax_h, 4) ||
        (inv_scale_h && !aligned(inv_scale_h, 4)))
        return fail(FP8_ERR_UNSUPPORTED, "fp8_swiglu_requant: misaligned pointer");
    hipError_t e = fp8k::launch_swiglu_requant(gu, M, F, absmax_h, compute_absmax, hq, hqt, inv_scale_h, stream);
    if (e != hipSuccess) return fail_hip("fp8_swiglu_requant", e);
    return FP8_OK;
}

fp8_status fp8_swiglu_backward(const void* gu, const void* dh, int64_t M, int64_t F, fp8_fmt fmt, float* absmax,
                               uint8_t* q, uint8_t* qt, float* scale, float* inv_scale, hipStream_t stream)
{
    t_last_error.clear();
    if (!gu || !dh || !absmax) return fail(FP8_ERR_INVALID, "fp8_swiglu_backward: null gu, dh or absmax");
    if (!q && !qt) return fail(FP8_ERR_INVALID, "fp8_swiglu_backward: at least one of q, qt is required");
    if (fmt != FP8_E4M3 && fmt != FP8_E5M2) return fail(FP8_ERR_INVALID, "fp8_swiglu_backward: bad format");
    if (F <= 0 || F > kMaxElems || !mul_ok(M, 2 * F, kMaxElems))
        return fail(FP8_ERR_INVALID, "fp8_swiglu_backward: bad shape");
    const int64_t n = M * F;
    const Range r[] = {{gu, 4 * n}, {dh, 2 * n}, {absmax, 4}, {q, q ? 2 * n : 0}, {qt, qt ? 2 * n : 0},
                       {scale, scale ? 4 : 0}, {inv_scale, inv_scale ? 4 : 0}};
    // the two inputs may alias each other; no output may alias anything
    for (int i = 2; i < 7; ++i)
        for (int j = 0; j < 7; ++j)
            if (i != j && overlap(r[i].p, r[i].n, r[j].p, r[j].n))
                return fail(FP8_ERR_INVALID, "fp8_swiglu_backward: overlapping buffers");
    if (F % 16) return fail(FP8_ERR_UNSUPPORTED, "fp8_swiglu_backward: F must be a multiple of 16");
    if (qt && M % 16) return fail(FP8_ERR_UNSUPPORTED, "fp8_swiglu_backward: M must be a multiple of 16 with qt");
    if (!aligned(gu, 16) || !aligned(dh, 16) || (q && !aligned(q, 16)) || (qt && !aligned(qt, 16)) ||
        !aligned(absmax, 4) || (scale && !aligned(scale, 4)) || (inv_scale && !aligned(inv_scale, 4)))
        return fail(FP8_ERR_UNSUPPORTED, "fp8_swiglu_backward: misaligned pointer");
    hipError_t e = fp8k::launch_swiglu_backward(gu, dh, M, F, (int)fmt, absmax, q, qt, scale, inv_scale, stream);
    if (e != hipSuccess) return fail_hip("fp8_swiglu_backward", e);
    return FP8_OK;
}

// Shared checks of the three GEMM calls, in the TN form out[P, Q] = A[P, R] . B[Q, R]^T.
// The block-scaled call passes need_inv = false (it has no per-tensor factors).
static fp8_status gemm_common(const char* name, const uint8_t* A, int fmt_a, const uint8_t* B, const float* inv_a,
                              const float* inv_b, void* out, int64_t P, int64_t Q, int64_t R, hipStream_t stream,
                              bool need_inv = true)
{
    char msg[160];
    if (!A || !B || (need_inv && (!inv_a || !inv_b)) || !out) {
        std::snprintf(msg, sizeof(msg), "%s: null pointer", name);
        return fail(FP8_ERR_INVALID, msg);
    }
    if (fmt_a != FP8_E4M3 && fmt_a != FP8_E5M2) {
        std::snprintf(msg, sizeof(msg), "%s: bad operand format", name);
        return fail(FP8_ERR_INVALID, msg);
    }
    if (P <= 0 || Q <= 0 || R <= 0) {
        std::snprintf(msg, sizeof(msg), "%s: dimensions must be positive", name);
        return fail(FP8_ERR_INVALID, msg);
    }
    // bound each dimension before forming any product (P * R, 2 * P * Q stay far below 2^63)
    if (P >= ((int64_t)1 << 30) || Q >= ((int64_t)1 << 30) || R >= ((int64_t)1 << 31)) {
        std::snprintf(msg, sizeof(msg), "%s: operand larger than 2 GiB", name);
        return fail(FP8_ERR_UNSUPPORTED, msg);
    }
    const Range r[] = {{A, P * R}, {B, Q * R}, {inv_a, need_inv ? 4 : 0}, {inv_b, need_inv ? 4 : 0},
                       {out, 2 * P * Q}};
    // the two inputs may alias each other (e.g. A == B); the output may alias nothing
    for (int i = 0; i < 4; ++i)
        if (overlap(r[i].p, r[i].n, r[4].p, r[4].n)) {
            std::snprintf(msg, sizeof(msg), "%s: output overlaps an input", name);
            return fail(FP8_ERR_INVALID, msg);
        }
    if (P % 16 || Q % 16 || R % 128 || P < 16 || Q < 16) {
        std::snprintf(msg, sizeof(msg), "%s: output dimensions must be multiples of 16, the reduction a multiple of 128",
                      name);
        return fail(FP8_ERR_UNSUPPORTED, msg);
    }
    if (P * R >= ((int64_t)1 << 31) || Q * R >= ((int64_t)1 << 31) || P >= ((int64_t)1 << 30) ||
        Q >= ((int64_t)1 << 30) || ((P + 255) / 256) * ((Q + 255) / 256) >= ((int64_t)1 << 31)) {
        std::snprintf(msg, sizeof(msg), "%s: operand larger than 2 GiB", name);
        return fail(FP8_ERR_UNSUPPORTED, msg);
    }
    if (!aligned(A, 16) || !aligned(B, 16) || !aligned(out, 16) || (need_inv && (!aligned(inv_a, 4) || !aligned(inv_b, 4)))) {
        std::snprintf(msg, sizeof(msg), "%s: misaligned pointer", name);
        return fail(FP8_ERR_UNSUPPORTED, msg);
    }
    (void)stream;
    return FP8_OK;
}

fp8_status fp8_gemm_fwd(const uint8_t* xq, const uint8_t* wq, const float* inv_sx, const float* inv_sw, void* y,
                        int64_t M, int64_t N, int64_t K, hipStream_t stream)
{
    t_last_error.clear();
    fp8_status st = gemm_common("fp8_gemm_fwd", xq, FP8_E4M3, wq, inv_sx, inv_sw, y, M, N, K, stream);
    if (st != FP8_OK) return st;
    // Y is stored non-temporally when it is too large to stay in the 256 MiB Infinity
    // Cache for the pass that reads it next while the operands are small enough to
    // stay there: then ordinary stores would only push out the operand panels the
    // launch keeps re-reading.  Measured on MI355X: the 14B-class gate/up forward
    // (453 MB out, 183 MB in) 9.6% faster, the step 1.6% shorter; with operands that
    // do not fit either (the 32B-class gate/up forward, 367 MB in) non-temporal
    // stores were 1% slower, and below 256 MiB of output (every 7B-class forward)
    // the next pass reads Y from the cache.
    const int64_t cache_bytes = (int64_t)256 << 20;
    const bool nt = 2 * M * N >= cache_bytes && (M + N) * K <= cache_bytes;
    hipError_t e = fp8k::launch_gemm_tn(xq, 0, 0, wq, 0, 0, inv_sx, inv_sw, y, M, N, K, nt, stream);
    if (e != hipSuccess) return fail_hip("fp8_gemm_fwd", e);
    return FP8_OK;
}

fp8_status fp8_gemm_fwd_swiglu_absmax(const uint8_t* xq, const uint8_t* wq, const float* inv_sx,
                                      const float* inv_sw, void* gu, float* absmax_h, int64_t M, int64_t F,
                                      int64_t K, hipStream_t stream)
{
    t_last_error.clear();
    const char* name = "fp8_gemm_fwd_swiglu_absmax";
    if (!absmax_h) return fail(FP8_ERR_INVALID, "fp8_gemm_fwd_swiglu_absmax: null absmax_h");
    if (F <= 0 || F > ((int64_t)1 << 29)) return fail(FP8_ERR_INVALID, "fp8_gemm_fwd_swiglu_absmax: bad F");
    fp8_status st = gemm_common(name, xq, FP8_E4M3, wq, inv_sx, inv_sw, gu, M, 2 * F, K, stream);
    if (st != FP8_OK) return st;
    const Range r[] = {{xq, M * K}, {wq, 2 * F * K}, {inv_sx, 4}, {inv_sw, 4}, {gu, 2 * M * 2 * F}};
    for (const Range& x : r)
        if (overlap(x.p, x.n, absmax_h, 4))
            return fail(FP8_ERR_INVALID, "fp8_gemm_fwd_swiglu_absmax: absmax_h overlaps another buffer");
    if (!aligned(absmax_h, 4)) return fail(FP8_ERR_UNSUPPORTED, "fp8_gemm_fwd_swiglu_absmax: misaligned absmax_h");
    if (F % 128 || M < 256)
        return fail(FP8_ERR_UNSUPPORTED, "fp8_gemm_fwd_swiglu_absmax: needs F % 128 == 0 and M >= 256");
    hipError_t e = fp8k::launch_gemm_gate_up(xq, wq, inv_sx, inv_sw, gu, absmax_h, M, F, K, stream);
    if (e != hipSuccess) return fail_hip(name, e);
    return FP8_OK;
}

fp8_status fp8_gemm_dgrad(const uint8_t* dyq, fp8_fmt dy_fmt, const uint8_t* wqt, const float* inv_sdy,
                          const float* inv_sw, void* dx, int64_t M, int64_t N, int64_t K, hipStream_t stream)
{
    t_last_error.clear();
    fp8_status st = gemm_common("fp8_gemm_dgrad", dyq, (int)dy_fmt, wqt, inv_sdy, inv_sw, dx, M, K, N, stream);
    if (st != FP8_OK) return st;
    hipError_t e = fp8k::launch_gemm_tn(dyq, (int)dy_fmt, 0, wqt, 0, 0, inv_sdy, inv_sw, dx, M, K, N, true, stream);
    if (e != hipSuccess) return fail_hip("fp8_gemm_dgrad", e);
    return FP8_OK;
}

fp8_status fp8_gemm_wgrad(const uint8_t* dyqt, fp8_fmt dy_fmt, const uint8_t* xqt, const float* inv_sdy,
                          const float* inv_sx, void* dw, int64_t M, int64_t N, int64_t K, hipStream_t stream)
{
    t_last_error.clear();
    fp8_status st = gemm_common("fp8_gemm_wgrad", dyqt, (int)dy_fmt, xqt, inv_sdy, inv_sx, dw, N, K, M, stream);
    if (st != FP8_OK) return st;
    hipError_t e = fp8k::launch_gemm_tn(dyqt, (int)dy_fmt, 0, xqt, 0, 0, inv_sdy, inv_sx, dw, N, K, M, true, stream);
    if (e != hipSuccess) return fail_hip("fp8_gemm_wgrad", e);
    return FP8_OK;
}

fp8_status fp8_gemm_backward(const uint8_t* dyq, const uint8_t* dyqt, fp8_fmt dy_fmt, const uint8_t* wqt,
                             const uint8_t* xqt, const float* inv_sdy, const float* inv_sw, const float* inv_sx,
                             void* dx, void* dw, int64_t M, int64_t N, int64_t K, hipStream_t stream)
{
    t_last_error.clear();
    fp8_status st = gemm_common("fp8_gemm_backward (dgrad)", dyq, (int)dy_fmt, wqt, inv_sdy, inv_sw, dx, M, K, N, stream);
    if (st != FP8_OK) return st;
    st = gemm_common("fp8_gemm_backward (wgrad)", dyqt, (int)dy_fmt, xqt, inv_sdy, inv_sx, dw, N, K, M, stream);
    if (st != FP8_OK) return st;
    const Range outs[] = {{dx, 2 * M * K}, {dw, 2 * N * K}};
    const Range ins[] = {{dyq, M * N}, {dyqt, M * N}, {wqt, K * N}, {xqt, K * M},
                         {inv_sdy, 4}, {inv_sw, 4}, {inv_sx, 4}};
    if (overlap(dx, 2 * M * K, dw, 2 * N * K))
        return fail(FP8_ERR_INVALID, "fp8_gemm_backward: dx and dw overlap");
    for (const Range& o : outs)
        for (const Range& i : ins)
            if (overlap(o.p, o.n, i.p, i.n)) return fail(FP8_ERR_INVALID, "fp8_gemm_backward: an output overlaps an input");
    hipError_t e = fp8k::launch_gemm_tn_pair(dyq, 0, wqt, 0, inv_sdy, inv_sw, dx, M, K, N, dyqt, 0, xqt, 0, inv_sdy,
                                             inv_sx, dw, N, K, M, (int)dy_fmt, 0, stream);
    if (e != hipSuccess) return fail_hip("fp8_gemm_backward", e);
    return FP8_OK;
}

// ---- the same products on the untransposed FP8 tensors (MN-major operands)

fp8_status fp8_gemm_dgrad_mn(const uint8_t* dyq, fp8_fmt dy_fmt, const uint8_t* wq, const float* inv_sdy,
                             const float* inv_sw, void* dx, int64_t M, int64_t N, int64_t K, hipStream_t stream)
{
    t_last_error.clear();
    fp8_status st = gemm_common("fp8_gemm_dgrad_mn", dyq, (int)dy_fmt, wq, inv_sdy, inv_sw, dx, M, K, N, stream);
    if (st != FP8_OK) return st;
    hipError_t e = fp8k::launch_gemm_tn(dyq, (int)dy_fmt, 0, wq, 0, 1, inv_sdy, inv_sw, dx, M, K, N, true, stream);
    if (e != hipSuccess) return fail_hip("fp8_gemm_dgrad_mn", e);
    return FP8_OK;
}

fp8_status fp8_gemm_wgrad_mn(const uint8_t* dyq, fp8_fmt dy_fmt, const uint8_t* xq, const float* inv_sdy,
                             const float* inv_sx, void* dw, int64_t M, int64_t N, int64_t K, hipStream_t stream)
{
    t_last_error.clear();
    fp8_status st = gemm_common("fp8_gemm_wgrad_mn", dyq, (int)dy_fmt, xq, inv_sdy, inv_sx, dw, N, K, M, stream);
    if (st != FP8_OK) return st;
    hipError_t e = fp8k::launch_gemm_tn(dyq, (int)dy_fmt, 1, xq, 0, 1, inv_sdy, inv_sx, dw, N, K, M, true, stream);
    if (e != hipSuccess) return fail_hip("fp8_gemm_wgrad_mn", e);
    return FP8_OK;
}

fp8_status fp8_gemm_backward_mn(const uint8_t* dyq, fp8_fmt dy_fmt, const uint8_t* wq, const uint8_t* xq,
                                const float* inv_sdy, const float* inv_sw, const float* inv_sx, void* dx, void* dw,
                                int64_t M, int64_t N, int64_t K, hipStream_t stream)
{
    t_last_error.clear();
    fp8_status st = gemm_common("fp8_gemm_backward_mn (dgrad)", dyq, (int)dy_fmt, wq, inv_sdy, inv_sw, dx, M, K, N,
                                stream);
    if (st != FP8_OK) return st;
    st = gemm_common("fp8_gemm_backward_mn (wgrad)", dyq, (int)dy_fmt, xq, inv_sdy, inv_sx, dw, N, K, M, stream);
    if (st != FP8_OK) return st;
    const Range outs[] = {{dx, 2 * M * K}, {dw, 2 * N * K}};
    const Range ins[] = {{dyq, M * N}, {wq, K * N}, {xq, K * M}, {inv_sdy, 4}, {inv_sw, 4}, {inv_sx, 4}};
    if (overlap(dx, 2 * M * K, dw, 2 * N * K))
        return fail(FP8_ERR_INVALID, "fp8_gemm_backward_mn: dx and dw overlap");
    for (const Range& o : outs)
        for (const Range& i : ins)
            if (overlap(o.p, o.n, i.p, i.n))
                return fail(FP8_ERR_INVALID, "fp8_gemm_backward_mn: an output overlaps an input");
    hipError_t e = fp8k::launch_gemm_tn_pair(dyq, 0, wq, 1, inv_sdy, inv_sw, dx, M, K, N, dyq, 1, xq, 1, inv_sdy,
                                             inv_sx, dw, N, K, M, (int)dy_fmt, 0, stream);
    if (e != hipSuccess) return fail_hip("fp8_gemm_backward_mn", e);
    return FP8_OK;
}

fp8_status fp8_mx_quantize(const void* x, int64_t rows, int64_t cols, fp8_fmt fmt, uint8_t* q, uint8_t* scales,
                           hipStream_t stream)
{
    t_last_error.clear();
    if (!x || !q || !scales) return fail(FP8_ERR_INVALID, "fp8_mx_quantize: null pointer");
    if (fmt != FP8_E4M3 && fmt != FP8_E5M2) return fail(FP8_ERR_INVALID, "fp8_mx_quantize: bad format");
    if (!mul_ok(rows, cols, kMaxElems)) return fail(FP8_ERR_INVALID, "fp8_mx_quantize: bad shape");
    const int64_t n = rows * cols;
    const Range r[] = {{x, 2 * n}, {q, n}, {scales, n / 32}};
    if (any_overlap(r)) return fail(FP8_ERR_INVALID, "fp8_mx_quantize: overlapping buffers");
    if (cols % 128) return fail(FP8_ERR_UNSUPPORTED, "fp8_mx_quantize: cols must be a multiple of 128");
    if (n / 32 >= ((int64_t)1 << 32)) return fail(FP8_ERR_UNSUPPORTED, "fp8_mx_quantize: more than 2^32 blocks");
    if (!aligned(x, 16) || !aligned(q, 16)) return fail(FP8_ERR_UNSUPPORTED, "fp8_mx_quantize: misaligned pointer");
    hipError_t e = fp8k::launch_mx_quantize(x, rows, cols, (int)fmt, q, scales, stream);
    if (e != hipSuccess) return fail_hip("fp8_mx_quantize", e);
    return FP8_OK;
}

fp8_status fp8_mx_quantize_t(const void* x, int64_t rows, int64_t cols, fp8_fmt fmt, uint8_t* qt, uint8_t* scales,
                             hipStream_t stream)
{
    t_last_error.clear();
    if (!x || !qt || !scales) return fail(FP8_ERR_INVALID, "fp8_mx_quantize_t: null pointer");
    if (fmt != FP8_E4M3 && fmt != FP8_E5M2) return fail(FP8_ERR_INVALID, "fp8_mx_quantize_t: bad format");
    if (!mul_ok(rows, cols, kMaxElems)) return fail(FP8_ERR_INVALID, "fp8_mx_quantize_t: bad shape");
    const int64_t n = rows * cols;
    const Range r[] = {{x, 2 * n}, {qt, n}, {scales, n / 32}};
    if (any_overlap(r)) return fail(FP8_ERR_INVALID, "fp8_mx_quantize_t: overlapping buffers");
    if (rows % 128 || cols % 128) return fail(FP8_ERR_UNSUPPORTED, "fp8_mx_quantize_t: rows and cols must be multiples of 128");
    if (!aligned(x, 16) || !aligned(qt, 16) || !aligned(scales, 4))
        return fail(FP8_ERR_UNSUPPORTED, "fp8_mx_quantize_t: misaligned pointer");
    hipError_t e = fp8k::launch_mx_quantize_t(x, rows, cols, (int)fmt, qt, scales, stream);
    if (e != hipSuccess) return fail_hip("fp8_mx_quantize_t", e);
    return FP8_OK;
}

fp8_status fp8_mx_quantize_both(const void* x, int64_t rows, int64_t cols, fp8_fmt fmt, uint8_t* q, uint8_t* sq,
                                uint8_t* qt, uint8_t* sqt, hipStream_t stream)
{
    t_last_error.clear();
    if (!x || !q || !sq || !qt || !sqt) return fail(FP8_ERR_INVALID, "fp8_mx_quantize_both: null pointer");
    if (fmt != FP8_E4M3 && fmt != FP8_E5M2) return fail(FP8_ERR_INVALID, "fp8_mx_quantize_both: bad format");
    if (!mul_ok(rows, cols, kMaxElems)) return fail(FP8_ERR_INVALID, "fp8_mx_quantize_both: bad shape");
    const int64_t n = rows * cols;
    const Range r[] = {{x, 2 * n}, {q, n}, {sq, n / 32}, {qt, n}, {sqt, n / 32}};
    if (any_overlap(r)) return fail(FP8_ERR_INVALID, "fp8_mx_quantize_both: overlapping buffers");
    if (rows % 128 || cols % 128) return fail(FP8_ERR_UNSUPPORTED, "fp8_mx_quantize_both: rows and cols must be multiples of 128");
    if (n / 32 >= ((int64_t)1 << 31)) return fail(FP8_ERR_UNSUPPORTED, "fp8_mx_quantize_both: tensor too large");
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(qt, 16) || !aligned(sq, 4) || !aligned(sqt, 4))
        return fail(FP8_ERR_UNSUPPORTED, "fp8_mx_quantize_both: misaligned pointer");
    hipError_t e = fp8k::launch_mx_quantize_both(x, rows, cols, (int)fmt, q, sq, qt, sqt, stream);
    if (e != hipSuccess) return fail_hip("fp8_mx_quantize_both", e);
    return FP8_OK;
}

fp8_status fp8_mx_swiglu_requant(const void* gu, int64_t M, int64_t F, uint8_t* hq, uint8_t* scales,
                                 hipStream_t stream)
{
    t_last_error.clear();
    if (!gu || !hq || !scales) return fail(FP8_ERR_INVALID, "fp8_mx_swiglu_requant: null pointer");
    if (M <= 0 || F <= 0 || !mul_ok(M, 2 * F, kMaxElems)) return fail(FP8_ERR_INVALID, "fp8_mx_swiglu_requant: bad shape");
    const Range r[] = {{gu, 4 * M * F}, {hq, M * F}, {scales, M * F / 32}};
    if (any_overlap(r)) return fail(FP8_ERR_INVALID, "fp8_mx_swiglu_requant: overlapping buffers");
    if (F % 128) return fail(FP8_ERR_UNSUPPORTED, "fp8_mx_swiglu_requant: F must be a multiple of 128");
    if (!aligned(gu, 16) || !aligned(hq, 16)) return fail(FP8_ERR_UNSUPPORTED, "fp8_mx_swiglu_requant: misaligned pointer");
    hipError_t e = fp8k::launch_mx_swiglu(gu, M, F, hq, scales, stream);
    if (e != hipSuccess) return fail_hip("fp8_mx_swiglu_requant", e);
    return FP8_OK;
}

fp8_status fp8_mx_gemm_fwd(const uint8_t* xq, const uint8_t* sx, fp8_fmt x_fmt, const uint8_t* wq, const uint8_t* sw,
                           void* y, int64_t M, int64_t N, int64_t K, hipStream_t stream)
{
    t_last_error.clear();
    const char* name = "fp8_mx_gemm_fwd";
    if (!sx || !sw) return fail(FP8_ERR_INVALID, "fp8_mx_gemm_fwd: null scales");
    fp8_status st = gemm_common(name, xq, (int)x_fmt, wq, nullptr, nullptr, y, M, N, K, stream, false);
    if (st != FP8_OK) return st;
    if (overlap(sx, M * (K / 32), y, 2 * M * N) || overlap(sw, N * (K / 32), y, 2 * M * N))
        return fail(FP8_ERR_INVALID, "fp8_mx_gemm_fwd: output overlaps the scales");
    if (M < 256 || N < 256) return fail(FP8_ERR_UNSUPPORTED, "fp8_mx_gemm_fwd: M and N must be at least 256");
    if (!aligned(sx, 4) || !aligned(sw, 4)) return fail(FP8_ERR_UNSUPPORTED, "fp8_mx_gemm_fwd: misaligned scales");
    hipError_t e = fp8k::launch_gemm_mx(xq, sx, (int)x_fmt, wq, sw, 0, y, M, N, K, stream);
    if (e != hipSuccess) return fail_hip(name, e);
    return FP8_OK;
}

fp8_status fp8_mx_gemm_backward(const uint8_t* dyq, const uint8_t* sdy, const uint8_t* dyqt, const uint8_t* sdyt,
                                fp8_fmt dy_fmt, const uint8_t* wqt, const uint8_t* swt, const uint8_t* xqt,
                                const uint8_t* sxt, void* dx, void* dw, int64_t M, int64_t N, int64_t K,
                                hipStream_t stream)
{
    t_last_error.clear();
    const char* name = "fp8_mx_gemm_backward";
    if (!sdy || !sdyt || !swt || !sxt) return fail(FP8_ERR_INVALID, "fp8_mx_gemm_backward: null scales");
    fp8_status st = gemm_common("fp8_mx_gemm_backward (dgrad)", dyq, (int)dy_fmt, wqt, nullptr, nullptr, dx, M, K, N,
                                stream, false);
    if (st != FP8_OK) return st;
    st = gemm_common("fp8_mx_gemm_backward (wgrad)", dyqt, (int)dy_fmt, xqt, nullptr, nullptr, dw, N, K, M, stream,
                     false);
    if (st != FP8_OK) return st;
    if (M < 256 || N < 256 || K < 256)
        return fail(FP8_ERR_UNSUPPORTED, "fp8_mx_gemm_backward: M, N and K must be at least 256");
    if (!aligned(sdy, 4) || !aligned(sdyt, 4) || !aligned(swt, 4) || !aligned(sxt, 4))
        return fail(FP8_ERR_UNSUPPORTED, "fp8_mx_gemm_backward: misaligned scales");
    if (overlap(dx, 2 * M * K, dw, 2 * N * K)) return fail(FP8_ERR_INVALID, "fp8_mx_gemm_backward: dx and dw overlap");
    const Range outs[] = {{dx, 2 * M * K}, {dw, 2 * N * K}};
    const Range ins[] = {{dyq, M * N},       {dyqt, M * N},       {wqt, K * N},       {xqt, K * M},
                         {sdy, M * N / 32}, {sdyt, M * N / 32}, {swt, K * N / 32}, {sxt, K * M / 32}};
    for (const Range& o : outs)
        for (const Range& i : ins)
            if (overlap(o.p, o.n, i.p, i.n))
                return fail(FP8_ERR_INVALID, "fp8_mx_gemm_backward: an output overlaps an input");
    hipError_t e = fp8k::launch_gemm_mx_pair(dyq, sdy, wqt, swt, dx, M, K, N, dyqt, sdyt, xqt, sxt, dw, N, K, M,
                                             (int)dy_fmt, stream);
    if (e != hipSuccess) return fail_hip(name, e);
    return FP8_OK;
}

// ---- the operators around the linears: norm, attention, loss

// No output of out[] may overlap an input of in[] or another output.
static bool outputs_overlap(const Range* out, int n_out, const Range* in, int n_in)
{
    for (int a = 0; a < n_out; ++a) {
        for (int b = a + 1; b < n_out; ++b)
            if (overlap(out[a].p, out[a].n, out[b].p, out[b].n)) return true;
        for (int b = 0; b < n_in; ++b)
            if (overlap(out[a].p, out[a].n, in[b].p, in[b].n)) return true;
    }
    return false;
}

static bool norm_shape_ok(int64_t rows, int64_t cols)
{
    return rows >= 1 && rows < ((int64_t)1 << 31) && cols >= 1 && cols <= 16384;
}

fp8_status fp8_norm_forward(const void* x, fp8_stream_type type, const void* add, const void* weight,
                            const void* bias, float eps, fp8_norm_kind kind, int64_t rows, int64_t cols, void* y,
                            void* sum, float* mean, float* rstd, float* absmax, hipStream_t stream)
{
    t_last_error.clear();
    if (type != FP8_STREAM_BF16 && type != FP8_STREAM_F32) return fail(FP8_ERR_INVALID, "fp8_norm_forward: bad stream type");
    if (kind != FP8_NORM_RMS && kind != FP8_NORM_LAYER) return fail(FP8_ERR_INVALID, "fp8_norm_forward: bad norm kind");
    const bool rms = kind == FP8_NORM_RMS, f32 = type == FP8_STREAM_F32;
    if (rows < 1 || cols < 1) return fail(FP8_ERR_INVALID, "fp8_norm_forward: rows and cols must be positive");
    if (!x || !weight || !y || !rstd || (!rms && !mean)) return fail(FP8_ERR_INVALID, "fp8_norm_forward: null pointer");
    if (rms && (mean || bias)) return fail(FP8_ERR_INVALID, "fp8_norm_forward: a root-mean-square norm has no mean and no bias");
    if (!add != !sum) return fail(FP8_ERR_INVALID, "fp8_norm_forward: add and sum go together");
    if (!(eps >= 0.0f)) return fail(FP8_ERR_INVALID, "fp8_norm_forward: eps must be at least 0");
    if (!norm_shape_ok(rows, cols)) return fail(FP8_ERR_UNSUPPORTED, "fp8_norm_forward: rows < 2^31 and cols <= 16384");
    const int64_t n = rows * cols, size = f32 ? 4 : 2;
    const Range in[] = {{x, n * size}, {add, 2 * n}, {weight, 2 * cols}, {bias, 2 * cols}};
    const Range out[] = {{y, 2 * n}, {sum, n * size}, {mean, 4 * rows}, {rstd, 4 * rows}, {absmax, 4}};
    if (outputs_overlap(out, 5, in, 4)) return fail(FP8_ERR_INVALID, "fp8_norm_forward: overlapping buffers");
    if (!aligned(x, 16) || !aligned(add, 16) || !aligned(weight, 16) || !aligned(bias, 16) || !aligned(y, 16) ||
        !aligned(sum, 16) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(absmax, 4))
        return fail(FP8_ERR_UNSUPPORTED, "fp8_norm_forward: misaligned pointer");
    hipError_t e = fp8k::launch_norm_forward(x, f32, add, weight, bias, eps, rms, rows, cols, y, sum, mean, rstd, absmax, stream);
    if (e != hipSuccess) return fail_hip("fp8_norm_forward", e);
    return FP8_OK;
}

fp8_status fp8_norm_backward_workspace(int64_t rows, int64_t cols, int64_t* bytes)
{
    t_last_error.clear();
    if (!bytes) return fail(FP8_ERR_INVALID, "fp8_norm_backward_workspace: null pointer");
    if (rows < 1 || cols < 1) return fail(FP8_ERR_INVALID, "fp8_norm_backward_workspace: rows and cols must be positive");
    if (!norm_shape_ok(rows, cols))
        return fail(FP8_ERR_UNSUPPORTED, "fp8_norm_backward_workspace: rows < 2^31 and cols <= 16384");
    *bytes = fp8k::norm_backward_workspace(rows, cols);
    return FP8_OK;
}

fp8_status fp8_norm_backward(const void* dy, const void* s, fp8_stream_type type, const void* weight,
                             const float* mean, const float* rstd, const void* dres, fp8_norm_kind kind,
                             int64_t rows, int64_t cols, void* dx, float* dweight, float* dbias, void* workspace,
                             int64_t workspace_bytes, hipStream_t stream)
{
    t_last_error.clear();
    if (type != FP8_STREAM_BF16 && type != FP8_STREAM_F32) return fail(FP8_ERR_INVALID, "fp8_norm_backward: bad stream type");
    if (kind != FP8_NORM_RMS && kind != FP8_NORM_LAYER) return fail(FP8_ERR_INVALID, "fp8_norm_backward: bad norm kind");
    const bool rms = kind == FP8_NORM_RMS, f32 = type == FP8_STREAM_F32;
    if (rows < 1 || cols < 1) return fail(FP8_ERR_INVALID, "fp8_norm_backward: rows and cols must be positive");
    if (!dy || !s || !weight || !rstd || !dx || !dweight || !workspace || (!rms && !mean))
        return fail(FP8_ERR_INVALID, "fp8_norm_backward: null pointer");
    if (rms && (mean || dbias)) return fail(FP8_ERR_INVALID, "fp8_norm_backward: a root-mean-square norm has no mean and no bias");
    if (!norm_shape_ok(rows, cols)) return fail(FP8_ERR_UNSUPPORTED, "fp8_norm_backward: rows < 2^31 and cols <= 16384");
    if (workspace_bytes < fp8k::norm_backward_workspace(rows, cols))
        return fail(FP8_ERR_INVALID, "fp8_norm_backward: workspace too small");
    const int64_t n = rows * cols, size = f32 ? 4 : 2;
    const Range in[] = {{dy, 2 * n}, {s, n * size}, {weight, 2 * cols}, {mean, 4 * rows}, {rstd, 4 * rows}, {dres, n * size}};
    const Range out[] = {{dx, n * size}, {dweight, 4 * cols}, {dbias, 4 * cols}, {workspace, workspace_bytes}};
    if (outputs_overlap(out, 4, in, 6)) return fail(FP8_ERR_INVALID, "fp8_norm_backward: overlapping buffers");
    if (!aligned(dy, 16) || !aligned(s, 16) || !aligned(weight, 16) || !aligned(dres, 16) || !aligned(dx, 16) ||
        !aligned(workspace, 16) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(dbias, 4))
        return fail(FP8_ERR_UNSUPPORTED, "fp8_norm_backward: misaligned pointer");
    hipError_t e = fp8k::launch_norm_backward(dy, s, f32, weight, mean, rstd, dres, rms, rows, cols, dx, dweight, dbias,
                                              static_cast<float*>(workspace), stream);
    if (e != hipSuccess) return fail_hip("fp8_norm_backward", e);
    return FP8_OK;
}

// A tensor of an attention call: its strides checked, and the bytes it spans.
struct Heads : fp8k::HeadLayout {
    uint16_t* p = nullptr;
    Range range() const { return {p, 2 * span()}; }
};

static fp8_status take_heads(const char* call, const char* name, const fp8_head_tensor* t, int64_t tokens,
                             int64_t heads, int64_t d, bool written, Heads& h)
{
    char msg[160];
    auto no = [&](fp8_status st, const char* what) {
        std::snprintf(msg, sizeof(msg), "%s: %s %s", call, name, what);
        return fail(st, msg);
    };
    if (!t || !t->data) return no(FP8_ERR_INVALID, "is a null pointer");
    h.p = static_cast<uint16_t*>(t->data);
    h.tokens = tokens;
    h.heads = heads;
    h.d = d;
    h.head = heads == 1 ? 0 : t->head_stride;                          // a single head's or token's stride moves nothing
    if (h.head < 0 || h.head > ((int64_t)1 << 40)) return no(FP8_ERR_INVALID, "has a bad head stride");
    h.row = fp8k::kernel_row(tokens, d, t->token_stride);
    if (h.row < d) return no(FP8_ERR_INVALID, "has tokens closer than head_dim");
    if (h.row >= fp8k::kMaxRow) return no(FP8_ERR_UNSUPPORTED, "has a token stride of 2^22 or more");
    if (h.row % 8 || h.head % 8) return no(FP8_ERR_UNSUPPORTED, "has strides that are not multiples of 8");
    if (!aligned(t->data, 16)) return no(FP8_ERR_UNSUPPORTED, "is not 16-byte aligned");
    if (written && !h.distinct()) return no(FP8_ERR_INVALID, "overlaps itself");
    return FP8_OK;
}

static bool heads_overlap(const Heads& a, const Heads& b)
{
    const intptr_t off = reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p);
    return fp8k::share_element(a, b, off / 2);             // both are 16-byte aligned
}

static bool heads_overlap(const Heads& a, const void* p, int64_t n)
{
    const Range r = a.range();
    return overlap(r.p, r.n, p, n);
}

static fp8_status attention_shape(const char* call, const fp8_attention_shape* s)
{
    char msg[160];
    auto no = [&](fp8_status st, const char* what) {
        std::snprintf(msg, sizeof(msg), "%s: %s", call, what);
        return fail(st, msg);
    };
    if (!s) return no(FP8_ERR_INVALID, "null shape");
    if (s->tokens_q < 1 || s->tokens_k < 1 || s->heads_q < 1 || s->heads_k < 1 || s->batch < 1 || s->head_dim < 1)
        return no(FP8_ERR_INVALID, "tokens, heads, head_dim and batch must be positive");
    if (s->tokens_q >= ((int64_t)1 << 31) || s->tokens_k >= ((int64_t)1 << 31) || s->heads_q > 65536 || s->batch > (1 << 24))
        return no(FP8_ERR_UNSUPPORTED, "more than 2^31 - 1 tokens, 2^16 heads or 2^24 sequences");
    if (s->heads_q % s->heads_k) return no(FP8_ERR_INVALID, "heads_q must be a multiple of heads_k");
    if (s->head_dim % 8 || s->head_dim > 128) return no(FP8_ERR_UNSUPPORTED, "head_dim must be a multiple of 8, at most 128");
    if (!s->bounds_q != !s->bounds_k) return no(FP8_ERR_INVALID, "bounds_q and bounds_k go together");
    if (!s->bounds_q && s->batch != 1) return no(FP8_ERR_INVALID, "several sequences need bounds");
    if (!aligned(s->bounds_q, 4) || !aligned(s->bounds_k, 4)) return no(FP8_ERR_UNSUPPORTED, "misaligned bounds");
    if (s->causal != 0 && s->causal != 1) return no(FP8_ERR_INVALID, "causal must be 0 or 1");
    if (!(s->scale > 0.0f) || s->scale > 3.0e38f) return no(FP8_ERR_INVALID, "scale must be positive and finite");
    if (s->tokens_q * s->heads_q / 16 >= 0x7FFFFFFF || !fp8k::attention_grid_ok(s->tokens_q, (int)s->batch, (int)s->heads_q) ||
        !fp8k::attention_grid_ok(s->tokens_k, (int)s->batch, (int)s->heads_k))
        return no(FP8_ERR_UNSUPPORTED, "too many rows for one launch");
    return FP8_OK;
}

static fp8k::AttentionArgs attention_args(const fp8_attention_shape& s)
{
    fp8k::AttentionArgs a{};
    a.tq = (int)s.tokens_q;
    a.tk = (int)s.tokens_k;
    a.hq = (int)s.heads_q;
    a.hk = (int)s.heads_k;
    a.d = (int)s.head_dim;
    a.batch = (int)s.batch;
    a.cu_q = s.bounds_q;
    a.cu_k = s.bounds_k;
    a.causal = s.causal;
    a.scale = s.scale;
    return a;
}

static int64_t attention_forward_bytes(const fp8_attention_shape& s)
{
    return fp8k::attention_forward_workspace(s.tokens_q, s.tokens_k, (int)s.heads_q, (int)s.heads_k, (int)s.head_dim,
                                              (int)s.batch);
}

fp8_status fp8_attention_forward_workspace(const fp8_attention_shape* shape, int64_t* bytes)
{
    t_last_error.clear();
    fp8_status st = attention_shape("fp8_attention_forward_workspace", shape);
    if (st != FP8_OK) return st;
    if (!bytes) return fail(FP8_ERR_INVALID, "fp8_attention_forward_workspace: null pointer");
    *bytes = attention_forward_bytes(*shape);
    return FP8_OK;
}

fp8_status fp8_attention_forward(const fp8_attention_shape* shape, const fp8_head_tensor* q,
                                 const fp8_head_tensor* k, const fp8_head_tensor* v, const fp8_head_tensor* out,
                                 float* lse, float* absmax, void* workspace, int64_t workspace_bytes,
                                 hipStream_t stream)
{
    t_last_error.clear();
    const char* call = "fp8_attention_forward";
    fp8_status st = attention_shape(call, shape);
    if (st != FP8_OK) return st;
    const fp8_attention_shape& s = *shape;
    Heads h[4];
    if ((st = take_heads(call, "q", q, s.tokens_q, s.heads_q, s.head_dim, false, h[0])) != FP8_OK ||
        (st = take_heads(call, "k", k, s.tokens_k, s.heads_k, s.head_dim, false, h[1])) != FP8_OK ||
        (st = take_heads(call, "v", v, s.tokens_k, s.heads_k, s.head_dim, false, h[2])) != FP8_OK ||
        (st = take_heads(call, "out", out, s.tokens_q, s.heads_q, s.head_dim, true, h[3])) != FP8_OK)
        return st;
    if (!lse) return fail(FP8_ERR_INVALID, "fp8_attention_forward: null lse");
    const int64_t need = attention_forward_bytes(s);
    if (need > 0 && !workspace) return fail(FP8_ERR_INVALID, "fp8_attention_forward: null workspace");
    if (workspace_bytes < need) return fail(FP8_ERR_INVALID, "fp8_attention_forward: workspace too small");
    if (!aligned(lse, 4) || !aligned(absmax, 4) || !aligned(workspace, 16))
        return fail(FP8_ERR_UNSUPPORTED, "fp8_attention_forward: misaligned lse, absmax or workspace");
    const Range flat[] = {{lse, 4 * s.heads_q * s.tokens_q}, {absmax, 4}, {workspace, workspace_bytes}};
    const Range in[] = {{s.bounds_q, 4 * (s.batch + 1)}, {s.bounds_k, 4 * (s.batch + 1)}};
    bool bad = outputs_overlap(flat, 3, in, 2);
    for (int i = 0; i < 4; ++i) {
        if (i < 3) bad = bad || heads_overlap(h[3], h[i]);
        for (const Range& r : flat) bad = bad || heads_overlap(h[i], r.p, r.n);
    }
    for (const Range& r : in) bad = bad || heads_overlap(h[3], r.p, r.n);
    if (bad) return fail(FP8_ERR_INVALID, "fp8_attention_forward: overlapping buffers");
    fp8k::AttentionArgs a = attention_args(s);
    a.q = h[0].p; a.q_row = h[0].row; a.q_head = h[0].head;
    a.k = h[1].p; a.k_row = h[1].row; a.k_head = h[1].head;
    a.v = h[2].p; a.v_row = h[2].row; a.v_head = h[2].head;
    a.out = h[3].p; a.out_row = h[3].row; a.out_head = h[3].head;
    a.lse = lse;
    a.absmax = reinterpret_cast<uint32_t*>(absmax);
    hipError_t e = fp8k::launch_attention_forward(a, workspace, stream);
    if (e != hipSuccess) return fail_hip(call, e);
    return FP8_OK;
}

static int64_t attention_workspace(const fp8_attention_shape& s)
{
    return fp8k::attention_backward_workspace(s.tokens_q, s.tokens_k, (int)s.heads_q, (int)s.heads_k, (int)s.head_dim,
                                              (int)s.batch);
}

fp8_status fp8_attention_backward_workspace(const fp8_attention_shape* shape, int64_t* bytes)
{
    t_last_error.clear();
    fp8_status st = attention_shape("fp8_attention_backward_workspace", shape);
    if (st != FP8_OK) return st;
    if (!bytes) return fail(FP8_ERR_INVALID, "fp8_attention_backward_workspace: null pointer");
    *bytes = attention_workspace(*shape);
    return FP8_OK;
}

fp8_status fp8_attention_backward(const fp8_attention_shape* shape, const fp8_head_tensor* dout,
                                  const fp8_head_tensor* q, const fp8_head_tensor* k, const fp8_head_tensor* v,
                                  const fp8_head_tensor* out, const float* lse, const fp8_head_tensor* dq,
                                  const fp8_head_tensor* dk, const fp8_head_tensor* dv, float* absmax,
                                  void* workspace, int64_t workspace_bytes, hipStream_t stream)
{
    t_last_error.clear();
    const char* call = "fp8_attention_backward";
    fp8_status st = attention_shape(call, shape);
    if (st != FP8_OK) return st;
    const fp8_attention_shape& s = *shape;
    Heads h[8];                                            // 0-4 read, 5-7 written
    if ((st = take_heads(call, "dout", dout, s.tokens_q, s.heads_q, s.head_dim, false, h[0])) != FP8_OK ||
        (st = take_heads(call, "q", q, s.tokens_q, s.heads_q, s.head_dim, false, h[1])) != FP8_OK ||
        (st = take_heads(call, "k", k, s.tokens_k, s.heads_k, s.head_dim, false, h[2])) != FP8_OK ||
        (st = take_heads(call, "v", v, s.tokens_k, s.heads_k, s.head_dim, false, h[3])) != FP8_OK ||
        (st = take_heads(call, "out", out, s.tokens_q, s.heads_q, s.head_dim, false, h[4])) != FP8_OK ||
        (st = take_heads(call, "dq", dq, s.tokens_q, s.heads_q, s.head_dim, true, h[5])) != FP8_OK ||
        (st = take_heads(call, "dk", dk, s.tokens_k, s.heads_k, s.head_dim, true, h[6])) != FP8_OK ||
        (st = take_heads(call, "dv", dv, s.tokens_k, s.heads_k, s.head_dim, true, h[7])) != FP8_OK)
        return st;
    if (!lse || !workspace) return fail(FP8_ERR_INVALID, "fp8_attention_backward: null lse or workspace");
    if (workspace_bytes < attention_workspace(s)) return fail(FP8_ERR_INVALID, "fp8_attention_backward: workspace too small");
    if (!aligned(lse, 4) || !aligned(absmax, 4) || !aligned(workspace, 16))
        return fail(FP8_ERR_UNSUPPORTED, "fp8_attention_backward: misaligned lse, absmax or workspace");
    const Range flat[] = {{absmax, 4}, {workspace, workspace_bytes}};
    const Range in[] = {{s.bounds_q, 4 * (s.batch + 1)}, {s.bounds_k, 4 * (s.batch + 1)}, {lse, 4 * s.heads_q * s.tokens_q}};
    bool bad = outputs_overlap(flat, 2, in, 3);
    for (int i = 0; i < 8; ++i) {
        for (int j = 5; j < 8; ++j) bad = bad || (i != j && heads_overlap(h[j], h[i]));
        for (const Range& r : flat) bad = bad || heads_overlap(h[i], r.p, r.n);
        if (i >= 5)
            for (const Range& r : in) bad = bad || heads_overlap(h[i], r.p, r.n);
    }
    if (bad) return fail(FP8_ERR_INVALID, "fp8_attention_backward: overlapping buffers");
    fp8k::AttentionArgs a = attention_args(s);
    a.dout = h[0].p; a.dout_row = h[0].row; a.dout_head = h[0].head;
    a.q = h[1].p; a.q_row = h[1].row; a.q_head = h[1].head;
    a.k = h[2].p; a.k_row = h[2].row; a.k_head = h[2].head;
    a.v = h[3].p; a.v_row = h[3].row; a.v_head = h[3].head;
    a.out = h[4].p; a.out_row = h[4].row; a.out_head = h[4].head;
    a.dq = h[5].p; a.dq_row = h[5].row; a.dq_head = h[5].head;
    a.dk = h[6].p; a.dk_row = h[6].row; a.dk_head = h[6].head;
    a.dv = h[7].p; a.dv_row = h[7].row; a.dv_head = h[7].head;
    a.lse = const_cast<float*>(lse);
    a.stats = static_cast<float*>(workspace);
    a.absmax = reinterpret_cast<uint32_t*>(absmax);
    hipError_t e = fp8k::launch_attention_backward(a, stream);
    if (e != hipSuccess) return fail_hip(call, e);
    return FP8_OK;
}

// ---- keys and values in a paged cache

// The struct's own checks; page_tokens as a power of two in `shift`.
static fp8_status cache_shape(const char* call, const fp8_kv_cache* c, int& shift)
{
    char msg[160];
    auto no = [&](fp8_status st, const char* what) {
        std::snprintf(msg, sizeof(msg), "%s: %s", call, what);
        return fail(st, msg);
    };
    if (!c) return no(FP8_ERR_INVALID, "null cache");
    if (c->pages < 1 || c->heads < 1 || c->head_dim < 1 || c->batch < 1 || c->blocks < 1 || c->tokens < 1 || c->page_tokens < 1)
        return no(FP8_ERR_INVALID, "pages, heads, page_tokens, head_dim, batch, blocks and tokens must be positive");
    shift = c->page_tokens == 16 ? 4 : c->page_tokens == 32 ? 5 : c->page_tokens == 64 ? 6 : c->page_tokens == 128 ? 7 : 0;
    if (!shift) return no(FP8_ERR_UNSUPPORTED, "page_tokens must be 16, 32, 64 or 128");
    if (c->head_dim % 8 || c->head_dim > 128) return no(FP8_ERR_UNSUPPORTED, "head_dim must be a multiple of 8, at most 128");
    if (c->pages >= ((int64_t)1 << 31) || c->heads > 65536 || c->batch > (1 << 20) || c->tokens >= ((int64_t)1 << 31))
        return no(FP8_ERR_UNSUPPORTED, "more than 2^31 - 1 pages or tokens, 2^16 heads or 2^20 sequences");
    if (c->blocks > ((int64_t)1 << 30) >> shift) return no(FP8_ERR_UNSUPPORTED, "rows of the table for more than 2^30 tokens");
    if (!c->bounds && c->tokens % c->batch)
        return no(FP8_ERR_INVALID, "tokens must be a multiple of batch without bounds");
    return FP8_OK;
}

// The pool, table, lengths and bounds of a call, as byte ranges.
static void cache_ranges(const fp8_kv_cache& c, Range (&r)[7])
{
    const int64_t scales = c.pages * c.heads, codes = scales * c.page_tokens * c.head_dim;
    const Range all[7] = {{c.k, codes}, {c.v, codes}, {c.k_scale, scales}, {c.v_scale, scales},
                          {c.table, 4 * c.batch * c.blocks}, {c.lengths, 4 * c.batch}, {c.bounds, 4 * (c.batch + 1)}};
    for (int i = 0; i < 7; ++i) r[i] = all[i];
}

static fp8_status cache_pointers(const char* call, const fp8_kv_cache& c)
{
    if (!c.k || !c.v || !c.k_scale || !c.v_scale || !c.table || !c.lengths)
        return fail(FP8_ERR_INVALID, std::string(call) + ": null pointer in the cache");
    if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.table, 4) || !aligned(c.lengths, 4) || !aligned(c.bounds, 4))
        return fail(FP8_ERR_UNSUPPORTED, std::string(call) + ": misaligned pointer in the cache");
    return FP8_OK;
}

static fp8k::CacheArgs cache_args(const fp8_kv_cache& c, int shift)
{
    fp8k::CacheArgs a{};
    a.k = c.k;
    a.v = c.v;
    a.k_scale = c.k_scale;
    a.v_scale = c.v_scale;
    a.table = c.table;
    a.lengths = c.lengths;
    a.cu = c.bounds;
    a.pages = c.pages;
    a.tokens = c.tokens;
    a.each = (int)(c.tokens / c.batch);
    a.heads = (int)c.heads;
    a.d = (int)c.head_dim;
    a.shift = shift;
    a.batch = (int)c.batch;
    a.blocks = (int)c.blocks;
    return a;
}

// Both directions between the call's keys and values and the cache.
static fp8_status cache_move(const char* call, const fp8_kv_cache* cache, const fp8_head_tensor* k,
                             const fp8_head_tensor* v, bool write, hipStream_t stream)
{
    t_last_error.clear();
    int shift = 0;
    fp8_status st = cache_shape(call, cache, shift);
    if (st != FP8_OK) return st;
    const fp8_kv_cache& c = *cache;
    if ((st = cache_pointers(call, c)) != FP8_OK) return st;
    Heads h[2];
    if ((st = take_heads(call, "k", k, c.tokens, c.heads, c.head_dim, !write, h[0])) != FP8_OK ||
        (st = take_heads(call, "v", v, c.tokens, c.heads, c.head_dim, !write, h[1])) != FP8_OK)
        return st;
    Range r[7];
    cache_ranges(c, r);
    bool bad = !write && heads_overlap(h[0], h[1]);
    for (int i = 0; i < 7; ++i) {
        for (const Heads& t : h)
            if (!write || i < 4) bad = bad || heads_overlap(t, r[i].p, r[i].n);
        for (int j = 0; write && j < 4; ++j) bad = bad || (i != j && overlap(r[i].p, r[i].n, r[j].p, r[j].n));
    }
    if (bad) return fail(FP8_ERR_INVALID, std::string(call) + ": overlapping buffers");
    fp8k::CacheArgs a = cache_args(c, shift);
    a.xk = h[0].p; a.xk_row = h[0].row; a.xk_head = h[0].head;
    a.xv = h[1].p; a.xv_row = h[1].row; a.xv_head = h[1].head;
    hipError_t e = write ? fp8k::launch_kv_cache_write(a, stream) : fp8k::launch_kv_cache_read(a, stream);
    if (e != hipSuccess) return fail_hip(call, e);
    return FP8_OK;
}

fp8_status fp8_kv_cache_write(const fp8_kv_cache* cache, const fp8_head_tensor* k, const fp8_head_tensor* v,
                              hipStream_t stream)
{
    return cache_move("fp8_kv_cache_write", cache, k, v, true, stream);
}

fp8_status fp8_kv_cache_read(const fp8_kv_cache* cache, const fp8_head_tensor* k, const fp8_head_tensor* v,
                             hipStream_t stream)
{
    return cache_move("fp8_kv_cache_read", cache, k, v, false, stream);
}

static fp8_status cached_shape(const char* call, const fp8_kv_cache* c, int64_t heads_q, int& shift)
{
    fp8_status st = cache_shape(call, c, shift);
    if (st != FP8_OK) return st;
    if (heads_q < 1 || heads_q % c->heads) return fail(FP8_ERR_INVALID, std::string(call) + ": heads_q must be a multiple of heads");
    if (heads_q > 65536 || c->tokens * heads_q >= ((int64_t)1 << 31) - 256)
        return fail(FP8_ERR_UNSUPPORTED, std::string(call) + ": more than 2^16 heads or 2^31 rows");
    if (!fp8k::attention_cached_grid_ok(c->tokens, (int)(heads_q / c->heads), (int)c->heads, (int)c->batch,
                                        (int)c->blocks, shift))
        return fail(FP8_ERR_UNSUPPORTED, std::string(call) + ": too many rows for one launch, or too many keys of all sequences");
    return FP8_OK;
}

static int64_t cached_bytes(const fp8_kv_cache& c, int64_t heads_q, int shift)
{
    return fp8k::attention_cached_workspace(c.tokens, (int)(heads_q / c.heads), (int)c.heads, (int)c.head_dim, (int)c.batch,
                                            (int)c.blocks, shift, c.bounds != nullptr);
}

fp8_status fp8_attention_cached_workspace(const fp8_kv_cache* cache, int64_t heads_q, int64_t* bytes)
{
    t_last_error.clear();
    int shift = 0;
    fp8_status st = cached_shape("fp8_attention_cached_workspace", cache, heads_q, shift);
    if (st != FP8_OK) return st;
    if (!bytes) return fail(FP8_ERR_INVALID, "fp8_attention_cached_workspace: null pointer");
    *bytes = cached_bytes(*cache, heads_q, shift);
    return FP8_OK;
}

fp8_status fp8_attention_cached(const fp8_kv_cache* cache, const fp8_head_tensor* q, const fp8_head_tensor* out,
                                int64_t heads_q, int causal, float scale, float* lse, float* absmax, void* workspace,
                                int64_t workspace_bytes, hipStream_t stream)
{
    t_last_error.clear();
    const char* call = "fp8_attention_cached";
    int shift = 0;
    fp8_status st = cached_shape(call, cache, heads_q, shift);
    if (st != FP8_OK) return st;
    const fp8_kv_cache& c = *cache;
    if ((st = cache_pointers(call, c)) != FP8_OK) return st;
    if (causal != 0 && causal != 1) return fail(FP8_ERR_INVALID, "fp8_attention_cached: causal must be 0 or 1");
    if (!(scale > 0.0f) || scale > 2.3e38f)                    // times log2 e it is finite
        return fail(FP8_ERR_INVALID, "fp8_attention_cached: scale must be positive and at most 2.3e38");
    Heads h[2];
    if ((st = take_heads(call, "q", q, c.tokens, heads_q, c.head_dim, false, h[0])) != FP8_OK ||
        (st = take_heads(call, "out", out, c.tokens, heads_q, c.head_dim, true, h[1])) != FP8_OK)
        return st;
    const int64_t need = cached_bytes(c, heads_q, shift);
    if (!lse) return fail(FP8_ERR_INVALID, "fp8_attention_cached: null lse");
    if (need > 0 && !workspace) return fail(FP8_ERR_INVALID, "fp8_attention_cached: null workspace");
    if (workspace_bytes < need) return fail(FP8_ERR_INVALID, "fp8_attention_cached: workspace too small");
    if (!aligned(lse, 4) || !aligned(absmax, 4) || !aligned(workspace, 16))
        return fail(FP8_ERR_UNSUPPORTED, "fp8_attention_cached: misaligned lse, absmax or workspace");
    Range in[7];
    cache_ranges(c, in);
    const Range flat[] = {{lse, 4 * heads_q * c.tokens}, {absmax, 4}, {workspace, workspace_bytes}};
    bool bad = outputs_overlap(flat, 3, in, 7) || heads_overlap(h[1], h[0]);
    for (const Range& r : flat) bad = bad || heads_overlap(h[0], r.p, r.n) || heads_overlap(h[1], r.p, r.n);
    for (const Range& r : in) bad = bad || heads_overlap(h[1], r.p, r.n);
    if (bad) return fail(FP8_ERR_INVALID, "fp8_attention_cached: overlapping buffers");
    fp8k::CachedAttentionArgs a{};
    a.c = cache_args(c, shift);
    a.q = h[0].p; a.q_row = h[0].row; a.q_head = h[0].head;
    a.out = h[1].p; a.out_row = h[1].row; a.out_head = h[1].head;
    a.lse = lse;
    a.absmax = reinterpret_cast<uint32_t*>(absmax);
    a.group = (int)(heads_q / c.heads);
    a.causal = causal;
    a.scale = scale;
    hipError_t e = fp8k::launch_attention_cached(a, workspace, stream);
    if (e != hipSuccess) return fail_hip(call, e);
    return FP8_OK;
}

static fp8_status loss_shape(const char* call, int64_t tokens, int64_t vocab, int64_t dim)
{
    char msg[160];
    if (tokens < 1 || vocab < 1 || dim < 1) {
        std::snprintf(msg, sizeof(msg), "%s: tokens, vocab and dim must be positive", call);
        return fail(FP8_ERR_INVALID, msg);
    }
    if (tokens >= (1 << 24) || vocab >= (1 << 24) || dim > 65536 || dim % 8) {
        std::snprintf(msg, sizeof(msg), "%s: tokens and vocab below 2^24, dim a multiple of 8 and at most 65536", call);
        return fail(FP8_ERR_UNSUPPORTED, msg);
    }
    return FP8_OK;
}

fp8_status fp8_linear_cross_entropy_forward_workspace(int64_t tokens, int64_t vocab, int64_t dim, int64_t* bytes)
{
    t_last_error.clear();
    fp8_status st = loss_shape("fp8_linear_cross_entropy_forward_workspace", tokens, vocab, dim);
    if (st != FP8_OK) return st;
    if (!bytes) return fail(FP8_ERR_INVALID, "fp8_linear_cross_entropy_forward_workspace: null pointer");
    *bytes = fp8k::loss_forward_workspace(tokens, vocab);
    return FP8_OK;
}

fp8_status fp8_linear_cross_entropy_forward(const void* x, const void* weight, const int64_t* target, int64_t tokens,
                                            int64_t vocab, int64_t dim, float* loss, float* lse, void* workspace,
                                            int64_t workspace_bytes, hipStream_t stream)
{
    t_last_error.clear();
    const char* call = "fp8_linear_cross_entropy_forward";
    fp8_status st = loss_shape(call, tokens, vocab, dim);
    if (st != FP8_OK) return st;
    if (!x || !weight || !target || !loss || !lse || !workspace)
        return fail(FP8_ERR_INVALID, "fp8_linear_cross_entropy_forward: null pointer");
    if (workspace_bytes < fp8k::loss_forward_workspace(tokens, vocab))
        return fail(FP8_ERR_INVALID, "fp8_linear_cross_entropy_forward: workspace too small");
    const Range in[] = {{x, 2 * tokens * dim}, {weight, 2 * vocab * dim}, {target, 8 * tokens}};
    const Range out[] = {{loss, 4 * tokens}, {lse, 4 * tokens}, {workspace, workspace_bytes}};
    if (outputs_overlap(out, 3, in, 3)) return fail(FP8_ERR_INVALID, "fp8_linear_cross_entropy_forward: overlapping buffers");
    if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(target, 8) || !aligned(loss, 4) || !aligned(lse, 4) ||
        !aligned(workspace, 16))
        return fail(FP8_ERR_UNSUPPORTED, "fp8_linear_cross_entropy_forward: misaligned pointer");
    hipError_t e = fp8k::launch_loss_forward(x, weight, target, tokens, vocab, dim, loss, lse, workspace, stream);
    if (e != hipSuccess) return fail_hip(call, e);
    return FP8_OK;
}

fp8_status fp8_linear_cross_entropy_backward_workspace(int64_t tokens, int64_t vocab, int64_t dim, int64_t* bytes)
{
    t_last_error.clear();
    fp8_status st = loss_shape("fp8_linear_cross_entropy_backward_workspace", tokens, vocab, dim);
    if (st != FP8_OK) return st;
    if (!bytes) return fail(FP8_ERR_INVALID, "fp8_linear_cross_entropy_backward_workspace: null pointer");
    *bytes = fp8k::loss_backward_workspace(tokens, vocab, dim);
    return FP8_OK;
}

fp8_status fp8_linear_cross_entropy_backward(const float* dloss, const void* x, const void* weight,
                                             const int64_t* target, const float* lse, int64_t tokens, int64_t vocab,
                                             int64_t dim, void* dx, void* dweight, void* workspace,
                                             int64_t workspace_bytes, hipStream_t stream)
{
    t_last_error.clear();
    const char* call = "fp8_linear_cross_entropy_backward";
    fp8_status st = loss_shape(call, tokens, vocab, dim);
    if (st != FP8_OK) return st;
    if (!dloss || !x || !weight || !target || !lse || !dx || !dweight || !workspace)
        return fail(FP8_ERR_INVALID, "fp8_linear_cross_entropy_backward: null pointer");
    if (workspace_bytes < fp8k::loss_backward_workspace(tokens, vocab, dim))
        return fail(FP8_ERR_INVALID, "fp8_linear_cross_entropy_backward: workspace too small");
    const Range in[] = {{dloss, 4 * tokens}, {x, 2 * tokens * dim}, {weight, 2 * vocab * dim}, {target, 8 * tokens}, {lse, 4 * tokens}};
    const Range out[] = {{dx, 2 * tokens * dim}, {dweight, 2 * vocab * dim}, {workspace, workspace_bytes}};
    if (outputs_overlap(out, 3, in, 5)) return fail(FP8_ERR_INVALID, "fp8_linear_cross_entropy_backward: overlapping buffers");
    if (!aligned(dloss, 4) || !aligned(x, 16) || !aligned(weight, 16) || !aligned(target, 8) || !aligned(lse, 4) ||
        !aligned(dx, 16) || !aligned(dweight, 16) || !aligned(workspace, 16))
        return fail(FP8_ERR_UNSUPPORTED, "fp8_linear_cross_entropy_backward: misaligned pointer");
    hipError_t e = fp8k::launch_loss_backward(dloss, x, weight, target, lse, tokens, vocab, dim, dx, dweight, workspace, stream);
    if (e != hipSuccess) return fail_hip(call, e);
    return FP8_OK;
}

fp8_status fp8_stream_copy(const void* src, void* dst, int64_t bytes, hipStream_t stream)
{
    t_last_error.clear();
    if (!src || !dst) return fail(FP8_ERR_INVALID, "fp8_stream_copy: null pointer");
    if (bytes <= 0 || bytes > 2 * kMaxElems) return fail(FP8_ERR_INVALID, "fp8_stream_copy: bytes must be in [1, 2^41]");
    if (bytes % 16 != 0 || !aligned(src, 16) || !aligned(dst, 16))
        return fail(FP8_ERR_UNSUPPORTED, "fp8_stream_copy: bytes a multiple of 16, both buffers 16-byte aligned");
    if (overlap(src, bytes, dst, bytes)) return fail(FP8_ERR_INVALID, "fp8_stream_copy: src and dst overlap");
    hipError_t e = fp8k::launch_stream_copy(src, dst, bytes, stream);
    if (e != hipSuccess) return fail_hip("fp8_stream_copy", e);
    return FP8_OK;
}

}  // extern "C"
