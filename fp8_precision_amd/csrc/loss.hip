// loss.hip -- cross entropy of a linear head over a large vocabulary, without ever
// holding the logits, for gfx950.
//
// With x [T, D], w [V, D] (bf16), z = x w^T and a target per token,
//   lse_t = log sum_v exp(z_tv),   loss_t = lse_t - z_t,target(t)
// and backward, g_tv = dloss_t (exp(z_tv - lse_t) - [v = target(t)]),
//   dx = g w,   dw = g^T x.
// A token whose target lies outside [0, V) has no target: loss 0 and no gradient, whatever its
// x: g's launch leaves a bit per token, by which dw's loads pass over its row (all three
// products, without and so: 4096 tokens, 32000 x 4096 2277 and 2297 us, 1001, 40007 x 1600 378
// and 384).
//
// Forward: the logits' product with the row statistics taken in its epilogue -- the
// maximum and the sum of exponentials of the wave's columns of each row -- and a
// second, small launch that joins them.  Backward: the vocabulary is walked in
// pieces; a piece's logits are computed again, turned into g (bf16) in the epilogue
// and written to a workspace, from which the piece's dw and its share of dx are
// taken.  dx is summed over the pieces in fp32.
//
// Bound by the matrix units (2 T V D operations forward, 6 T V D backward) except for
// few tokens, where reading w bounds.  The product kernel: 256 columns by 256, 128 or
// 64 rows per workgroup of 4 waves, one wave per SIMD; reduction steps of 64
// elements in two LDS stages filled by 16-byte direct-to-LDS buffer loads issued a
// step and more ahead; fragments double-buffered in registers across two barriers per
// step; persistent workgroups in an XCD-major walk that load the next tile's first
// stages before the epilogue.  The chip runs these products at its power limit, so the
// instruction matters: v_mfma_f32_16x16x32_bf16; 32x32x16 kept the matrix units 65%
// busy instead of 58% at the same stage of this kernel and yet ran 3% slower, its clock
// at 1.88 GHz instead of 2.26.
// Operands are read along the reduction ("K": x and w for the logits, g for dx) or
// across it ("MN": w for dx, g and x for dw) through transposing LDS reads, so no
// transposed copy of anything exists.  Rows, columns and reduction elements past an
// operand's end read as zero (the buffer's size, or an offset outside it).
//
// g is rounded to bf16, as an operand of the matrix units -- divided by the largest
// |dloss| of a token with a target, which the products' epilogues multiply in again: with one dloss for all tokens
// (the mean), its own rounding would be a common error of every gradient, up to 2^-8.
// z, the statistics and every sum stay in fp32.  The sums are formed in a fixed order: no atomics.
#include "fp8_device.hpp"
#include "fp8_internal.hpp"

namespace fp8k {

namespace {

typedef __bf16 lb16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 lb16x2 __attribute__((ext_vector_type(2)));
typedef float lf32x2 __attribute__((ext_vector_type(2)));
typedef float lf32x4 __attribute__((ext_vector_type(4)));
typedef short ls16x4 __attribute__((ext_vector_type(4)));
typedef unsigned int lu32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) ls16x4 lds_ls16x4;
typedef __attribute__((address_space(3))) lu32x4 lds_lu32x4;

constexpr float kLossLog2e = 1.44269504088896340736f;
constexpr float kLossLn2 = 0.69314718055994530942f;
constexpr float kLossInf = __builtin_inff();
constexpr int kStep = 64;                 // reduction elements of a step (128 bytes)
constexpr int kOutside = (int)0x80000000; // an offset past every buffer's size

// Fragment: 16 rows x 32 reduction elements, 8 per lane.
union LossFrag {
    lu32x4 u;
    lb16x8 b;
    ls16x4 s[2];
};

__device__ __forceinline__ uint32_t loss_pair(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(lf32x2{a, b}, lb16x2));
}

__device__ __forceinline__ void loss_to_lds(uint32_t voff, const lu32x4& desc, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :
                 : "v"(voff), "s"(desc), "s"(lds)
                 : "memory", "m0");
}

__device__ __forceinline__ lu32x4 loss_desc(const uint8_t* base, int64_t bytes)
{
    const uint64_t b = (uint64_t)base;
    const int64_t n = bytes < 0 ? 0 : bytes > 0x7FFFFFFF ? 0x7FFFFFFF : bytes;
    lu32x4 d;
    d[0] = __builtin_amdgcn_readfirstlane((uint32_t)b);
    d[1] = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32) & 0xFFFFu);
    d[2] = __builtin_amdgcn_readfirstlane((uint32_t)n);
    d[3] = 0x00020000u;
    return d;
}

// One operand: element (i, r) of the product's row (or column) i and reduction index r
// at p + i * pitch + r (K) or p + r * pitch + i (MN).
struct Side {
    const uint16_t* p;
    int64_t pitch;
};

// Loads of one operand's EXT rows (columns) of the tile for one wave.  The LDS image:
//   K:  EXT rows of 128 bytes, 16-byte chunk c of row r at c ^ (r >> 1 & 7) ^ (r & 1) << 2;
//   MN: 64 rows (reduction) of 2 EXT bytes, chunk c of row r at
//       c ^ ((r & 3) << 1 | (r >> 3 & 1) << 3):
// so that the 16 rows of a plain read, and the 32-byte pieces of 8 rows that half a
// wave's transposing read takes, spread over all banks.
template <bool MN, int EXT>
struct Feed {
    static constexpr int kLoads = EXT / 32;                  // 1 KB each
    const uint8_t* base;
    int64_t pitch, left;                                     // bytes; of the matrix from base on
    uint32_t voff[kLoads];
    int chunk[2];                                            // K: the lane's chunk for even and odd loads

    __device__ __forceinline__ void init(const Side& s, int origin, int extent, int total_r, int r0, int wave, int lane)
    {
        pitch = s.pitch * 2;
        if (!MN) {
            base = reinterpret_cast<const uint8_t*>(s.p) + (int64_t)origin * pitch + (int64_t)r0 * 2;
            left = (int64_t)(extent - origin) * pitch - (int64_t)r0 * 2;
#pragma unroll
            for (int ii = 0; ii < kLoads; ++ii) {
                const int r = wave * (EXT / 4) + ii * 8 + (lane >> 3);
                chunk[ii & 1] = (lane & 7) ^ ((r >> 1) & 7) ^ ((r & 1) << 2);
                voff[ii] = (uint32_t)(r * (int)pitch) + (uint32_t)chunk[ii & 1] * 16u;
            }
        } else {
            constexpr int kRowLanes = EXT / 8, kRows = 64 / kRowLanes;   // lanes per row, rows per load
            base = reinterpret_cast<const uint8_t*>(s.p) + (int64_t)r0 * pitch + (int64_t)origin * 2;
            left = (int64_t)(total_r - r0) * pitch - (int64_t)origin * 2;
#pragma unroll
            for (int ii = 0; ii < kLoads; ++ii) {
                const int r = wave * 16 + ii * kRows + lane / kRowLanes;
                const int c = (lane % kRowLanes) ^ ((r & 3) << 1 | (r >> 3 & 1) << 3);
                voff[ii] = origin + c * 8 < extent ? (uint32_t)(r * (int)pitch) + (uint32_t)c * 16u : (uint32_t)kOutside;
            }
        }
    }

    // Load ii's offset, past the buffer where the reduction row's bit is not in `live` (of
    // the step's 64 rows): the row then reads as zero.  `dead` is dead_rows(live).
    __device__ __forceinline__ static uint32_t dead_rows(uint64_t live, int wave, int lane)
    {
        return (uint32_t)(~live >> (wave * 16)) >> (lane / (EXT / 8));
    }
    __device__ __forceinline__ uint32_t offset(int ii, uint32_t dead) const
    {
        return voff[ii] | (dead << (31 - ii * (512 / EXT)) & (uint32_t)kOutside);
    }

    // From here on every load is of the reduction's last step, which has in_step < kStep
    // elements: lanes past them read zero.
    __device__ __forceinline__ void trim(int in_step)
    {
        if (!MN) {
#pragma unroll
            for (int ii = 0; ii < kLoads; ++ii)
                if (chunk[ii & 1] * 8 >= in_step) voff[ii] = (uint32_t)kOutside;
        }
    }
    __device__ __forceinline__ lu32x4 desc(int kt) const
    {
        const int64_t on = MN ? (int64_t)kt * kStep * pitch : (int64_t)kt * kStep * 2;
        return loss_desc(base + on, left - on);
    }
};

// This lane's addresses in an operand image of the first stage, for the wave's 16-row
// blocks from `first` on; block i and reduction elements 32 k .. are at
//   K:  at[k] + 2048 i;   MN:  at[i] + 32 k rows, and 4 rows on.
template <bool MN, int EXT, int N>
struct Reader {
    uint32_t at[MN ? N : 2];
    __device__ __forceinline__ void init(uint32_t image, int first, int lane)
    {
        const int g = lane >> 4, l = lane & 15;
        if (!MN) {
            const int f = ((l >> 1) & 7) ^ ((l & 1) << 2);
            at[0] = image + (first * 16 + l) * 128 + ((g ^ f) * 16);
            at[1] = image + (first * 16 + l) * 128 + ((g ^ f ^ 4) * 16);
        } else {
            const int f = (l >> 2) << 1 | (g & 1) << 3;
#pragma unroll
            for (int i = 0; i < N; ++i)
                at[MN ? i : 0] = image + (8 * g + (l >> 2)) * (EXT * 2) + (((2 * (first + i) + (l & 3) / 2) ^ f) * 16) +
                                 (l & 1) * 8;
        }
    }
    __device__ __forceinline__ LossFrag read(uint32_t stage, int i, int k) const
    {
        LossFrag f;
        if (!MN) {
            f.u = *((const lds_lu32x4*)(uintptr_t)(at[k] + stage) + i * 128);
        } else {
            lds_ls16x4* p = (lds_ls16x4*)(uintptr_t)(at[MN ? i : 0] + stage) + k * (32 * EXT / 4);
            f.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
            f.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p + EXT);
        }
        return f;
    }
};

// s_waitcnt immediate: at most n vector memory operations in flight.
constexpr int wait_loads(int n) { return 0x0F70 | (n & 15) | (n >> 4) << 14; }

// A barrier that waits for nothing but the waves themselves: what a wave has to have done
// before it is waited for explicitly.  No LDS access is moved over it.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

// Memory that nothing writes while the kernel runs, read through the scalar cache.
typedef const __attribute__((address_space(4))) uint64_t* ScalarWords;

// What a launch's epilogue does with the tile's sums.
enum { kStats = 0, kGrad = 1, kSum = 2, kStore = 3 };

struct LossArgs {
    Side a, b;
    int P, Q, R;                          // rows, columns, reduction
    int tiles_m, tiles_n, units;          // units: tiles * splits
    int steps, per;                       // reduction steps in all and per split
    int first, halves;                    // halves: this launch's units are the two 128-row halves of
                                          // the 256-row units from `first` on
    // statistics and gradient
    const int64_t* target;
    const float* lse;
    const float* dloss;
    float* unit;                          // the largest |dloss| of a target, found with g and left to its products' epilogues
    float2* stats;                        // [column block][T]: maximum, sum of exponentials
    float* hit;                           // [T]: the target's logit
    uint64_t* live;                       // a bit per token: it has a target (found with g, for dw)
    int v0, vocab;                        // the piece's first column in the vocabulary, and its size
    // outputs
    uint16_t* out;                        // bf16, pitch out_pitch: g, dw, or dx once complete
    int64_t out_pitch;
    int out_cols;                         // g: columns written (Q rounded up; those past Q get 0)
    float* sum;                           // [splits][P][Q] fp32 partial dx
    int fresh, last;                      // sum: nothing to add to yet; write bf16 to out
};

struct Unit {
    int m0, n0, r0, kt, split;
    int turn;                             // the reduction step it begins with
};

}  // namespace

namespace {
// Workgroups per CU: two where the accumulators are small.
constexpr int loss_per_cu(int mi, int nj) { return mi * nj <= 16 ? 2 : 1; }
}  // namespace

// MI x NJ blocks of 16 x 16 per wave, GM x GN waves, NS stages.  MI355X: the logits of 4096
// tokens, 32000 x 4096 748 us (1.44 PFLOP/s; the library's product of the size 718 to 728), of
// 8192, 65521 x 5120 3.74 ms (1.47); the backward's three products 2.25 ms (1.43) and 383 us
// for 1001 tokens, 40007 x 1600.  At the power limit; what stands between these and the
// library is the epilogue and the last round's idle units.
template <int MI, int NJ, int GM, int GN, int NS, bool LA, bool LB, int EPI>
__global__ void __launch_bounds__(256, loss_per_cu(MI, NJ)) loss_product_kernel(const LossArgs g)
{
    constexpr int BM = 16 * MI * GM, BN = 16 * NJ * GN;
    static_assert(GM * GN == 4, "four waves");
    constexpr int kA = BM * 128, kStage = kA + BN * 128;
    constexpr int kLoads = BM / 32 + BN / 32;
    constexpr int kEpi = EPI == kGrad || EPI == kStore ? 16 * 16 * NJ * 2 : 0;   // a wave's 16 rows of bf16
    constexpr int kHalf = MI / 2;
    // Few rows: bound by reading w, whose rows are often a power of two apart; workgroups
    // that all begin with a row's start would then read the same few of the memory's
    // channels at any one time, so each begins with another step of the reduction (16
    // tokens, 32000 x 4096, the weight in memory: 64 us with one beginning, 51 so; 128
    // tokens, 50000 x 2048: 57.6 and 46.5; with tiles of 256 rows it loses, 87 and 94).
    constexpr bool kTurn = BM <= 128 && !LA && !LB;
    // dw: the reduction runs over the tokens.  g is 0 for those without a target, but their x
    // may be anything, and 0 times an infinity is not 0: their rows of x are not read.
    constexpr bool kLive = LA;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[NS * kStage + 4 * kEpi];
    // the tile's rows: target (-1: none), dloss, lse in powers of two
    __shared__ int row_target[BM];
    __shared__ float row_scale[BM], row_lse[BM];

    const int G = gridDim.x;
    int slot = blockIdx.x;
    if (G % 8 == 0) slot = (blockIdx.x % 8) * (G / 8) + blockIdx.x / 8;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / GN, wn = wave % GN;
    const uint32_t lds0 = (uint32_t)(uintptr_t)smem;

    auto unit_of = [&](int u) {
        Unit w;
        const int tiles = g.tiles_m * g.tiles_n, id = g.halves ? g.first + u / 2 : u;
        w.split = id / tiles;
        const int t = id - w.split * tiles;
        // groups of 8 tile rows, each walked column by column: 32 neighbours are 8 x 4 tiles
        const int group = t / (8 * g.tiles_n), in = t - group * 8 * g.tiles_n;
        const int rows = min(8, g.tiles_m - group * 8);
        w.m0 = (group * 8 + in % rows) * BM;
        if (g.halves) w.m0 = 2 * w.m0 + (u & 1) * BM;
        w.n0 = (in / rows) * BN;
        const int s0 = w.split * g.per;
        w.r0 = s0 * kStep;
        w.kt = min(g.steps - s0, g.per);
        w.turn = kTurn && !g.halves && g.R % kStep == 0 ? w.n0 / BN % w.kt : 0;
        return w;
    };
    // step kt of the unit, and the load descriptors' step
    auto turned = [&](const Unit& w, int kt) {
        kt += w.turn;
        return kTurn && kt >= w.kt ? kt - w.kt : kt;
    };

    Feed<LA, BM> fa;
    Feed<LB, BN> fb;
    Reader<LA, BM, MI> ra;
    Reader<LB, BN, NJ> rb;
    ra.init(lds0, wm * MI, lane);
    rb.init(lds0 + kA, wn * NJ, lane);
    lf32x4 acc[MI][NJ];
    LossFrag bq[NJ][2], alo[kHalf][2], ahi[kHalf][2];

    // before the first load of step kt: if it is the reduction's last and not a whole one
    auto trim = [&](const Unit& w, int kt) {
        const int in_step = g.R - w.r0 - kt * kStep;
        if (in_step < kStep) {
            fa.trim(in_step);
            fb.trim(in_step);
        }
    };
    auto live_rows = [&](const Unit& w, int kt) -> uint64_t {
        return ((ScalarWords)(uintptr_t)g.live)[__builtin_amdgcn_readfirstlane(w.r0 / kStep + kt)];
    };
    auto start = [&](const Unit& w) {
        int ln = lane;
        asm volatile("" : "+v"(ln));      // what follows from the lane is computed per tile, not held across them
        fa.init(g.a, w.m0, g.P, g.R, w.r0, wave, ln);
        fb.init(g.b, w.n0, g.Q, g.R, w.r0, wave, ln);
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const int kt = min(s, w.kt - 1);
            trim(w, kt);
            const lu32x4 da = fa.desc(turned(w, kt)), db = fb.desc(turned(w, kt));
            const uint32_t dead = kLive ? fb.dead_rows(live_rows(w, kt), wave, ln) : 0;
#pragma unroll
            for (int x = 0; x < BM / 32; ++x)
                loss_to_lds(fa.voff[x], da,
                            __builtin_amdgcn_readfirstlane(lds0 + s * kStage + (wave * (BM / 32) + x) * 1024));
#pragma unroll
            for (int x = 0; x < BN / 32; ++x)
                loss_to_lds(kLive ? fb.offset(x, dead) : fb.voff[x], db,
                            __builtin_amdgcn_readfirstlane(lds0 + s * kStage + kA + (wave * (BN / 32) + x) * 1024));
        }
    };
    // Instruction t of a half step: B block t / (2 kHalf), A block t / 2 % kHalf, the first or
    // second 32 of the 64 reduction elements (one accumulator's two instructions in a row
    // measured 2% faster than kHalf apart).  An instruction takes 16 cycles and the wave
    // issues another at most every 4, so reads and loads are dealt over the slots one at a
    // time, and the loads over the whole step: a CU takes a 1 KB load every 16 cycles, and
    // all 64 of a step in one half of it made every instruction behind them wait.
    constexpr int kSlots = 2 * kHalf * NJ, kFree = kSlots / 4;
    constexpr int kLoadsA = BM / 32, kLoadsB = BN / 32;
    // The first half of a step: A blocks 0 .. kHalf - 1, while the others are read.  B was
    // read in the half before; once every wave has it (slot kFree), B of the step NS ahead is
    // loaded into its place.
    // Their rows' word was read in the half0 before, after a wait for LDS reads and ahead of
    // the next: a scalar load in flight makes every wait for an LDS read one for all.
    uint64_t live = 0;
    auto half0 = [&](uint32_t cur, const lu32x4& db, const Unit& w, int next) {
        const uint32_t dead = kLive ? fb.dead_rows(live, wave, lane) : 0;
#pragma unroll
        for (int t = 0; t < kSlots; ++t) {
            const int j = t / (2 * kHalf), k = t % 2, i = t / 2 % kHalf;
            if (t == kFree) {
                __builtin_amdgcn_s_waitcnt(0xC07F);          // this wave's reads
                lds_barrier();
                if (kLive) live = live_rows(w, next);
            }
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bq[j][k].b, alo[i][k].b, acc[i][j], 0, 0, 0);
#pragma unroll
            for (int x = 0; x < 2 * kHalf; ++x)
                if (t == x * kSlots * 3 / (8 * kHalf)) ahi[x / 2][x % 2] = ra.read(cur, kHalf + x / 2, x % 2);
#pragma unroll
            for (int x = 0; x < kLoadsB; ++x)
                if (t == kFree + x * (kSlots - kFree) / kLoadsB)
                    loss_to_lds(kLive ? fb.offset(x, dead) : fb.voff[x], db,
                                __builtin_amdgcn_readfirstlane(lds0 + cur + kA + (wave * kLoadsB + x) * 1024));
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // The second half: the next step's fragments replace those that are done with, and A of
    // the step NS ahead is loaded into this step's place.
    auto half1 = [&](bool more, uint32_t cur, uint32_t nxt, const lu32x4& da) {
#pragma unroll
        for (int t = 0; t < kSlots; ++t) {
            const int j = t / (2 * kHalf), k = t % 2, i = t / 2 % kHalf;
            acc[kHalf + i][j] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(bq[j][k].b, ahi[i][k].b, acc[kHalf + i][j], 0, 0, 0);
            if (more) {
                if (i == kHalf - 1) bq[j][k] = rb.read(nxt, j, k);
#pragma unroll
                for (int x = 0; x < 2 * kHalf; ++x)
                    if (t == x * kSlots / (2 * kHalf)) alo[x / 2][x % 2] = ra.read(nxt, x / 2, x % 2);
#pragma unroll
                for (int x = 0; x < kLoadsA; ++x)
                    if (t == x * kSlots / kLoadsA + 1)
                        loss_to_lds(fa.voff[x], da,
                                    __builtin_amdgcn_readfirstlane(lds0 + cur + (wave * kLoadsA + x) * 1024));
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    // The rows' values are loaded before the tile's first operand loads and stored to LDS
    // before the next tile's, so that waiting for them never waits for a prefetch.
    int my_target = -1;
    float my_scale = 0.0f, my_lse = 0.0f;
    auto fetch_rows = [&](const Unit& w) {
        if (EPI != kStats && EPI != kGrad) return;
        const int m = w.m0 + (int)threadIdx.x;
        my_target = -1;
        if ((int)threadIdx.x < BM && m < g.P) {
            const int64_t t = g.target[m];
            if (t >= 0 && t < g.vocab) my_target = (int)t;
            if (EPI == kGrad) {
                my_scale = g.dloss[m];
                my_lse = g.lse[m];
            }
        }
    };
    // The largest finite |dloss| of a token with a target (1 if there is none above 0).  g's
    // launches find it, every workgroup for itself (a launch of its own took 2 to 5 us), and
    // leave it in memory.
    float by = 1.0f;
    if (EPI == kGrad) {
        __shared__ uint32_t part[4];
        uint32_t top = 0;
#pragma unroll 8
        for (int i = threadIdx.x; i < g.P; i += 256) {
            const uint32_t v = __float_as_uint(g.dloss[i]) & 0x7FFFFFFFu;
            const bool has = (uint64_t)g.target[i] < (uint64_t)g.vocab;
            top = max(top, has && v < 0x7F800000u ? v : 0u);
        }
        top = wave_max_u32(top);
        if (lane == 0) part[wave] = top;
        __syncthreads();
        top = max(max(part[0], part[1]), max(part[2], part[3]));
        if (top != 0) by = __uint_as_float(top);
        if (blockIdx.x == 0 && threadIdx.x == 0) *g.unit = by;
    } else if (EPI != kStats) {
        by = *g.unit;
    }
    auto keep_rows = [&](const Unit& w) {
        if ((EPI != kStats && EPI != kGrad) || (int)threadIdx.x >= BM) return;
        if (EPI == kGrad && w.n0 == 0 && w.m0 + wave * 64 < g.P) {
            const uint64_t has = __ballot(my_target >= 0);
            if (lane == 0) g.live[w.m0 / 64 + wave] = has;
        }
        row_target[threadIdx.x] = my_target;
        if (EPI == kGrad) {
            row_scale[threadIdx.x] = my_target < 0 ? 0.0f : my_scale / by;
            row_lse[threadIdx.x] = my_target < 0 ? 0.0f : my_lse * kLossLog2e;
        }
    };

    int u = slot;
    if (u >= g.units) return;
    Unit w = unit_of(u);
    fetch_rows(w);
    start(w);
    for (;;) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[i][j] = lf32x4{0, 0, 0, 0};
        // the first stage has landed once at most the later ones' loads are in flight
        __builtin_amdgcn_s_waitcnt(wait_loads((NS - 1) * kLoads));
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) bq[j][k] = rb.read(0, j, k);
#pragma unroll
            for (int i = 0; i < kHalf; ++i) alo[i][k] = ra.read(0, i, k);
        }
        uint32_t cur = 0;                                    // the stage, in bytes from the first
        // (past the last step its loads are repeated into places that are read no more, so
        // that the count of loads in flight stays the same)
        int ahead = min(NS, w.kt - 1);
        trim(w, ahead);
        if (kLive) live = live_rows(w, ahead);
        half0(cur, fb.desc(turned(w, ahead)), w, min(NS + 1, w.kt - 1));
        for (int kt = 0; kt + 1 < w.kt; ++kt) {
            const uint32_t nxt = cur + kStage == NS * kStage ? 0 : cur + kStage;
            // the next step's loads of this wave (later: whole steps and one B), and its reads
            __builtin_amdgcn_s_waitcnt(wait_loads((NS - 2) * kLoads + kLoadsB) & 0xF0FF);
            lds_barrier();                                   // everyone's; this step's A is read
            half1(true, cur, nxt, fa.desc(turned(w, ahead)));
            ahead = min(kt + 1 + NS, w.kt - 1);
            trim(w, ahead);
            half0(nxt, fb.desc(turned(w, ahead)), w, min(kt + 2 + NS, w.kt - 1));
            cur = nxt;
        }
        __builtin_amdgcn_s_waitcnt(wait_loads(0));
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
        half1(false, 0, 0, lu32x4{0, 0, 0, 0});
        keep_rows(w);
        __syncthreads();

        const Unit done = w;
        u += G;
        if (u < g.units) {
            w = unit_of(u);
            fetch_rows(w);
            start(w);
        }

        // Sums of rows i and up stay in accumulation registers until row i is taken: moved
        // earlier (as the compiler would) they spill what the next tile's loads need.
        auto hold = [&](int i) {
            if constexpr (MI * NJ == 64) {
#pragma unroll
                for (int x = 0; x < MI; ++x)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        if (x >= i) asm volatile("" : "+a"(acc[x][j]));
            }
        };
        hold(0);
        // lane: row 16 i + lane % 16 of the wave's tile, columns 16 j + 4 (lane / 16) + e
        int ln = lane;
        asm volatile("" : "+v"(ln));
        const int r16 = ln & 15, q4 = ln >> 4;
        const int m_wave = done.m0 + wm * 16 * MI, n_wave = done.n0 + wn * 16 * NJ;
        if (EPI == kStats) {
            if (n_wave < g.Q) {
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    hold(i);
                    const int m = m_wave + 16 * i + r16;
                    float top = -kLossInf;
                    if (n_wave + 16 * NJ > g.Q) {            // only a row's last block
#pragma unroll
                        for (int j = 0; j < NJ; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (n_wave + 16 * j + 4 * q4 + e >= g.Q) acc[i][j][e] = -kLossInf;
                    }
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) top = fmaxf(top, acc[i][j][e]);
                    top = fmaxf(top, __shfl_xor(top, 16, 64));
                    top = fmaxf(top, __shfl_xor(top, 32, 64));
                    const float by = top == -kLossInf ? 0.0f : top * kLossLog2e;
                    float s = 0.0f;
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s += __builtin_amdgcn_exp2f(fmaf(acc[i][j][e], kLossLog2e, -by));
                    s += __shfl_xor(s, 16, 64);
                    s += __shfl_xor(s, 32, 64);
                    if (m < g.P) {
                        if (q4 == 0) g.stats[(int64_t)(n_wave / (16 * NJ)) * g.P + m] = make_float2(top, s);
                        const int at = row_target[m - done.m0] - n_wave;
                        if (at >= 0 && at < 16 * NJ) {
#pragma unroll
                            for (int j = 0; j < NJ; ++j)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (at == 16 * j + 4 * q4 + e) g.hit[m] = acc[i][j][e];
                        }
                    }
                }
            }
        } else if (EPI == kSum) {
            float* sum = g.sum + (int64_t)done.split * g.P * g.Q;
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                hold(i);
                const int m = m_wave + 16 * i + r16;
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const int n = n_wave + 16 * j + 4 * q4;
                    if (m < g.P && n < g.Q) {               // Q is a multiple of 8: 4 columns at a time
                        float4* at = reinterpret_cast<float4*>(sum + (int64_t)m * g.Q + n);
                        float4 v = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
                        if (!g.fresh) {
                            const float4 o = *at;
                            v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
                        }
                        if (g.last)
                            *reinterpret_cast<uint2*>(g.out + (int64_t)m * g.out_pitch + n) =
                                make_uint2(loss_pair(v.x * by, v.y * by), loss_pair(v.z * by, v.w * by));
                        else
                            *at = v;
                    }
                }
            }
        } else {
            // 16 rows at a time through the wave's LDS, written as 16 NJ-column row segments
            const uint32_t ew = lds0 + NS * kStage + wave * kEpi;
            constexpr int kRowB = 32 * NJ, kSeg = 2 * NJ;    // bytes and 16-byte chunks of a row
            const int cols = EPI == kGrad ? g.out_cols : g.Q;
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                hold(i);
                if (EPI == kGrad) {
                    const int row = m_wave - done.m0 + 16 * i + r16, t = row_target[row];
                    const float scale = row_scale[row], lse2 = row_lse[row];
                    // p dloss, 0 for a token without a target (whatever its logits are)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float p = scale * __builtin_amdgcn_exp2f(fmaf(acc[i][j][e], kLossLog2e, -lse2));
                            acc[i][j][e] = t < 0 ? 0.0f : p;
                        }
                    const int at = t < 0 ? -1 : t - g.v0 - n_wave;   // the target's column within the wave's
                    if (__any(at >= 0 && at < 16 * NJ)) {
#pragma unroll
                        for (int j = 0; j < NJ; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (at == 16 * j + 4 * q4 + e) acc[i][j][e] -= scale;
                    }
                    if (n_wave + 16 * NJ > g.Q) {
#pragma unroll
                        for (int j = 0; j < NJ; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (n_wave + 16 * j + 4 * q4 + e >= g.Q) acc[i][j][e] = 0.0f;
                    }
                }
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const int c = (2 * j + (q4 >> 1)) ^ (r16 & (kSeg - 1));
                    typedef unsigned int u2 __attribute__((ext_vector_type(2)));
                    typedef __attribute__((address_space(3))) u2 lds_u2;
                    *(lds_u2*)(uintptr_t)(ew + r16 * kRowB + c * 16 + (q4 & 1) * 8) =
                        EPI == kGrad ? u2{loss_pair(acc[i][j][0], acc[i][j][1]), loss_pair(acc[i][j][2], acc[i][j][3])}
                                     : u2{loss_pair(acc[i][j][0] * by, acc[i][j][1] * by),
                                          loss_pair(acc[i][j][2] * by, acc[i][j][3] * by)};
                }
                __builtin_amdgcn_wave_barrier();             // one wave's LDS accesses stay in order
#pragma unroll
                for (int k = 0; k < NJ / 2; ++k) {           // 64 lanes x 16 bytes each
                    const int idx = k * 64 + ln, rr = idx / kSeg, c = idx % kSeg;
                    const lu32x4 v = *(const lds_lu32x4*)(uintptr_t)(ew + rr * kRowB + ((c ^ (rr & (kSeg - 1))) * 16));
                    const int m = m_wave + 16 * i + rr, n = n_wave + c * 8;
                    if (m < g.P && n < cols) *reinterpret_cast<lu32x4*>(g.out + (int64_t)m * g.out_pitch + n) = v;
                }
                __builtin_amdgcn_wave_barrier();
            }
        }
        if (u >= g.units) break;
    }
}

// lse and loss of R rows per workgroup (16, or 2 where there are few) from their column
// blocks' statistics: 1024 / R lanes take a row's blocks in turn and are joined 8 at a
// time, in order.
template <int R>
__global__ void __launch_bounds__(1024)
loss_join_kernel(const float2* __restrict__ stats, int blocks, const float* __restrict__ hit,
                 const int64_t* __restrict__ target, int T, int64_t vocab, float* __restrict__ loss,
                 float* __restrict__ lse)
{
    constexpr int kLanes = 1024 / R;      // a power of 8
    __shared__ float2 part[kLanes][R];
    const int r = threadIdx.x % R, k = threadIdx.x / R, m = blockIdx.x * R + r;
    float top = -kLossInf, s = 0.0f;
    auto join = [&](float2 o) {
        // a NaN maximum or sum stays NaN
        const float up = o.x > top ? o.x : top;
        const float base = up == -kLossInf ? 0.0f : up;
        s = s * __builtin_amdgcn_exp2f((top - base) * kLossLog2e) + o.y * __builtin_amdgcn_exp2f((o.x - base) * kLossLog2e);
        top = up;
    };
    if (m < T) {
#pragma unroll 4
        for (int b = k; b < blocks; b += kLanes) join(stats[(int64_t)b * T + m]);
    }
    part[k][r] = make_float2(top, s);
    for (int left = kLanes; left > 1; left /= 8) {
        const int n = left / 8;
        __syncthreads();
        top = -kLossInf;
        s = 0.0f;
        if (k < n)
            for (int i = 0; i < 8; ++i) join(part[k * 8 + i][r]);
        __syncthreads();
        if (k < n) part[k][r] = make_float2(top, s);
    }
    if (k == 0 && m < T) {
        const float z = (top == -kLossInf ? 0.0f : top) + __builtin_amdgcn_logf(s) * kLossLn2;
        const int64_t t = target[m];
        lse[m] = z;
        loss[m] = t >= 0 && t < vocab ? z - hit[m] : 0.0f;
    }
}

// A gradient from its splits' partial sums, added in order and rounded: 4 elements per thread.
__global__ void __launch_bounds__(256)
loss_add_kernel(const float4* __restrict__ sum, int splits, int64_t n4, const float* __restrict__ unit,
                uint2* __restrict__ out)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n4) return;
    float4 t = sum[i];
#pragma unroll 8
    for (int s = 1; s < splits; ++s) {
        const float4 o = sum[(int64_t)s * n4 + i];
        t = make_float4(t.x + o.x, t.y + o.y, t.z + o.z, t.w + o.w);
    }
    const float by = *unit;
    out[i] = make_uint2(loss_pair(t.x * by, t.y * by), loss_pair(t.z * by, t.w * by));
}

// ---------------------------------------------------------------------- plan and launches

namespace {

// Rows of a tile: the fewest that T needs, for few tokens.
int tile_rows(int64_t T) { return T <= 64 ? 64 : T <= 128 ? 128 : 256; }

// The same for the logits, which take the smallest tiles (64 x 128) also where these are
// no more than the CUs.  MI355X, forward, larger tiles / these: 298 tokens, 1933 x 2960
// 38.6 / 21.4 us; 100, 4000 x 4096 48.8 / 25.2; 128, 8000 x 1024 20.3 / 14.6.  With two to
// a CU they lose: 200, 16000 x 4096 53.6 / 113.8.
int logit_rows(int64_t T, int64_t V)
{
    return (T + 63) / 64 * ((V + 127) / 128) <= device_cu_count() ? 64 : tile_rows(T);
}
int column_block(int rows) { return rows == 64 ? 32 : 128; }       // a wave's columns of the logits

int64_t up_to(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

// The backward pass's pieces of the vocabulary: as few as keep a piece's g at or under
// 256 MiB (or 4096 columns), of one size, whole tiles.  Fewer pieces read and write the
// fp32 sums of dx less often: 8192 tokens, 65521 x 5120, in pieces of 128 / 256 / 512 MiB
// took 12.56 / 12.19 / 12.07 ms; the workspace is what larger ones cost.
int64_t piece_columns(int64_t T, int64_t V)
{
    const int64_t most = std::max<int64_t>(4096, ((int64_t)256 << 20) / (2 * T));
    const int64_t pieces = (V + most - 1) / most;
    return up_to((V + pieces - 1) / pieces, 256);
}

// dx has T / rows x D / 256 tiles; where they would leave CUs idle its reduction over
// the (first, largest) piece is split among that many workgroups.  Every split has at
// least one of its reduction steps; those of a smaller last piece may be fewer, and
// their partial sums then stand as the earlier pieces left them.
int dx_splits(int64_t T, int64_t D, int64_t piece)
{
    const int64_t tiles = (T + tile_rows(T) - 1) / tile_rows(T) * ((D + 255) / 256);
    const int64_t steps = (piece + kStep - 1) / kStep;
    const int64_t s = std::max<int64_t>(1, std::min<int64_t>(device_cu_count() / tiles, steps / 8));
    const int64_t per = (steps + s - 1) / s;
    return (int)((steps + per - 1) / per);
}

// dw of a small vocabulary likewise: where the vocabulary is one piece and its tiles fill at
// most half of the CUs, its reduction over the tokens is split (8 or more steps each) and
// the partial sums are joined.  The split saves 56 us of 131 with 8039 tokens, 1246 x 272,
// and 46 of 169 with 8192, 256 x 4096 (MI355X).
int dw_splits(int64_t T, int64_t V, int64_t D, int64_t piece)
{
    const int64_t tiles = (V + 255) / 256 * ((D + 255) / 256), steps = (T + kStep - 1) / kStep;
    if (piece < V || 2 * tiles > device_cu_count()) return 1;
    const int64_t s = std::max<int64_t>(1, std::min<int64_t>(device_cu_count() / tiles, steps / 8));
    const int64_t per = (steps + s - 1) / s;
    return (int)((steps + per - 1) / per);
}

struct Space {                            // the workspace's parts, in bytes from its start
    int64_t g, sum, unit, live, wsum, total;
    int64_t piece;
    int splits, wsplits;                  // of dx, of dw
};

Space backward_space(int64_t T, int64_t V, int64_t D)
{
    Space s;
    s.piece = piece_columns(T, V);
    s.splits = dx_splits(T, D, std::min(s.piece, V));
    s.g = 0;
    s.sum = up_to(T * s.piece * 2, 256);
    s.unit = s.sum + up_to(T * D * 4 * s.splits, 256);
    s.wsplits = dw_splits(T, V, D, s.piece);
    s.live = s.unit + 256;
    s.wsum = s.live + up_to((T + 63) / 64 * 8, 256);
    s.total = s.wsum + (s.wsplits > 1 ? V * D * 4 * s.wsplits : 0);
    return s;
}

template <int MI, int NJ, int GM, int GN, int NS, bool LA, bool LB, int EPI>
hipError_t launch_product(const LossArgs& g, hipStream_t stream)
{
    const int grid = std::min(g.units, device_cu_count() * loss_per_cu(MI, NJ));
    return launch(loss_product_kernel<MI, NJ, GM, GN, NS, LA, LB, EPI>, dim3((unsigned)grid), dim3(256), stream, g);
}

// Which tiles a product runs on.  Few rows (64 or 128) take tiles of as many.  256-row
// tiles run in rounds of one per CU; when those past the last full round would fill at
// most half of one, they run as halves in a launch of their own (8192 x 8192 x 5120, 640
// tiles: 2.5 rounds instead of 3).
template <bool LA, bool LB, int EPI>
hipError_t product(LossArgs g, int rows, int splits, hipStream_t stream)
{
    const bool narrow = !LB && rows == 64;               // logits of few tokens: 64 x 128
    const bool shallow = LA && rows == 128;              // dw of few tokens: 128 x 128
    const int cols = narrow || shallow ? 128 : 256;
    g.tiles_m = (g.P + rows - 1) / rows;
    g.tiles_n = (g.Q + cols - 1) / cols;
    g.steps = (g.R + kStep - 1) / kStep;
    g.per = (g.steps + splits - 1) / splits;
    g.units = g.tiles_m * g.tiles_n * ((g.steps + g.per - 1) / g.per);
    if constexpr (!LA) {
        if constexpr (!LB) {
            if (rows == 64) return launch_product<4, 2, 1, 4, 3, LA, LB, EPI>(g, stream);
        } else {
            if (rows == 64) return launch_product<4, 4, 1, 4, 2, LA, LB, EPI>(g, stream);
        }
        if (rows == 128) return launch_product<4, 8, 2, 2, 2, LA, LB, EPI>(g, stream);
    } else {
        if constexpr (EPI == kStore)
            if (rows == 128) return launch_product<4, 4, 2, 2, 2, LA, LB, EPI>(g, stream);
    }
    const int cus = device_cu_count(), tail = g.units % cus;
    const bool split = tail > 0 && 2 * tail <= cus;
    const int whole = split ? g.units - tail : g.units;
    if (whole > 0) {
        g.units = whole;
        const hipError_t e = launch_product<8, 8, 2, 2, 2, LA, LB, EPI>(g, stream);
        if (e != hipSuccess || !split) return e;
    }
    g.first = whole;
    g.halves = 1;
    g.units = 2 * tail;
    return launch_product<4, 8, 2, 2, 2, LA, LB, EPI>(g, stream);
}

}  // namespace

int64_t loss_forward_workspace(int64_t T, int64_t V)
{
    const int cb = column_block(logit_rows(T, V));
    return up_to((V + cb - 1) / cb * T * 8, 256) + T * 4;
}

int64_t loss_backward_workspace(int64_t T, int64_t V, int64_t D) { return backward_space(T, V, D).total; }

hipError_t launch_loss_forward(const void* x, const void* w, const int64_t* target, int64_t T, int64_t V, int64_t D,
                               float* loss, float* lse, void* workspace, hipStream_t stream)
{
    const int rows = logit_rows(T, V), cb = column_block(rows);
    const int blocks = (int)((V + cb - 1) / cb);
    LossArgs g{};
    g.a = {static_cast<const uint16_t*>(x), D};
    g.b = {static_cast<const uint16_t*>(w), D};
    g.P = (int)T;
    g.Q = (int)V;
    g.R = (int)D;
    g.target = target;
    g.vocab = (int)V;
    g.stats = static_cast<float2*>(workspace);
    g.hit = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + up_to((int64_t)blocks * T * 8, 256));
    const hipError_t e = product<false, false, kStats>(g, rows, 1, stream);
    if (e != hipSuccess) return e;
    const int joined = rows == 64 ? 2 : 16;
    return launch(rows == 64 ? loss_join_kernel<2> : loss_join_kernel<16>, dim3((unsigned)((T + joined - 1) / joined)),
                  dim3(1024), stream, static_cast<const float2*>(g.stats), blocks, static_cast<const float*>(g.hit), target, (int)T, V, loss,
                  lse);
}

hipError_t launch_loss_backward(const float* dloss, const void* x, const void* w, const int64_t* target,
                                const float* lse, int64_t T, int64_t V, int64_t D, void* dx, void* dw,
                                void* workspace, hipStream_t stream)
{
    const Space sp = backward_space(T, V, D);
    const int rows = tile_rows(T);
    uint16_t* gm = static_cast<uint16_t*>(workspace);
    float* sum = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + sp.sum);
    float* unit = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + sp.unit);
    uint64_t* live = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(workspace) + sp.live);
    float* wsum = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + sp.wsum);
    hipError_t e = hipSuccess;
    const Side xs{static_cast<const uint16_t*>(x), D};
    int splits = sp.splits;
    for (int64_t v0 = 0; v0 < V; v0 += sp.piece) {
        const int64_t n = std::min(sp.piece, V - v0);
        const Side ws{static_cast<const uint16_t*>(w) + v0 * D, D}, gs{gm, sp.piece};
        LossArgs g{};
        g.a = xs;
        g.b = ws;
        g.P = (int)T;
        g.Q = (int)n;
        g.R = (int)D;
        g.target = target;
        g.lse = lse;
        g.dloss = dloss;
        g.unit = unit;
        g.live = live;
        g.v0 = (int)v0;
        g.vocab = (int)V;
        g.out = gm;
        g.out_pitch = sp.piece;
        g.out_cols = (int)up_to(n, 8);
        e = product<false, false, kGrad>(g, logit_rows(T, n), 1, stream);
        if (e != hipSuccess) return e;

        LossArgs d{};
        d.a = gs;
        d.b = ws;
        d.P = (int)T;
        d.Q = (int)D;
        d.R = (int)n;
        d.sum = sum;
        d.unit = unit;
        d.out = static_cast<uint16_t*>(dx);
        d.out_pitch = D;
        d.fresh = v0 == 0;
        d.last = splits == 1 && v0 + n == V;
        e = product<false, true, kSum>(d, rows, splits, stream);
        if (e != hipSuccess) return e;

        LossArgs h{};
        h.a = gs;
        h.b = xs;
        h.P = (int)n;
        h.Q = (int)D;
        h.R = (int)T;
        h.unit = unit;
        h.live = live;
        h.out = static_cast<uint16_t*>(dw) + v0 * D;
        h.out_pitch = D;
        if (sp.wsplits > 1) {
            h.sum = wsum;
            h.fresh = 1;
            e = product<true, true, kSum>(h, 256, sp.wsplits, stream);
        } else {
            e = product<true, true, kStore>(h, T <= kStep ? 128 : 256, 1, stream);
        }
        if (e != hipSuccess) return e;
    }
    auto add = [&](const float* parts, int count, int64_t n, void* out) {
        return launch(loss_add_kernel, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), stream,
                      reinterpret_cast<const float4*>(parts), count, n / 4, static_cast<const float*>(unit),
                      static_cast<uint2*>(out));
    };
    if (sp.wsplits > 1) e = add(wsum, sp.wsplits, V * D, dw);
    if (e == hipSuccess && splits > 1) e = add(sum, splits, T * D, dx);
    return e;
}

}  // namespace fp8k
