// moe_mat_tile.h -- tiles of the experts' products in bf16: the forward product and both of its
// gradients (moe_matmul.hip, moe_matmul_grad.hip). One kernel makes all three, whose operands differ in
// how they lie in memory next to the axis that is summed over:
//   forward   out[r, n] = sum_i a[s(r), i] w[e, n, i]     both along the sum;
//   rows      da[r, i]  = sum_n dy[r, n] w[e, n, i]       w across it: read out of LDS transposed;
//   weights   dw[e, n, i] = sum_r dy[r, n] a[s(r), i]     both across it, and the sum ends with the
//                                                         expert's rows.
#ifndef MOE_MAT_TILE_H
#define MOE_MAT_TILE_H

#include <atomic>
#include <type_traits>

#include "moe_block.h"
#include "moe_tiles.h"

namespace {

using namespace moe_dev;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

enum Mode { kForward, kRowsBack, kWeightsBack };

struct MatArgs {
    const __bf16* rows;        // a; dy; dy
    const __bf16* cols;        // w; w; a
    const int32_t* row_token;
    const int32_t* offsets;
    const float* bias;
    const void* extra;         // residual (out's type); pre (bf16), for the activation's gradient
    void* out;
    __bf16* pre;               // out, forward only
    int32_t a_rows, R, E;
    int32_t N;                 // columns of the result
    int32_t M;                 // weights: rows of an expert's result
    int32_t D;                 // forward, rows: terms of a sum
    int32_t act;
    int32_t n_blocks;          // tiles side by side over N
    int32_t max_tiles;         // row tiles, at most
    double inv_blocks;         // 1 / n_blocks
    int32_t m_blocks;          // weights: tiles of an expert over M
    int32_t splits;            // parts that a sum is made in, each a result of its own
};

// Rows of expert e and the first of them, as expert_rows() of the other products, which the tiles'
// functions find here for these arguments. Offsets are read as constants: for the same e in every lane
// that is a scalar load, which is not waited for together with the loads into LDS.
__device__ __forceinline__ int32_t expert_rows(const MatArgs& p, int32_t e, int32_t* lo)
{
    if (!p.offsets) {
        *lo = 0;
        return p.R;
    }
    typedef const __attribute__((address_space(4))) int32_t* constants;
    const constants at = (constants)(uintptr_t)p.offsets;
    *lo = min(max(at[e], 0), p.R);
    return min(max(at[e + 1], *lo), p.R) - *lo;
}

constexpr uint32_t kOut = 0xFFFFFFF0u;   // offset behind every buffer: such a load gives zeros
constexpr int kXcds = 8;                 // workgroup b runs on XCD b % 8
constexpr int kCus = 256;
constexpr int kStepK = 128;              // bytes of a line in a stage: 64 terms of the sum

// ------------------------------------------------------------------------------- epilogues --
// GELU's tanh form is v / (1 + exp(-t)), t = 2 sqrt(2 / pi) (v + 0.044715 v^3).
constexpr float kGelu = 1.59576912f, kCube = 0.044715f;

// 1 / (1 + exp(-t)), with the rounding of t log2 e added back to first order, as in logistic(). Below
// -87, where it leaves the normal numbers, it is 0.
__device__ __forceinline__ float sigmoid(float t)
{
    constexpr float hi = -1.44269502f, lo = -1.92596299e-8f;
    const float x = t * hi;
    const float rest = (__builtin_fmaf(t, hi, -x) + t * lo) * 0.693147182f;
    const float e = __builtin_amdgcn_exp2f(x);
    const float r = __builtin_amdgcn_rcpf(1.0f + (t > 87.0f ? 0.0f : __builtin_fmaf(e, rest, e)));
    return t < -87.0f ? 0.0f : r;
}

__device__ __forceinline__ float activate(float v, int32_t act)
{
    if (act == MOE_MAT_RELU)
        return v < 0.0f ? 0.0f : v;
    if (act == MOE_MAT_SILU)
        return silu<true>(v);
    if (act == MOE_MAT_GELU)
        return logistic<true>(v, kGelu * __builtin_fmaf(kCube * v * v, v, v));
    return v;
}

// The activation's slope at v: s (1 + v (1 - s)) of SiLU, s (1 + v (1 - s) t') of GELU. Both are 0
// and 1 to fp32 from 100 on, where v is taken for its bound; a NaN stays one. Where s is taken for 0
// the slope is below 4e-36.
__device__ __forceinline__ float slope(float v, int32_t act)
{
    if (act == MOE_MAT_RELU)
        return v > 0.0f ? 1.0f : v == v ? 0.0f : v;
    const float w = fminf(fmaxf(v, -100.0f), 100.0f);
    const bool gelu = act == MOE_MAT_GELU;
    const float s = sigmoid(gelu ? kGelu * __builtin_fmaf(kCube * w * w, w, w) : w);
    const float dt = gelu ? kGelu * __builtin_fmaf(3.0f * kCube * w, w, 1.0f) : 1.0f;
    const float d = s * __builtin_fmaf(w * dt, 1.0f - s, 1.0f);
    return v == v ? d : v;
}

// Four values at p, `left` of them there; `vec`: all rows of theirs lie on 4-element borders.
__device__ __forceinline__ f32x4 load4(const float* p, int32_t left, bool vec)
{
    if (vec && left >= 4)
        return *reinterpret_cast<const f32x4*>(p);
    f32x4 v;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        v[c] = c < left ? p[c] : 0.0f;
    return v;
}

__device__ __forceinline__ f32x4 load4(const __bf16* p, int32_t left, bool vec)
{
    f32x4 v;
    if (vec && left >= 4) {
        const bf16x4 b = *reinterpret_cast<const bf16x4*>(p);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            v[c] = (float)b[c];
        return v;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
        v[c] = c < left ? (float)p[c] : 0.0f;
    return v;
}

// The thread's number where the compiler does not know it for that: what is made from it is made there,
// in place of before the loop over the tiles, where it would hold registers through all products.
__device__ __forceinline__ int thread_here()
{
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

// ---- tiles ----
struct Work {
    Tile t;                    // weights: row0 is a row of the expert's result
    int32_t step0, step1;      // steps of the sum
    int32_t split;
    int32_t first, count;      // weights: the expert's rows
};

// The steps of part `split` of a sum of `steps`. Weights: of an expert's rows, which may be none, or fewer
// steps than parts; a part without steps gets one behind the end, whose rows are not there. The other sums are
// as long for every tile, and choose() gives each part four steps at least: there a step behind the end would
// read the next rows.
__device__ __forceinline__ void part_of(const MatArgs& p, int32_t split, int32_t steps, Work* w)
{
    w->split = split;
    w->step0 = p.splits > 1 ? (int32_t)((int64_t)steps * split / p.splits) : 0;
    w->step1 = p.splits > 1 ? (int32_t)((int64_t)steps * (split + 1) / p.splits) : steps;
    if (w->step1 <= w->step0) {                               // nothing: a step behind the end, zeros
        w->step0 = steps;
        w->step1 = steps + 1;
    }
}

// Tile `at` of the experts' weights: expert by expert, four blocks of M by all blocks of N at a time,
// those of M fastest, so that tiles that run together on an XCD share their operands in its L2.
template <int BM>
__device__ __forceinline__ Work weights_at(const MatArgs& p, int32_t at)
{
    Work w;
    const int32_t all = p.max_tiles * p.n_blocks, split = p.splits > 1 ? at / all : 0;
    at -= split * all;
    const int32_t row = quotient(at, p.n_blocks, p.inv_blocks);
    w.t.e = __builtin_amdgcn_readfirstlane(row / p.m_blocks);
    const int32_t local = at - w.t.e * p.m_blocks * p.n_blocks;
    const int32_t group = quotient(local, 4 * p.n_blocks, p.inv_blocks / 4);
    const int32_t in = local - group * 4 * p.n_blocks;
    const int32_t side = min(4, p.m_blocks - group * 4);
    w.t.n = side == 4 ? in >> 2 : side == 3 ? (int32_t)((uint32_t)in / 3u) : side == 2 ? in >> 1 : in;
    const int32_t block = group * 4 + in - w.t.n * side;
    w.t.row0 = block * BM;
    w.t.rows = min(BM, p.M - block * BM);
    w.count = __builtin_amdgcn_readfirstlane(expert_rows(p, w.t.e, &w.first));
    w.first = __builtin_amdgcn_readfirstlane(w.first);
    part_of(p, split, (w.count + 63) / 64, &w);
    return w;
}

// Results of a wavefront's fragments, row lane % 32 and columns 8 i + 4 (lane / 32) + c of fragment
// g in v[g][i], through a little LDS of its own and out as whole lines: 16-byte piece c of row r
// lies in slot c ^ (r % 8). Rows of whole 64 bytes are stored past the caches (weights of 20 experts of 1000
// x 2064 in fp32, with the other gradients, 98 us for 110, 32 experts of 4096 x 2048 1% either way); others
// through them, where the L2 puts together what two tiles write of 64 bytes (weights of 60 experts of 264 x
// 5016 in fp32 74 us for 158).
template <int UNIT, typename OUT, int F>
__device__ __forceinline__ void store_unit(int8_t* unit, const typename Four<OUT>::type (&v)[F][4],
                                           OUT* base, __amdgpu_buffer_rsrc_t buffer, bool wide, bool past,
                                           int32_t ld, int32_t n_end, int32_t tr, int32_t n1,
                                           uint32_t rows, int lane)
{
    constexpr int kRow = F * 32 * (int)sizeof(OUT), kRows = UNIT / kRow < 32 ? UNIT / kRow : 32;
    constexpr int kStores = kRows * kRow / 1024, kPieces = kRow / 16;
    static_assert(kStores >= 1, "unit");
    const int r32 = lane & 31, half = lane >> 5;
    const auto at16 = [&](int r, int c) {                     // piece c of row r
        return unit + r * kRow + (c ^ (r & (kPieces - 1) & 7)) * 16;
    };
#pragma unroll 1
    for (int phase = 0; phase < 32 / kRows; ++phase) {
        asm volatile("" ::: "memory");                        // LDS serves a wavefront in order
        if (r32 / kRows == phase) {
            const int r = r32 % kRows;
#pragma unroll
            for (int g = 0; g < F; ++g)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int byte = (32 * g + 8 * i + 4 * half) * (int)sizeof(OUT);
                    *reinterpret_cast<typename Four<OUT>::type*>(at16(r, byte / 16) + byte % 16) =
                        v[g][i];
                }
        }
        asm volatile("" ::: "memory");
        const int32_t tr0 = tr + phase * kRows;
        const uint32_t ok = rows >> phase * kRows;
        if (wide) {
#pragma unroll
            for (int s = 0; s < kStores; ++s) {
                const int r = s * (kRows / kStores) + lane / kPieces, c = lane % kPieces;
                const u32x4 out = *reinterpret_cast<const u32x4*>(at16(r, c));
                const int32_t n = n1 + c * (16 / (int)sizeof(OUT));
                const uint32_t to = ((uint32_t)(tr0 + r) * (uint32_t)ld + (uint32_t)n) *
                                    (uint32_t)sizeof(OUT);
                const uint32_t at = (ok >> r & 1) && n < n_end ? to : kOut;
                if (past)
                    store_buffer(out, buffer, at);
                else
                    __builtin_amdgcn_raw_buffer_store_b128(out, buffer, at, 0, 0);
            }
        } else {                                              // a value a lane, side by side
            constexpr int kCols = F * 32;
#pragma unroll 1
            for (int s = 0; s < kRows * kCols / 64; ++s) {
                const int r = s * (64 / kCols) + lane / kCols, c = lane % kCols;
                const int byte = c * (int)sizeof(OUT);
                const OUT out = *reinterpret_cast<const OUT*>(at16(r, byte / 16) + byte % 16);
                if ((ok >> r & 1) && n1 + c < n_end)
                    base[(int64_t)(tr0 + r) * ld + n1 + c] = out;
            }
        }
    }
}

// `left` of four values at p (or all, if more).
template <typename OUT>
__device__ __forceinline__ void store4(OUT* p, typename Four<OUT>::type v, int32_t left)
{
    if (left >= 4 && (uintptr_t)p % sizeof(v) == 0) {
        *reinterpret_cast<typename Four<OUT>::type*>(p) = v;
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (c < left)
                p[c] = v[c];
    }
}

template <typename OUT>
__device__ __forceinline__ typename Four<OUT>::type round4(f32x4 y)
{
    typename Four<OUT>::type v;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        v[c] = (OUT)y[c];
    return v;
}

// Where a result's rows go: the tile's first row at base, a row in `parts` parts of n columns.
template <typename OUT>
struct Sink {
    OUT* base;
    int32_t ld;
    bool wide, past;
    __amdgpu_buffer_rsrc_t buffer;

    __device__ __forceinline__ Sink(OUT* out, int64_t row0, int32_t rows, int32_t n, int32_t parts)
    {
        const int32_t columns = parts * n;
        base = out + row0 * columns;
        ld = columns;
        wide = n % (16 / (int)sizeof(OUT)) == 0 && (uintptr_t)out % 16 == 0 && columns <= (1 << 20);
        past = n * (int64_t)sizeof(OUT) % 64 == 0 && (uintptr_t)out % 64 == 0;
        buffer = __builtin_amdgcn_make_buffer_rsrc(
            base, 0, (int32_t)((uint32_t)rows * (uint32_t)columns * (uint32_t)sizeof(OUT)),
            0x00020000);
    }
};

// An operand whose lines lie across the sum: a stage holds 64 lines of COLS columns. A wavefront's
// load brings 1024 bytes, two or four lines. ds_read_b64_tr_b16 hands lane i of 16 the column i of
// four lines of 16 columns (32 bytes); unit u of line c lies in unit u ^ flip(c), so that the four
// lines of 16 lanes, and the two units of 32, fall on different banks.
template <int COLS>
struct Across {
    static constexpr int kPieces = COLS / 8, kLines = 64 / kPieces;   // of a load
    static_assert(COLS == 128 || COLS == 256, "eight units of 32 bytes at least");

    __device__ __forceinline__ static int flip(int line) { return (line & 1) * 2 ^ (line >> 1 & 1) * 5; }
};

// The operands' 16 bytes of a lane: 8 terms of the sum for one row or column of a fragment.
__device__ __forceinline__ bf16x8 read_along(const int8_t* p)
{
    return *reinterpret_cast<const bf16x8*>(p);
}

template <int COLS>
__device__ __forceinline__ bf16x8 read_across(const int8_t* p)
{
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * COLS * 2));
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, v);
}

// A tile of BM rows by BN columns by WM x WN wavefronts, each of BM / WM by BN / WN of it: the operands'
// roles are exchanged in the instruction (columns left, rows right), so that a lane's sums are four columns
// side by side of one row. A step is 64 terms of the sum: a stage of 128 bytes a line, filled by loads that
// go straight to LDS, STAGES of them around. Operands along the sum: 16-byte piece c of line r lies in slot c
// ^ (r / 2 % 8), which keeps the reads of 16 bytes off each other's banks (no conflicts counted; with r % 8
// half of the LDS cycles were conflicts, in the same time). The four quarters of a step are read one
// quarter ahead of their products, and the loads of a stage are spread out over the two quarters behind
// its barrier (2% less time than all at once). Loads out of range write zeros, so the ends of sums, rows
// that take no part and channels beyond the last cost no instructions. Sums stay in fp32 from the first
// product to the epilogue; pre, out and da are rounded to their type once, at the end.
// Bound by LDS and the matrix cores together: a 256 x 256 step takes 1.71 us, its products alone 0.86 at
// 2.5 PFLOP/s. 8192 x 8192 x 8192 in forward form 926 us when taken apart (868 to
// 912 since), without the loads 770, without the LDS reads 784, without the products 516: each takes over
// half of the time and they overlap as far as two stages of 64 KB allow (a third does not fit). The
// gradients of 8192^3: rows 870 to 910, weights 905 to 970 (a library product 779).
// FULL: with pre, a residual, or an activation other than SwiGLU (rows: with an activation's
// gradient), whose registers the other calls do not have to give up.
template <int MODE, int BM, int BN, int WM, int WN, int STAGES, bool SWIGLU, bool FULL,
          typename OUT>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_mat_tile(MatArgs p)
{
    constexpr bool kRowsAcross = MODE == kWeightsBack, kColsAcross = MODE != kForward;
    constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
    constexpr int MF = BM / WM / 32, NF = BN / WN / 32;       // 32 x 32 fragments of a wavefront
    constexpr int kLoadsA = BM / 8 / kWaves, kLoadsW = BN / 8 / kWaves;
    constexpr int kLoads = kLoadsA + kLoadsW;
    constexpr int kStage = (BM + BN) * kStepK;
    constexpr int kGroup = 4;
    static_assert(MF * WM * 32 == BM && NF * WN * 32 == BN, "tile");
    static_assert(kLoadsA * 8 * kWaves == BM && kLoadsW * 8 * kWaves == BN, "loads");
    static_assert(STAGES >= 2, "a stage ahead");
    static_assert(MODE == kForward || !SWIGLU, "only the forward product pairs channels");
    static_assert(MODE != kWeightsBack || STAGES == 2, "row tokens have come with the stage before");
    // results of a wavefront: fragments side by side, and the units they are stored in
    constexpr int kUnit = STAGES * kStage + kWaves * 2048 + 8192 <= 163840 ? 2048 : 1024;
    constexpr int kOutF = SWIGLU ? NF / 2 : NF, kUnitF = kOutF < 2 || sizeof(OUT) == 4 ? 1 : 2;
    constexpr int kStores = MF * (kOutF / kUnitF) * kUnitF * 32 * 32 * (int)sizeof(OUT) / 1024;
    static_assert(NF == 2 && BM <= kThreads, "results");
    static_assert((STAGES - 2) * kLoads + kStores <= 63, "vmcnt has six bits");
    extern __shared__ __attribute__((aligned(1024))) int8_t s_stage[];
    __shared__ __attribute__((aligned(16))) int8_t s_unit[kWaves][kUnit];
    __shared__ __attribute__((aligned(16))) float s_bias[BN];
    __shared__ uint32_t s_ok[BM / 32];                        // a bit for each row to be written
    constexpr int kRing = 8;
    static_assert(STAGES + 2 <= kRing, "tiles between the loads and the products");
    __shared__ Work s_work[kRing];
    int32_t* s_prefix = reinterpret_cast<int32_t*>(s_stage + STAGES * kStage);   // [E + 1]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // workgroup b runs on XCD b % 8: each XCD takes a run of consecutive tiles, all of them, or, where
    // the experts' rows make tiles unequal, of those that run at a time
    int32_t first, last, stride, all = 0;                     // all: tiles of a part
    if (MODE == kWeightsBack) {
        last = p.max_tiles * p.n_blocks * p.splits;
        stride = gridDim.x;
        first = (blockIdx.x % kXcds) * (gridDim.x / kXcds) + blockIdx.x / kXcds;
    } else {
        all = tile_prefix<kThreads, BM>(p, s_prefix) * p.n_blocks;
        const int32_t whole = all * p.splits;
        const int32_t share = (whole + kXcds - 1) / kXcds;
        stride = gridDim.x / kXcds;
        first = (blockIdx.x % kXcds) * share + blockIdx.x / kXcds;
        last = min((int32_t)(blockIdx.x % kXcds + 1) * share, whole);
    }
    if (first >= last)
        return;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int8_t*)s_stage;
    const int32_t n_w = SWIGLU ? 2 * p.N : p.N;

    // The loads run ahead of the products through the same tiles: their own place in them
    const int line = lane >> 3;                               // operands along the sum
    const int piece = 16 * ((lane & 7) ^ (4 * (wave & 1) + (line >> 1)));
    static_assert(kWaves % 2 == 0, "a wavefront's lines are all even or odd eights");
    typedef Across<(kRowsAcross ? BM : 128)> RowsT;
    typedef Across<(kColsAcross ? BN : 128)> ColsT;
    const auto line_a = [&](int i) {
        return kRowsAcross ? (i * kWaves + wave) * RowsT::kLines + lane / RowsT::kPieces
                           : 8 * (i * kWaves + wave) + line;
    };
    const auto line_w = [&](int i) {
        return kColsAcross ? (i * kWaves + wave) * ColsT::kLines + lane / ColsT::kPieces
                           : 8 * (i * kWaves + wave) + line;
    };
    u32x4 abuf, wbuf;
    uint32_t avo[kLoadsA], wvo[kLoadsW];                      // offsets at the tile's first step
    int32_t arow[kLoadsA], wrow[kLoadsW];                     // rows read ahead, used a step later
    int32_t load_tile = first, load_step = 0, load_nth = 0;
    Work lw;
    uint32_t load_to = lds0 + wave * 1024;
    int32_t ahead = 0;                                        // stages loaded and not yet begun
    int32_t older = 0;                                        // of these, before the last stores
    const auto tokens = [&]() {                               // of the rows of the next step
        if (MODE == kWeightsBack && p.row_token && lw.count > 0) {
            const int32_t r0 = load_step * 64;
#pragma unroll
            for (int i = 0; i < kLoadsA; ++i)
                arow[i] = p.row_token[lw.first + min(r0 + line_a(i), lw.count - 1)];
#pragma unroll
            for (int i = 0; i < kLoadsW; ++i)
                wrow[i] = p.row_token[lw.first + min(r0 + line_w(i), lw.count - 1)];
        }
    };
    const auto aim = [&]() {
        if (MODE == kWeightsBack) {
            lw = weights_at<BM>(p, load_tile);
        } else {
            const int32_t split = p.splits > 1 ? load_tile / all : 0;
            lw.t = tile_at<BM, kGroup>(p, s_prefix, load_tile - split * all);
            part_of(p, split, (p.D + 63) / 64, &lw);
        }
        load_step = lw.step0;
        if (tid == 0)
            s_work[load_nth % kRing] = lw;
        ++load_nth;
        const Tile& t = lw.t;
        const int32_t n0 = t.n * (SWIGLU ? BN / 2 : BN);
        if (kRowsAcross) {
#pragma unroll
            for (int i = 0; i < kLoadsA; ++i) {
                const int u = lane % RowsT::kPieces ^ RowsT::flip(line_a(i)) * 2;
                const int32_t n = t.row0 + 8 * u;
                avo[i] = (uint32_t)(n < p.M ? n : t.row0) * 2u;
            }
        } else {
            abuf = MODE == kForward && p.row_token
                       ? buffer_of(p.rows, (uint32_t)((int64_t)p.a_rows * p.D * 2))
                       : buffer_of(p.rows + (int64_t)t.row0 * p.D, (uint32_t)t.rows * (uint32_t)p.D * 2u);
#pragma unroll
            for (int i = 0; i < kLoadsA; ++i)
                arow[i] = min(line_a(i), t.rows - 1);
            if (MODE == kForward && p.row_token) {
#pragma unroll
                for (int i = 0; i < kLoadsA; ++i)
                    arow[i] = p.row_token[t.row0 + arow[i]];
            }
        }
        if (kColsAcross) {
            if (MODE == kRowsBack)
                wbuf = buffer_of(p.cols + (int64_t)t.e * p.D * p.N, (uint32_t)((int64_t)p.D * p.N * 2));
#pragma unroll
            for (int i = 0; i < kLoadsW; ++i) {
                const int u = lane % ColsT::kPieces ^ ColsT::flip(line_w(i)) * 2;
                const int32_t n = n0 + 8 * u;
                wvo[i] = (uint32_t)(n < p.N ? n : n0) * 2u;
                if (MODE == kRowsBack)
                    wvo[i] += (uint32_t)line_w(i) * (uint32_t)p.N * 2u;
            }
        } else {
            wbuf = buffer_of(p.cols + (int64_t)t.e * n_w * p.D, (uint32_t)((int64_t)n_w * p.D * 2));
#pragma unroll
            for (int i = 0; i < kLoadsW; ++i) {
                const int32_t c = line_w(i);
                // with SwiGLU every other 32 channels are the up channels of the 32 before
                int32_t n = SWIGLU ? n0 + c / 64 * 32 + c % 32 : n0 + c;
                n = min(n, p.N - 1) + (SWIGLU && (c & 32) ? p.N : 0);
                wvo[i] = (uint32_t)n * (uint32_t)p.D * 2u + piece;
            }
        }
    };
    // A stage is asked for in three steps: begin(), its kLoads loads one by one, end().
    bool some = false;                                        // there is a stage left to ask for
    uint32_t ao[kLoadsA], wo[kLoadsW], step_at = 0, step_by = 0;
    bool behind = false, ends = false;
    const auto begin = [&]() {
        some = load_tile < last;
        if (!some)
            return;
        if (MODE == kWeightsBack) {
            const int32_t r0 = load_step * 64, left = max(0, min(64, lw.count - r0));
            const int64_t row = (int64_t)lw.first + r0;
            abuf = buffer_of(p.rows + row * p.M, (uint32_t)left * (uint32_t)p.M * 2u);
            wbuf = p.row_token ? buffer_of(p.cols, (uint32_t)((int64_t)p.a_rows * p.N * 2))
                               : buffer_of(p.cols + row * p.N, (uint32_t)left * (uint32_t)p.N * 2u);
            // all offsets before the first load: the compiler waits for the tokens where they are
            // used, and would wait there for the loads that went out before
            if (p.row_token) {
#pragma unroll
                for (int i = 0; i < kLoadsA; ++i) {
                    const int32_t c = line_a(i);
                    const bool in = c < left && (uint32_t)arow[i] < (uint32_t)p.a_rows;
                    ao[i] = in ? avo[i] + (uint32_t)c * (uint32_t)p.M * 2u : kOut;
                }
#pragma unroll
                for (int i = 0; i < kLoadsW; ++i) {
                    const bool in = line_w(i) < left && (uint32_t)wrow[i] < (uint32_t)p.a_rows;
                    wo[i] = in ? wvo[i] + (uint32_t)wrow[i] * (uint32_t)p.N * 2u : kOut;
                }
            } else {
#pragma unroll
                for (int i = 0; i < kLoadsA; ++i)
                    ao[i] = line_a(i) < left ? avo[i] + (uint32_t)line_a(i) * (uint32_t)p.M * 2u : kOut;
#pragma unroll
                for (int i = 0; i < kLoadsW; ++i)
                    wo[i] = line_w(i) < left ? wvo[i] + (uint32_t)line_w(i) * (uint32_t)p.N * 2u : kOut;
            }
#pragma unroll
            for (int i = 0; i < kLoadsA; ++i)
                asm volatile("" : "+v"(ao[i]));
#pragma unroll
            for (int i = 0; i < kLoadsW; ++i)
                asm volatile("" : "+v"(wo[i]));
        } else {
            // the tokens are waited for here, before the loads, with two stages in every step: what is
            // under way from memory has come then, and the compiler does not wait again where it
            // cannot tell
            if (STAGES == 2 || load_step == lw.step0) {
#pragma unroll
                for (int i = 0; i < kLoadsA; ++i)
                    asm volatile("" : "+v"(arow[i]));
            }
            if (load_step == lw.step0) {
#pragma unroll
                for (int i = 0; i < kLoadsA; ++i) {
                    int32_t r = arow[i];
                    if (MODE == kForward && p.row_token)
                        r = (uint32_t)r < (uint32_t)p.a_rows ? r : 0;     // its results are not stored
                    avo[i] = (uint32_t)r * (uint32_t)p.D * 2u + piece;
                }
            }
            ends = load_step == (p.D + 63) / 64 - 1;          // terms behind the sum's end are zeros
            behind = ends && load_step * 64 + piece / 2 >= p.D;
            step_at = (uint32_t)load_step * kStepK;
            step_by = kColsAcross ? (uint32_t)load_step * 64u * (uint32_t)p.N * 2u : step_at;
        }
    };
    const auto load = [&](int i) {
        if (!some)
            return;
        if (i < kLoadsA) {
            const uint32_t off = MODE == kWeightsBack ? ao[i] : behind ? kOut : avo[i] + step_at;
            load_lds(abuf, off, 0, load_to + i * kWaves * 1024);
        } else {
            i -= kLoadsA;
            const bool out = kColsAcross ? ends && load_step * 64 + line_w(i) >= p.D : behind;
            const uint32_t off = MODE == kWeightsBack ? wo[i] : out ? kOut : wvo[i] + step_by;
            load_lds(wbuf, off, 0, load_to + BM * kStepK + i * kWaves * 1024);
        }
    };
    const auto end = [&]() {
        if (!some)
            return;
        load_to += kStage;
        if (load_to >= lds0 + STAGES * kStage)
            load_to -= STAGES * kStage;
        ++ahead;
        if (++load_step == lw.step1) {
            load_tile += stride;
            if (load_tile < last)
                aim();
        }
        if (load_tile < last)
            tokens();
    };
    const auto issue = [&]() {
        begin();
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            load(i);
        end();
    };

    const int wm = MF > 1 ? wave / WN : wave % WM, wn = MF > 1 ? wave % WN : wave / WM;
    const int r32 = lane & 31, half = lane >> 5;
    f32x16 acc[MF][NF];
    // this lane's slots of the four quarters of a step: along the sum one for each quarter (32 rows
    // further on for each fragment), across it one for each fragment (16 lines on for each quarter)
    int slot[4], aslot[MF], wslot[NF];
#pragma unroll
    for (int q = 0; q < 4; ++q)
        slot[q] = r32 * kStepK + 16 * ((2 * q + half) ^ (r32 >> 1 & 7));
    const int across = 8 * half + ((lane & 15) >> 2);         // line of the quarter
#pragma unroll
    for (int m = 0; m < MF; ++m)
        aslot[m] = across * BM * 2 + 8 * (lane & 3) +
                   32 * ((2 * (wm * MF + m) + (lane >> 4 & 1)) ^ RowsT::flip(across));
#pragma unroll
    for (int f = 0; f < NF; ++f)
        wslot[f] = across * BN * 2 + 8 * (lane & 3) +
                   32 * ((2 * (wn * NF + f) + (lane >> 4 & 1)) ^ ColsT::flip(across));
    int at = 0;                                               // the stage that is multiplied
    bf16x8 wv[2][NF], av[2][MF];
    const auto read_a = [&](int m, int q) {
        if constexpr (kRowsAcross)
            return read_across<BM>(s_stage + at + aslot[m] + q * 16 * BM * 2);
        else
            return read_along(s_stage + at + (wm * MF + m) * 32 * kStepK + slot[q]);
    };
    const auto read_w = [&](int f, int q) {
        if constexpr (kColsAcross)
            return read_across<BN>(s_stage + at + BM * kStepK + wslot[f] + q * 16 * BN * 2);
        else
            return read_along(s_stage + at + (BM + (wn * NF + f) * 32) * kStepK + slot[q]);
    };
    const auto read = [&](int set, int q) {                   // quarter q of the stage
#pragma unroll
        for (int f = 0; f < NF; ++f)
            wv[set][f] = read_w(f, q);
#pragma unroll
        for (int m = 0; m < MF; ++m)
            av[set][m] = read_a(m, q);
    };
    // Multiplies operand set `cur` while quarter q goes into the other set. Fragments of rows that
    // the tile does not have are left out. Reads stay spread out among the products, and so are the
    // loads of half a stage, if any.
    int32_t frags = MF;
    const auto multiply = [&](int cur, int q, auto which) {
        constexpr int kHalf = decltype(which)::value;
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            const bool live = MF == 1 || m < frags;
#pragma unroll
            for (int i = 0; i < NF; ++i) {
                if (kHalf >= 0) {
                    constexpr int kPlaces = 2 * MF * NF;
                    const int place = (kHalf * MF + m) * NF + i;
#pragma unroll
                    for (int n = place * kLoads / kPlaces; n < (place + 1) * kLoads / kPlaces; ++n)
                        load(n);
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (!live)
                    continue;
                const int f = m & 1 ? NF - 1 - i : i;
                acc[m][f] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wv[cur][f], av[cur][m],
                                                                    acc[m][f], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
                if (q >= 0 && i == 0)
                    av[1 - cur][m] = read_a(m, q);
                if (q >= 0 && m == 0)
                    wv[1 - cur][i] = read_w(i, q);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    constexpr std::integral_constant<int, -1> kNone{};
    constexpr std::integral_constant<int, 0> kFirst{};
    constexpr std::integral_constant<int, 1> kSecond{};
    // this wavefront's loads of the next stage have landed
    const auto landed = [&]() {
        if (ahead < STAGES - 1)
            wait_loads<0>();
        else if (older > 0)                                   // without the stores behind it
            wait_loads<(STAGES - 2) * kLoads + kStores>();
        else
            wait_loads<(STAGES - 2) * kLoads>();
        --older;
    };
    const auto after = [&](int stage) { return stage + kStage == STAGES * kStage ? 0 : stage + kStage; };

    aim();
    tokens();
#pragma unroll
    for (int s = 0; s < STAGES; ++s)
        issue();
    wait_loads<0>();
    ahead -= 1;
    wait_workgroup();
    for (int32_t tile = first, nth = 0; tile < last; tile += stride, ++nth) {
        const Work& work = s_work[nth % kRing];
        const int32_t steps = __builtin_amdgcn_readfirstlane(work.step1 - work.step0);
        const int32_t split = __builtin_amdgcn_readfirstlane(work.split);
        if (steps == 1)                                       // no wait in the loop keeps the
            wait_workgroup();                                 // tiles' rows and biases apart
        Tile t;
        t.e = __builtin_amdgcn_readfirstlane(work.t.e);
        t.row0 = __builtin_amdgcn_readfirstlane(work.t.row0);
        t.rows = __builtin_amdgcn_readfirstlane(work.t.rows);
        t.n = __builtin_amdgcn_readfirstlane(work.t.n);
        const int32_t n0 = t.n * (SWIGLU ? BN / 2 : BN);
        // a thread's row of the tile, and its channels' biases, put into LDS at the tile's end
        const bool mine = tid < t.rows;
        int32_t src = 0;
        if (MODE != kWeightsBack && p.row_token && mine)
            src = p.row_token[t.row0 + tid];
        float bias[(BN + kThreads - 1) / kThreads] = {};
        if (MODE == kForward && p.bias) {
#pragma unroll
            for (int i = 0; i < (BN + kThreads - 1) / kThreads; ++i) {
                const int32_t c = min(i * kThreads + tid, BN - 1);
                const int32_t n = min(SWIGLU ? n0 + c / 64 * 32 + c % 32 : n0 + c, p.N - 1);
                bias[i] = p.bias[(int64_t)t.e * n_w + n + (SWIGLU && (c & 32) ? p.N : 0)];
            }
        }
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
            for (int f = 0; f < NF; ++f)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    acc[m][f][i] = 0.0f;
        read(0, 0);
        frags = __builtin_amdgcn_readfirstlane(min(MF, (t.rows - wm * MF * 32 + 31) / 32));
        // A step multiplies the four quarters of its stage; before the last of them the next stage has
        // to be there and everybody has read this one, whose place is loaded again from then on.
        const auto turn = [&](int32_t step) {
            const int next = after(at);
            landed();
            if (step == 0) {                                  // waited for here, where loads are anyway
                asm volatile("" : "+v"(src));
#pragma unroll
                for (int i = 0; i < (BN + kThreads - 1) / kThreads; ++i)
                    asm volatile("" : "+v"(bias[i]));
            }
            wait_workgroup();
            --ahead;
            at = next;
            begin();
            multiply(1, 0, kFirst);
            multiply(0, 1, kSecond);
            end();
        };
        multiply(0, 1, kNone);
        for (int32_t step = 0; step < steps - 1; ++step) {
            multiply(1, 2, kNone);
            multiply(0, 3, kNone);
            turn(step);
        }
        multiply(1, 2, kNone);
        multiply(0, 3, kNone);
        multiply(1, -1, kNone);
        const int next = after(at);
        if (ahead > 0)
            landed();
        const uint64_t oks = __ballot(mine && (uint32_t)src < (uint32_t)(MODE == kWeightsBack ? 1 : p.a_rows));
        if (lane < 2 && wave * 2 + lane < BM / 32)
            s_ok[wave * 2 + lane] = (uint32_t)(oks >> (32 * lane));
        if (MODE == kForward && p.bias) {
#pragma unroll
            for (int i = 0; i < (BN + kThreads - 1) / kThreads; ++i)
                if (i * kThreads + tid < BN)
                    s_bias[i * kThreads + tid] = bias[i];
        }
        wait_workgroup();
        older = 0;
        if (ahead > 0) {
            --ahead;
            issue();
            older = ahead;
        }
        at = next;

        // Results, while the next tile's first stages are on their way. Stores of whole rows count the
        // same for every wavefront, so that landed() can wait for the loads before them without them.
        const bool paired = MODE == kRowsBack && FULL && p.act == MOE_MAT_SWIGLU;
        const int64_t row0 = MODE == kWeightsBack ? ((int64_t)split * p.E + t.e) * p.M + t.row0
                                                  : (int64_t)split * p.R + t.row0;
        const Sink<OUT> out(static_cast<OUT*>(p.out), row0, t.rows, p.N, paired ? 2 : 1);
        const Sink<__bf16> pre(p.pre, row0, t.rows, p.N, SWIGLU ? 2 : 1);
        if (!out.wide || paired || (FULL && p.pre))
            older = 0;
        const int lane = thread_here() & 63, r32 = lane & 31, half = lane >> 5;
        int8_t* unit = s_unit[wave];
        const bool vec = p.N % 4 == 0 && (uintptr_t)p.extra % 16 == 0;
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            const uint32_t rows = s_ok[wm * MF + m];
            const int32_t tr = (wm * MF + m) * 32;
            const bool live = rows >> r32 & 1;
#pragma unroll
            for (int u = 0; u < kOutF; u += kUnitF) {
                const int32_t n1 = n0 + (wn * kOutF + u) * 32;
                typename Four<OUT>::type v[kUnitF][4], v2[kUnitF][4];   // columns 8 i + 4 half
                bf16x4 gate[kUnitF][4], up[kUnitF][4];
#pragma unroll
                for (int g = 0; g < kUnitF; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int f = SWIGLU ? 2 * (u + g) : u + g;
                        const int32_t n = n1 + 32 * g + 8 * i + 4 * half;
                        f32x4 y, z;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            y[c] = acc[m][f][4 * i + c];
                            z[c] = acc[m][f + SWIGLU][4 * i + c];
                        }
                        if (MODE == kForward) {
                            if (p.bias) {
                                const float* s = s_bias + (wn * NF + f) * 32 + 8 * i + 4 * half;
                                y += *reinterpret_cast<const f32x4*>(s);
                                if (SWIGLU)
                                    z += *reinterpret_cast<const f32x4*>(s + 32);
                            }
                            if (FULL && p.pre) {
                                gate[g][i] = round4<__bf16>(y);
                                if (SWIGLU)
                                    up[g][i] = round4<__bf16>(z);
                            }
                            if (SWIGLU) {
                                y = swiglu(y, z);
                            } else if (FULL && p.act != MOE_MAT_NONE) {
#pragma unroll
                                for (int c = 0; c < 4; ++c)
                                    y[c] = activate(y[c], p.act);
                            }
                            if (FULL && p.extra)
                                y += load4(static_cast<const OUT*>(p.extra) +
                                               (row0 + tr + r32) * p.N + n,
                                           live ? p.N - n : 0, vec);
                        }
                        if (MODE == kRowsBack && FULL) {
                            const int32_t left = live ? p.N - n : 0;
                            const __bf16* q = static_cast<const __bf16*>(p.extra) +
                                              (row0 + tr + r32) * (paired ? 2 * p.N : p.N) + n;
                            const f32x4 x = load4(q, left, vec);
                            if (paired) {
                                const f32x4 x2 = load4(q + p.N, left, vec);
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    z[c] = y[c] * activate(x[c], MOE_MAT_SILU);
                                    y[c] = y[c] * x2[c] * slope(x[c], MOE_MAT_SILU);
                                }
                                v2[g][i] = round4<OUT>(z);
                            } else {
#pragma unroll
                                for (int c = 0; c < 4; ++c)
                                    y[c] *= slope(x[c], p.act);
                            }
                        }
                        v[g][i] = round4<OUT>(y);
                    }
                if (MODE == kForward && FULL && p.pre) {
                    store_unit<kUnit, __bf16, kUnitF>(unit, gate, pre.base, pre.buffer, pre.wide, pre.past,
                                                      pre.ld, p.N, tr, n1, rows, lane);
                    if (SWIGLU)
                        store_unit<kUnit, __bf16, kUnitF>(unit, up, pre.base, pre.buffer, pre.wide,
                                                          pre.past, pre.ld, n_w, tr, p.N + n1, rows, lane);
                }
                store_unit<kUnit, OUT, kUnitF>(unit, v, out.base, out.buffer, out.wide, out.past, out.ld, p.N,
                                               tr, n1, rows, lane);
                if (MODE == kRowsBack && FULL && paired)
                    store_unit<kUnit, OUT, kUnitF>(unit, v2, out.base, out.buffer, out.wide, out.past, out.ld,
                                                   2 * p.N, tr, p.N + n1, rows, lane);
            }
        }
    }
}

// WGS: persistent workgroups of a CU; kOnce: a workgroup for each tile, taken up as CUs come free.
constexpr int kOnce = 1 << 20;

template <int MODE, int BM, int BN, int WM, int WN, int STAGES, int WGS, bool SWIGLU,
          bool FULL, typename OUT>
inline moe_status_t launch_tile(MatArgs p, hipStream_t stream)
{
    constexpr int kThreads = 64 * WM * WN, kStages = STAGES * (BM + BN) * kStepK;
    p.n_blocks = (int32_t)div_up(p.N, SWIGLU ? BN / 2 : BN);
    p.inv_blocks = 1.0 / p.n_blocks;
    p.m_blocks = MODE == kWeightsBack ? (int32_t)div_up(p.M, BM) : 0;
    const int64_t rows = MODE == kWeightsBack ? (int64_t)p.E * p.m_blocks : most_tiles(p, BM);
    const int64_t tiles = rows * p.n_blocks * p.splits;
    if (tiles > INT32_MAX / 2)
        return MOE_ERR_UNSUPPORTED;
    int64_t most = (int64_t)kCus * WGS;                       // and below 2^31 threads
    if (most > INT32_MAX / kThreads / kXcds * kXcds)
        most = INT32_MAX / kThreads / kXcds * kXcds;
    const int64_t blocks = tiles < most ? div_up(tiles, kXcds) * kXcds : most;
    p.max_tiles = (int32_t)rows;
    const auto kernel = k_mat_tile<MODE, BM, BN, WM, WN, STAGES, SWIGLU, FULL, OUT>;
    if (kStages > 49152) {                                    // once a device is enough
        static std::atomic<uint64_t> allowed{0};
        int dev = 0;
        if (hipGetDevice(&dev) != hipSuccess)
            return MOE_ERR_HIP;
        const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
        if (!(allowed.load(std::memory_order_relaxed) & bit)) {
            if (hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                    kStages + (MOE_MAX_EXPERTS + 1) * 4) != hipSuccess)
                return MOE_ERR_HIP;
            allowed.fetch_or(bit, std::memory_order_relaxed);
        }
    }
    const int prefix = MODE == kWeightsBack ? 0 : (p.E + 1) * 4;
    kernel<<<(unsigned)blocks, kThreads, kStages + prefix, stream>>>(p);
    return launched();
}

// The tile shapes, and what a step of 64 terms and a tile's beginning and end take (us, as measured with
// every slot taken; `alone` with one workgroup a CU): 16384 channels by 4096 rows in one expert, K = 512
// and 2048. Large tiles read less for each product (256 x 256: 1.25 PFLOP/s; 128 x 256: 1.0; 64 x 256:
// 0.85), small ones waste less on experts with few rows and fill the GPU sooner (98 rows of 60 experts,
// rows' gradient by 5016 of 264: 67 us by 256 x 256, 38 by 64 x 256; 32768 rows of 32 experts by 2048 of
// 4096: 525 and 804).
struct TileCost {
    int32_t bm, bn, slots;
    float step, alone, tile;
};
constexpr TileCost kMatTiles[3][5] = {
    {{256, 256, 256, 1.71f, 1.35f, 8.1f}, {128, 256, 256, 1.07f, 0.90f, 3.8f},
     {128, 128, 512, 1.03f, 0.82f, 5.0f}, {64, 256, 256, 0.62f, 0.62f, 3.5f},
     {32, 128, 512, 0.52f, 0.50f, 3.3f}},
    {{256, 256, 256, 1.71f, 1.33f, 8.0f}, {128, 256, 256, 1.07f, 0.88f, 3.8f},
     {128, 128, 512, 1.10f, 0.82f, 4.5f}, {64, 256, 256, 0.70f, 0.66f, 3.0f},
     {32, 128, 512, 0.66f, 0.55f, 3.0f}},
    {{256, 256, 256, 1.77f, 1.60f, 9.0f}, {128, 256, 256, 1.16f, 1.16f, 4.5f},
     {128, 128, 512, 1.16f, 1.00f, 5.0f}, {0, 0, 0, 0.0f, 0.0f, 0.0f}, {0, 0, 0, 0.0f, 0.0f, 0.0f}},
};

// How a product is made: its tile shape, and the parts of its sums. The least time by the
// figures above: rounds of tiles over the slots, where an expert's last tile (weights: step) is half full
// on average; the host knows the rows of all experts, not of each. Parts go through memory in fp32 and
// are joined by a launch of its own, 4 us and their bytes, which only few tiles with long sums are worth
// (4096 rows by 384 channels of 7168: 48 us in 4 parts, 72 in one); at most 16 parts and 256 MB of them, the
// size of the Infinity Cache.
struct Plan {
    int shape;
    int32_t splits;
    int64_t part_bytes;        // of all parts, 0 for one
};

constexpr int64_t kMostPartBytes = (int64_t)256 << 20;

template <int MODE>
inline Plan choose(int32_t R, int32_t E, int32_t M, int64_t n_w, int32_t D)
{
    const int64_t experts = E < R ? E : R;
    const double depth = MODE == kWeightsBack ? (double)R / E / 64 + 0.5 : (double)div_up(D, 64);
    const int64_t bytes = (MODE == kWeightsBack ? (int64_t)E * M : (int64_t)R) * n_w * 4;
    Plan best = {0, 1, 0};
    double least = 0.0;
    for (int splits = 1; splits <= 16; splits *= 2) {
        if (splits > 1 && (depth < 4.0 * splits || bytes * splits > kMostPartBytes))
            break;
        for (int i = 0; i < 5 && kMatTiles[MODE][i].bm; ++i) {
            const TileCost& c = kMatTiles[MODE][i];
            int64_t tiles;
            if (MODE == kWeightsBack)
                tiles = E * div_up(M, c.bm);
            else if (E == 1)
                tiles = div_up(R, c.bm);
            else
                tiles = R / c.bm + experts / 2 > experts ? R / c.bm + experts / 2 : experts;
            tiles *= div_up(n_w, c.bn) * splits;
            double time = (double)div_up(tiles, c.slots) *
                          (depth / splits * (tiles <= 256 ? c.alone : c.step) + c.tile);
            if (splits > 1)                                   // the join: a launch, and its bytes
                time += 4.0 + (double)bytes * (splits + 1) / 4e6;
            if ((splits == 1 && i == 0) || time < least) {
                best = {i, splits, splits > 1 ? bytes * splits : 0};
                least = time;
            }
        }
    }
    return best;
}

template <int MODE, bool SWIGLU, bool FULL, typename OUT>
inline moe_status_t launch_shape(int shape, const MatArgs& p, hipStream_t stream)
{
    if constexpr (MODE == kWeightsBack) {
        switch (shape) {
        case 0: return launch_tile<MODE, 256, 256, 2, 4, 2, 1, SWIGLU, FULL, OUT>(p, stream);
        case 1: return launch_tile<MODE, 128, 256, 2, 4, 2, 1, SWIGLU, FULL, OUT>(p, stream);
        default: return launch_tile<MODE, 128, 128, 2, 2, 2, 2, SWIGLU, FULL, OUT>(p, stream);
        }
    } else {
        switch (shape) {
        case 0: return launch_tile<MODE, 256, 256, 2, 4, 2, 1, SWIGLU, FULL, OUT>(p, stream);
        case 1: return launch_tile<MODE, 128, 256, 2, 4, 3, 1, SWIGLU, FULL, OUT>(p, stream);
        case 2: return launch_tile<MODE, 128, 128, 2, 2, 2, 2, SWIGLU, FULL, OUT>(p, stream);
        case 3: return launch_tile<MODE, 64, 256, 2, 4, 3, 1, SWIGLU, FULL, OUT>(p, stream);
        default: return launch_tile<MODE, 32, 128, 1, 2, 3, kOnce, SWIGLU, FULL, OUT>(p, stream);
        }
    }
}

// Weights of an expert that a product takes.
inline bool fits(int64_t n_w, int32_t K)
{
    return K % 8 == 0 && n_w <= MOE_MAT_MAX_SIZE && K <= MOE_MAT_MAX_SIZE && n_w * K * 2 < (int64_t)1 << 32;
}

// The limits that all three products share.
inline moe_status_t check_sizes(int32_t a_rows, const int32_t* row_token, const int32_t* offsets, int32_t R,
                         int32_t E, int32_t N, int64_t n_w, int32_t K, int32_t act)
{
    if (R < 0 || a_rows < 0 || E < 1 || N < 1 || K < 1 || act < MOE_MAT_NONE || act > MOE_MAT_GELU ||
        (!offsets && E != 1) || (!row_token && R > a_rows) || (row_token && R > 0 && a_rows < 1))
        return MOE_ERR_INVALID;
    if (E > MOE_MAX_EXPERTS || !fits(n_w, K) ||
        (row_token && (int64_t)a_rows * K * 2 >= ((int64_t)1 << 32)))
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

inline MatArgs mat_args(const void* rows, const void* cols, const int32_t* row_token, const int32_t* offsets,
                 int32_t a_rows, int32_t R, int32_t E)
{
    MatArgs p = {};
    p.rows = static_cast<const __bf16*>(rows);
    p.cols = static_cast<const __bf16*>(cols);
    p.row_token = row_token;
    p.offsets = offsets;
    p.a_rows = a_rows;
    p.R = R;
    p.E = E;
    p.splits = 1;
    return p;
}

}  // namespace

#endif  // MOE_MAT_TILE_H
