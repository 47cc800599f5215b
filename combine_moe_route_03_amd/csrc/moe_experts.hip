// moe_experts.hip -- 8-bit rows with a scale for each token, and the experts' product in 8-bit
// integers (declared in include/moe_layer.h).
//   k_quant_rows   q = rint(127 x / max |x|), scale = max |x| / 127: one pass, bound by HBM.
//   k_matmul_tile  y_rn = (sum_i a_ri w_eni) a_scale_r w_scale_en, and SwiGLU of two channels: tiles
//                  of 32 to 256 rows of one expert. With few rows an expert the weights' bytes bound
//                  it (128 tokens over 256 experts: 7.4 GB in 1.19 ms, 6.2 TB/s), with many the
//                  matrix cores and the LDS that feeds them (8192^3: 456 to 500 us on different
//                  boxes, 2.2 to 2.4 POPS).
//   k_matmul_few   the same where there are too few tiles to fill the GPU: the wavefronts of a
//                  workgroup share K (one row by 29 MB of weights: 7.7 us).
#include <atomic>

#include "moe_layer.h"
#include "moe_tiles.h"

namespace {

using namespace moe_dev;

// ------------------------------------------------------------------------------ 8-bit rows --
// a = max |x|, q = rint(127 x / a), scale = a / 127. Each row is read once, held in registers
// between its maximum and its codes, and bound by HBM: 2 (bf16) or 4 (fp32) bytes in and one out
// for an element. G lanes take a row, with up to NV vectors of 8 elements a lane in flight at once.
// Rows beyond 512 lanes of 8 vectors are read a second time, from the cache.
constexpr int kQuantVec = 8;
constexpr int kXcds = 8;                 // workgroup b runs on XCD b % 8
constexpr int kCus = 256;

// Eight elements as they are in memory.
struct Bf16x8 {
    typedef uint16_t elem;
    static constexpr bool kWide = true;      // 127 x is formed, and a divides it
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u32x4 x;

    __device__ __forceinline__ void load(const elem* __restrict__ p)
    {
        x = *reinterpret_cast<const u32x4*>(p);
    }

    // The largest magnitude: magnitudes compare as their bits do, NaN and infinity come out on top.
    __device__ __forceinline__ uint32_t top() const
    {
        u16x2 m = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t b = x[i] & 0x7FFF7FFFu;
            m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, b));
        }
        return (uint32_t)(m[0] > m[1] ? m[0] : m[1]) << 16;
    }

    __device__ __forceinline__ float value(int i) const
    {
        return __uint_as_float(i & 1 ? x[i / 2] & 0xFFFF0000u : x[i / 2] << 16);
    }
};

struct F32x8 {
    typedef float elem;
    static constexpr bool kWide = false;     // 127 / a is formed, and multiplies x
    u32x4 x[2];

    __device__ __forceinline__ void load(const elem* __restrict__ p)
    {
        x[0] = reinterpret_cast<const u32x4*>(p)[0];
        x[1] = reinterpret_cast<const u32x4*>(p)[1];
    }

    __device__ __forceinline__ uint32_t top() const
    {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = max(m, x[i / 4][i % 4] & 0x7FFFFFFFu);
        return m;
    }

    __device__ __forceinline__ float value(int i) const
    {
        return __uint_as_float(x[i / 4][i % 4]);
    }
};

// A row's largest magnitude, and what its codes are made with: x and a are taken times `up`, a power
// of two (1 but for extreme a), which keeps 127 x and the reciprocals in range.
struct Scaling {
    float a, inv, up;
};

// The lowest byte of fl(q + 1.5 * 2^23), for four q and four more: there the whole number nearest
// to q stands in the lowest bits, halves to even.
__device__ __forceinline__ u32x2 low_bytes(const float t[8])
{
    u32x2 c;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        c[i] = __builtin_amdgcn_perm(__float_as_uint(t[4 * i + 1]), __float_as_uint(t[4 * i]),
                                     0x0C0C0400u) |
               __builtin_amdgcn_perm(__float_as_uint(t[4 * i + 3]), __float_as_uint(t[4 * i + 2]),
                                     0x04000C0Cu);
    return c;
}
constexpr float kWhole = 12582912.0f;

// bf16: with 15 and 8 bits, 127 x / a is a half exactly, or at least 2^-16 of itself away from one.
// One step of division (remainder, exact, times the reciprocal) brings the quotient to within an ulp
// and an exact half to itself, so every code is right. (Exact halves are common: x = a / 2 is one.
// Sent to a slower exact path they made it 45 us for 32768 rows of 2048.)
__device__ __forceinline__ u32x2 codes8(const Bf16x8& v, const Scaling& s, bool* border)
{
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = v.value(i) * (127.0f * s.up);
        const float q = x * s.inv;
        t[i] = __builtin_fmaf(__builtin_fmaf(-q, s.a, x), s.inv, q) + kWhole;
    }
    *border = false;
    return low_bytes(t);
}

// fp32: x inv, inv = fl(127 / a), is off by at most 127 * 2^-24 < 7.6e-6 from 127 x / a. Where one
// of the elements lies that near to a half, or the row is scaled, all 8 are left to exact_codes8().
__device__ __forceinline__ u32x2 codes8(const F32x8& v, const Scaling& s, bool* border)
{
    float t[8], far = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = v.value(i);
        t[i] = __builtin_fmaf(x, s.inv, kWhole);
        far = fmaxf(far, __builtin_fabsf(__builtin_fmaf(x, s.inv, kWhole - t[i])));
    }
    *border = far > 0.49999f || s.up != 1.0f;
    return low_bytes(t);
}

// Next to a half the whole number r below the quotient or the one above it: 127 x - r a decides,
// which fp64 holds exactly: 127 x has 31 bits, r a too, and there x >= a / 254, so both are
// multiples of ulp(a) 2^-8 below 2 a.
__device__ __forceinline__ u32x2 exact_codes8(const F32x8& v, const Scaling& s)
{
    u32x2 c = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = v.value(i) * s.up, q = x * s.inv;
        float r = rintf(q);
        if (__builtin_fabsf(q - r) > 0.4999f) {
            r = floorf(q);
            const double d = 2.0 * (127.0 * (double)x - (double)r * (double)s.a) - (double)s.a;
            if (d > 0.0 || (d == 0.0 && ((int32_t)r & 1)))
                r += 1.0f;
        }
        c[i / 4] |= ((uint32_t)(int32_t)r & 0xFFu) << (8 * (i % 4));
    }
    return c;
}

__device__ __forceinline__ u32x2 exact_codes8(const Bf16x8& v, const Scaling& s)
{
    bool border;
    return codes8(v, s, &border);
}

template <typename V, int G, int NV>
__global__ __launch_bounds__(G < 256 ? 256 : G) void k_quant_rows(
    const typename V::elem* __restrict__ x, int32_t R, int32_t H,
    const int32_t* __restrict__ n_rows, int8_t* __restrict__ q, float* __restrict__ scale)
{
    constexpr int kThreads = G < 256 ? 256 : G;
    constexpr int kRows = kThreads / G;                       // rows of a workgroup at a time
    constexpr int kWavesPerRow = G / 64;                      // 0: several rows in a wavefront
    __shared__ uint32_t s_max[2][kThreads / 64];
    const int tid = threadIdx.x, g = tid % G;
    const int32_t rows = n_rows ? min(max(n_rows[0], 0), R) : R;
    const int nvec = H / kQuantVec;
    int flip = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < rows; r0 += (int64_t)gridDim.x * kRows) {
        const int64_t row = r0 + tid / G;
        const bool live = row < rows;
        const typename V::elem* p = x + row * H;
        V v[NV];
        uint32_t m = 0u;
        if (live) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (g + i * G < nvec)
                    v[i].load(p + (int64_t)(g + i * G) * kQuantVec);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (g + i * G < nvec)
                    m = max(m, v[i].top());
            for (int i = g + NV * G; i < nvec; i += G) {
                V t;
                t.load(p + (int64_t)i * kQuantVec);
                m = max(m, t.top());
            }
        }
        // bits of magnitudes up to that of NaN order as floats do not: reduced as integers
#pragma unroll
        for (int d = 1; d < (G < 64 ? G : 64); d <<= 1)
            m = max(m, (uint32_t)__shfl_xor((int)m, d));
        if (kWavesPerRow > 1) {
            if ((tid & 63) == 0)
                s_max[flip][tid >> 6] = m;
            __syncthreads();
            const int w0 = tid / G * kWavesPerRow;
#pragma unroll
            for (int w = 0; w < kWavesPerRow; ++w)
                m = max(m, s_max[flip][w0 + w]);
            flip ^= 1;
        }
        if (!live)
            continue;
        Scaling sc = {__uint_as_float(m), 0.0f, 1.0f};
        float s = 1.0f;
        if (m >= 0x7F800000u) {
            s = __uint_as_float(0x7FC00000u);
        } else if (m) {
            s = sc.a / 127.0f;
            if (sc.a < 5.42101086e-20f)                       // 2^-64
                sc.up = 18446744073709551616.0f;              // 2^64
            else if (V::kWide && sc.a > 1.26765060e+30f)      // 2^100
                sc.up = 5.42101086e-20f;
            sc.a *= sc.up;
            sc.inv = (V::kWide ? 1.0f : 127.0f) / sc.a;
        }
        if (g == 0)
            scale[row] = s;
        const bool zero = sc.inv == 0.0f;
        int8_t* out = q + row * H;
        uint32_t again = 0u;                                  // a bit for each vector
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (g + i * G < nvec) {
                bool border;
                const u32x2 c = codes8(v[i], sc, &border);
                again |= (uint32_t)(border && !zero) << i;
                *reinterpret_cast<u32x2*>(out + (int64_t)(g + i * G) * kQuantVec) =
                    zero ? u32x2{0u, 0u} : c;
            }
        // the few vectors with an element next to a half, from memory, so that this stays small
        while (again) {
            const int at = g + (__ffs((int)again) - 1) * G;
            again &= again - 1u;
            V t;
            t.load(p + (int64_t)at * kQuantVec);
            *reinterpret_cast<u32x2*>(out + (int64_t)at * kQuantVec) = exact_codes8(t, sc);
        }
        for (int i = g + NV * G; i < nvec; i += G) {
            V t;
            t.load(p + (int64_t)i * kQuantVec);
            *reinterpret_cast<u32x2*>(out + (int64_t)i * kQuantVec) =
                zero ? u32x2{0u, 0u} : exact_codes8(t, sc);
        }
    }
}

template <typename V, int G, int NV>
void launch_quant_g(const void* x, int32_t R, int32_t H, const int32_t* n_rows, int8_t* q,
                    float* scale, hipStream_t stream)
{
    constexpr int kThreads = G < 256 ? 256 : G;
    const int64_t blocks = div_up(R, kThreads / G);
    const int64_t most = 1 << 20;
    k_quant_rows<V, G, NV><<<(unsigned)(blocks < most ? blocks : most), kThreads, 0, stream>>>(
        static_cast<const typename V::elem*>(x), R, H, n_rows, q, scale);
}

// Lanes of a row: few enough that each has two to four vectors in flight, so many that a row's
// registers leave room for other rows. 32768 rows in bf16: 1408 elements 30 us with 64 lanes, 33
// with 128, 37 with 256; 2048: 40, 39, 44; 4096: 81, 73, 73 (5.5 TB/s), 91 with 512; 4096 rows of
// 7168: 20, 20, 18, 18. In fp32, as chosen here, 32768 rows of 4096 take 125 us (5.4 TB/s).
template <typename V>
void launch_quant(const void* x, int32_t R, int32_t H, const int32_t* n_rows, int8_t* q,
                  float* scale, hipStream_t stream)
{
    if (H <= 512)
        launch_quant_g<V, 16, 4>(x, R, H, n_rows, q, scale, stream);
    else if (H <= 1536)
        launch_quant_g<V, 64, 4>(x, R, H, n_rows, q, scale, stream);
    else if (H <= 2048)
        launch_quant_g<V, 128, 2>(x, R, H, n_rows, q, scale, stream);
    else if (H <= 4096)
        launch_quant_g<V, 128, 4>(x, R, H, n_rows, q, scale, stream);
    else if (H <= 8192)
        launch_quant_g<V, 512, 2>(x, R, H, n_rows, q, scale, stream);
    else
        launch_quant_g<V, 512, 8>(x, R, H, n_rows, q, scale, stream);
}

// ------------------------------------------------------------------------ experts' product --
struct MatmulArgs {
    const int8_t* a;
    const float* a_scale;
    const int32_t* row_token;
    const int8_t* w;
    const float* w_scale;
    const int32_t* offsets;
    void* out;
    int32_t a_rows, R, E, N, K;
    int32_t n_blocks;          // workgroups side by side over the channels
    int32_t max_tiles;         // row tiles, at most
    double inv_blocks;         // 1 / n_blocks
};

// Few rows an expert: bound by reading the weights, each once. A workgroup takes up to 16 MF rows
// of one expert and 16 NF channels; its wavefronts share the K axis out by 128-byte pieces, read
// weights and rows straight into MFMA operands, and add their int32 sums up through LDS (integers:
// any order gives the same). v_mfma_i32_16x16x64_i8 with the weights as the left operand: lane l
// gives channel l % 16 and 16 bytes of K at 16 (l / 16), and gets row l % 16 with channels
// 4 (l / 16) + i, so that its four results lie side by side in memory.
template <int MF, int NF, int WAVES, int U, bool SWIGLU, typename OUT>
__global__ __launch_bounds__(64 * WAVES) void k_matmul_few(MatmulArgs p)
{
    constexpr int kFrags = MF * NF;
    __shared__ i32x4 s_acc[WAVES][kFrags][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t nb = blockIdx.x % p.n_blocks;
    const Tile tile = find_tile<16 * MF>(p, blockIdx.x / p.n_blocks);
    if (tile.rows == 0)
        return;
    const int r16 = lane & 15, kq = lane >> 4;
    const int32_t n_w = SWIGLU ? 2 * p.N : p.N;               // channels of w
    const int8_t* we = p.w + (int64_t)tile.e * n_w * p.K;

    // channels: fragment f covers 16 from n0 + 16 f; with SwiGLU even fragments hold the gate and
    // the odd ones the same channels' up
    const int32_t n0 = nb * (SWIGLU ? 8 * NF : 16 * NF);
    const int8_t* wp[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
        int32_t n = SWIGLU ? n0 + 16 * (f / 2) + r16 : n0 + 16 * f + r16;
        n = min(n, p.N - 1) + (SWIGLU && (f & 1) ? p.N : 0);
        wp[f] = we + (int64_t)n * p.K;
    }
    const int8_t* ap[MF];
#pragma unroll
    for (int m = 0; m < MF; ++m) {
        const int32_t r = tile.row0 + min(16 * m + r16, tile.rows - 1);
        int32_t src = p.row_token ? p.row_token[r] : r;
        src = (uint32_t)src < (uint32_t)p.a_rows ? src : 0;   // its results are not stored
        ap[m] = p.a + (int64_t)src * p.K;
    }
    // the fragment (with SwiGLU the pair) that this wavefront will join and store: its scales are
    // read ahead
    constexpr int kStep = SWIGLU ? 2 : 1;
    static_assert(kFrags <= WAVES * kStep, "one for a wavefront");
    const int mine = wave * kStep;
    const int32_t at_row = 16 * (mine / NF) + r16;
    const int32_t row = tile.row0 + min(at_row, tile.rows - 1);
    const int32_t src = p.row_token ? p.row_token[row] : row;
    const int32_t n = n0 + (SWIGLU ? 8 : 16) * (mine % NF) + 4 * kq;
    const int32_t left = p.N - n;
    const bool stores = mine < kFrags && at_row < tile.rows &&
                        (uint32_t)src < (uint32_t)p.a_rows && left > 0;
    float sa = 0.0f, sw[4], su[4];
    if (stores) {
        const float* s = p.w_scale + (int64_t)tile.e * n_w + n;
        sa = p.a_scale[src];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            sw[c] = s[c < left ? c : 0];
            su[c] = SWIGLU ? s[p.N + (c < left ? c : 0)] : 0.0f;
        }
    }
    i32x4 acc[MF][NF];
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int f = 0; f < NF; ++f)
            acc[m][f] = i32x4{0, 0, 0, 0};

    for (int32_t k0 = wave * 128; k0 < p.K; k0 += U * WAVES * 128) {
        i32x4 wv[2 * U][NF], av[2 * U][MF];
#pragma unroll
        for (int h = 0; h < 2 * U; ++h) {
            const int32_t at = k0 + h / 2 * WAVES * 128 + 64 * (h % 2) + 16 * kq;
            const bool in = at < p.K;                         // K is a multiple of 16
            const int32_t from = in ? at : 0;
#pragma unroll
            for (int f = 0; f < NF; ++f)
                wv[h][f] = *reinterpret_cast<const i32x4*>(wp[f] + from);
#pragma unroll
            for (int m = 0; m < MF; ++m) {
                av[h][m] = *reinterpret_cast<const i32x4*>(ap[m] + from);
                av[h][m] = in ? av[h][m] : i32x4{0, 0, 0, 0};
            }
        }
#pragma unroll
        for (int h = 0; h < 2 * U; ++h)
#pragma unroll
            for (int m = 0; m < MF; ++m)
#pragma unroll
                for (int f = 0; f < NF; ++f)
                    acc[m][f] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[h][f], av[h][m],
                                                                      acc[m][f], 0, 0, 0);
    }
    // the wavefronts' sums of each fragment (with SwiGLU of each pair) are joined by one of them
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int f = 0; f < NF; ++f)
            s_acc[wave][m * NF + f][lane] = acc[m][f];
    __syncthreads();
    if (!stores)
        return;
    i32x4 sum[2];
#pragma unroll
    for (int g = 0; g < kStep; ++g) {
        sum[g] = s_acc[0][mine + g][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w)
            sum[g] += s_acc[w][mine + g][lane];
    }
    OUT* out = static_cast<OUT*>(p.out) + (int64_t)row * p.N + n;
    typedef typename Four<OUT>::type four;
    f32x4 y, up;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        y[c] = (float)sum[0][c] * sa * sw[c];
        up[c] = (float)sum[kStep - 1][c] * sa * su[c];
    }
    if (SWIGLU)
        y = swiglu(y, up);
    four v;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        v[c] = (OUT)y[c];
    if (left >= 4 && (uintptr_t)out % sizeof(four) == 0) {
        *reinterpret_cast<four*>(out) = v;
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (c < left)
                out[c] = v[c];
    }
}

// ---- tiles ----
// Persistent workgroups take tiles of BM rows by BN channels. K goes through LDS stages of 128 bytes
// a row, filled by loads that go straight to LDS. A wavefront's load brings 8 lines of 128 bytes:
// lane l the 16-byte piece (l % 8) ^ (l / 8) of line l / 8, so that piece c of line r lies in slot
// c ^ (r % 8) and the operand reads (the same piece of consecutive lines) fall on different banks.
// Operands of a quarter step are read while the quarter before is multiplied, and the loads go on
// into the next tile: its first stages are asked for before a tile's results are written.
//   A step of a 256 x 256 tile is 2048 cycles of MFMA (v_mfma_i32_32x32x32_i8, 8 wavefronts of 128 x
// 64), and 2048 of LDS at 128 bytes a cycle: 64 KiB in, 192 KiB out. Of 8192^3, 496 us, 410 are left
// without the LDS reads, 316 without the products, 303 with the loads alone. Steps of 64 bytes (half
// lines a load, twice the barriers) take 562 us against 509, four wavefronts of 128 x 128 (less LDS,
// one wavefront a SIMD) 510 against 488, loads spread among the products 484 against 477.
//   A tile's beginning waits: its rows' tokens and its channels' scales come by ordinary loads, and
// the compiler waits for the first of them before the first product, in every instance. vmcnt counts
// in order, so the last tile's stores and the stages read ahead are waited for with it; aim(), which
// reads offsets and row tokens, waits as well. Where a tile has few steps this shows (16 steps, 384
// experts: 1.12 ms for 0.95 of bytes). The 256 x 256 instances also keep 6 to 11 registers in scratch,
// which they read at a tile's beginning and end, not among the products.
constexpr int kStepK = 128;

template <int BM, int BN, int WM, int WN, int STAGES, bool PIN, bool SWIGLU, typename OUT>
__global__ __launch_bounds__(64 * WM * WN) void k_matmul_tile(MatmulArgs p)
{
    constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
    constexpr int MF = BM / WM / 32, NF = BN / WN / 32;       // 32 x 32 fragments of a wavefront
    constexpr int kLoadsA = BM / 8 / kWaves, kLoadsW = BN / 8 / kWaves;
    constexpr int kLoads = kLoadsA + kLoadsW;
    constexpr int kStage = (BM + BN) * kStepK;
    constexpr int kGroup = 4;
    static_assert(MF * WM * 32 == BM && NF * WN * 32 == BN, "tile");
    static_assert(kLoadsA * 8 * kWaves == BM && kLoadsW * 8 * kWaves == BN, "loads");
    static_assert(NF % 2 == 0 && STAGES >= 2, "pairs of fragments");
    // results of a wavefront: fragments side by side, and the units they are stored in
    constexpr int kUnit = 1024;
    constexpr int kOutF = SWIGLU ? NF / 2 : NF, kUnitF = kOutF < 2 ? 1 : 2;
    constexpr int kUnitRow = kUnitF * 32 * (int)sizeof(OUT);
    constexpr int kUnitRows = kUnit / kUnitRow < 32 ? kUnit / kUnitRow : 32;
    constexpr int kUnitStores = kUnitRows * kUnitRow / 1024;
    constexpr int kStores = MF * (32 / kUnitRows) * (kOutF / kUnitF) * kUnitStores;
    static_assert(kOutF % kUnitF == 0 && kUnitStores >= 1 && BM <= kThreads, "results");
    static_assert((STAGES - 2) * kLoads + kStores <= 63, "vmcnt has six bits");
    extern __shared__ __attribute__((aligned(1024))) int8_t s_stage[];
    __shared__ __attribute__((aligned(16))) int8_t s_unit[kWaves][kUnit];
    __shared__ __attribute__((aligned(16))) float s_ws[BN];
    __shared__ float s_as[BM];
    __shared__ uint32_t s_ok[BM / 32];                        // a bit for each row to be written
    constexpr int kRing = 8;
    static_assert(STAGES + 2 <= kRing, "tiles between the loads and the products");
    __shared__ Tile s_tile[kRing];
    int32_t* s_prefix = reinterpret_cast<int32_t*>(s_stage + STAGES * kStage);   // [E + 1]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int32_t all = tile_prefix<kThreads, BM>(p, s_prefix) * p.n_blocks;
    // workgroup b runs on XCD b % 8: each XCD takes a run of consecutive tiles
    const int32_t share = (all + kXcds - 1) / kXcds;
    const int32_t stride = gridDim.x / kXcds;
    const int32_t first = (blockIdx.x % kXcds) * share + blockIdx.x / kXcds;
    const int32_t last = min((int32_t)(blockIdx.x % kXcds + 1) * share, all);
    if (first >= last)
        return;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int8_t*)s_stage;
    const int32_t n_w = SWIGLU ? 2 * p.N : p.N;
    const int32_t steps = (p.K + kStepK - 1) / kStepK;
    const bool ragged = p.K % kStepK != 0;

    // The loads run ahead of the products through the same tiles: their own place in them
    const int line = lane >> 3, piece = 16 * ((lane & 7) ^ line);
    const bool behind = (p.K & ~(kStepK - 1)) + piece >= p.K; // in a ragged last step
    u32x4 abuf, wbuf;
    uint32_t avo[kLoadsA], wvo[kLoadsW];
    int32_t arow[kLoadsA];                                    // read at aim(), used a step later
    int32_t load_tile = first, load_step = 0, load_nth = 0;
    uint32_t load_to = lds0 + wave * 1024;
    int32_t ahead = 0;                                        // stages loaded and not yet begun
    int32_t older = 0;                                        // of these, before the last stores
    const auto aim = [&]() {
        const Tile t = tile_at<BM, kGroup>(p, s_prefix, load_tile);
        if (tid == 0)
            s_tile[load_nth % kRing] = t;
        ++load_nth;
        abuf = p.row_token ? buffer_of(p.a, (uint32_t)((int64_t)p.a_rows * p.K))
                           : buffer_of(p.a + (int64_t)t.row0 * p.K, (uint32_t)(t.rows * p.K));
        wbuf = buffer_of(p.w + (int64_t)t.e * n_w * p.K, (uint32_t)((int64_t)n_w * p.K));
#pragma unroll
        for (int i = 0; i < kLoadsA; ++i) {
            const int32_t m = min(8 * (i * kWaves + wave) + line, t.rows - 1);
            arow[i] = p.row_token ? p.row_token[t.row0 + m] : m;
        }
        const int32_t n0 = t.n * (SWIGLU ? BN / 2 : BN);
#pragma unroll
        for (int i = 0; i < kLoadsW; ++i) {
            const int32_t c = 8 * (i * kWaves + wave) + line;
            // with SwiGLU every other 32 channels are the up channels of the 32 before
            int32_t n = SWIGLU ? n0 + c / 64 * 32 + c % 32 : n0 + c;
            n = min(n, p.N - 1) + (SWIGLU && (c & 32) ? p.N : 0);
            wvo[i] = (uint32_t)n * (uint32_t)p.K + piece;
        }
    };
    const auto issue = [&]() {
        if (load_tile >= last)
            return;
        const uint32_t at = (uint32_t)load_step * kStepK;
        if (load_step == 0) {
#pragma unroll
            for (int i = 0; i < kLoadsA; ++i) {
                int32_t r = arow[i];
                if (p.row_token)
                    r = (uint32_t)r < (uint32_t)p.a_rows ? r : 0;     // its results are not stored
                avo[i] = (uint32_t)r * (uint32_t)p.K + piece;
            }
        }
        // pieces behind the end of K repeat the step's first one, and are zeroed in LDS later
        const uint32_t back = ragged && load_step == steps - 1 && behind ? piece : 0u;
#pragma unroll
        for (int i = 0; i < kLoadsA; ++i)
            load_lds(abuf, avo[i] - back, at, load_to + i * kWaves * 1024);
#pragma unroll
        for (int i = 0; i < kLoadsW; ++i)
            load_lds(wbuf, wvo[i] - back, at, load_to + BM * kStepK + i * kWaves * 1024);
        load_to += kStage;
        if (load_to >= lds0 + STAGES * kStage)
            load_to -= STAGES * kStage;
        ++ahead;
        if (++load_step == steps) {
            load_step = 0;
            load_tile += stride;
            if (load_tile < last)
                aim();
        }
    };

    const int wm = MF > 1 ? wave / WN : wave % WM, wn = MF > 1 ? wave % WN : wave / WM;
    const int r32 = lane & 31, half = lane >> 5;
    typedef int32_t i32x16 __attribute__((ext_vector_type(16)));
    i32x16 acc[MF][NF];
    // this lane's slots of the four 32-byte quarters of a step
    int slot[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
        slot[q] = r32 * kStepK + 16 * ((2 * q + half) ^ (r32 & 7));
    int at = 0;                                               // the stage that is multiplied
    i32x4 wv[2][NF], av[2][MF];
    const auto read = [&](int set, int q) {                   // quarter q of the stage
        const int8_t* sw = s_stage + at + (BM + wn * NF * 32) * kStepK + slot[q];
        const int8_t* sa = s_stage + at + wm * MF * 32 * kStepK + slot[q];
#pragma unroll
        for (int f = 0; f < NF; ++f)
            wv[set][f] = *reinterpret_cast<const i32x4*>(sw + f * 32 * kStepK);
#pragma unroll
        for (int m = 0; m < MF; ++m)
            av[set][m] = *reinterpret_cast<const i32x4*>(sa + m * 32 * kStepK);
    };
    // Multiplies operand set `cur` while quarter q goes into the other set. Fragments of rows that
    // the tile does not have are left out (the wavefronts of its upper rows are spread over the four
    // SIMDs, so that gains time: 512 rows an expert, 404 -> 380 us). PIN: the reads stay spread out
    // among the products, where the compiler would group them (8192^3: 511 -> 471 us; with few
    // products a step it loses).
    int32_t frags = MF;
    const auto multiply = [&](int cur, int q) {
        const int8_t* sw = s_stage + at + (BM + wn * NF * 32) * kStepK + slot[q < 0 ? 0 : q];
        const int8_t* sa = s_stage + at + wm * MF * 32 * kStepK + slot[q < 0 ? 0 : q];
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            if (MF > 1 && m >= frags)
                continue;
#pragma unroll
            for (int i = 0; i < NF; ++i) {
                const int f = m & 1 ? NF - 1 - i : i;
                acc[m][f] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wv[cur][f], av[cur][m],
                                                                  acc[m][f], 0, 0, 0);
                if (PIN)
                    __builtin_amdgcn_sched_barrier(0);
                if (q >= 0 && i == 0)
                    av[1 - cur][m] = *reinterpret_cast<const i32x4*>(sa + m * 32 * kStepK);
                if (q >= 0 && m == 0)
                    wv[1 - cur][i] = *reinterpret_cast<const i32x4*>(sw + i * 32 * kStepK);
                if (PIN)
                    __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    // this wavefront's loads of the next stage have landed; `partial`: it is a ragged last step
    const auto landed = [&](int32_t next, bool partial) {
        if (ahead < STAGES - 1)
            wait_loads<0>();
        else if (older > 0)                                   // without the stores behind it
            wait_loads<(STAGES - 2) * kLoads + kStores>();
        else
            wait_loads<(STAGES - 2) * kLoads>();
        --older;
        if (partial && behind) {
#pragma unroll
            for (int i = 0; i < kLoadsA; ++i)
                *reinterpret_cast<i32x4*>(s_stage + next + (i * kWaves + wave) * 1024 + 16 * lane) =
                    i32x4{0, 0, 0, 0};
        }
    };
    const auto after = [&](int stage) { return stage + kStage == STAGES * kStage ? 0 : stage + kStage; };

    aim();
#pragma unroll
    for (int s = 0; s < STAGES; ++s)
        issue();
    if (ahead == STAGES)                                      // the first stage only
        wait_loads<(STAGES - 1) * kLoads>();
    else
        wait_loads<0>();
    ahead -= 1;
    if (ragged && steps == 1 && behind) {
#pragma unroll
        for (int i = 0; i < kLoadsA; ++i)
            *reinterpret_cast<i32x4*>(s_stage + (i * kWaves + wave) * 1024 + 16 * lane) =
                i32x4{0, 0, 0, 0};
    }
    wait_workgroup();
    for (int32_t tile = first, nth = 0; tile < last; tile += stride, ++nth) {
        if (steps == 1)                                       // no wait in the loop keeps the
            wait_workgroup();                                 // tiles' scales apart
        Tile t;
        t.e = __builtin_amdgcn_readfirstlane(s_tile[nth % kRing].e);
        t.row0 = __builtin_amdgcn_readfirstlane(s_tile[nth % kRing].row0);
        t.rows = __builtin_amdgcn_readfirstlane(s_tile[nth % kRing].rows);
        t.n = __builtin_amdgcn_readfirstlane(s_tile[nth % kRing].n);
        // scales: a thread's row of the tile, and its channels, put into LDS at the tile's end
        const int32_t n0 = t.n * (SWIGLU ? BN / 2 : BN);
        const bool mine = tid < t.rows;
        const int32_t row = t.row0 + (mine ? tid : 0);
        const int32_t src = p.row_token ? p.row_token[row] : row;
        float ws[(BN + kThreads - 1) / kThreads];
#pragma unroll
        for (int i = 0; i < (BN + kThreads - 1) / kThreads; ++i) {
            const int32_t c = min(i * kThreads + tid, BN - 1);
            const int32_t n = min(SWIGLU ? n0 + c / 64 * 32 + c % 32 : n0 + c, p.N - 1);
            ws[i] = p.w_scale[(int64_t)t.e * n_w + n + (SWIGLU && (c & 32) ? p.N : 0)];
        }
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
            for (int f = 0; f < NF; ++f)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    acc[m][f][i] = 0;
        read(0, 0);
        frags = __builtin_amdgcn_readfirstlane(
            min(MF, (t.rows - wm * MF * 32 + 31) / 32));
        bool ok = false;
        float as = 0.0f;
        const auto scale = [&]() {
            ok = mine && (uint32_t)src < (uint32_t)p.a_rows;
            as = p.a_scale[ok ? src : 0];
        };
        if (steps < 3)
            scale();
        for (int32_t step = 0; step < steps - 1; ++step) {
            multiply(0, 1);
            multiply(1, 2);
            multiply(0, 3);
            const int next = after(at);
            landed(next, ragged && step == steps - 2);
            wait_workgroup();                                 // and this stage is read
            --ahead;
            if (step == 1)                                    // (the row came at the beginning)
                scale();
            issue();
            at = next;
            multiply(1, 0);
        }
        multiply(0, 1);
        multiply(1, 2);
        multiply(0, 3);
        multiply(1, -1);
        const int next = after(at);
        if (ahead > 0)
            landed(next, ragged && steps == 1);
        if (tid < BM)
            s_as[tid] = as;
        const uint64_t oks = __ballot(ok);
        if (lane < 2 && wave * 2 + lane < BM / 32)
            s_ok[wave * 2 + lane] = (uint32_t)(oks >> (32 * lane));
#pragma unroll
        for (int i = 0; i < (BN + kThreads - 1) / kThreads; ++i)
            if (i * kThreads + tid < BN)
                s_ws[i * kThreads + tid] = ws[i];
        wait_workgroup();
        older = 0;
        if (ahead > 0) {
            --ahead;
            issue();
            older = ahead;
        }
        at = next;

        // Results, while the next tile's first stages are on their way: the lane's fp32 values are
        // rounded, go through a little LDS of the wavefront's own, and come back as rows of 128
        // bytes (bf16) for 16-byte stores; 16-byte piece c of row r lies in slot c ^ (r % 8).
        // Stores of whole rows count the same for every wavefront, so that landed() can wait for the
        // loads before them without them; the next tile's ordinary loads still wait for them, see
        // above. (Stored from the accumulators two bytes at a time, the
        // results of 8192^3 took 150 of 621 us; with the stores waited for at once, 50 of 470.)
        constexpr int kPieces = kUnitRow / 16;
        const bool wide = p.N % (16 / (int)sizeof(OUT)) == 0 && (uintptr_t)p.out % 16 == 0 &&
                          p.N <= (1 << 20);
        OUT* base = static_cast<OUT*>(p.out) + (int64_t)t.row0 * p.N;
        const __amdgpu_buffer_rsrc_t obuf = __builtin_amdgcn_make_buffer_rsrc(
            base, 0, (int32_t)((uint32_t)t.rows * (uint32_t)p.N * (uint32_t)sizeof(OUT)), 0x00020000);
        int8_t* unit = s_unit[wave];
        if (!wide)
            older = 0;
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            const float sa = s_as[(wm * MF + m) * 32 + r32];
            const uint32_t rows = s_ok[wm * MF + m];
#pragma unroll
            for (int u = 0; u < kOutF; u += kUnitF) {
                typename Four<OUT>::type v[kUnitF][4];        // channels 8 i + 4 half
#pragma unroll
                for (int g = 0; g < kUnitF; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int f = SWIGLU ? 2 * (u + g) : u + g;
                        const float* sw = s_ws + (wn * NF + f) * 32 + 8 * i + 4 * half;
                        const f32x4 s0 = *reinterpret_cast<const f32x4*>(sw);
                        const f32x4 s1 = *reinterpret_cast<const f32x4*>(SWIGLU ? sw + 32 : sw);
                        f32x4 y, up;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            y[c] = (float)acc[m][f][4 * i + c] * sa * s0[c];
                            up[c] = (float)acc[m][f + SWIGLU][4 * i + c] * sa * s1[c];
                        }
                        if (SWIGLU)
                            y = swiglu(y, up);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            v[g][i][c] = (OUT)y[c];
                    }
#pragma unroll 1
                for (int phase = 0; phase < 32 / kUnitRows; ++phase) {
                    asm volatile("" ::: "memory");            // LDS serves a wavefront in order
                    if (r32 / kUnitRows == phase) {
                        const int r = r32 % kUnitRows;
#pragma unroll
                        for (int g = 0; g < kUnitF; ++g)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int byte = (32 * g + 8 * i + 4 * half) * (int)sizeof(OUT);
                                *reinterpret_cast<typename Four<OUT>::type*>(
                                    unit + r * kUnitRow +
                                    ((byte / 16 ^ (r & (kPieces - 1) & 7)) * 16) + byte % 16) =
                                    v[g][i];
                            }
                    }
                    asm volatile("" ::: "memory");
                    const auto at16 = [&](int r, int c) {     // piece c of row r
                        return unit + r * kUnitRow + (c ^ (r & (kPieces - 1) & 7)) * 16;
                    };
                    const int32_t n1 = n0 + (wn * kOutF + u) * 32;
                    const int32_t tr0 = (wm * MF + m) * 32 + phase * kUnitRows;
                    const uint32_t ok_rows = rows >> phase * kUnitRows;
                    if (wide) {
#pragma unroll
                        for (int s = 0; s < kUnitStores; ++s) {
                            const int r = s * (kUnitRows / kUnitStores) + lane / kPieces;
                            const int c = lane % kPieces;
                            const u32x4 out = *reinterpret_cast<const u32x4*>(at16(r, c));
                            const int32_t n = n1 + c * (16 / (int)sizeof(OUT));
                            const uint32_t to = (uint32_t)((tr0 + r) * p.N + n) *
                                                (uint32_t)sizeof(OUT);
                            store_buffer(out, obuf,
                                         (ok_rows >> r & 1) && n < p.N ? to : 0xFFFFFFF0u);
                        }
                    } else {                                  // a value a lane, side by side
                        constexpr int kCols = kUnitF * 32;
                        constexpr int kUnroll = sizeof(OUT) == 2 ? 4 : 1;   // (registers)
#pragma unroll kUnroll
                        for (int s = 0; s < kUnitRows * kCols / 64; ++s) {
                            const int r = s * (64 / kCols) + lane / kCols, c = lane % kCols;
                            const int byte = c * (int)sizeof(OUT);
                            const OUT out = *reinterpret_cast<const OUT*>(at16(r, byte / 16) +
                                                                          byte % 16);
                            if ((ok_rows >> r & 1) && n1 + c < p.N)
                                base[(int64_t)(tr0 + r) * p.N + n1 + c] = out;
                        }
                    }
                }
            }
        }
    }
}

template <int MF, int NF, int WAVES, int U, bool SWIGLU, typename OUT>
moe_status_t launch_few(MatmulArgs p, hipStream_t stream)
{
    p.n_blocks = (int32_t)div_up(p.N, SWIGLU ? 8 * NF : 16 * NF);
    const int64_t blocks = most_tiles(p, 16 * MF) * p.n_blocks;
    if (blocks * 64 * WAVES > INT32_MAX)
        return MOE_ERR_UNSUPPORTED;
    k_matmul_few<MF, NF, WAVES, U, SWIGLU, OUT><<<(unsigned)blocks, 64 * WAVES, 0, stream>>>(p);
    return launched();
}

// WGS: persistent workgroups of a CU; kOnce: a workgroup for each tile, taken up as CUs come free.
constexpr int kOnce = 1 << 20;

template <int BM, int BN, int WM, int WN, int STAGES, bool PIN, int WGS, bool SWIGLU, typename OUT>
moe_status_t launch_tile(MatmulArgs p, hipStream_t stream)
{
    constexpr int kThreads = 64 * WM * WN, kStages = STAGES * (BM + BN) * kStepK;
    p.n_blocks = (int32_t)div_up(p.N, SWIGLU ? BN / 2 : BN);
    p.inv_blocks = 1.0 / p.n_blocks;
    const int64_t tiles = most_tiles(p, BM) * p.n_blocks;
    if (tiles > INT32_MAX / 2)
        return MOE_ERR_UNSUPPORTED;
    int64_t most = (int64_t)kCus * WGS;                       // and below 2^31 threads
    if (most > INT32_MAX / kThreads / kXcds * kXcds)
        most = INT32_MAX / kThreads / kXcds * kXcds;
    const int64_t blocks = tiles < most ? div_up(tiles, kXcds) * kXcds : most;
    p.max_tiles = (int32_t)most_tiles(p, BM);
    const auto kernel = k_matmul_tile<BM, BN, WM, WN, STAGES, PIN, SWIGLU, OUT>;
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
    kernel<<<(unsigned)blocks, kThreads, kStages + (p.E + 1) * 4, stream>>>(p);
    return launched();
}

// The tile shapes, and what a step of 128 bytes of K and a tile's beginning and end take (us, as
// measured with every slot taken; `alone` with one workgroup a CU): 16384 channels by 4096 rows in
// one expert, K = 2048 and 8192. Large tiles read less for each product (256 x 256: 2.2 POPS; 128 x
// 256: 2.0; 64 x 256: 1.4), small ones waste less on experts with few rows and fill the GPU sooner.
struct TileCost {
    int32_t bm, bn, slots;
    float step, alone, tile;
};
constexpr TileCost kTiles[] = {
    {256, 256, 256, 1.75f, 1.50f, 7.0f},
    {128, 256, 256, 1.08f, 0.95f, 4.3f},
    {128, 128, 512, 1.30f, 0.90f, 2.0f},
    {64, 256, 256, 0.72f, 0.72f, 2.5f},
    {32, 128, 512, 0.75f, 0.50f, 1.5f},
};

// The shape with the least time by these figures: rounds of tiles over the slots, where an expert's
// last tile is half full on average. The host knows the rows of all experts, not of each.
inline int choose_tile(const MatmulArgs& p, int64_t n_w)
{
    const double steps = (double)div_up(p.K, kStepK);
    const int64_t experts = p.E < p.R ? p.E : p.R;
    int best = 0;
    double least = 0.0;
    for (int i = 0; i < 5; ++i) {
        const TileCost& c = kTiles[i];
        int64_t tiles = p.offsets ? p.R / c.bm + experts / 2 : div_up(p.R, c.bm);
        if (tiles < experts)
            tiles = experts;
        tiles *= div_up(n_w, c.bn);
        const double step = tiles <= 256 ? c.alone : c.step;
        const double time = (double)div_up(tiles, c.slots) * (steps * step + c.tile);
        if (i == 0 || time < least) {
            best = i;
            least = time;
        }
    }
    return best;
}

// Few tiles leave most of the GPU idle and their K axis in one workgroup: there the wavefronts of a
// workgroup share K, and 16 or 32 channels make a workgroup (one row by 4096 channels, K = 7168:
// 7.7 us against 28; 64 rows: 17 against 28; 128 rows, 128 tiles of 32 x 128: 32 against 28).
constexpr int64_t kFewTiles = 128;

template <bool SWIGLU, typename OUT>
moe_status_t launch_matmul(const MatmulArgs& p, hipStream_t stream)
{
    const int64_t n_w = SWIGLU ? 2 * (int64_t)p.N : p.N;
    const int64_t experts = p.E < p.R ? p.E : p.R;
    const int64_t rows = div_up(p.R, experts);
    if (most_tiles(p, 32) * div_up(n_w, 128) < kFewTiles) {
        if (rows > 16)
            return launch_few<2, 2, 8, 4, SWIGLU, OUT>(p, stream);
        if (SWIGLU || most_tiles(p, 16) * div_up(n_w, 16) > 512)
            return launch_few<1, 2, 8, 4, SWIGLU, OUT>(p, stream);
        return launch_few<1, SWIGLU ? 2 : 1, 8, SWIGLU ? 4 : 2, SWIGLU, OUT>(p, stream);
    }
    switch (choose_tile(p, n_w)) {
    case 0: return launch_tile<256, 256, 2, 4, 2, true, 1, SWIGLU, OUT>(p, stream);
    case 1: return launch_tile<128, 256, 2, 4, 3, true, 1, SWIGLU, OUT>(p, stream);
    case 2: return launch_tile<128, 128, 2, 2, 2, true, 2, SWIGLU, OUT>(p, stream);
    case 3: return launch_tile<64, 256, 2, 4, 3, false, 1, SWIGLU, OUT>(p, stream);
    default: return launch_tile<32, 128, 1, 2, 3, false, kOnce, SWIGLU, OUT>(p, stream);
    }
}

}  // namespace

extern "C" {

moe_status_t moe_quant_rows(const void* x, moe_dtype_t x_dtype, int32_t R, int32_t H,
                            const int32_t* n_rows, int8_t* q, float* scale, hipStream_t stream)
{
    if (R < 0 || H < 1)
        return MOE_ERR_INVALID;
    if ((x_dtype != MOE_F32 && x_dtype != MOE_BF16) || H % 16 != 0)
        return MOE_ERR_UNSUPPORTED;
    if (R > 0 && (!x || !q || !scale))
        return MOE_ERR_INVALID;
    if (!aligned_to((const char*)x, 16) || !aligned_to(q, 16) || !aligned_to(scale, 4))
        return MOE_ERR_UNSUPPORTED;
    if (R == 0)
        return MOE_OK;
    if (x_dtype == MOE_BF16)
        launch_quant<Bf16x8>(x, R, H, n_rows, q, scale, stream);
    else
        launch_quant<F32x8>(x, R, H, n_rows, q, scale, stream);
    return launched();
}

moe_status_t moe_expert_matmul_i8(const int8_t* a, const float* a_scale, int32_t a_rows,
                                  const int32_t* row_token, const int8_t* w, const float* w_scale,
                                  const int32_t* expert_offsets, int32_t R, int32_t E, int32_t N,
                                  int32_t K, moe_act_t act, void* out, moe_dtype_t out_dtype,
                                  hipStream_t stream)
{
    if (R < 0 || a_rows < 0 || E < 1 || N < 1 || K < 1 ||
        (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU) || (!expert_offsets && E != 1) ||
        (!row_token && R > a_rows) || (row_token && R > 0 && a_rows < 1))
        return MOE_ERR_INVALID;
    const int64_t n_w = act == MOE_ACT_SWIGLU ? 2 * (int64_t)N : N;
    if ((out_dtype != MOE_F32 && out_dtype != MOE_BF16) || K % 16 != 0 || K > MOE_MATMUL_MAX_K ||
        E > MOE_MAX_EXPERTS || n_w * K >= ((int64_t)1 << 32) ||
        (row_token && (int64_t)a_rows * K >= ((int64_t)1 << 32)))
        return MOE_ERR_UNSUPPORTED;
    if (R > 0 && (!a || !a_scale || !w || !w_scale || !out))
        return MOE_ERR_INVALID;
    if (!aligned_to(a, 16) || !aligned_to(w, 16) ||
        !aligned_to((const char*)out, out_dtype == MOE_F32 ? 4 : 2))
        return MOE_ERR_UNSUPPORTED;
    if (R == 0)
        return MOE_OK;
    MatmulArgs p;
    p.a = a;
    p.a_scale = a_scale;
    p.row_token = row_token;
    p.w = w;
    p.w_scale = w_scale;
    p.offsets = expert_offsets;
    p.out = out;
    p.a_rows = a_rows;
    p.R = R;
    p.E = E;
    p.N = N;
    p.K = K;
    p.n_blocks = 0;
    p.max_tiles = 0;
    p.inv_blocks = 0.0;
    const bool bf16 = out_dtype == MOE_BF16;
    if (act == MOE_ACT_SWIGLU)
        return bf16 ? launch_matmul<true, __bf16>(p, stream) : launch_matmul<true, float>(p, stream);
    return bf16 ? launch_matmul<false, __bf16>(p, stream) : launch_matmul<false, float>(p, stream);
}

}  // extern "C"
