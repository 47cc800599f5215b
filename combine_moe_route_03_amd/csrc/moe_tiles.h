// moe_tiles.h -- what the products over the experts' rows share: tiles of rows and where they are,
// loads that go straight to LDS, stores of whole lines, and the SwiGLU of four channels.
//
// `Args` of a product holds at least
//   const int32_t* offsets;    [E + 1] first row of each expert, or null: all R rows are expert 0's
//   int32_t R, E;
//   int32_t n_blocks;          workgroups side by side over the channels
//   int32_t max_tiles;         row tiles, at most
//   double inv_blocks;         1 / n_blocks
#ifndef MOE_TILES_H
#define MOE_TILES_H

#include "moe_device.h"
#include "moe_route.h"

namespace moe_dev {

// Rows [row0, row0 + rows) of expert e, channel block n; rows = 0: nothing to do.
struct Tile {
    int32_t e, row0, rows, n;
};

// Rows of expert e and the first of them. Offsets are clamped into [0, R], so no value of theirs
// leads outside the rows.
template <typename Args>
__device__ __forceinline__ int32_t expert_rows(const Args& p, int32_t e, int32_t* lo)
{
    if (!p.offsets) {
        *lo = 0;
        return p.R;
    }
    *lo = min(max(p.offsets[e], 0), p.R);
    return min(max(p.offsets[e + 1], *lo), p.R) - *lo;
}

// Row tile `index` of all experts' tiles of BM rows, found by each wavefront for itself: a lane
// adds up the tiles of its share of the experts, a scan over the lanes finds the share that holds
// the index.
template <int BM, typename Args>
__device__ __forceinline__ Tile find_tile(const Args& p, int32_t index)
{
    const int lane = threadIdx.x & 63;
    int32_t mine = 0, lo = 0;
    if (p.E == 1) {
        const int32_t rows = expert_rows(p, 0, &lo);
        return Tile{0, lo + index * BM, max(0, min(BM, rows - index * BM)), 0};
    }
    const int per = (p.E + 63) / 64;
    const int e0 = min(lane * per, p.E), e1 = min(e0 + per, p.E);
    for (int e = e0; e < e1; ++e)
        mine += (expert_rows(p, e, &lo) + BM - 1) / BM;
    int32_t upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t o = __shfl_up(upto, d);
        if (lane >= d)
            upto += o;
    }
    const int32_t before = upto - mine;
    const uint64_t holds = __ballot(before <= index && index < upto);
    if (holds == 0)
        return Tile{0, 0, 0, 0};
    const int at = __ffsll((unsigned long long)holds) - 1;
    int32_t e = __builtin_amdgcn_readlane(e0, at);
    int32_t left = index - __builtin_amdgcn_readlane(before, at), n;
    for (;; ++e) {
        n = expert_rows(p, e, &lo);
        const int32_t tiles = (n + BM - 1) / BM;
        if (left < tiles)
            break;
        left -= tiles;
    }
    return Tile{e, __builtin_amdgcn_readfirstlane(lo + left * BM),
                __builtin_amdgcn_readfirstlane(min(BM, n - left * BM)), 0};
}

// v / (1 + exp(-t)), with exp(x) = 2^(x log2 e): the product's rounding, |t| 2^-24 of the result, is
// added back to first order; v_exp_f32 and v_rcp_f32 are good to one ulp. FAR: any t. Above
// x = 96, where 1 is nothing next to exp, both work on its root and the result is v / sqrt(exp) /
// sqrt(exp): exp itself overflows from x = 128 (t -88.7) and its reciprocal is flushed from 126, but
// silu, where v is t, is a normal number down to -92. Beyond |x| = 192 the root goes without its
// correction, which an infinite x would make infinite or NaN.
template <bool FAR>
__device__ __forceinline__ float logistic(float v, float t)
{
    constexpr float hi = -1.44269502f, lo = -1.92596299e-8f;
    const float x = t * hi;
    const float rest = (__builtin_fmaf(t, hi, -x) + t * lo) * 0.693147182f;
    if (!FAR) {
        const float e = __builtin_amdgcn_exp2f(x);
        return v * __builtin_amdgcn_rcpf(1.0f + __builtin_fmaf(e, rest, e));
    }
    const bool far = x > 96.0f;
    const float half = far ? 0.5f : 1.0f;
    const float e = __builtin_amdgcn_exp2f(x * half);
    const float s = __builtin_fabsf(x) > 192.0f ? e : __builtin_fmaf(e, rest * half, e);
    const float r = __builtin_amdgcn_rcpf((far ? 0.0f : 1.0f) + s);
    return v * r * (far ? r : 1.0f);
}

template <bool FAR>
__device__ __forceinline__ float silu(float gate)
{
    return logistic<FAR>(gate, gate);
}

// silu(gate) * up of four channels. Gates up to 64 have the same bits by both forms, so a row's
// results do not depend on what else is in its wavefront. (The form for any gate alone: 16384 rows
// over 4 experts, 4096 channels of K = 512, 140 us against 130; 2048 tokens over 64 experts of 2048
// by 4096 390 against 377.)
__device__ __forceinline__ f32x4 swiglu(f32x4 gate, f32x4 up)
{
    const float most = fmaxf(fmaxf(__builtin_fabsf(gate[0]), __builtin_fabsf(gate[1])),
                             fmaxf(__builtin_fabsf(gate[2]), __builtin_fabsf(gate[3])));
    f32x4 y;
    if (__builtin_expect(!__any(most > 64.0f), 1)) {          // a NaN may go either way
#pragma unroll
        for (int c = 0; c < 4; ++c)
            y[c] = silu<false>(gate[c]) * up[c];
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            y[c] = silu<true>(gate[c]) * up[c];
    }
    return y;
}

// Four results as they are kept in memory.
template <typename OUT>
struct Four {
    typedef f32x4 type;
};
template <>
struct Four<__bf16> {
    typedef bf16x4 type;
};

__device__ __forceinline__ u32x4 buffer_of(const void* base, uint32_t bytes)
{
    const uint64_t b = (uint64_t)(uintptr_t)base;
    u32x4 r;
    r[0] = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b);
    r[1] = (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(b >> 32) & 0xFFFFu));
    r[2] = (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes);
    r[3] = 0x00020000u;
    return r;
}

// 16 bytes a lane from `buffer` at voff + soff to LDS at lds + 16 * lane. In asm, since the
// compiler would wait for all such loads before every LDS read; it has no register output, and
// wait_loads() waits for it. The compiler puts the LDS address into m0 itself, so that it knows what
// is in there. It does not see that the asm is a memory instruction, so the wait states before one are
// here: one after the write of m0, five after a vector instruction that wrote a scalar operand (a
// descriptor made by readfirstlane, or taken back by readlane from where scalars are spilled to).
__device__ __forceinline__ void load_lds(u32x4 buffer, uint32_t voff, uint32_t soff, uint32_t lds)
{
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :: "{m0}"(lds), "v"(voff), "s"(buffer), "s"(soff) : "memory");
}

// All but the PENDING youngest of this wavefront's loads are in LDS.
template <int PENDING>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" :: "n"(PENDING) : "memory");
}

// This wavefront's LDS accesses are done, and so are those of the others of the workgroup.
__device__ __forceinline__ void wait_workgroup()
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// 16 bytes to `buffer` at voff, dropped where that is out of its range. Not for the caches: the
// next kernel reads the results from their start, and only the last ones would still be there.
__device__ __forceinline__ void store_buffer(u32x4 v, __amdgpu_buffer_rsrc_t buffer, uint32_t voff)
{
    __builtin_amdgcn_raw_buffer_store_b128(v, buffer, voff, 0, 2 /* nt */);
}

// Exclusive prefix of the experts' row tiles into prefix[0 .. E] (every thread calls), and their
// total; 0 if that is more than rising offsets can give.
template <int THREADS, int BM, typename Args>
__device__ __forceinline__ int32_t tile_prefix(const Args& p, int32_t* prefix)
{
    __shared__ int64_t s_wave[THREADS / 64];
    const int tid = threadIdx.x;
    const int per = (p.E + THREADS - 1) / THREADS;
    const int e0 = min(tid * per, p.E), e1 = min(e0 + per, p.E);
    const auto tiles = [&](int32_t e) {
        int32_t lo;
        const int32_t n = expert_rows(p, e, &lo);
        return n / BM + (n % BM != 0);
    };
    int64_t mine = 0;
    for (int e = e0; e < e1; ++e)
        mine += tiles(e);
    int64_t upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up((long long)upto, d);
        if ((tid & 63) >= d)
            upto += o;
    }
    if ((tid & 63) == 63)
        s_wave[tid >> 6] = upto;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) {
        if (w < (tid >> 6))
            upto += s_wave[w];
        total += s_wave[w];
    }
    if (total > p.max_tiles)
        return 0;
    int32_t at = (int32_t)(upto - mine);
    for (int e = e0; e < e1; ++e) {
        prefix[e] = at;
        at += tiles(e);
    }
    if (tid == 0)
        prefix[p.E] = (int32_t)total;
    __syncthreads();
    return __builtin_amdgcn_readfirstlane((int32_t)total);
}

// x / n of the same value in every lane, x >= 0, by inv = 1 / n in fp64: off by one at most.
__device__ __forceinline__ int32_t quotient(int32_t x, int32_t n, double inv)
{
    int32_t q = __builtin_amdgcn_readfirstlane((int32_t)((double)x * inv));
    const int32_t r = x - q * n;
    q -= r < 0;
    q += r >= n;
    return q;
}

// Tile `at` of all: expert by expert, GROUP row tiles by all channel blocks at a time, row tiles
// fastest, so that tiles that run together on an XCD share weights and rows in its L2.
template <int BM, int GROUP, typename Args>
__device__ __forceinline__ Tile tile_at(const Args& p, const int32_t* prefix, int32_t at)
{
    static_assert(GROUP == 4, "side is at most 4");
    const int32_t index = quotient(at, p.n_blocks, p.inv_blocks);
    int32_t e = -1;
    for (int j = 0; j < p.E; j += 64) {
        const int i = j + (threadIdx.x & 63);
        e += __popcll(__ballot(i < p.E && prefix[i] <= index));
    }
    const int32_t before = __builtin_amdgcn_readfirstlane(prefix[e]);
    const int32_t tiles = __builtin_amdgcn_readfirstlane(prefix[e + 1]) - before;
    const int32_t local = at - before * p.n_blocks;
    const int32_t group = quotient(local, GROUP * p.n_blocks, p.inv_blocks / GROUP);
    const int32_t in = local - group * GROUP * p.n_blocks;
    const int32_t side = min(GROUP, tiles - group * GROUP);
    Tile t;
    t.e = e;
    t.n = side == 4 ? in >> 2 : side == 3 ? (int32_t)((uint32_t)in / 3u) : side == 2 ? in >> 1 : in;
    const int32_t m = group * GROUP + in - t.n * side;
    int32_t lo;
    const int32_t n = expert_rows(p, e, &lo);
    t.row0 = __builtin_amdgcn_readfirstlane(lo + m * BM);
    t.rows = __builtin_amdgcn_readfirstlane(min(BM, n - m * BM));
    return t;
}

// Workgroups for tiles of bm rows: the row tiles of all experts are at most R / bm and one more for
// each expert that has rows.
template <typename Args>
inline int64_t most_tiles(const Args& p, int32_t bm)
{
    return p.offsets ? p.R / bm + (p.E < p.R ? p.E : p.R) : div_up(p.R, bm);
}

inline moe_status_t launched()
{
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe_dev

#endif  // MOE_TILES_H
