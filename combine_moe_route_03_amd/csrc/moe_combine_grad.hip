// moe_combine_grad.hip -- the gradient of the weighted combine (declared in include/moe_block.h):
//   dy[row of (t, j)] = w_tj dout_t,  dw_tj = <dout_t, y[row of (t, j)]>.
// A token's dout is read once, into registers, and each of its rows of y once: bound by HBM.
#include "moe_block.h"
#include "moe_device.h"

namespace {

using namespace moe_dev;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// NT: past the caches, for what is read once and is more than they hold.
template <bool NT, typename V>
__device__ __forceinline__ V load16(const V* p)
{
    if constexpr (NT)
        return __builtin_nontemporal_load(p);
    else
        return *p;
}

// Eight elements as they are in memory.
template <typename T>
struct Eight;

template <>
struct Eight<__bf16> {
    u32x4 x;

    template <bool NT>
    __device__ __forceinline__ void load(const __bf16* p)
    {
        x = load16<NT>(reinterpret_cast<const u32x4*>(p));
    }

    __device__ __forceinline__ float value(int i) const
    {
        return __uint_as_float(i & 1 ? x[i / 2] & 0xFFFF0000u : x[i / 2] << 16);
    }

    __device__ __forceinline__ static void store(__bf16* p, const float (&v)[8])
    {
        bf16x8 b;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            b[i] = (__bf16)v[i];
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, b), reinterpret_cast<u32x4*>(p));
    }
};

template <>
struct Eight<float> {
    f32x4 x[2];

    template <bool NT>
    __device__ __forceinline__ void load(const float* p)
    {
        x[0] = load16<NT>(reinterpret_cast<const f32x4*>(p));
        x[1] = load16<NT>(reinterpret_cast<const f32x4*>(p) + 1);
    }

    __device__ __forceinline__ float value(int i) const { return x[i / 4][i % 4]; }

    __device__ __forceinline__ static void store(float* p, const float (&v)[8])
    {
        __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4*>(p));
        __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, reinterpret_cast<f32x4*>(p) + 1);
    }
};

struct CombineGradArgs {
    const void* dout;
    const void* y;
    const int32_t* token_row;
    const float* w;
    int32_t T, H, k;
    void* dy;
    float* dw;
    int32_t share, shares;     // slots of a workgroup, and how many shares a token's slots make
};

// WAVES wavefronts take a token, or `share` of its slots; a lane holds up to NV pieces of 8 elements of
// dout, rows longer than that are taken in turns. The slots' products are joined over the wavefronts at
// the end, in order. 4096 tokens, k = 8, 7168 bf16: 175 to 202 us (5.7 to 4.9 TB/s, half of it written) with
// 8 wavefronts of two pieces, 217 with 4 of four, 320 with 2 of seven; two slots' rows on their way at a
// time 204. fp32 rows 405 to 446 us (4.9 to 4.5 TB/s), 128 tokens 16.
template <typename YT, typename OT, int WAVES, int NV, bool NT>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) void k_combine_grad(CombineGradArgs a)
{
    constexpr int kTokens = WAVES == 1 ? 4 : 1, kLanes = 64 * WAVES;
    __shared__ float s_dot[MOE_MAX_TOPK][WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l = tid % kLanes;
    const int pieces = a.H / 8;
    const int32_t R = a.T * a.k;
    for (int64_t i = (int64_t)blockIdx.x * kTokens + (WAVES == 1 ? wave : 0); i < (int64_t)a.T * a.shares;
         i += (int64_t)gridDim.x * kTokens) {
        const int64_t t = a.shares == 1 ? i : i / a.shares;
        const int j0 = (int)(i - t * a.shares) * a.share, j1 = min(j0 + a.share, a.k);
        const int32_t my_row = lane < a.k ? a.token_row[t * a.k + lane] : -1;
        const float my_w = a.dy && lane < a.k ? a.w[t * a.k + lane] : 0.0f;
        float my_dot = 0.0f;                                  // lane j: this wavefront's part of slot j
        for (int p0 = 0; p0 < pieces; p0 += kLanes * NV) {
            Eight<OT> d[NV];
#pragma unroll
            for (int n = 0; n < NV; ++n)
                if (p0 + n * kLanes + l < pieces)
                    d[n].template load<false>(static_cast<const OT*>(a.dout) + t * a.H +
                                              (int64_t)(p0 + n * kLanes + l) * 8);
            for (int j = j0; j < j1; ++j) {
                const int32_t row = __builtin_amdgcn_readlane(my_row, j);
                if ((uint32_t)row >= (uint32_t)R)
                    continue;
                const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(my_w), j));
                const int64_t base = (int64_t)row * a.H;
                Eight<YT> y[NV];
                if (a.dw) {
#pragma unroll
                    for (int n = 0; n < NV; ++n)
                        if (p0 + n * kLanes + l < pieces)
                            y[n].template load<NT>(static_cast<const YT*>(a.y) + base +
                                                   (int64_t)(p0 + n * kLanes + l) * 8);
                }
                float dot = 0.0f;
#pragma unroll
                for (int n = 0; n < NV; ++n)
                    if (p0 + n * kLanes + l < pieces) {
                        float v[8];
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            v[c] = w * d[n].value(c);
                        if (a.dy)
                            Eight<YT>::store(static_cast<YT*>(a.dy) + base +
                                                 (int64_t)(p0 + n * kLanes + l) * 8, v);
                        if (a.dw) {
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                dot = __builtin_fmaf(d[n].value(c), y[n].value(c), dot);
                        }
                    }
                if (a.dw) {
                    dot = group_sum<64>(dot);
                    my_dot += lane == j ? dot : 0.0f;
                }
            }
        }
        if (!a.dw)
            continue;
        if (WAVES == 1) {
            if (lane >= j0 && lane < j1)
                a.dw[t * a.k + lane] = my_dot;
        } else {
            if (lane >= j0 && lane < j1)
                s_dot[lane][wave] = my_dot;
            __syncthreads();
            if (tid >= j0 && tid < j1) {
                float sum = 0.0f;
#pragma unroll
                for (int w = 0; w < WAVES; ++w)
                    sum += s_dot[tid][w];
                a.dw[t * a.k + tid] = sum;
            }
            __syncthreads();
        }
    }
}

// Few tokens: their slots are shared out over workgroups, which read dout again, from the L2, until there
// are four of them for a CU (128 tokens, k = 8, 7168: 20 -> 6.3 us). Batches that the Infinity Cache holds
// are read through the caches, larger ones past them (512 tokens 21.5 and 25 us; 4096 tokens 207 and 202).
template <typename YT, typename OT, int WAVES, int NV>
void launch_combine_grad(CombineGradArgs a, hipStream_t stream)
{
    constexpr int kTokens = WAVES == 1 ? 4 : 1, kThreads = WAVES == 1 ? 256 : 64 * WAVES;
    a.share = a.k;
    while (a.share > 1 && div_up(a.T * div_up(a.k, a.share), kTokens) < 1024)
        a.share = (a.share + 1) / 2;
    a.shares = (int32_t)div_up(a.k, a.share);
    const int64_t need = div_up((int64_t)a.T * a.shares, kTokens), most = 1 << 20;
    const unsigned blocks = (unsigned)(need < most ? need : most);
    if (2 * (int64_t)sizeof(YT) * a.T * a.k * a.H > (int64_t)256 << 20)
        k_combine_grad<YT, OT, WAVES, NV, true><<<blocks, kThreads, 0, stream>>>(a);
    else
        k_combine_grad<YT, OT, WAVES, NV, false><<<blocks, kThreads, 0, stream>>>(a);
}

// One wavefront of two pieces, four of one and eight of two for 4096 tokens, k = 8, in us: bf16 H = 256 8.5, 13.5
// and 25; 1024 30, 31 and 48; 1032 29, 25 and 31; 2048 79, 56 and 60; 2056 80, 70 and 64; 7168 190, 186 and 188.
// fp32 H = 256 16, 21 and 36; 520 27, 25 and 30; 1024 64, 62 and 62; 1032 78, 70 and 69; 2048 122, 126 and 121;
// 2056 158, 146 and 136; 7168 433, 454 and 438. Of 128 tokens by 7168 14, 8.7 and 8.2 (bf16).
template <typename YT, typename OT>
void launch_combine_grad(const CombineGradArgs& a, hipStream_t stream)
{
    if (a.H <= 1024)
        launch_combine_grad<YT, OT, 1, 2>(a, stream);
    else if (a.H <= 2048)
        launch_combine_grad<YT, OT, 4, 1>(a, stream);
    else
        launch_combine_grad<YT, OT, 8, 2>(a, stream);
}

}  // namespace

extern "C" {

moe_status_t moe_combine_grad(const void* dout, moe_dtype_t dout_dtype, const void* y,
                              moe_dtype_t y_dtype, const int32_t* token_row, const float* topk_w,
                              int32_t T, int32_t H, int32_t k, void* dy, float* dtopk_w,
                              hipStream_t stream)
{
    if (T < 0 || H < 1 || k < 1 || (int64_t)T * k > INT32_MAX || (T > 0 && !dy && !dtopk_w))
        return MOE_ERR_INVALID;
    if ((dout_dtype != MOE_F32 && dout_dtype != MOE_BF16) ||
        (y_dtype != MOE_F32 && y_dtype != MOE_BF16) || H % 8 != 0 || k > MOE_MAX_TOPK)
        return MOE_ERR_UNSUPPORTED;
    if (T > 0 && (!dout || !token_row || (dtopk_w && !y) || (dy && !topk_w)))
        return MOE_ERR_INVALID;
    if (!aligned_to((const char*)dout, 16) || !aligned_to((const char*)y, 16) ||
        !aligned_to((const char*)dy, 16) || !aligned_to(token_row, 4) || !aligned_to(topk_w, 4) ||
        !aligned_to(dtopk_w, 4))
        return MOE_ERR_UNSUPPORTED;
    if (T == 0)
        return MOE_OK;
    const CombineGradArgs a = {dout, y, token_row, topk_w, T, H, k, dy, dtopk_w, k, 1};
    if (y_dtype == MOE_BF16)
        dout_dtype == MOE_BF16 ? launch_combine_grad<__bf16, __bf16>(a, stream)
                               : launch_combine_grad<__bf16, float>(a, stream);
    else
        dout_dtype == MOE_BF16 ? launch_combine_grad<float, __bf16>(a, stream)
                               : launch_combine_grad<float, float>(a, stream);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
