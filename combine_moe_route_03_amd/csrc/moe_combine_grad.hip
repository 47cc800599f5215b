// moe_combine_grad.hip -- the gradient of the weighted combine (declared in include/moe_block.h):
//   dy[row of (t, j)] = w_tj dout_t,  dw_tj = <dout_t, y[row of (t, j)]>.
// A token's dout is read once, into registers, and each of its rows of y once: bound by HBM.
#include "moe_block.h"
#include "moe_device.h"

namespace {

using namespace moe_dev;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Eight elements as they are in memory.
template <typename T>
struct Eight;

template <>
struct Eight<__bf16> {
    u32x4 x;

    __device__ __forceinline__ void load(const __bf16* p)
    {
        x = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
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

    __device__ __forceinline__ void load(const float* p)
    {
        x[0] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
        x[1] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p) + 1);
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
};

// WAVES wavefronts take a token; a lane holds up to NV pieces of 8 elements of dout, rows longer than
// that are taken in turns. The slots' products are joined over the wavefronts at a turn's end.
template <typename YT, typename OT, int WAVES, int NV>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) void k_combine_grad(CombineGradArgs a)
{
    constexpr int kTokens = WAVES == 1 ? 4 : 1, kLanes = 64 * WAVES;
    __shared__ float s_dot[MOE_MAX_TOPK][WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l = tid % kLanes;
    const int pieces = a.H / 8;
    const int32_t R = a.T * a.k;
    for (int64_t t = (int64_t)blockIdx.x * kTokens + (WAVES == 1 ? wave : 0); t < a.T;
         t += (int64_t)gridDim.x * kTokens) {
        for (int p0 = 0; p0 < pieces; p0 += kLanes * NV) {
            Eight<OT> d[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (p0 + i * kLanes + l < pieces)
                    d[i].load(static_cast<const OT*>(a.dout) + t * a.H +
                              (int64_t)(p0 + i * kLanes + l) * 8);
            for (int j = 0; j < a.k; ++j) {
                const int32_t row = a.token_row[t * a.k + j];
                const bool in = (uint32_t)row < (uint32_t)R;
                const float w = a.dy ? a.w[t * a.k + j] : 0.0f;
                float dot = 0.0f;
                if (in) {
                    const int64_t base = (int64_t)row * a.H;
                    Eight<YT> y[NV];
                    if (a.dw) {
#pragma unroll
                        for (int i = 0; i < NV; ++i)
                            if (p0 + i * kLanes + l < pieces)
                                y[i].load(static_cast<const YT*>(a.y) + base +
                                          (int64_t)(p0 + i * kLanes + l) * 8);
                    }
#pragma unroll
                    for (int i = 0; i < NV; ++i)
                        if (p0 + i * kLanes + l < pieces) {
                            float v[8];
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                v[c] = w * d[i].value(c);
                            if (a.dy)
                                Eight<YT>::store(static_cast<YT*>(a.dy) + base +
                                                     (int64_t)(p0 + i * kLanes + l) * 8, v);
                            if (a.dw) {
#pragma unroll
                                for (int c = 0; c < 8; ++c)
                                    dot = __builtin_fmaf(d[i].value(c), y[i].value(c), dot);
                            }
                        }
                }
                if (!a.dw)
                    continue;
                dot = group_sum<64>(dot);
                if (lane == 0) {
                    if (WAVES == 1)
                        a.dw[t * a.k + j] = p0 == 0 ? dot : a.dw[t * a.k + j] + dot;
                    else
                        s_dot[j][wave] = p0 == 0 ? dot : s_dot[j][wave] + dot;
                }
            }
        }
        if (WAVES > 1 && a.dw) {
            __syncthreads();
            if (tid < a.k) {
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

template <typename YT, typename OT>
void launch_combine_grad(const CombineGradArgs& a, hipStream_t stream)
{
    const int64_t most = 1 << 20;
    if (a.H <= 1024) {
        const int64_t blocks = div_up(a.T, 4);
        k_combine_grad<YT, OT, 1, 2><<<(unsigned)(blocks < most ? blocks : most), 256, 0, stream>>>(a);
    } else {
        const int64_t blocks = a.T;
        k_combine_grad<YT, OT, 4, 4><<<(unsigned)(blocks < most ? blocks : most), 256, 0, stream>>>(a);
    }
}

}  // namespace

extern "C" {

moe_status_t moe_combine_grad(const void* dout, moe_dtype_t dout_dtype, const void* y,
                              moe_dtype_t y_dtype, const int32_t* token_row, const float* topk_w,
                              int32_t T, int32_t H, int32_t k, void* dy, float* dtopk_w,
                              hipStream_t stream)
{
    if (T < 0 || H < 1 || k < 1 || (int64_t)T * k > INT32_MAX || (!dy && !dtopk_w))
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
    const CombineGradArgs a = {dout, y, token_row, topk_w, T, H, k, dy, dtopk_w};
    if (y_dtype == MOE_BF16)
        dout_dtype == MOE_BF16 ? launch_combine_grad<__bf16, __bf16>(a, stream)
                               : launch_combine_grad<__bf16, float>(a, stream);
    else
        dout_dtype == MOE_BF16 ? launch_combine_grad<float, __bf16>(a, stream)
                               : launch_combine_grad<float, float>(a, stream);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
