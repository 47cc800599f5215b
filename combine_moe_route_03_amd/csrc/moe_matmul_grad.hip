// moe_matmul_grad.hip -- the gradients of the experts' product in bf16 (declared in include/moe_block.h):
// of its rows, with the gradient of the activation that made them in the epilogue, of its weights, and of
// its bias. The products are the tiles of moe_mat_tile.h.
#include <initializer_list>

#include "moe_mat_tile.h"

namespace {

// ---- bias gradient ----
// Column sums of dy over an expert's rows: 16 lanes hold 128 columns, 16 rows of a workgroup at a
// time, each lane's rows in order and the 16 joined in order.
__global__ __launch_bounds__(256) void k_bias_grad(MatArgs p, float* __restrict__ dbias)
{
    __shared__ float s_sum[16][128];
    const int tid = threadIdx.x, g = tid & 15, slot = tid >> 4;
    const int32_t e = blockIdx.x / p.n_blocks, n = (blockIdx.x % p.n_blocks) * 128 + 8 * g;
    int32_t lo;
    const int32_t count = expert_rows(p, e, &lo);
    float sum[8] = {};
    if (n < p.N)
        for (int32_t r = slot; r < count; r += 16) {
            if (p.row_token && (uint32_t)p.row_token[lo + r] >= (uint32_t)p.a_rows)
                continue;
            const bf16x8 v = *reinterpret_cast<const bf16x8*>(p.rows + (int64_t)(lo + r) * p.N + n);
#pragma unroll
            for (int c = 0; c < 8; ++c)
                sum[c] += (float)v[c];
        }
#pragma unroll
    for (int c = 0; c < 8; ++c)
        s_sum[slot][8 * g + c] = sum[c];
    __syncthreads();
    const int32_t col = (blockIdx.x % p.n_blocks) * 128 + tid;
    if (tid < 128 && col < p.N) {
        float all = 0.0f;
#pragma unroll
        for (int s = 0; s < 16; ++s)
            all += s_sum[s][tid];
        dbias[(int64_t)e * p.N + col] = all;
    }
}

template <typename OUT>
moe_status_t launch_rows(const MatArgs& p, hipStream_t stream)
{
    const int shape = choose_tile<kRowsBack>(p, p.N);
    return p.act != MOE_MAT_NONE ? launch_shape<kRowsBack, false, true, OUT>(shape, p, stream)
                                 : launch_shape<kRowsBack, false, false, OUT>(shape, p, stream);
}

template <typename OUT>
moe_status_t launch_weights(const MatArgs& p, hipStream_t stream)
{
    return launch_shape<kWeightsBack, false, false, OUT>(choose_tile<kWeightsBack>(p, p.N), p, stream);
}

}  // namespace

extern "C" {

size_t moe_matmul_grad_workspace_bytes(int32_t R, int32_t E, int32_t N, int32_t K)
{
    return R < 0 || E < 1 || N < 1 || K < 1 ? 0 : 256;
}

moe_status_t moe_expert_matmul_grad(const void* dy, const void* a, int32_t a_rows,
                                    const int32_t* row_token, const void* w,
                                    const int32_t* expert_offsets, int32_t R, int32_t E, int32_t N,
                                    int32_t K, moe_mat_act_t act, const void* pre, void* da,
                                    moe_dtype_t da_dtype, void* dw, moe_dtype_t dw_dtype,
                                    float* dbias, void* workspace, size_t workspace_bytes,
                                    hipStream_t stream)
{
    moe_status_t st = check_sizes(a_rows, row_token, expert_offsets, R, E, N, N, K, act);
    if (st != MOE_OK)
        return st;
    if (!da && !dw && !dbias)
        return MOE_ERR_INVALID;
    if (N % 8 != 0 || (da && da_dtype != MOE_F32 && da_dtype != MOE_BF16) ||
        (dw && dw_dtype != MOE_F32 && dw_dtype != MOE_BF16) ||
        (act == MOE_MAT_SWIGLU && K > MOE_MAT_MAX_SIZE / 2))
        return MOE_ERR_UNSUPPORTED;
    if (R > 0 && (!dy || (da && (!w || (act != MOE_MAT_NONE && !pre))) || (dw && !a)))
        return MOE_ERR_INVALID;
    if (!workspace || workspace_bytes < moe_matmul_grad_workspace_bytes(R, E, N, K))
        return MOE_ERR_WORKSPACE;
    for (const void* q : {dy, a, w, (const void*)da, (const void*)dw, (const void*)workspace})
        if (!aligned_to((const char*)q, 16))
            return MOE_ERR_UNSUPPORTED;
    if (!aligned_to((const char*)pre, 2) || !aligned_to(dbias, 4))
        return MOE_ERR_UNSUPPORTED;
    if (da && R > 0) {
        MatArgs p = mat_args(dy, w, row_token, expert_offsets, a_rows, R, E);
        p.extra = pre;
        p.out = da;
        p.N = K;
        p.D = N;
        p.act = act;
        st = da_dtype == MOE_BF16 ? launch_rows<__bf16>(p, stream)
                                  : launch_rows<float>(p, stream);
        if (st != MOE_OK)
            return st;
    }
    if (dw) {
        MatArgs p = mat_args(dy, a, row_token, expert_offsets, a_rows, R, E);
        p.out = dw;
        p.N = K;
        p.M = N;
        st = dw_dtype == MOE_BF16 ? launch_weights<__bf16>(p, stream)
                                  : launch_weights<float>(p, stream);
        if (st != MOE_OK)
            return st;
    }
    if (dbias) {
        MatArgs p = mat_args(dy, nullptr, row_token, expert_offsets, a_rows, R, E);
        p.N = N;
        p.n_blocks = (int32_t)div_up(N, 128);
        k_bias_grad<<<(unsigned)(E * p.n_blocks), 256, 0, stream>>>(p, dbias);
        st = launched();
    }
    return st;
}

}  // extern "C"
