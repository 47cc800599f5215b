// moe_matmul_grad.hip -- the gradients of the experts' product in bf16 (declared in include/moe_block.h):
// of its rows, with the gradient of the activation that made them in the epilogue, of its weights, and of
// its bias. The products are the tiles of moe_mat_tile.h.
#include <initializer_list>

#include "moe_mat_tile.h"

namespace {

// ---- sums in parts ----
// Adds up `splits` parts in order; four columns a thread. Rows of a: those of an expert, with the
// activation's gradient; weights: all. Parts and sums are fp32, results are rounded once. Bound by the
// parts' bytes: 64 rows by 384 channels of 7168, rows' gradient 10 us with it, weights' 11.
template <bool ROWS, typename OUT>
__global__ __launch_bounds__(256) void k_join_parts(MatArgs p, const f32x4* __restrict__ parts,
                                                    int64_t total)
{
    const int32_t quads = p.N / 4;
    int32_t lo = 0, hi = p.R;
    if (ROWS && p.offsets) {
        lo = min(max(p.offsets[0], 0), p.R);
        hi = min(max(p.offsets[p.E], 0), p.R);
    }
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / quads;
        const int32_t n = 4 * (int32_t)(i - row * quads);
        if (ROWS && (row < lo || row >= hi ||
                     (p.row_token && (uint32_t)p.row_token[row] >= (uint32_t)p.a_rows)))
            continue;
        f32x4 y = parts[i];
        for (int s = 1; s < p.splits; ++s)
            y += parts[s * total + i];
        typedef typename Four<OUT>::type four;
        if (ROWS && p.act == MOE_MAT_SWIGLU) {
            const __bf16* q = static_cast<const __bf16*>(p.extra) + row * 2 * p.N + n;
            const f32x4 gate = load4(q, 4, false), up = load4(q + p.N, 4, false);
            f32x4 z;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                z[c] = y[c] * activate(gate[c], MOE_MAT_SILU);
                y[c] = y[c] * up[c] * slope(gate[c], MOE_MAT_SILU);
            }
            OUT* out = static_cast<OUT*>(p.out) + row * 2 * p.N + n;
            *reinterpret_cast<four*>(out) = round4<OUT>(y);
            *reinterpret_cast<four*>(out + p.N) = round4<OUT>(z);
            continue;
        }
        if (ROWS && p.act != MOE_MAT_NONE) {
            const f32x4 x = load4(static_cast<const __bf16*>(p.extra) + row * p.N + n, 4, false);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                y[c] *= slope(x[c], p.act);
        }
        *reinterpret_cast<four*>(static_cast<OUT*>(p.out) + 4 * i) = round4<OUT>(y);
    }
}

template <bool ROWS, typename OUT>
moe_status_t launch_join(const MatArgs& p, const void* parts, int64_t rows, hipStream_t stream)
{
    const int64_t total = rows * (p.N / 4), need = div_up(total, 256), most = 8192;
    k_join_parts<ROWS, OUT><<<(unsigned)(need < most ? need : most), 256, 0, stream>>>(
        p, static_cast<const f32x4*>(parts), total);
    return launched();
}

// ---- bias gradient ----
// Column sums of dy over an expert's rows: 16 lanes hold 128 columns, 16 rows of a workgroup at a time and
// eight of each lane on their way, each lane's rows in order and the 16 joined in order. The rows of an
// expert are shared out over `splits` workgroups, whose sums are joined by a launch of its own. Bound by
// latency where there are few rows, else by reading dy: 2331 rows of 20 experts by 1000 12.7 us with the
// launch of the join (uneven experts without parts 18), 4096 rows by 384 12.6, 32768 rows of 256 experts by
// 4096 44.7 (floor 41).
__global__ __launch_bounds__(256) void k_bias_grad(MatArgs p, float* __restrict__ out)
{
    constexpr int kFlight = 8;
    __shared__ float s_sum[16][128];
    const int tid = threadIdx.x, g = tid & 15, slot = tid >> 4;
    const int32_t block = blockIdx.x % p.n_blocks, part = blockIdx.x / p.n_blocks;
    const int32_t split = part % p.splits, e = part / p.splits;
    const int32_t n = block * 128 + 8 * g;
    int32_t lo;
    const int32_t count = expert_rows(p, e, &lo);
    const int32_t r0 = (int32_t)((int64_t)count * split / p.splits);
    const int32_t r1 = (int32_t)((int64_t)count * (split + 1) / p.splits);
    float sum[8] = {};
    if (n < p.N)
        for (int32_t r = r0 + slot; r < r1; r += 16 * kFlight) {
            bool in[kFlight];
            bf16x8 v[kFlight];
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                in[i] = r + 16 * i < r1;
                if (p.row_token && in[i])
                    in[i] = (uint32_t)p.row_token[lo + r + 16 * i] < (uint32_t)p.a_rows;
            }
#pragma unroll
            for (int i = 0; i < kFlight; ++i)
                if (in[i])
                    v[i] = *reinterpret_cast<const bf16x8*>(p.rows + (int64_t)(lo + r + 16 * i) * p.N + n);
#pragma unroll
            for (int i = 0; i < kFlight; ++i)
                if (in[i]) {
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        sum[c] += (float)v[i][c];
                }
        }
#pragma unroll
    for (int c = 0; c < 8; ++c)
        s_sum[slot][8 * g + c] = sum[c];
    __syncthreads();
    const int32_t col = block * 128 + tid;
    if (tid < 128 && col < p.N) {
        float all = 0.0f;
#pragma unroll
        for (int s = 0; s < 16; ++s)
            all += s_sum[s][tid];
        out[((int64_t)split * p.E + e) * p.N + col] = all;
    }
}

__global__ __launch_bounds__(256) void k_join_bias(const float* __restrict__ parts, int64_t total,
                                                   int32_t splits, float* __restrict__ dbias)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        float sum = parts[i];
#pragma unroll 8
        for (int s = 1; s < splits; ++s)
            sum += parts[s * total + i];
        dbias[i] = sum;
    }
}

// Workgroups for the rows of an expert: four a CU in all, of 16 rows at least where experts have the same
// number, and 64 at most, whose sums the join adds up one by one (4096 rows by 384: 62 us with 256).
int32_t bias_splits(int32_t R, int32_t E, int32_t N)
{
    int64_t s = 1024 / ((int64_t)E * div_up(N, 128));
    if (s > (int64_t)R / E / 16)
        s = (int64_t)R / E / 16;
    return s < 1 ? 1 : s > 64 ? 64 : (int32_t)s;
}

template <typename OUT>
moe_status_t launch_rows(MatArgs p, void* parts, hipStream_t stream)
{
    const Plan plan = choose<kRowsBack>(p.R, p.E, 0, p.N, p.D);
    if (plan.splits == 1)
        return p.act != MOE_MAT_NONE ? launch_shape<kRowsBack, false, true, OUT>(plan.shape, p, stream)
                                     : launch_shape<kRowsBack, false, false, OUT>(plan.shape, p, stream);
    MatArgs q = p;
    q.splits = p.splits = plan.splits;
    q.out = parts;
    q.act = MOE_MAT_NONE;
    const moe_status_t st = launch_shape<kRowsBack, false, false, float>(plan.shape, q, stream);
    return st != MOE_OK ? st : launch_join<true, OUT>(p, parts, p.R, stream);
}

template <typename OUT>
moe_status_t launch_weights(MatArgs p, void* parts, hipStream_t stream)
{
    const Plan plan = choose<kWeightsBack>(p.R, p.E, p.M, p.N, 0);
    if (plan.splits == 1)
        return launch_shape<kWeightsBack, false, false, OUT>(plan.shape, p, stream);
    MatArgs q = p;
    q.splits = p.splits = plan.splits;
    q.out = parts;
    const moe_status_t st = launch_shape<kWeightsBack, false, false, float>(plan.shape, q, stream);
    return st != MOE_OK ? st : launch_join<false, OUT>(p, parts, (int64_t)p.E * p.M, stream);
}

}  // namespace

extern "C" {

size_t moe_matmul_grad_workspace_bytes(int32_t R, int32_t E, int32_t N, int32_t K)
{
    if (R < 0 || E < 1 || N < 1 || K < 1 || E > MOE_MAX_EXPERTS || N > MOE_MAT_MAX_SIZE ||
        K > MOE_MAT_MAX_SIZE)
        return 0;
    int64_t bytes = 256;
    if (R > 0) {
        const int64_t rows = choose<kRowsBack>(R, E, 0, K, N).part_bytes;
        const int64_t weights = choose<kWeightsBack>(R, E, N, K, 0).part_bytes;
        const int64_t splits = bias_splits(R, E, N), bias = splits > 1 ? splits * E * N * 4 : 0;
        for (const int64_t b : {rows, weights, bias})
            bytes = b > bytes ? b : bytes;
    }
    return (size_t)bytes;
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
    if (R > 0 && !da && !dw && !dbias)
        return MOE_ERR_INVALID;
    if (N % 8 != 0 || (da && da_dtype != MOE_F32 && da_dtype != MOE_BF16) ||
        (dw && dw_dtype != MOE_F32 && dw_dtype != MOE_BF16) ||
        (act == MOE_MAT_SWIGLU && K > MOE_MAT_MAX_SIZE / 2) ||
        (dbias && E * div_up(N, 128) > INT32_MAX / 256))      // one workgroup of 256 for each
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
        st = da_dtype == MOE_BF16 ? launch_rows<__bf16>(p, workspace, stream)
                                  : launch_rows<float>(p, workspace, stream);
        if (st != MOE_OK)
            return st;
    }
    if (dw) {
        MatArgs p = mat_args(dy, a, row_token, expert_offsets, a_rows, R, E);
        p.out = dw;
        p.N = K;
        p.M = N;
        st = dw_dtype == MOE_BF16 ? launch_weights<__bf16>(p, workspace, stream)
                                  : launch_weights<float>(p, workspace, stream);
        if (st != MOE_OK)
            return st;
    }
    if (dbias) {
        MatArgs p = mat_args(dy, nullptr, row_token, expert_offsets, a_rows, R, E);
        p.N = N;
        p.n_blocks = (int32_t)div_up(N, 128);
        p.splits = R > 0 ? bias_splits(R, E, N) : 1;
        float* parts = p.splits > 1 ? static_cast<float*>(workspace) : dbias;
        k_bias_grad<<<(unsigned)(E * p.splits * p.n_blocks), 256, 0, stream>>>(p, parts);
        if (p.splits > 1) {
            const int64_t total = (int64_t)E * N, need = div_up(total, 256);
            k_join_bias<<<(unsigned)(need < 4096 ? need : 4096), 256, 0, stream>>>(parts, total, p.splits,
                                                                                 dbias);
        }
        st = launched();
    }
    return st;
}

}  // extern "C"
