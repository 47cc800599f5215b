// moe_matmul.hip -- the experts' product in bf16 with its epilogue (declared in include/moe_block.h):
// out = act(a w^T + bias) + residual over the rows of each expert. Where there are rows for them, the tiles
// of moe_mat_tile.h; below, k_mat_few.
#include "moe_mat_tile.h"

namespace {

// ---- few rows ----
// Bound by reading the weights, each once: a workgroup takes up to 16 rows of one expert and 16 channels
// (with SwiGLU, gate and up of 16); its eight wavefronts share the sum out by 128-byte pieces, read
// weights and rows straight into operands, and add their fp32 sums up through LDS, in wavefront order:
// no wait in the loop but for the operands, and eight times the loads on their way that a tile with all
// of the sum to itself has. 8 rows of 8 experts by 2 x 1024 channels of 2048 14.9 us (floor at 6.5 TB/s
// 10.3), one token by 384 of 7168 9.7. v_mfma_f32_16x16x32_bf16 with the weights as the left operand: lane
// l gives channel l % 16 and 16 bytes of the sum at 16 (l / 16), and gets row l % 16 with channels
// 4 (l / 16) + i.
template <int WAVES, int U, bool SWIGLU, typename OUT>
__global__ __launch_bounds__(64 * WAVES) void k_mat_few(MatArgs p)
{
    constexpr int NF = SWIGLU ? 2 : 1;                        // fragments
    __shared__ f32x4 s_acc[WAVES][NF][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t nb = blockIdx.x % p.n_blocks;
    const Tile tile = find_tile<16>(p, blockIdx.x / p.n_blocks);
    if (tile.rows == 0)
        return;
    const int r16 = lane & 15, kq = lane >> 4;
    const int32_t n_w = SWIGLU ? 2 * p.N : p.N;               // channels of w
    const __bf16* we = p.cols + (int64_t)tile.e * n_w * p.D;

    const int32_t n0 = nb * 16;                               // SwiGLU: the first fragment's is the gate,
    const __bf16* wp[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
        const int32_t n = min(n0 + r16, p.N - 1) + f * p.N;   // the other's the same channels' up
        wp[f] = we + (int64_t)n * p.D;
    }
    const int32_t row = tile.row0 + min(r16, tile.rows - 1);
    const int32_t src = p.row_token ? p.row_token[row] : row;
    const bool there = (uint32_t)src < (uint32_t)p.a_rows;    // else its results are not stored
    const __bf16* ap = p.rows + (int64_t)(there ? src : 0) * p.D;
    // the first wavefront joins the sums and stores
    const int32_t n = n0 + 4 * kq;
    const int32_t left = p.N - n;
    const bool stores = wave == 0 && r16 < tile.rows && there && left > 0;
    const bool vec = p.N % 4 == 0;
    f32x4 b0 = {0.0f, 0.0f, 0.0f, 0.0f}, b1 = b0, res = b0;
    if (stores && p.bias) {
        const float* b = p.bias + (int64_t)tile.e * n_w + n;
        b0 = load4(b, left, false);
        if (SWIGLU)
            b1 = load4(b + p.N, left, false);
    }
    if (stores && p.extra)
        res = load4(static_cast<const OUT*>(p.extra) + (int64_t)row * p.N + n, left,
                    vec && (uintptr_t)p.extra % 16 == 0);
    f32x4 acc[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f)
        acc[f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    for (int32_t k0 = wave * 64; k0 < p.D; k0 += U * WAVES * 64) {
        bf16x8 wv[2 * U][NF], av[2 * U];
#pragma unroll
        for (int h = 0; h < 2 * U; ++h) {
            const int32_t at = k0 + h / 2 * WAVES * 64 + 32 * (h % 2) + 8 * kq;
            const bool in = at < p.D;                         // D is a multiple of 8
            const bf16x8 none = {};
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                wv[h][f] = *reinterpret_cast<const bf16x8*>(wp[f] + (in ? at : 0));
                wv[h][f] = in ? wv[h][f] : none;
            }
            av[h] = *reinterpret_cast<const bf16x8*>(ap + (in ? at : 0));
            av[h] = in ? av[h] : none;
        }
#pragma unroll
        for (int h = 0; h < 2 * U; ++h)
#pragma unroll
            for (int f = 0; f < NF; ++f)
                acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[h][f], av[h], acc[f], 0, 0, 0);
    }
#pragma unroll
    for (int f = 0; f < NF; ++f)
        s_acc[wave][f][lane] = acc[f];
    __syncthreads();
    if (!stores)
        return;
    f32x4 sum[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
        sum[f] = s_acc[0][f][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w)
            sum[f] += s_acc[w][f][lane];
    }
    f32x4 y = sum[0] + b0, up = sum[NF - 1] + b1;
    if (p.pre) {
        __bf16* q = p.pre + (int64_t)row * n_w + n;
        store4(q, round4<__bf16>(y), left);
        if (SWIGLU)
            store4(q + p.N, round4<__bf16>(up), left);
    }
    if (SWIGLU) {
        y = swiglu(y, up);
    } else if (p.act != MOE_MAT_NONE) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            y[c] = activate(y[c], p.act);
    }
    if (p.extra)
        y += res;
    store4(static_cast<OUT*>(p.out) + (int64_t)row * p.N + n, round4<OUT>(y), left);
}

// ---- sums in parts ----
// Adds up `splits` parts [R, n_w] in order and does what else there is to a result: four columns of a row
// a thread. Parts stay in fp32, so that out is rounded once here too. Bound by their bytes and a launch: 64
// rows by 384 channels of 7168 in 16 parts 13.0 us with it (4.5 of them), 32.8 without parts (16 loads
// one behind the other: 17.0); 4096 rows in 4 parts 48 and 72.
template <bool SWIGLU, typename OUT>
__global__ __launch_bounds__(256) void k_join_forward(MatArgs p, const float* __restrict__ parts)
{
    const int32_t quads = (p.N + 3) / 4, n_w = SWIGLU ? 2 * p.N : p.N;
    const int64_t total = (int64_t)p.R * quads, part = (int64_t)p.R * n_w;
    const bool vec = p.N % 4 == 0, vec_extra = vec && (uintptr_t)p.extra % 16 == 0;
    const int32_t lo = p.offsets ? min(max(p.offsets[0], 0), p.R) : 0;
    const int32_t hi = p.offsets ? min(max(p.offsets[p.E], 0), p.R) : p.R;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / quads;
        const int32_t n = 4 * (int32_t)(i - row * quads), left = p.N - n;
        if (row < lo || row >= hi ||
            (p.row_token && (uint32_t)p.row_token[row] >= (uint32_t)p.a_rows))
            continue;
        const float* q = parts + row * n_w + n;
        f32x4 y = load4(q, left, vec), z = y;
        if (SWIGLU)
            z = load4(q + p.N, left, vec);
#pragma unroll 5
        for (int s = 1; s < p.splits; ++s) {
            y += load4(q + s * part, left, vec);
            if (SWIGLU)
                z += load4(q + s * part + p.N, left, vec);
        }
        if (p.bias) {
            int32_t e = 0, end = p.E;                         // the row's expert
            while (end - e > 1) {
                const int32_t mid = (e + end) / 2;
                if (p.offsets[mid] <= row)
                    e = mid;
                else
                    end = mid;
            }
            const float* b = p.bias + (int64_t)e * n_w + n;
            y += load4(b, left, false);
            if (SWIGLU)
                z += load4(b + p.N, left, false);
        }
        if (p.pre) {
            __bf16* pre = p.pre + row * n_w + n;
            store4(pre, round4<__bf16>(y), left);
            if (SWIGLU)
                store4(pre + p.N, round4<__bf16>(z), left);
        }
        if (SWIGLU) {
            y = swiglu(y, z);
        } else if (p.act != MOE_MAT_NONE) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                y[c] = activate(y[c], p.act);
        }
        if (p.extra)
            y += load4(static_cast<const OUT*>(p.extra) + row * p.N + n, left, vec_extra);
        store4(static_cast<OUT*>(p.out) + row * p.N + n, round4<OUT>(y), left);
    }
}

// At most 2 * 8 of its workgroups for each of less than 256 tiles of few().
template <bool SWIGLU, typename OUT>
moe_status_t launch_few(MatArgs p, hipStream_t stream)
{
    constexpr int kWaves = 8;
    p.n_blocks = (int32_t)div_up(p.N, 16);
    const int64_t blocks = most_tiles(p, 16) * p.n_blocks;
    k_mat_few<kWaves, SWIGLU ? 4 : 2, SWIGLU, OUT><<<(unsigned)blocks, 64 * kWaves, 0, stream>>>(p);
    return launched();
}

// Experts with no more rows than a matrix instruction takes, and tiles (of 32 rows by 128 channels) for
// less than a workgroup a CU: k_mat_few; else the tiles of moe_mat_tile.h, here and there (us): 16 rows by
// 2048 channels of 2048 (16 tiles) 8.4 and 11.6, by 16384 of 1024 (128) 10.0 and 14.2, 8 rows of 64 experts
// by 2 x 1408 of 2048 (176) 19.1 and 21.5, 16 rows by 32768 of 1024 (256) 16.9 and 14.2, one token by 32768
// of 2048 (256) 28 and 26, 32 rows of 128 experts by 2 x 1024 of 2048 (528) 43 and 34. 32 channels a
// workgroup: 8.7, 13.4 and 24 us for the first, second and fourth.
constexpr int64_t kFewTiles = 256;

bool few(int32_t R, int32_t E, int64_t n_w)
{
    const int64_t experts = E < R ? E : R;
    const int64_t tiles = E == 1 ? div_up(R, 32) : R / 32 + experts;
    return div_up(R, experts) <= 16 && tiles * div_up(n_w, 128) < kFewTiles;
}

template <bool SWIGLU, typename OUT>
moe_status_t launch_forward(const MatArgs& p, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    const int64_t n_w = SWIGLU ? 2 * (int64_t)p.N : p.N;
    if (few(p.R, p.E, n_w)) {
        return launch_few<SWIGLU, OUT>(p, stream);
    }
    const Plan plan = choose<kForward>(p.R, p.E, 0, n_w, p.D);
    if (plan.splits > 1) {
        if (!workspace || workspace_bytes < (size_t)plan.part_bytes)
            return MOE_ERR_WORKSPACE;
        MatArgs q = p, j = p;
        q.splits = j.splits = plan.splits;
        q.N = (int32_t)n_w;
        q.out = workspace;
        q.act = MOE_MAT_NONE;
        q.bias = nullptr;
        q.extra = nullptr;
        q.pre = nullptr;
        const moe_status_t st = launch_shape<kForward, false, false, float>(plan.shape, q, stream);
        if (st != MOE_OK)
            return st;
        const int64_t need = div_up((int64_t)p.R * div_up(p.N, 4), 256), most = 8192;
        k_join_forward<SWIGLU, OUT><<<(unsigned)(need < most ? need : most), 256, 0, stream>>>(
            j, static_cast<const float*>(workspace));
        return launched();
    }
    if (p.pre || p.extra || (!SWIGLU && p.act != MOE_MAT_NONE))
        return launch_shape<kForward, SWIGLU, true, OUT>(plan.shape, p, stream);
    return launch_shape<kForward, SWIGLU, false, OUT>(plan.shape, p, stream);
}

}  // namespace

extern "C" {

size_t moe_expert_matmul_workspace_bytes(int32_t R, int32_t E, int32_t channels, int32_t K)
{
    if (R < 1 || E < 1 || channels < 1 || K < 1 || E > MOE_MAX_EXPERTS || !fits(channels, K) ||
        few(R, E, channels))
        return 0;
    return (size_t)choose<kForward>(R, E, 0, channels, K).part_bytes;
}

moe_status_t moe_expert_matmul(const void* a, int32_t a_rows, const int32_t* row_token,
                               const void* w, const float* bias, const int32_t* expert_offsets,
                               int32_t R, int32_t E, int32_t N, int32_t K, moe_mat_act_t act,
                               const void* residual, void* pre, void* out, moe_dtype_t out_dtype,
                               void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    const int64_t n_w = act == MOE_MAT_SWIGLU ? 2 * (int64_t)N : N;
    const moe_status_t st = check_sizes(a_rows, row_token, expert_offsets, R, E, N, n_w, K, act);
    if (st != MOE_OK)
        return st;
    if (out_dtype != MOE_F32 && out_dtype != MOE_BF16)
        return MOE_ERR_UNSUPPORTED;
    if (R > 0 && (!a || !w || !out))
        return MOE_ERR_INVALID;
    const int each = out_dtype == MOE_F32 ? 4 : 2;
    if (!aligned_to((const char*)a, 16) || !aligned_to((const char*)w, 16) || !aligned_to(bias, 4) ||
        !aligned_to((const char*)out, each) || !aligned_to((const char*)residual, each) ||
        !aligned_to((const char*)pre, 2) || !aligned_to((const char*)workspace, 16))
        return MOE_ERR_UNSUPPORTED;
    if (R == 0)
        return MOE_OK;
    MatArgs p = mat_args(a, w, row_token, expert_offsets, a_rows, R, E);
    p.bias = bias;
    p.extra = residual;
    p.out = out;
    p.pre = static_cast<__bf16*>(pre);
    p.N = N;
    p.D = K;
    p.act = act;
    if (act == MOE_MAT_SWIGLU)
        return out_dtype == MOE_BF16 ? launch_forward<true, __bf16>(p, workspace, workspace_bytes, stream)
                                     : launch_forward<true, float>(p, workspace, workspace_bytes, stream);
    return out_dtype == MOE_BF16 ? launch_forward<false, __bf16>(p, workspace, workspace_bytes, stream)
                                 : launch_forward<false, float>(p, workspace, workspace_bytes, stream);
}

}  // extern "C"
