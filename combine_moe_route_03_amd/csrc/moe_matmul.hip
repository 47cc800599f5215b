// moe_matmul.hip -- the experts' product in bf16 with its epilogue (declared in include/moe_block.h):
// out = act(a w^T + bias) + residual over the rows of each expert. Where there are rows for them, the tiles
// of moe_mat_tile.h; below, k_mat_few.
#include "moe_mat_tile.h"

namespace {

// ---- few rows ----
// Bound by reading the weights, each once: a workgroup takes up to 16 MF rows of one expert and 16 NF
// channels; its wavefronts share the sum out by 128-byte pieces, read weights and rows straight into
// operands, and add their fp32 sums up through LDS, in wavefront order. v_mfma_f32_16x16x32_bf16 with
// the weights as the left operand: lane l gives channel l % 16 and 16 bytes of the sum at 16 (l / 16),
// and gets row l % 16 with channels 4 (l / 16) + i.
template <int MF, int NF, int WAVES, int U, bool SWIGLU, typename OUT>
__global__ __launch_bounds__(64 * WAVES) void k_mat_few(MatArgs p)
{
    constexpr int kFrags = MF * NF;
    __shared__ f32x4 s_acc[WAVES][kFrags][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t nb = blockIdx.x % p.n_blocks;
    const Tile tile = find_tile<16 * MF>(p, blockIdx.x / p.n_blocks);
    if (tile.rows == 0)
        return;
    const int r16 = lane & 15, kq = lane >> 4;
    const int32_t n_w = SWIGLU ? 2 * p.N : p.N;               // channels of w
    const __bf16* we = p.cols + (int64_t)tile.e * n_w * p.D;

    // channels: fragment f covers 16 from n0 + 16 f; with SwiGLU even fragments hold the gate and
    // the odd ones the same channels' up
    const int32_t n0 = nb * (SWIGLU ? 8 * NF : 16 * NF);
    const __bf16* wp[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
        int32_t n = SWIGLU ? n0 + 16 * (f / 2) + r16 : n0 + 16 * f + r16;
        n = min(n, p.N - 1) + (SWIGLU && (f & 1) ? p.N : 0);
        wp[f] = we + (int64_t)n * p.D;
    }
    const __bf16* ap[MF];
#pragma unroll
    for (int m = 0; m < MF; ++m) {
        const int32_t r = tile.row0 + min(16 * m + r16, tile.rows - 1);
        int32_t src = p.row_token ? p.row_token[r] : r;
        src = (uint32_t)src < (uint32_t)p.a_rows ? src : 0;   // its results are not stored
        ap[m] = p.rows + (int64_t)src * p.D;
    }
    // the fragment (with SwiGLU the pair) that this wavefront will join and store
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
    f32x4 acc[MF][NF];
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int f = 0; f < NF; ++f)
            acc[m][f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    for (int32_t k0 = wave * 64; k0 < p.D; k0 += U * WAVES * 64) {
        bf16x8 wv[2 * U][NF], av[2 * U][MF];
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
#pragma unroll
            for (int m = 0; m < MF; ++m) {
                av[h][m] = *reinterpret_cast<const bf16x8*>(ap[m] + (in ? at : 0));
                av[h][m] = in ? av[h][m] : none;
            }
        }
#pragma unroll
        for (int h = 0; h < 2 * U; ++h)
#pragma unroll
            for (int m = 0; m < MF; ++m)
#pragma unroll
                for (int f = 0; f < NF; ++f)
                    acc[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[h][f], av[h][m],
                                                                        acc[m][f], 0, 0, 0);
    }
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int f = 0; f < NF; ++f)
            s_acc[wave][m * NF + f][lane] = acc[m][f];
    __syncthreads();
    if (!stores)
        return;
    f32x4 sum[2];
#pragma unroll
    for (int g = 0; g < kStep; ++g) {
        sum[g] = s_acc[0][mine + g][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w)
            sum[g] += s_acc[w][mine + g][lane];
    }
    f32x4 y = sum[0] + b0, up = sum[kStep - 1] + b1;
    const auto put = [&](auto* to, auto v) {
        if (left >= 4 && (uintptr_t)to % sizeof(v) == 0) {
            *reinterpret_cast<decltype(v)*>(to) = v;
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (c < left)
                    to[c] = v[c];
        }
    };
    if (p.pre) {
        __bf16* q = p.pre + (int64_t)row * n_w + n;
        put(q, round4<__bf16>(y));
        if (SWIGLU)
            put(q + p.N, round4<__bf16>(up));
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
    put(static_cast<OUT*>(p.out) + (int64_t)row * p.N + n, round4<OUT>(y));
}

template <int MF, int NF, int WAVES, int U, bool SWIGLU, typename OUT>
moe_status_t launch_few(MatArgs p, hipStream_t stream)
{
    p.n_blocks = (int32_t)div_up(p.N, SWIGLU ? 8 * NF : 16 * NF);
    const int64_t blocks = most_tiles(p, 16 * MF) * p.n_blocks;
    if (blocks * 64 * WAVES > INT32_MAX)
        return MOE_ERR_UNSUPPORTED;
    k_mat_few<MF, NF, WAVES, U, SWIGLU, OUT><<<(unsigned)blocks, 64 * WAVES, 0, stream>>>(p);
    return launched();
}

// Few tiles leave most of the GPU idle and their sum in one workgroup: there the wavefronts of a workgroup
// share it, and 16 or 32 channels make a workgroup.
constexpr int64_t kFewTiles = 128;

template <bool SWIGLU, typename OUT>
moe_status_t launch_forward(const MatArgs& p, hipStream_t stream)
{
    const int64_t n_w = SWIGLU ? 2 * (int64_t)p.N : p.N;
    if (most_tiles(p, 32) * div_up(n_w, 128) < kFewTiles) {
        if (div_up(p.R, p.E < p.R ? p.E : p.R) > 16)
            return launch_few<2, 2, 8, 4, SWIGLU, OUT>(p, stream);
        if (SWIGLU || most_tiles(p, 16) * div_up(n_w, 16) > 512)
            return launch_few<1, 2, 8, 4, SWIGLU, OUT>(p, stream);
        return launch_few<1, SWIGLU ? 2 : 1, 8, SWIGLU ? 4 : 2, SWIGLU, OUT>(p, stream);
    }
    const int shape = choose<kForward>(p.R, p.E, 0, n_w, p.D).shape;
    if (p.pre || p.extra || (!SWIGLU && p.act != MOE_MAT_NONE))
        return launch_shape<kForward, SWIGLU, true, OUT>(shape, p, stream);
    return launch_shape<kForward, SWIGLU, false, OUT>(shape, p, stream);
}

}  // namespace

extern "C" {

moe_status_t moe_expert_matmul(const void* a, int32_t a_rows, const int32_t* row_token,
                               const void* w, const float* bias, const int32_t* expert_offsets,
                               int32_t R, int32_t E, int32_t N, int32_t K, moe_mat_act_t act,
                               const void* residual, void* pre, void* out, moe_dtype_t out_dtype,
                               hipStream_t stream)
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
        !aligned_to((const char*)pre, 2))
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
        return out_dtype == MOE_BF16 ? launch_forward<true, __bf16>(p, stream)
                                     : launch_forward<true, float>(p, stream);
    return out_dtype == MOE_BF16 ? launch_forward<false, __bf16>(p, stream)
                                 : launch_forward<false, float>(p, stream);
}

}  // extern "C"
