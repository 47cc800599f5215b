// moe_gate.hip -- scored routing, its gradient, and the update of its bias (declared in
// include/moe_block.h).
#include "moe_block.h"
#include "moe_rows.h"

namespace {

using namespace moe_dev;

struct RouteArgs {
    const float* logits;
    const float* bias;
    int32_t T, E, k, score, groups, kept, top, renorm;
    float scale;
    int32_t* idx;
    float* w;
};

// ----------------------------------------------------------------------------------- routing --
__device__ __forceinline__ double shfl_xor(double v, int d) { return __shfl_xor(v, d); }

// The larger value, equal ones by the lower number.
struct Best {
    double v;
    int i;

    __device__ __forceinline__ void take(double w, int j)
    {
        if (w > v || (w == v && j < i)) {
            v = w;
            i = j;
        }
    }

    __device__ __forceinline__ void join_wave()
    {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1)
            take(shfl_xor(v, d), __shfl_xor(i, d));
    }
};

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        v += shfl_xor(v, d);
    return v;
}

// A token by one wavefront in 64 bits. c: E doubles of LDS, the wavefront's own.
__device__ __forceinline__ void route_exact(const RouteArgs& a, int64_t t, double* c)
{
    const int lane = threadIdx.x & 63;
    const float* l = a.logits + t * a.E;
    double m = 0.0, z = 1.0;
    if (a.score == MOE_SCORE_SOFTMAX) {
        float top = -INFINITY;
        for (int e = lane; e < a.E; e += 64)
            top = fmaxf(top, l[e]);
        top = group_max<64>(top);
        m = top == -INFINITY ? 0.0 : (double)top;
        double sum = 0.0;
        for (int e = lane; e < a.E; e += 64)
            sum += exp((double)l[e] - m);
        z = wave_sum(sum);
    }
    const auto score_of = [&](float x) {
        if (a.score == MOE_SCORE_SOFTMAX)
            return x == -INFINITY ? 0.0 : exp((double)x - m) / z;
        return 1.0 / (1.0 + exp(-(double)x));
    };
    for (int e = lane; e < a.E; e += 64) {
        const float x = l[e];
        double v = score_of(x) + (a.bias ? (double)a.bias[e] : 0.0);
        if (x == -INFINITY || !(v == v))
            v = -INFINITY;
        c[e] = v;
    }
    __syncthreads();
    const int per = a.E / a.groups;
    uint64_t open = ~0ull;                                    // a bit for each kept group
    if (a.groups > 1) {
        double sum = -INFINITY;
        if (lane < a.groups) {
            // the group's `top` largest, each the best behind the one before
            double prev = INFINITY;
            int at = -1;
            sum = 0.0;
            for (int j = 0; j < a.top; ++j) {
                Best b = {-INFINITY, 1 << 20};
                for (int i = 0; i < per; ++i) {
                    const double v = c[lane * per + i];
                    if (v < prev || (v == prev && i > at))
                        b.take(v, i);
                }
                prev = b.v;
                at = b.i;
                sum += b.v;
            }
            if (!(sum == sum))
                sum = -INFINITY;
        }
        open = 0ull;
        bool taken = lane >= a.groups;
        for (int j = 0; j < a.kept; ++j) {
            Best b = {-INFINITY, 1 << 20};
            if (!taken)
                b.take(sum, lane);
            b.join_wave();
            open |= 1ull << b.i;
            taken = taken || lane == b.i;
        }
    }
    uint32_t gone = 0u;                                       // a bit for each of the lane's experts
    int mine = 0;
    for (int j = 0; j < a.k; ++j) {
        Best b = {-INFINITY, 1 << 20};
        for (int i = 0; lane + 64 * i < a.E; ++i) {
            const int e = lane + 64 * i;
            if (!(gone >> i & 1) && (open >> (a.groups > 1 ? e / per : 0) & 1))
                b.take(c[e], e);
        }
        b.join_wave();
        if ((b.i & 63) == lane)
            gone |= 1u << (b.i / 64);
        if (lane == j)
            mine = b.i;
    }
    const double s = lane < a.k ? score_of(l[mine]) : 0.0;
    const double sum = a.renorm ? wave_sum(s) : 1.0;
    if (lane < a.k) {
        a.idx[t * a.k + lane] = mine;
        a.w[t * a.k + lane] = (float)((sum == 0.0 ? 0.0 : s / sum) * (double)a.scale);
    }
}

__global__ __launch_bounds__(64) void k_route_scored(RouteArgs a)
{
    __shared__ double s_c[MOE_MAX_EXPERTS];
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        route_exact(a, t, s_c);
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------------- gradient --
struct ScoredGradArgs {
    const float* logits;
    const int32_t* idx;
    const float* dw;
    const float* add;
    int32_t T, E, k;
    float scale;
    float* out;
};

__device__ __forceinline__ float sigmoid_of(float x)
{
    const float e = exp_neg(-__builtin_fabsf(x));             // at most 1
    const float r = 1.0f / (1.0f + e);
    return x >= 0.0f ? r : e * r;                             // (a NaN takes the second)
}

// Softmax weights that are not renormalised: every expert's logit takes part. G lanes take a token;
// with q_e the sum of dw_j over the slots of expert e, put together in LDS of the group's own,
// dl_e = scale p_e (q_e - sum_i p_i q_i).
template <int G, int NV, int VEC>
__global__ __launch_bounds__(256) void k_scored_grad_all(ScoredGradArgs a)
{
    const int tid = threadIdx.x, g = tid & (G - 1);
    __shared__ __attribute__((aligned(16))) float s_row[256 * NV * VEC];
    float* row = s_row + tid / G * (G * NV * VEC);
    const int64_t groups = (int64_t)gridDim.x * (256 / G);
    for (int64_t t = (int64_t)blockIdx.x * (256 / G) + tid / G; t < a.T; t += groups) {
        Row<G, NV, VEC> p, r;
        int32_t id = g < a.k ? a.idx[t * a.k + g] : -1;
        float dw = g < a.k ? a.dw[t * a.k + g] : 0.0f;
        p.load(a.logits + t * a.E, g, a.E);
        if (a.add)
            r.load(a.add + t * a.E, g, a.E);
        softmax_row(p);
#pragma unroll
        for (int i = 0; i < NV * VEC; ++i)
            row[Row<G, NV, VEC>::expert(g, i)] = 0.0f;
        asm volatile("" ::: "memory");                        // LDS serves a wavefront in order
        if ((uint32_t)id < (uint32_t)a.E)
            __hip_atomic_fetch_add(row + id, dw, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        for (int j = g + G; j < a.k; j += G) {                // more slots than lanes
            id = a.idx[t * a.k + j];
            if ((uint32_t)id < (uint32_t)a.E)
                __hip_atomic_fetch_add(row + id, a.dw[t * a.k + j], __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_WORKGROUP);
        }
        asm volatile("" ::: "memory");
        float q[NV * VEC], dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NV * VEC; ++i) {
            q[i] = row[Row<G, NV, VEC>::expert(g, i)];
            dot = __builtin_fmaf(p.v[i], q[i], dot);
        }
        asm volatile("" ::: "memory");
        dot = group_sum<G>(dot);
#pragma unroll
        for (int i = 0; i < NV * VEC; ++i)
            r.v[i] = __builtin_fmaf(a.scale * p.v[i], q[i] - dot, a.add ? r.v[i] : 0.0f);
        r.store(a.out + t * a.E, g, a.E);
    }
}

// The other weights: only the chosen logits take part. With S the sum of the chosen scores and v_j =
// s_j / S, dl_j = scale v_j (dw_j - sum_i v_i dw_i), times 1 - s_j for the sigmoid; without the sum,
// dl_j = scale s_j (1 - s_j) dw_j. Scores go into the quotients relative to that of the largest
// chosen logit (for the sigmoid where that is negative), so that none of them vanishes. G lanes take a
// token, lane j the slots j, j + G, ...; the terms are added to the row in LDS of the group's own.
template <int G, int NV, int VEC, bool SIGMOID, bool RENORM>
__global__ __launch_bounds__(256) void k_scored_grad(ScoredGradArgs a)
{
    const int tid = threadIdx.x, g = tid & (G - 1);
    __shared__ __attribute__((aligned(16))) float s_row[256 * NV * VEC];
    float* row = s_row + tid / G * (G * NV * VEC);
    const int64_t groups = (int64_t)gridDim.x * (256 / G);
    struct Slot {
        int32_t id;
        float dw, x;
    };
    for (int64_t t = (int64_t)blockIdx.x * (256 / G) + tid / G; t < a.T; t += groups) {
        const auto slot = [&](int j) {
            Slot s = {-1, 0.0f, -INFINITY};
            if (j < a.k) {
                s.id = a.idx[t * a.k + j];
                s.dw = a.dw[t * a.k + j];
                if ((uint32_t)s.id < (uint32_t)a.E)
                    s.x = a.logits[t * a.E + s.id];
                else
                    s.id = -1;
            }
            return s;
        };
        Row<G, NV, VEC> r;
        if (a.add) {
            r.load(a.add + t * a.E, g, a.E);
        } else {
#pragma unroll
            for (int i = 0; i < NV * VEC; ++i)
                r.v[i] = 0.0f;
        }
        const Slot first = slot(g);
#pragma unroll
        for (int i = 0; i < NV * VEC; ++i)
            row[Row<G, NV, VEC>::expert(g, i)] = r.v[i];
        float top = 0.0f, inv = 1.0f, dot = 0.0f;
        const auto share = [&](const Slot& s) {               // v_j but for the sum
            if (!SIGMOID)
                return exp_neg(s.x - top);
            return top < 0.0f ? exp_neg(s.x - top) * sigmoid_of(-s.x) : sigmoid_of(s.x);
        };
        if (RENORM) {
            top = first.x;
            for (int j = g + G; j < a.k; j += G)
                top = fmaxf(top, slot(j).x);
            top = group_max<G>(top);
            top = top == -INFINITY ? 0.0f : top;
            float sum = 0.0f;
            if (first.id >= 0) {
                sum = share(first);
                dot = sum * first.dw;
            }
            for (int j = g + G; j < a.k; j += G) {
                const Slot s = slot(j);
                if (s.id >= 0) {
                    const float v = share(s);
                    sum += v;
                    dot = __builtin_fmaf(v, s.dw, dot);
                }
            }
            sum = group_sum<G>(sum);
            inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            dot = group_sum<G>(dot) * inv;
        }
        const auto term = [&](const Slot& s) {
            float d = a.scale * (RENORM ? share(s) * inv * (s.dw - dot) : sigmoid_of(s.x) * s.dw);
            return SIGMOID ? d * sigmoid_of(-s.x) : d;
        };
        asm volatile("" ::: "memory");                        // LDS serves a wavefront in order
        if (first.id >= 0)
            __hip_atomic_fetch_add(row + first.id, term(first), __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_WORKGROUP);
        for (int j = g + G; j < a.k; j += G) {                // more slots than lanes
            const Slot s = slot(j);
            if (s.id >= 0)
                __hip_atomic_fetch_add(row + s.id, term(s), __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_WORKGROUP);
        }
        asm volatile("" ::: "memory");
#pragma unroll
        for (int i = 0; i < NV * VEC; ++i)
            r.v[i] = row[Row<G, NV, VEC>::expert(g, i)];
        asm volatile("" ::: "memory");
        r.store(a.out + t * a.E, g, a.E);
    }
}

// --------------------------------------------------------------------------------- bias update --
__global__ __launch_bounds__(256) void k_bias_update(const float* bias,
                                                     const int32_t* __restrict__ counts, int32_t E,
                                                     float rate, float* out)
{
    __shared__ int64_t s_sum[4];
    const int tid = threadIdx.x;
    const int64_t row = (int64_t)blockIdx.x * E;
    int64_t sum = 0;
    for (int e = tid; e < E; e += 256)
        sum += counts[row + e];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        sum += __shfl_xor((long long)sum, d);
    if ((tid & 63) == 0)
        s_sum[tid >> 6] = sum;
    __syncthreads();
    sum = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
    for (int e = tid; e < E; e += 256) {
        const int64_t over = sum - (int64_t)E * counts[row + e];
        out[row + e] = bias[row + e] + (over > 0 ? rate : over < 0 ? -rate : 0.0f);
    }
}

template <int G, int NV, int VEC>
void launch_grad(Row<G, NV, VEC>, const ScoredGradArgs& a, int score, bool renorm, hipStream_t stream)
{
    const int64_t need = div_up(a.T, 256 / G), most = 4096;
    const unsigned blocks = (unsigned)(need < most ? need : most);
    if (score == MOE_SCORE_SOFTMAX && !renorm)
        k_scored_grad_all<G, NV, VEC><<<blocks, 256, 0, stream>>>(a);
    else if (score == MOE_SCORE_SOFTMAX)
        k_scored_grad<G, NV, VEC, false, true><<<blocks, 256, 0, stream>>>(a);
    else if (renorm)
        k_scored_grad<G, NV, VEC, true, true><<<blocks, 256, 0, stream>>>(a);
    else
        k_scored_grad<G, NV, VEC, true, false><<<blocks, 256, 0, stream>>>(a);
}

inline moe_status_t launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

moe_status_t check_sizes(int32_t T, int32_t E, int32_t k, int32_t score, float scale)
{
    if (T < 0 || E < 1 || k < 1 || (int64_t)T * k > INT32_MAX || !(scale - scale == 0.0f) ||
        (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID))
        return MOE_ERR_INVALID;
    if (E > MOE_MAX_EXPERTS || k > MOE_MAX_TOPK)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace

extern "C" {

moe_status_t moe_route_scored(const float* logits, const float* bias, int32_t T, int32_t E,
                              int32_t k, moe_score_t score, int32_t n_groups, int32_t topk_groups,
                              int32_t group_top, int32_t renormalize, float scale,
                              int32_t* topk_idx, float* topk_w, hipStream_t stream)
{
    const moe_status_t st = check_sizes(T, E, k, score, scale);
    if (st == MOE_ERR_INVALID || n_groups < 1 || E % n_groups != 0 || topk_groups < 1 ||
        topk_groups > n_groups || (n_groups > 1 && (group_top < 1 || group_top > E / n_groups)) ||
        k > (int64_t)topk_groups * (E / n_groups))
        return MOE_ERR_INVALID;
    if (st != MOE_OK || n_groups > MOE_MAX_GROUPS)
        return MOE_ERR_UNSUPPORTED;
    if (T > 0 && (!logits || !topk_idx || !topk_w))
        return MOE_ERR_INVALID;
    if (!aligned_to(logits, 4) || !aligned_to(bias, 4) || !aligned_to(topk_idx, 4) ||
        !aligned_to(topk_w, 4))
        return MOE_ERR_UNSUPPORTED;
    if (T == 0)
        return MOE_OK;
    RouteArgs a = {logits, bias, T, E, k, score, n_groups, topk_groups, group_top, renormalize != 0,
                   scale, topk_idx, topk_w};
    const int32_t most = 1 << 16;
    k_route_scored<<<(unsigned)(T < most ? T : most), 64, 0, stream>>>(a);
    return launched();
}

moe_status_t moe_route_scored_grad(const float* logits, const int32_t* topk_idx,
                                   const float* dtopk_w, const float* add, int32_t T, int32_t E,
                                   int32_t k, moe_score_t score, int32_t renormalize, float scale,
                                   float* dlogits, hipStream_t stream)
{
    const moe_status_t st = check_sizes(T, E, k, score, scale);
    if (st != MOE_OK)
        return st;
    if (T > 0 && (!logits || !topk_idx || !dtopk_w || !dlogits))
        return MOE_ERR_INVALID;
    if (!aligned_to(logits, 4) || !aligned_to(topk_idx, 4) || !aligned_to(dtopk_w, 4) ||
        !aligned_to(add, 4) || !aligned_to(dlogits, 4))
        return MOE_ERR_UNSUPPORTED;
    if (T == 0)
        return MOE_OK;
    const ScoredGradArgs a = {logits, topk_idx, dtopk_w, add, T, E, k, scale, dlogits};
    with_row(E, E % 4 == 0 && aligned_to(logits, 16) && aligned_to(add, 16) && aligned_to(dlogits, 16),
             [&](auto row) { launch_grad(row, a, score, renormalize != 0, stream); });
    return launched();
}

moe_status_t moe_bias_update(const float* bias, const int32_t* expert_counts, int32_t L, int32_t E,
                             float rate, float* out, hipStream_t stream)
{
    if (L < 0 || E < 1)
        return MOE_ERR_INVALID;
    if (E > MOE_MAX_EXPERTS || L > INT32_MAX / 256)
        return MOE_ERR_UNSUPPORTED;
    if (L > 0 && (!bias || !expert_counts || !out))
        return MOE_ERR_INVALID;
    if (!aligned_to(bias, 4) || !aligned_to(expert_counts, 4) || !aligned_to(out, 4))
        return MOE_ERR_UNSUPPORTED;
    if (L == 0)
        return MOE_OK;
    k_bias_update<<<(unsigned)L, 256, 0, stream>>>(bias, expert_counts, E, rate, out);
    return launched();
}

}  // extern "C"
