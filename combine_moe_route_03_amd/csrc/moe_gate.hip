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
// Scores and choices are made in 64 bits (an fp64 instruction takes as long as an fp32 one here), so that
// the order of the choices is that of the definition and the weights are rounded once. G lanes take a
// token, lane g the experts g, g + G, ...; T tokens of E experts are read once, and past small batches the
// vector instructions bound it, most of them the exponentials (about 25 each) and the k rounds.

// exp(x) = 2^n exp(r), |r| <= ln 2 / 2, by the series to r^12, which leaves out less than 2^-52. NEAR: for
// |x| <= kNear only, where 2^n is an addition to the exponent's bits; else 0 below -800 and infinity
// above 800.
constexpr double kNear = 690.0;

template <bool NEAR>
__device__ __forceinline__ double exp_wide(double x)
{
    constexpr double kWhole = 6755399441055744.0;             // 1.5 * 2^52: n stands in the low bits
    if (!NEAR)
        x = fmin(fmax(x, -800.0), 800.0);
    const double t = __builtin_fma(x, 1.4426950408889634, kWhole), n = t - kWhole;
    const double r = __builtin_fma(-n, 2.3190468138462996e-17, __builtin_fma(-n, 0.6931471805599453, x));
    double p = 1.0 / 479001600.0;
    constexpr double c[] = {1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0, 1.0 / 40320.0,
                            1.0 / 5040.0, 1.0 / 720.0, 1.0 / 120.0, 1.0 / 24.0, 1.0 / 6.0, 0.5, 1.0, 1.0};
#pragma unroll
    for (int i = 0; i < 12; ++i)
        p = __builtin_fma(p, r, c[i]);
    const int whole = (int)(uint32_t)__double_as_longlong(t);
    if (!NEAR)
        return ldexp(p, whole);
    return __longlong_as_double(__double_as_longlong(p) + ((long long)whole << 52));
}

// 1 / d for 1 <= d < 2^1000: two steps of Newton's from v_rcp_f64's 2^-26 or so.
__device__ __forceinline__ double reciprocal(double d)
{
    double r = __builtin_amdgcn_rcp(d);
    r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
    return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v)
{
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    return __longlong_as_double(
        (long long)((uint64_t)dpp_u32<CTRL>((uint32_t)(b >> 32)) << 32 | dpp_u32<CTRL>((uint32_t)b)));
}

// Reductions over a group of 16 or 64 lanes, the result in each of them, in a fixed order: within 16
// lanes by DPP, beyond by shuffles.
template <int G, typename Op>
__device__ __forceinline__ uint32_t reduce_u32(uint32_t v, Op op)
{
    v = op(v, dpp_u32<0xB1>(v));
    v = op(v, dpp_u32<0x4E>(v));
    v = op(v, dpp_u32<0x141>(v));
    v = op(v, dpp_u32<0x140>(v));
    if (G == 64) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = op(r[0], r[1]);
        const auto q = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = op(q[0], q[1]);
    }
    return v;
}

template <int G, typename Op>
__device__ __forceinline__ double reduce_f64(double v, Op op)
{
    v = op(v, dpp_f64<0xB1>(v));
    v = op(v, dpp_f64<0x4E>(v));
    v = op(v, dpp_f64<0x141>(v));
    v = op(v, dpp_f64<0x140>(v));
    if (G == 64) {
        v = op(v, __shfl_xor(v, 16));
        v = op(v, __shfl_xor(v, 32));
    }
    return v;
}

// Floats as unsigned integers of the same order, all above 0.
__device__ __forceinline__ uint32_t ordered(float v)
{
    const uint32_t u = __float_as_uint(v);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// This group's bits of a ballot.
template <int G>
__device__ __forceinline__ uint64_t group_ballot(bool b)
{
    const uint64_t all = __ballot(b);
    return G == 64 ? all : all >> (threadIdx.x & 48) & 0xFFFFu;
}

// Maximum and minimum of two numbers that are no NaN, one instruction each (the compiler makes sure of that
// with two more for every operand from memory).
__device__ __forceinline__ double larger(double u, double v)
{
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(u), "v"(v));
    return r;
}

__device__ __forceinline__ double smaller(double u, double v)
{
    double r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(u), "v"(v));
    return r;
}

// Choices behind every other (masked experts), and those that take no part.
constexpr double kBehind = -1.7976931348623157e308;

// Experts of kept groups among G lanes' c (in LDS, group by group with a double between, which spreads
// the lanes' reads over the banks): a bit for each group.
template <int G>
__device__ __forceinline__ uint64_t kept_groups(const RouteArgs& a, const double* c, double* score)
{
    const int g = threadIdx.x & (G - 1), per = a.E / a.groups;
    double sum = -INFINITY;
    if (g < a.groups) {
        const double* mine = c + g * (per + 1);
        if (a.top <= 2) {
            double t1 = -INFINITY, t2 = -INFINITY;
            const auto take = [&](double v) {
                t2 = larger(t2, smaller(t1, v));
                t1 = larger(t1, v);
            };
            int i = 0;
            for (; i + 8 <= per; i += 8) {
                double v[8];
#pragma unroll
                for (int n = 0; n < 8; ++n)
                    v[n] = mine[i + n];
#pragma unroll
                for (int n = 0; n < 8; ++n)
                    take(v[n]);
            }
            for (; i < per; ++i)
                take(mine[i]);
            sum = a.top == 1 ? t1 : t1 + t2;
        } else {                                              // each the best behind the one before
            double prev = INFINITY;
            int at = -1;
            sum = 0.0;
            for (int j = 0; j < a.top; ++j) {
                double best = -INFINITY;
                int where = per;
                for (int i = 0; i < per; ++i) {
                    const double v = mine[i];
                    if ((v < prev || (v == prev && i > at)) && (v > best || where == per)) {
                        best = v;
                        where = i;
                    }
                }
                prev = best;
                at = where;
                sum += best;
            }
        }
        sum = sum > -1e300 ? sum : kBehind;                   // with a masked expert: behind the others
        score[g] = sum;
    }
    asm volatile("" ::: "memory");                            // LDS serves a wavefront in order
    int rank = 0;
    for (int j = 0; j < a.groups; ++j) {
        const double v = score[j];
        rank += v > sum || (v == sum && j < g);
    }
    asm volatile("" ::: "memory");
    return group_ballot<G>(g < a.groups && rank < a.kept);
}

// P experts a lane. The k rounds go by 27 bits of c as fp32 and 5 of the lane's expert number, which makes
// a lane's keys different, and by the three largest of each lane, so that a round is a maximum over lanes.
// What they chose is held against the choices in 64 bits: the order of the chosen, and that no other one
// comes before the last. Where that fails (two choices within 2^-19 of each other, or more than three of
// the chosen with one lane: a token in 100 for 8 of 256) the rounds run again in 64 bits. Clearing a chosen
// key among all of a lane's and taking their maximum again, round by round: a tenth more
// instructions (256 experts, 16384 tokens: 22.5 us for 21).
template <int G, int P>
__global__ __launch_bounds__(256) void k_route_scored(RouteArgs a)
{
    static_assert(P <= 32 && (G == 16 || G == 64), "five bits; rows of DPP");
    extern __shared__ double s_choice[];                      // [256 / G][E + groups + 1], [256 / G][groups]
    const int tid = threadIdx.x, g = tid & (G - 1);
    const int64_t t = (int64_t)blockIdx.x * (256 / G) + tid / G;
    const bool valid = t < a.T;
    const float* l = a.logits + (valid ? t : 0) * a.E;
    const int stride = a.E + a.groups + 1;
    double* lc = s_choice + tid / G * stride;
    const int per = a.E / a.groups;
    const uint32_t magic = ((1u << 20) + per - 1) / per;      // e / per for e < 1024
    float x[P], b[P];                                         // read without a branch each
#pragma unroll
    for (int p = 0; p < P; ++p)
        x[p] = l[min(g + G * p, a.E - 1)];
#pragma unroll
    for (int p = 0; p < P; ++p)
        b[p] = a.bias ? a.bias[min(g + G * p, a.E - 1)] : 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p)
        x[p] = g + G * p < a.E ? x[p] : -INFINITY;
    double c[P], m = 0.0, z = 1.0;
    if (a.score == MOE_SCORE_SOFTMAX) {
        float top = -INFINITY;
#pragma unroll
        for (int p = 0; p < P; ++p)
            top = fmaxf(top, x[p]);
        top = group_max<G>(top);
        m = top == -INFINITY ? 0.0 : (double)top;
    }
    bool far = false;                                         // NaN among it
#pragma unroll
    for (int p = 0; p < P; ++p)
        far = far || (!(fabs((double)x[p] - m) <= kNear) && x[p] != -INFINITY);
    far = __any(far);
    if (a.score == MOE_SCORE_SOFTMAX) {
        double sum = 0.0;
        if (__builtin_expect(!far, 1)) {
#pragma unroll
            for (int p = 0; p < P; ++p)
                c[p] = exp_wide<true>(x[p] == -INFINITY ? 0.0 : (double)x[p] - m);
        } else {
#pragma unroll
            for (int p = 0; p < P; ++p)
                c[p] = exp_wide<false>((double)x[p] - m);
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
            c[p] = x[p] == -INFINITY ? 0.0 : c[p];
            sum += c[p];
        }
        sum = reduce_f64<G>(sum, [](double u, double v) { return u + v; });
        z = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
        for (int p = 0; p < P; ++p)
            c[p] *= z;
    } else if (__builtin_expect(!far, 1)) {
#pragma unroll
        for (int p = 0; p < P; ++p)
            c[p] = reciprocal(1.0 + exp_wide<true>(x[p] == -INFINITY ? 0.0 : -(double)x[p]));
    } else {
#pragma unroll
        for (int p = 0; p < P; ++p)
            c[p] = 1.0 / (1.0 + exp_wide<false>(-(double)x[p]));
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int e = g + G * p;
        c[p] += (double)b[p];
        c[p] = x[p] == -INFINITY || !(c[p] >= kBehind) ? kBehind : fmin(c[p], -kBehind);
        c[p] = e < a.E ? c[p] : -INFINITY;
        lc[e < a.E ? e + (int)((uint32_t)e * magic >> 20) : stride - 1] = c[p];   // (the last: unused)
    }
    asm volatile("" ::: "memory");
    if (a.groups > 1) {
        const uint64_t open = kept_groups<G>(a, lc, s_choice + 256 / G * stride + tid / G * a.groups);
#pragma unroll
        for (int p = 0; p < P; ++p)
            if (!(open >> ((uint32_t)(g + G * p) * magic >> 20 & 63) & 1))
                c[p] = -INFINITY;
    }
    uint32_t best[3] = {0u, 0u, 0u};                          // the lane's, largest first
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const uint32_t key = c[p] == -INFINITY ? 0u : (ordered((float)c[p]) & ~31u) | (31 - p);
        best[2] = max(best[2], min(best[1], key));
        best[1] = max(best[1], min(best[0], key));
        best[0] = max(best[0], key);
    }
    int mine = 0;                                             // lane j: the expert of slot j
    bool wrong = false;
    for (int j = 0; j < a.k; ++j) {
        const uint32_t top = reduce_u32<G>(best[0], [](uint32_t u, uint32_t v) { return max(u, v); });
        const int w = __ffsll((unsigned long long)group_ballot<G>(best[0] == top)) - 1;
        wrong = wrong || top == 0u;
        if (g == j && top != 0u)
            mine = w + G * (31 - (int)(top & 31u));
        const bool pop = g == w;
        best[0] = pop ? best[1] : best[0];
        best[1] = pop ? best[2] : best[1];
        best[2] = pop ? 0u : best[2];
    }
    const auto choice_of = [&](int e) { return lc[e + (int)((uint32_t)e * magic >> 20)]; };
    const double chosen = g < a.k ? choice_of(mine) : 0.0;
    const double next = __shfl(chosen, (tid & 63) + 1), last = __shfl(chosen, (tid & 63 & ~(G - 1)) + a.k - 1);
    const int next_id = __shfl(mine, (tid & 63) + 1), last_id = __shfl(mine, (tid & 63 & ~(G - 1)) + a.k - 1);
    wrong = wrong || (g < a.k - 1 && !(chosen > next || (chosen == next && mine < next_id)));
    int before = 0;
#pragma unroll
    for (int p = 0; p < P; ++p)
        before += c[p] > last || (c[p] == last && g + G * p < last_id);
    before = (int)reduce_u32<G>((uint32_t)before, [](uint32_t u, uint32_t v) { return u + v; });
    wrong = wrong || before != a.k - 1;
    if (__builtin_expect(__any(wrong), 0)) {                  // by 64 bits, every token of the wavefront
        uint32_t gone = 0u;
        for (int j = 0; j < a.k; ++j) {
            double best = -INFINITY;
            int at = -1;
#pragma unroll
            for (int p = 0; p < P; ++p)
                if (!(gone >> p & 1) && c[p] > best) {
                    best = c[p];
                    at = p;
                }
            const double top = reduce_f64<G>(best, [](double u, double v) { return fmax(u, v); });
            const uint32_t id = reduce_u32<G>(at >= 0 && best == top ? (uint32_t)(g + G * at) : 0xFFFFFFFFu,
                                              [](uint32_t u, uint32_t v) { return min(u, v); });
            if (g == j)
                mine = (int)id;
            if (at >= 0 && id == (uint32_t)(g + G * at))
                gone |= 1u << at;
        }
    }
    double s = 0.0;
    if (g < a.k) {
        const float lx = l[mine];
        if (a.score == MOE_SCORE_SOFTMAX)
            s = lx == -INFINITY ? 0.0 : exp_wide<false>((double)lx - m) * z;
        else
            s = 1.0 / (1.0 + exp_wide<false>(-(double)lx));
    }
    double sum = 1.0;
    if (a.renorm)
        sum = reduce_f64<G>(s, [](double u, double v) { return u + v; });
    if (valid && g < a.k) {
        a.idx[t * a.k + g] = mine;
        a.w[t * a.k + g] = (float)((sum == 0.0 ? 0.0 : s / sum) * (double)a.scale);
    }
}

// A launch takes 2^31 threads: from 2^32 on the runtime takes the number of threads modulo 2^32, without an
// error. 2^27 tokens of 16 lanes, 2^25 of 64.
template <int G, int P>
void launch_route(RouteArgs a, hipStream_t stream)
{
    constexpr int32_t kTokens = (1 << 23) * (256 / G);
    const size_t lds = (size_t)(256 / G) * (a.E + 2 * a.groups + 1) * sizeof(double);
    int32_t left = a.T;
    for (; left > kTokens; left -= kTokens) {
        a.T = kTokens;
        k_route_scored<G, P><<<kTokens / (256 / G), 256, lds, stream>>>(a);
        a.logits += (int64_t)kTokens * a.E;
        a.idx += (int64_t)kTokens * a.k;
        a.w += (int64_t)kTokens * a.k;
    }
    a.T = left;
    k_route_scored<G, P><<<(unsigned)div_up(left, 256 / G), 256, lds, stream>>>(a);
}

// 16 lanes a token take two thirds of the instructions, or half, of a wavefront a token, which spreads few
// tokens over more SIMDs: 64 experts, 8 chosen, 4096 tokens 6.0 and 5.9 us, 65536 22 and 52; 160 experts
// in groups 8.1 and 8.9, 43 and 85; 256 experts in groups 11.3 and 9.8, 16384 tokens 24 and 29; 384
// experts, 65536 tokens 89 and 92.
constexpr int32_t kWideTokens = 4096;

void launch_route(const RouteArgs& a, hipStream_t stream)
{
    if (a.T >= (a.E <= 160 ? kWideTokens : 2 * kWideTokens) && a.E <= 256 && a.k <= 16 && a.groups <= 16) {
        if (a.E <= 32) launch_route<16, 2>(a, stream);
        else if (a.E <= 64) launch_route<16, 4>(a, stream);
        else if (a.E <= 128) launch_route<16, 8>(a, stream);
        else if (a.E <= 160) launch_route<16, 10>(a, stream);
        else launch_route<16, 16>(a, stream);
        return;
    }
    if (a.E <= 64) launch_route<64, 1>(a, stream);
    else if (a.E <= 128) launch_route<64, 2>(a, stream);
    else if (a.E <= 256) launch_route<64, 4>(a, stream);
    else if (a.E <= 384) launch_route<64, 6>(a, stream);
    else if (a.E <= 512) launch_route<64, 8>(a, stream);
    else launch_route<64, 16>(a, stream);
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
// dl_e = scale p_e (q_e - sum_i p_i q_i). That difference is small for the first expert of a token that is
// sure of it (p 1 - 1e-6: 1e-6 q), so q counts from that expert's, which leaves the others' part of the sum:
// with c the q of the p over 1/2, if there is one, it is (q_e - c) - sum_i p_i (q_i - c). Logits are read once
// and the gradient is written once, with p made again from them in fp32: 65536 tokens of 256 experts, 8
// chosen, 21.2 to 22.2 us, 6.5 to 6.2 TB/s, HBM's rate.
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
        float q[NV * VEC], dot = 0.0f, from = 0.0f;
#pragma unroll
        for (int i = 0; i < NV * VEC; ++i) {
            q[i] = row[Row<G, NV, VEC>::expert(g, i)];
            from += p.v[i] > 0.5f ? q[i] : 0.0f;
        }
        asm volatile("" ::: "memory");
        from = group_sum<G>(from);
#pragma unroll
        for (int i = 0; i < NV * VEC; ++i) {
            q[i] -= from;
            dot = __builtin_fmaf(p.v[i], q[i], dot);
        }
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
// chosen logit (for the sigmoid where that is negative), so that none of them vanishes, and dw counts
// from that of the v over 1/2, if there is one, as above. G lanes take a token, lane j the slots j, j + G,
// ...; the terms are added to the row in LDS of the group's own, which is written whole, zeros and all. Its
// writes and a chain of two loads (ids, then their logits) bound it: 4096 tokens of 384 experts with a
// gradient to add 4.4 us, 2.9 TB/s, most of it in the Infinity Cache.
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
        float top = 0.0f, inv = 1.0f, dot = 0.0f, from = 0.0f;
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
            const float v = first.id >= 0 ? share(first) : 0.0f;
            float sum = v;
            for (int j = g + G; j < a.k; j += G) {
                const Slot s = slot(j);
                if (s.id >= 0)
                    sum += share(s);
            }
            sum = group_sum<G>(sum);
            inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            from = v * inv > 0.5f ? first.dw : 0.0f;
            for (int j = g + G; j < a.k; j += G) {
                const Slot s = slot(j);
                if (s.id >= 0 && share(s) * inv > 0.5f)
                    from += s.dw;
            }
            from = group_sum<G>(from);
            dot = first.id >= 0 ? v * (first.dw - from) : 0.0f;
            for (int j = g + G; j < a.k; j += G) {
                const Slot s = slot(j);
                if (s.id >= 0)
                    dot = __builtin_fmaf(share(s), s.dw - from, dot);
            }
            dot = group_sum<G>(dot) * inv;
        }
        const auto term = [&](const Slot& s) {
            float d = a.scale * (RENORM ? share(s) * inv * (s.dw - from - dot) : sigmoid_of(s.x) * s.dw);
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
// bias + rate sign(mean count - count), a workgroup a layer: E count against the sum of counts, in 64-bit
// integers, so that the sign is exact. A launch and two chained loads: 2.0 us for a layer of 384 experts,
// 4.8 for 48 layers of 256.
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
    launch_route(a, stream);
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
