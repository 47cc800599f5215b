// moe_balance.hip -- the router's balance loss, its per-expert counts, and the gradient of the
// router's logits (declared in include/moe_layer.h).
//
// For a sequence of n tokens with kept-slot counts c_e and probability sums P_e = sum_t p_te,
//   loss = alpha / S * E / (k n^2) * sum_e c_e P_e,   d loss / d l_te = f p_te (c_e - sum_i c_i p_ti)
// with f = alpha / S * E / (k n^2), since d p_i / d l_e = p_i (delta_ie - p_e). The forward pass
// reads the logits once, the backward pass reads them again (4 bytes an element, against writing
// and reading the probabilities) and writes the gradient once. Small batches are bound by their
// launches, long ones by the vector instructions next to HBM: of 256 experts a token takes 93 in the
// forward pass and 245 in the backward one with the weights' part, which keeps the SIMDs busy for 11
// of its 16 us and for 28 of its 31 us (65536 tokens, k = 8).
#include "moe_layer.h"
#include "moe_rows.h"

namespace {

using namespace moe_dev;

constexpr int kLossThreads = 1024;
constexpr int kLossWaves = kLossThreads / 64;
constexpr int kGradThreads = 256;
constexpr int kMaxLossBlocks = 512;      // workgroups of the forward pass, two a CU
constexpr int kLossTokens = 32;          //   of no fewer tokens than two a wavefront
// One workgroup and one launch up to so many tokens: a token costs its 93 instructions on one CU
// (256 experts: 0.038 us), a second launch about 4 us of the GPU and 3 of the host. us by one launch
// and by two, launches alone: 64 tokens 4.2 and 8.0 (64 experts), 5.8 and 8.7 (256), 9.2 and 11.0
// (1024); 192 tokens 5.2 and 8.2, 11.1 and 9.1, 19.8 and 11.1. (With more than 64 experts the limit by
// these figures would be lower, with fewer higher.)
constexpr int kDirectTokens = 192;
constexpr int kFinishExperts = 32;       // experts of a finishing workgroup
constexpr int kFinishThreads = 512;      //   by 16 slices of the partial sums
constexpr int kFinishSlices = kFinishThreads / kFinishExperts;

struct LossArgs {
    const float* logits;
    const int32_t* idx;
    const uint8_t* mask;
    int32_t L;                // tokens of a sequence
    int32_t E, k, S;
    int32_t nb;               // workgroups of a sequence
    int32_t chunk;            // tokens of a workgroup
    float* part_sum;          // [S * nb, E]
    int32_t* part_count;      // [S * nb, E]
    int32_t* part_tokens;     // [S * nb]
    double* part_loss;        // [S * finishing workgroups of a sequence]
    uint32_t* ticket;
    float alpha;
    float* loss;
    int32_t* counts;
    float* sums;
    int32_t* tokens;
};

// The loss's factor of a sequence: alpha / S * E / (k n^2), 0 for a sequence of padding.
__device__ __forceinline__ double seq_factor(float alpha, int32_t S, int32_t E, int32_t k,
                                             int32_t n)
{
    return n > 0 ? (double)alpha * E / ((double)S * k * ((double)n * n)) : 0.0;
}

// One workgroup sums a chunk of one sequence's tokens: every group of G lanes takes a token at a
// time and keeps its experts' sums in registers, LDS joins the groups in a fixed order, and integer
// LDS atomics count the chunk's ids (their order changes nothing). DIRECT: the only workgroup of
// the call finishes the loss itself.
template <int G, int NV, int VEC, bool DIRECT>
__global__ __launch_bounds__(kLossThreads) void k_balance_partial(LossArgs a)
{
    constexpr int kGroups = kLossThreads / G;
    constexpr int kPer = 64 / G;                      // groups of a wavefront
    extern __shared__ float lds[];
    float* red = lds;                                 // [kLossWaves, E]
    int32_t* hist = reinterpret_cast<int32_t*>(lds + kLossWaves * a.E);
    __shared__ int32_t s_tokens;
    __shared__ double s_loss[kLossWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int g = lane & (G - 1), grp = tid / G;
    const int s = blockIdx.x / a.nb, b = blockIdx.x % a.nb;
    const int64_t first = (int64_t)s * a.L + (int64_t)b * a.chunk;
    const int n = min(a.chunk, a.L - b * a.chunk);    // at least one, or the whole batch is empty
    if (!DIRECT && blockIdx.x == 0 && tid == 0)
        *a.ticket = 0u;
    for (int e = tid; e < a.E; e += kLossThreads)
        hist[e] = 0;
    if (tid == 0)
        s_tokens = 0;
    __syncthreads();

    const int64_t items = (int64_t)n * a.k;
    for (int64_t i = tid; i < items; i += kLossThreads) {
        const int32_t e = a.idx[first * a.k + i];
        if ((uint32_t)e < (uint32_t)a.E && (!a.mask || a.mask[first + i / a.k]))
            atomicAdd(&hist[e], 1);
    }

    Row<G, NV, VEC> sum;
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i)
        sum.v[i] = 0.0f;
    int seen = 0;
    // rows in flight; two workgroups a CU leave 64 registers
    constexpr int U = (DIRECT ? 2 : 1) * (NV * VEC <= 4 ? 4 : NV * VEC <= 8 ? 2 : 1);
    for (int t0 = grp; t0 < n; t0 += U * kGroups) {
        Row<G, NV, VEC> r[U];
        bool use[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + u * kGroups;
            use[u] = t < n && (!a.mask || a.mask[first + t]);
            if (use[u])
                r[u].load(a.logits + (first + t) * a.E, g, a.E);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!use[u])
                continue;
            softmax_row(r[u]);
#pragma unroll
            for (int i = 0; i < NV * VEC; ++i)
                sum.v[i] += r[u].v[i];
            ++seen;
        }
    }
    if (g == 0 && seen)
        atomicAdd(&s_tokens, seen);
    // groups of a wavefront (lanes G apart hold the same experts), then the wavefronts through LDS
#pragma unroll
    for (int d = 1; d < kPer; d <<= 1) {
#pragma unroll
        for (int i = 0; i < NV * VEC; ++i)
            sum.v[i] += __shfl_xor(sum.v[i], d * G);
    }
    if (lane < G) {
#pragma unroll
        for (int i = 0; i < NV * VEC; ++i) {
            const int e = Row<G, NV, VEC>::expert(g, i);
            if (e < a.E)
                red[wave * a.E + e] = sum.v[i];
        }
    }
    __syncthreads();
    const int tokens = s_tokens;
    double dot = 0.0;
    for (int e = tid; e < a.E; e += kLossThreads) {
        float p = 0.0f;
#pragma unroll
        for (int w = 0; w < kLossWaves; ++w)
            p += red[w * a.E + e];
        if (DIRECT) {
            a.sums[e] = p;
            a.counts[e] = hist[e];
            dot += (double)p * hist[e];
        } else {
            a.part_sum[(int64_t)blockIdx.x * a.E + e] = p;
            a.part_count[(int64_t)blockIdx.x * a.E + e] = hist[e];
        }
    }
    if (!DIRECT) {
        if (tid == 0)
            a.part_tokens[blockIdx.x] = tokens;
        return;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        dot += __shfl_xor(dot, d);
    if (lane == 0)
        s_loss[wave] = dot;
    __syncthreads();
    if (tid == 0) {
        double all = 0.0;
        for (int w = 0; w < kLossWaves; ++w)
            all += s_loss[w];
        a.loss[0] = (float)(all * seq_factor(a.alpha, 1, a.E, a.k, tokens));
        a.tokens[0] = tokens;
    }
}

// Sums the workgroups' parts of 32 experts of one sequence (16 slices side by side, joined in
// order, fp64) and its share of the loss; the last workgroup to finish adds the shares up in their
// order. The shares cross XCDs, whose L2s are not coherent, so they are stored and loaded at
// device scope.
__global__ __launch_bounds__(kFinishThreads) void k_balance_finish(LossArgs a, int32_t eb)
{
    __shared__ double s_sum[kFinishThreads];
    __shared__ int32_t s_count[kFinishThreads];
    __shared__ int32_t s_tokens;
    __shared__ bool s_last;
    const int tid = threadIdx.x;
    const int s = blockIdx.x / eb, c = blockIdx.x % eb;
    const int e = c * kFinishExperts + tid % kFinishExperts, slice = tid / kFinishExperts;
    int32_t tokens = 0;
    for (int b = tid; b < a.nb; b += kFinishThreads)
        tokens += a.part_tokens[(int64_t)s * a.nb + b];
    if (tid == 0)
        s_tokens = 0;
    double p = 0.0;
    int32_t n = 0;
    if (e < a.E) {
        const float* sum = a.part_sum + (int64_t)s * a.nb * a.E + e;
        const int32_t* count = a.part_count + (int64_t)s * a.nb * a.E + e;
        // eight parts in flight: up to 128 of them take one round
        for (int b0 = slice; b0 < a.nb; b0 += 8 * kFinishSlices) {
            float x[8];
            int32_t c[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t at = (int64_t)min(b0 + i * kFinishSlices, a.nb - 1) * a.E;
                x[i] = sum[at];
                c[i] = count[at];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (b0 + i * kFinishSlices < a.nb) {
                    p += x[i];
                    n += c[i];
                }
        }
    }
    s_sum[tid] = p;
    s_count[tid] = n;
    __syncthreads();
    if (tokens)
        atomicAdd(&s_tokens, tokens);
    __syncthreads();
    tokens = s_tokens;
    double dot = 0.0;
    if (tid < kFinishExperts && e < a.E) {
#pragma unroll 1
        for (int i = 1; i < kFinishSlices; ++i) {
            p += s_sum[i * kFinishExperts + tid];
            n += s_count[i * kFinishExperts + tid];
        }
        a.sums[(int64_t)s * a.E + e] = (float)p;
        a.counts[(int64_t)s * a.E + e] = n;
        dot = p * n;
    }
    __syncthreads();
    if (tid < kFinishExperts)
        s_sum[tid] = dot;
    __syncthreads();
    if (tid == 0) {
        double all = 0.0;
#pragma unroll 8
        for (int i = 0; i < kFinishExperts; ++i)
            all += s_sum[i];
        if (c == 0)
            a.tokens[s] = tokens;
        all *= seq_factor(a.alpha, a.S, a.E, a.k, tokens);
        __hip_atomic_store(&a.part_loss[blockIdx.x], all, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
        s_last = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_ACQ_REL,
                                        __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last)
        return;
    double all = 0.0;
    for (int64_t i = tid; i < (int64_t)gridDim.x; i += kFinishThreads)
        all += __hip_atomic_load(&a.part_loss[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    s_sum[tid] = all;
    __syncthreads();
    for (int d = kFinishThreads / 2; d; d >>= 1) {
        if (tid < d)
            s_sum[tid] += s_sum[tid + d];
        __syncthreads();
    }
    if (tid == 0)
        a.loss[0] = (float)s_sum[0];
}

__global__ __launch_bounds__(256) void k_balance_empty(LossArgs a)
{
    const int64_t n = (int64_t)a.S * a.E;
    for (int64_t i = blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        a.counts[i] = 0;
        a.sums[i] = 0.0f;
        if (i < a.S)
            a.tokens[i] = 0;
        if (i == 0)
            a.loss[0] = 0.0f;
    }
}

struct GradArgs {
    const float* logits;
    const int32_t* idx;
    const float* w;
    const float* dw;
    const uint8_t* mask;
    const int32_t* counts;
    const int32_t* tokens;
    const float* dloss;
    int32_t T, L, E, k, S;
    float alpha;
    float* out;
};

// G lanes take a token at a time: softmax of its logits, the two reductions, one store (past the
// caches: 65536 tokens of 256 experts 29 us against 38 with plain stores; two or four tokens in
// flight for a group cost more in occupancy than they hide, 33 and 48 us). The counts enter as
// c - m with the integer m nearest to the mean count k n / E: the probabilities add up to one, so m
// drops out, and the difference p (c - sum c p) loses nothing to cancellation (the plain difference
// loses log2(c / |c - mean|) bits). A group keeps its sequence's centred counts in registers while
// its tokens stay in the sequence.
//   The weights' term goes through LDS of the group's own: the row is put there, the lanes of the
// slots add theirs to it, and it is taken back (comparing every slot with every lane's experts in
// registers took 17 us more at 65536 tokens, k = 8).
template <int G, int NV, int VEC>
__global__ __launch_bounds__(kGradThreads) void k_route_grad(GradArgs a)
{
    const int tid = threadIdx.x;
    const int g = tid & (G - 1);
    __shared__ __attribute__((aligned(16))) float s_row[kGradThreads * NV * VEC];
    float* row = s_row + tid / G * (G * NV * VEC);
    const int64_t groups = (int64_t)gridDim.x * (kGradThreads / G);
    const float dloss = a.dloss ? a.dloss[0] : 1.0f;
    int cur = -1;
    float f = 0.0f;
    Row<G, NV, VEC> c;
    for (int64_t t = (int64_t)blockIdx.x * (kGradThreads / G) + tid / G; t < a.T; t += groups) {
        Row<G, NV, VEC> r;
        const bool slot = a.dw && g < a.k;
        int32_t id = slot ? a.idx[t * a.k + g] : -1;
        float w = slot ? a.w[t * a.k + g] : 0.0f;
        float dw = slot ? a.dw[t * a.k + g] : 0.0f;
        if (a.counts && (!a.mask || a.mask[t])) {
            r.load(a.logits + t * a.E, g, a.E);
            const int s = (int)((uint32_t)t / (uint32_t)a.L);
            if (s != cur) {
                cur = s;
                const int32_t n = a.tokens[s];
                const int32_t m = (int32_t)(((int64_t)a.k * n + a.E / 2) / a.E);
                f = (float)((double)dloss * seq_factor(a.alpha, a.S, a.E, a.k, n));
#pragma unroll
                for (int i = 0; i < NV * VEC; ++i) {
                    const int e = Row<G, NV, VEC>::expert(g, i);
                    c.v[i] = e < a.E ? (float)(a.counts[(int64_t)s * a.E + e] - m) : 0.0f;
                }
            }
            softmax_row(r);
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < NV * VEC; ++i)
                dot = __builtin_fmaf(c.v[i], r.v[i], dot);
            dot = group_sum<G>(dot);
#pragma unroll
            for (int i = 0; i < NV * VEC; ++i)
                r.v[i] = f * (r.v[i] * (c.v[i] - dot));
        } else {
#pragma unroll
            for (int i = 0; i < NV * VEC; ++i)
                r.v[i] = 0.0f;
        }
        if (a.dw) {
            float part = w * dw;
            for (int j = g + G; j < a.k; j += G)
                part = __builtin_fmaf(a.w[t * a.k + j], a.dw[t * a.k + j], part);
            const float all = group_sum<G>(part);
#pragma unroll
            for (int i = 0; i < NV * VEC; ++i)
                row[Row<G, NV, VEC>::expert(g, i)] = r.v[i];
            asm volatile("" ::: "memory");                    // LDS serves a wavefront in order
            if ((uint32_t)id < (uint32_t)a.E)
                __hip_atomic_fetch_add(row + id, w * (dw - all), __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_WORKGROUP);
            for (int j = g + G; j < a.k; j += G) {            // more slots than lanes
                id = a.idx[t * a.k + j];
                if ((uint32_t)id < (uint32_t)a.E)
                    __hip_atomic_fetch_add(row + id, a.w[t * a.k + j] * (a.dw[t * a.k + j] - all),
                                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
            }
            asm volatile("" ::: "memory");
#pragma unroll
            for (int i = 0; i < NV * VEC; ++i)
                r.v[i] = row[Row<G, NV, VEC>::expert(g, i)];
        }
        r.store(a.out + t * a.E, g, a.E);
    }
}

// Workgroups of a sequence, and their tokens: as many as fill the GPU, but chunks of no fewer than
// two tokens a wavefront; a small batch is one chunk.
struct LossPlan {
    int32_t nb, chunk;
    size_t sum, count, tokens, loss, ticket, bytes;
};

LossPlan loss_plan(int32_t T, int32_t E, int32_t S)
{
    LossPlan p;
    const int64_t L = T / S;
    int64_t nb = kMaxLossBlocks / (S < kMaxLossBlocks ? S : kMaxLossBlocks);
    if (nb > div_up(L, kLossTokens))
        nb = div_up(L, kLossTokens);
    if (nb < 1 || (S == 1 && L <= kDirectTokens))
        nb = 1;
    p.chunk = (int32_t)div_up(L > 0 ? L : 1, nb);
    p.nb = (int32_t)(L > 0 ? div_up(L, p.chunk) : 1);
    const auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
    const size_t parts = (size_t)S * p.nb;
    p.sum = 0;
    p.count = up(parts * E * 4);
    p.tokens = p.count + up(parts * E * 4);
    p.loss = p.tokens + up(parts * 4);
    p.ticket = p.loss + up((size_t)S * div_up(E, kFinishExperts) * 8);
    p.bytes = p.ticket + 256;
    return p;
}

template <int G, int NV, int VEC>
void launch_loss(Row<G, NV, VEC>, const LossArgs& a, hipStream_t stream)
{
    const size_t lds = (size_t)(kLossWaves + 1) * a.E * 4;
    if (a.S == 1 && a.nb == 1) {
        k_balance_partial<G, NV, VEC, true><<<1, kLossThreads, lds, stream>>>(a);
        return;
    }
    k_balance_partial<G, NV, VEC, false><<<(unsigned)(a.S * a.nb), kLossThreads, lds, stream>>>(a);
    const int32_t eb = (int32_t)div_up(a.E, kFinishExperts);
    k_balance_finish<<<(unsigned)((int64_t)a.S * eb), kFinishThreads, 0, stream>>>(a, eb);
}

template <int G, int NV, int VEC>
void launch_grad(Row<G, NV, VEC>, const GradArgs& a, hipStream_t stream)
{
    const int64_t blocks = div_up(a.T, kGradThreads / G);
    const int64_t most = 4096;
    k_route_grad<G, NV, VEC><<<(unsigned)(blocks < most ? blocks : most), kGradThreads, 0,
                               stream>>>(a);
}

moe_status_t check_batch(int32_t T, int32_t E, int32_t k, int32_t S)
{
    if (T < 0 || E < 1 || k < 1 || S < 1 || T % S != 0 || (int64_t)T * k > INT32_MAX)
        return MOE_ERR_INVALID;
    if (E > MOE_MAX_EXPERTS || k > MOE_MAX_TOPK || S > MOE_MAX_SEQS)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

moe_status_t launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

}  // namespace

extern "C" {

size_t moe_balance_workspace_bytes(int32_t T, int32_t E, int32_t n_seqs)
{
    return check_batch(T, E, 1, n_seqs) == MOE_OK ? loss_plan(T, E, n_seqs).bytes : 0;
}

moe_status_t moe_balance_loss(const float* logits, const int32_t* topk_idx,
                              const uint8_t* token_mask, int32_t T, int32_t E, int32_t k,
                              int32_t n_seqs, float alpha, float* loss, int32_t* expert_counts,
                              float* prob_sums, int32_t* seq_tokens, void* workspace,
                              size_t workspace_bytes, hipStream_t stream)
{
    const moe_status_t st = check_batch(T, E, k, n_seqs);
    if (st != MOE_OK)
        return st;
    if (!loss || !expert_counts || !prob_sums || !seq_tokens || (T > 0 && (!logits || !topk_idx)))
        return MOE_ERR_INVALID;
    const LossPlan p = loss_plan(T, E, n_seqs);
    if (!workspace || workspace_bytes < p.bytes)
        return MOE_ERR_WORKSPACE;
    if (!aligned_to((const char*)workspace, 16) || !aligned_to(logits, 4))
        return MOE_ERR_UNSUPPORTED;
    char* ws = static_cast<char*>(workspace);
    LossArgs a;
    a.logits = logits;
    a.idx = topk_idx;
    a.mask = token_mask;
    a.L = T / n_seqs;
    a.E = E;
    a.k = k;
    a.S = n_seqs;
    a.nb = p.nb;
    a.chunk = p.chunk;
    a.part_sum = reinterpret_cast<float*>(ws + p.sum);
    a.part_count = reinterpret_cast<int32_t*>(ws + p.count);
    a.part_tokens = reinterpret_cast<int32_t*>(ws + p.tokens);
    a.part_loss = reinterpret_cast<double*>(ws + p.loss);
    a.ticket = reinterpret_cast<uint32_t*>(ws + p.ticket);
    a.alpha = alpha;
    a.loss = loss;
    a.counts = expert_counts;
    a.sums = prob_sums;
    a.tokens = seq_tokens;
    if (T == 0)
        k_balance_empty<<<256, 256, 0, stream>>>(a);
    else
        with_row(E, E % 4 == 0 && aligned_to(logits, 16),
                 [&](auto row) { launch_loss(row, a, stream); });
    return launched();
}

moe_status_t moe_route_grad(const float* logits, const int32_t* topk_idx, const float* topk_w,
                            const float* dtopk_w, const uint8_t* token_mask,
                            const int32_t* expert_counts, const int32_t* seq_tokens,
                            const float* dloss, int32_t T, int32_t E, int32_t k, int32_t n_seqs,
                            float alpha, float* dlogits, hipStream_t stream)
{
    const moe_status_t st = check_batch(T, E, k, n_seqs);
    if (st != MOE_OK)
        return st;
    if (!expert_counts != !seq_tokens || !topk_w != !dtopk_w || (!expert_counts && !topk_w))
        return MOE_ERR_INVALID;
    if (T > 0 && (!dlogits || (expert_counts && !logits) || (topk_w && !topk_idx)))
        return MOE_ERR_INVALID;
    if (T == 0)
        return MOE_OK;
    GradArgs a;
    a.logits = logits;
    a.idx = topk_idx;
    a.w = topk_w;
    a.dw = dtopk_w;
    a.mask = token_mask;
    a.counts = expert_counts;
    a.tokens = seq_tokens;
    a.dloss = dloss;
    a.T = T;
    a.L = T / n_seqs;
    a.E = E;
    a.k = k;
    a.S = n_seqs;
    a.alpha = alpha;
    a.out = dlogits;
    with_row(E, E % 4 == 0 && aligned_to(logits, 16) && aligned_to(dlogits, 16),
             [&](auto row) { launch_grad(row, a, stream); });
    return launched();
}

}  // extern "C"
