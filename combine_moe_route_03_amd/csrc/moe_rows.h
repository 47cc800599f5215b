// moe_rows.h -- a row of logits in the registers of a group of lanes, and its softmax.
#ifndef MOE_ROWS_H
#define MOE_ROWS_H

#include "moe_device.h"

namespace moe_dev {

// A row of E fp32 values over the G lanes of a group: lane g holds elements (v * G + g) * VEC + c.
// Rows of other than a multiple of 4 experts, or not 16-byte aligned, take VEC = 1.
template <int G, int NV, int VEC>
struct Row {
    float v[NV * VEC];

    static __device__ __forceinline__ int expert(int g, int i)
    {
        return ((i / VEC) * G + g) * VEC + i % VEC;
    }

    __device__ __forceinline__ void load(const float* __restrict__ p, int g, int E)
    {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (i * G + g) * VEC;
            if (VEC == 4) {
                const f32x4 x = e < E ? *reinterpret_cast<const f32x4*>(p + e)
                                      : f32x4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    v[i * VEC + c] = x[c];
            } else {
                v[i] = e < E ? p[e] : -INFINITY;
            }
        }
    }

    __device__ __forceinline__ void store(float* __restrict__ p, int g, int E) const
    {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (i * G + g) * VEC;
            if (e >= E)
                continue;
            if (VEC == 4) {
                f32x4 x;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    x[c] = v[i * VEC + c];
                __builtin_nontemporal_store(x, reinterpret_cast<f32x4*>(p + e));
            } else {
                __builtin_nontemporal_store(v[i], p + e);
            }
        }
    }
};

// exp(x) for x <= 0 as 2^(x log2 e), log2 e in two parts: off by |x| 2^-24 for the product's
// rounding, and by one ulp of v_exp_f32. Results below 2^-126 are zero; next to the row's largest
// term, which is 1, they are nothing.
__device__ __forceinline__ float exp_neg(float x)
{
    return __builtin_amdgcn_exp2f(__builtin_fmaf(x, 1.44269502f, x * 1.92596299e-8f));
}

// Turns logits into probabilities in place. A row of -infinity only gets zeros; a NaN or +infinity
// makes the row NaN (the maximum ignores NaN, the sum does not).
template <int G, int NV, int VEC>
__device__ __forceinline__ void softmax_row(Row<G, NV, VEC>& r)
{
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i)
        m = fmaxf(m, r.v[i]);
    m = group_max<G>(m);
    if (m == -INFINITY)
        m = 0.0f;                        // exp(-infinity - 0) = 0, and a NaN stays one
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i) {
        r.v[i] = exp_neg(r.v[i] - m);
        s += r.v[i];
    }
    s = group_sum<G>(s);
    const float inv = s == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(s);    // one ulp
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i)
        r.v[i] *= inv;
}

// Calls f with the row shape of E experts: rows that can be read 16 bytes at a time take as few
// lanes as hold them by fours, so that small E puts several tokens into a wavefront.
template <typename F>
inline void with_row(int32_t E, bool vec, F f)
{
    if (vec) {
        if (E <= 8) f(Row<2, 1, 4>());
        else if (E <= 16) f(Row<4, 1, 4>());
        else if (E <= 32) f(Row<8, 1, 4>());
        else if (E <= 64) f(Row<16, 1, 4>());
        else if (E <= 128) f(Row<32, 1, 4>());
        else if (E <= 256) f(Row<64, 1, 4>());
        else if (E <= 512) f(Row<64, 2, 4>());
        else f(Row<64, 4, 4>());
    } else {
        if (E <= 64) f(Row<64, 1, 1>());
        else if (E <= 128) f(Row<64, 2, 1>());
        else if (E <= 256) f(Row<64, 4, 1>());
        else if (E <= 512) f(Row<64, 8, 1>());
        else f(Row<64, 16, 1>());
    }
}

}  // namespace moe_dev

#endif  // MOE_ROWS_H
