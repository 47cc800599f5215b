// moe_device.h -- device and host helpers shared by the operators next to routing.
#ifndef MOE_DEVICE_H
#define MOE_DEVICE_H

#include <hip/hip_runtime.h>

#include <stdint.h>

namespace moe_dev {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v)
{
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL,
                                                                 0xF, 0xF, false));
}

// Reduction over groups of G lanes (a power of two), the result in every lane of the group:
// quad_perm [1,0,3,2] and [2,3,0,1], then row_half_mirror and row_mirror pair lanes whose partial
// results are already uniform; beyond a 16-lane row v_permlane16_swap and v_permlane32_swap hand
// every lane both halves' results. The order is fixed.
template <int G, typename Op>
__device__ __forceinline__ float group_reduce(float v, Op op)
{
    if (G >= 2)
        v = op(v, dpp_f32<0xB1>(v));
    if (G >= 4)
        v = op(v, dpp_f32<0x4E>(v));
    if (G >= 8)
        v = op(v, dpp_f32<0x141>(v));
    if (G >= 16)
        v = op(v, dpp_f32<0x140>(v));
    if (G >= 32) {
        const uint32_t b = __float_as_uint(v);
        const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
        v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    if (G >= 64) {
        const uint32_t b = __float_as_uint(v);
        const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
        v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    return v;
}

template <int G>
__device__ __forceinline__ float group_sum(float v)
{
    return group_reduce<G>(v, [](float a, float b) { return a + b; });
}

template <int G>
__device__ __forceinline__ float group_max(float v)
{
    return group_reduce<G>(v, [](float a, float b) { return fmaxf(a, b); });
}

template <typename T>
inline bool aligned_to(const T* p, uintptr_t n)
{
    return (uintptr_t)p % n == 0;
}

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace moe_dev

#endif  // MOE_DEVICE_H
