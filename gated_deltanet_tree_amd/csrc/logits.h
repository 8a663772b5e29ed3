// Rows of logits as the kernels that stream them read them: eight at a time from the 16-byte boundary at
// or below a row's start, NaN as -inf (gfx950, wave64).
#pragma once

#include "gdn_device.h"

namespace gdn {

constexpr float kInf = __builtin_inff();

// Rows may start at any element: groups of eight are counted from the 16-byte boundary at or
// below the row's start.
template <typename T> __device__ __forceinline__ int misaligned(const T *row) {
    return int((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
}

template <typename T> __device__ __forceinline__ float logit(T x) {
    const float f = to_f32<T>(x);
    return f == f ? f : -kInf;  // NaN: never drawn
}

// Logits 8 g - mis .. 8 g - mis + 7 of a row, -inf outside [0, V).
template <typename T>
__device__ __forceinline__ void load_group(const T *row, int mis, int g, int V, float *x) {
    const int first = 8 * g - mis;
    if (first >= 0 && first + 8 <= V) {
        if constexpr (sizeof(T) == 2) {
            const uint4 v = *reinterpret_cast<const uint4 *>(row + first);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = bf16_lo(w[i]);
                x[2 * i + 1] = bf16_hi(w[i]);
            }
        } else {
            const float4 a = reinterpret_cast<const float4 *>(row + first)[0];
            const float4 b = reinterpret_cast<const float4 *>(row + first)[1];
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] == x[i] ? x[i] : -kInf;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = first + i >= 0 && first + i < V ? logit(row[first + i]) : -kInf;
    }
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor(x, d));
    return x;
}
__device__ __forceinline__ int wave_min(int x) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x = min(x, __shfl_xor(x, d));
    return x;
}
template <typename F> __device__ __forceinline__ F wave_sum(F x) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
    return x;
}

}  // namespace gdn
