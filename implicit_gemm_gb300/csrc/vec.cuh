// Loads and stores of V consecutive elements of a storage type as fp32 values.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace wg {

template <typename T>
constexpr bool is_half = false;
template <>
constexpr bool is_half<__half> = true;

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// V elements of T, moved by one access of at most 16 bytes each (two for eight
// fp32 elements).  The address is aligned to min(16, V * sizeof(T)) bytes.
template <typename T, int V>
struct alignas((V * sizeof(T)) > 16 ? 16 : V * sizeof(T)) Vec {
    T v[V];
};

template <typename T, int V>
__device__ __forceinline__ void load_f32(const T* p, float (&f)[V])
{
    if constexpr (V == 8 && sizeof(T) == 2) {
        // Two elements per word: the halves of a bf16 word are fp32 values but for a shift or a mask.
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (!is_half<T>) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                f[2 * i] = h.x, f[2 * i + 1] = h.y;
            }
        }
        return;
    }
    const Vec<T, V> x = *reinterpret_cast<const Vec<T, V>*>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_f32<T>(x.v[i]);
}

template <typename T, int V>
__device__ __forceinline__ void store_f32(T* p, const float (&f)[V])
{
    Vec<T, V> x;
#pragma unroll
    for (int i = 0; i < V; ++i) x.v[i] = from_f32<T>(f[i]);
    *reinterpret_cast<Vec<T, V>*>(p) = x;
}

}  // namespace wg
