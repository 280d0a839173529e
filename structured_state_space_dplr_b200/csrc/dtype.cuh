// dtype.cuh -- the element types of the token-major operators (s4_dtype) and
// their conversions. All arithmetic is in float; a value is rounded to 16
// bits (to nearest even) once, where it is stored.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <cstring>

namespace s4 {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }

template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// V consecutive elements in one load or store of V * sizeof(T) bytes, aligned to that
template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
    T v[V];
};
template <typename T, int V>
__device__ __forceinline__ void load_pack(const T *p, float (&o)[V]) {
    const Pack<T, V> r = *reinterpret_cast<const Pack<T, V> *>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = to_f(r.v[i]);
}
// the same of a pack in shared memory or registers, two 16-bit values at a time
__device__ __forceinline__ void to_f2(uint32_t w, float &a, float &b, __nv_bfloat16) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void to_f2(uint32_t w, float &a, float &b, __half) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    a = f.x;
    b = f.y;
}
template <typename T, int V>
__device__ __forceinline__ void unpack(const Pack<T, V> &r, float (&o)[V]) {
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {
        uint32_t w[V / 2];
        memcpy(w, &r, sizeof(w));
#pragma unroll
        for (int i = 0; i < V / 2; ++i) to_f2(w[i], o[2 * i], o[2 * i + 1], T{});
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = to_f(r.v[i]);
    }
}
template <typename T, int V>
__device__ __forceinline__ void store_pack(T *p, const float (&o)[V]) {
    Pack<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = from_f<T>(o[i]);
    *reinterpret_cast<Pack<T, V> *>(p) = r;
}

}  // namespace s4
