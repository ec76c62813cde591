// Storage types of the training kernels: fp32, fp64, bfloat16 and binary16
// elements, read and written in vectors and computed on in fp32 (fp64 for fp64).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace cgtp {

template <typename S>
struct Compute {
    using type = float;
};
template <>
struct Compute<double> {
    using type = double;
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ double widen(double x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float widen(__half x) { return __half2float(x); }

// Rounded to nearest, ties to even.
template <typename S>
__device__ __forceinline__ S narrow(typename Compute<S>::type x);
template <>
__device__ __forceinline__ float narrow<float>(float x) {
    return x;
}
template <>
__device__ __forceinline__ double narrow<double>(double x) {
    return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half narrow<__half>(float x) {
    return __float2half_rn(x);
}

// V consecutive elements, moved as one access (16 bytes at most).
template <typename S, int V>
struct alignas(sizeof(S) * V) Pack {
    S v[V];
};

template <typename S, int V>
__device__ __forceinline__ Pack<S, V> load_pack(const S* p) {
    return *reinterpret_cast<const Pack<S, V>*>(p);
}
template <typename S, int V>
__device__ __forceinline__ void store_pack(S* p, const Pack<S, V>& x) {
    *reinterpret_cast<Pack<S, V>*>(p) = x;
}

}  // namespace cgtp
