// Storage types of the training kernels: fp32, fp64, bfloat16 and binary16
// elements, read and written in vectors and computed on in fp32 (fp64 for fp64).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace cgtp {

// Launches a kernel of a chain: it may begin, up to its wait_for_previous(),
// while the kernel before it on the stream still runs (one that has called
// let_next_start()), which hides the launch.
template <typename... K, typename... A>
cudaError_t launch_chained(void (*kernel)(K...), dim3 grid, dim3 block, cudaStream_t s,
                           A... args) {
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = block;
    c.stream = s;
    c.attrs = &early;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, static_cast<K>(args)...);
}
// Until the kernel before this one is done and its writes are seen.
__device__ __forceinline__ void wait_for_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

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

// V consecutive elements, moved as one access (16 bytes at most) and held as
// they lie in memory: 16-bit elements stay two to a register until one is used
// (as an array of 16-bit values each would take a register of its own: the
// gradient of 16,384 rows of 4096 took 572 us so, with spills, and 282 us not).
template <typename S, int V, bool Halves = (sizeof(S) == 2 && V % 2 == 0)>
struct alignas(sizeof(S) * V) Pack {
    using C = typename Compute<S>::type;
    S v[V];
    __device__ __forceinline__ C get(int i) const { return widen(v[i]); }
    __device__ __forceinline__ void set(const C (&x)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = narrow<S>(x[i]);
    }
    __device__ __forceinline__ void fill(C x) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = narrow<S>(x);
    }
};

__device__ __forceinline__ float half_of(uint32_t w, int i, __nv_bfloat16) {
    return __uint_as_float(i ? w & 0xFFFF0000u : w << 16);
}
__device__ __forceinline__ float half_of(uint32_t w, int i, __half) {
    return __half2float(__ushort_as_half((unsigned short)(i ? w >> 16 : w & 0xFFFFu)));
}
__device__ __forceinline__ uint32_t halves_of(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint32_t halves_of(float a, float b, __half) {
    const __half2 p = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
}

template <typename S, int V>
struct alignas(sizeof(S) * V) Pack<S, V, true> {
    using C = float;
    uint32_t w[V / 2];
    __device__ __forceinline__ float get(int i) const { return half_of(w[i / 2], i & 1, S{}); }
    __device__ __forceinline__ void set(const float (&x)[V]) {
#pragma unroll
        for (int i = 0; i < V; i += 2) w[i / 2] = halves_of(x[i], x[i + 1], S{});
    }
    __device__ __forceinline__ void fill(float x) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) w[i] = halves_of(x, x, S{});
    }
};

template <typename S, int V>
__device__ __forceinline__ Pack<S, V> load_pack(const S* p) {
    return *reinterpret_cast<const Pack<S, V>*>(p);
}
template <typename S, int V>
__device__ __forceinline__ void store_pack(S* p, const Pack<S, V>& x) {
    *reinterpret_cast<Pack<S, V>*>(p) = x;
}

// A store that the caches need not keep.
template <typename S, int V>
__device__ __forceinline__ void stream_pack(S* p, const Pack<S, V>& x) {
    if constexpr (sizeof(S) * V == 16)
        __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(&x));
    else
        store_pack(p, x);
}

// Asynchronous copies to shared memory of 4, 8 or 16 bytes.
template <int N>
__device__ __forceinline__ void copy_async(void* shared, const void* src) {
    const uint32_t dst = (uint32_t)__cvta_generic_to_shared(shared);
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N)
                     : "memory");
}
__device__ __forceinline__ void copies_end_group() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Two values that go through the arithmetic together: one packed instruction
// for each pair of fp32 operations.
template <typename C>
struct Two {
    C x, y;
};
__device__ __forceinline__ unsigned long long bits_of(Two<float> a) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
    return r;
}
__device__ __forceinline__ Two<float> two_of(unsigned long long r) {
    Two<float> a;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
    return a;
}
__device__ __forceinline__ Two<float> fma(Two<float> a, Two<float> b, Two<float> c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(bits_of(a)), "l"(bits_of(b)), "l"(bits_of(c)));
    return two_of(r);
}
__device__ __forceinline__ Two<float> operator*(Two<float> a, Two<float> b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits_of(a)), "l"(bits_of(b)));
    return two_of(r);
}
__device__ __forceinline__ Two<float> operator+(Two<float> a, Two<float> b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits_of(a)), "l"(bits_of(b)));
    return two_of(r);
}
__device__ __forceinline__ Two<double> fma(Two<double> a, Two<double> b, Two<double> c) {
    return {::fma(a.x, b.x, c.x), ::fma(a.y, b.y, c.y)};
}
__device__ __forceinline__ Two<double> operator*(Two<double> a, Two<double> b) {
    return {a.x * b.x, a.y * b.y};
}
__device__ __forceinline__ Two<double> operator+(Two<double> a, Two<double> b) {
    return {a.x + b.x, a.y + b.y};
}

// Elements 2i and 2i + 1 of a pack.
template <typename S, int V>
__device__ __forceinline__ Two<typename Compute<S>::type> two_at(const Pack<S, V>& p, int i) {
    return {p.get(2 * i), p.get(2 * i + 1)};
}
template <typename S, int V>
__device__ __forceinline__ void set_twos(Pack<S, V>& p, const Two<typename Compute<S>::type> (&v)[V / 2]) {
    typename Compute<S>::type x[V];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) x[2 * i] = v[i].x, x[2 * i + 1] = v[i].y;
    p.set(x);
}

}  // namespace cgtp
