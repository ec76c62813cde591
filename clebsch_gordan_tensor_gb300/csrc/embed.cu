// Embedding lookup and its gradient (sm_103a).
//
//   out[n] = s table[index[n]]          grad_table[v] = s sum_{index[n] = v} g[n]
//
// The lookup is a copy of rows.  The gradient sorts the indices (stable radix
// sort, eight bits a pass, key V for padding) and walks the sorted positions in
// chunks of equal length, so that a frequent row costs no more than many rare
// ones: a chunk adds up each run of equal keys in registers, writes the rows
// whose run it holds whole, and leaves the first and the last run, where they
// cross its ends, as partial rows that a second kernel joins in order.  No
// atomics on floating-point values: the same inputs give the same bits.
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.hpp"
#include "storage.cuh"

namespace cgtp {

__device__ int cgtp_embed_error;  // nonzero: an index of V or more was met

namespace {

// ------------------------------------------------------------- lookup --

// A group of T lanes copies a tile of T * V columns of one row.
template <typename S, typename I, int V>
__global__ void __launch_bounds__(256)
embed_forward_kernel(int64_t n, int64_t v, int64_t d, int T, int64_t tiles,
                     const I* __restrict__ index, const S* __restrict__ table,
                     typename Compute<S>::type scale, S* __restrict__ out, int64_t stride) {
    const int64_t groups = (int64_t)gridDim.x * (256 / T);
    const int t = threadIdx.x % T;
    for (int64_t w = (int64_t)blockIdx.x * (256 / T) + threadIdx.x / T; w < n * tiles;
         w += groups) {
        const int64_t row = w / tiles, col = (w % tiles * T + t) * V;
        if (col >= d) continue;
        const int64_t i = index[row];
        Pack<S, V> p;
        typename Compute<S>::type x[V];
        if (i >= 0 && i < v) {
            p = load_pack<S, V>(table + i * d + col);
#pragma unroll
            for (int k = 0; k < V; ++k) x[k] = p.get(k) * scale;
        } else {
            if (i >= v && t == 0) cgtp_embed_error = 1;
#pragma unroll
            for (int k = 0; k < V; ++k) x[k] = 0;
        }
        p.set(x);
        store_pack(out + row * stride + col, p);
    }
}

// --------------------------------------------------------------- sort --

constexpr int kTile = 2048;  // positions of a CTA in a pass
constexpr int kSortThreads = 256, kSortWarps = kSortThreads / 32;
constexpr int kPerWarp = kTile / kSortWarps;

template <typename I>
__device__ __forceinline__ uint32_t key_of(I i, uint32_t v) {
    if (i < 0) return v;
    if ((uint64_t)i >= v) {
        cgtp_embed_error = 1;
        return v;
    }
    return (uint32_t)i;
}
// Keys of later passes are made already.
struct Sorted {
    uint32_t key;
};
__device__ __forceinline__ uint32_t key_of(Sorted s, uint32_t) { return s.key; }

template <typename I>
__global__ void __launch_bounds__(kSortThreads)
sort_count_kernel(uint32_t n, uint32_t v, int shift, const I* __restrict__ in,
                  uint32_t* __restrict__ hist) {
    __shared__ uint32_t count[256];
    count[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t first = blockIdx.x * kTile;
    for (int j = threadIdx.x; j < kTile && first + j < n; j += kSortThreads)
        atomicAdd(&count[key_of(in[first + j], v) >> shift & 255u], 1u);
    __syncthreads();
    hist[threadIdx.x * gridDim.x + blockIdx.x] = count[threadIdx.x];
}

// Exclusive sums of len values, one CTA.
__global__ void __launch_bounds__(1024)
sort_scan_kernel(uint32_t len, uint32_t* __restrict__ hist) {
    __shared__ uint32_t warp_sum[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t each = (len + 1023) / 1024;
    const uint32_t first = min(threadIdx.x * each, len), last = min(first + each, len);
    uint32_t s = 0;
    for (uint32_t i = first; i < last; ++i) s += hist[i];
    uint32_t inc = s;
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        uint32_t w = warp_sum[lane], x;
        for (int o = 1; o < 32; o <<= 1) {
            x = __shfl_up_sync(0xFFFFFFFFu, w, o);
            if (lane >= o) w += x;
        }
        warp_sum[lane] = w;
    }
    __syncthreads();
    uint32_t run = inc - s + (warp ? warp_sum[warp - 1] : 0);
    for (uint32_t i = first; i < last; ++i) {
        const uint32_t x = hist[i];
        hist[i] = run;
        run += x;
    }
}

// Stable: a warp owns consecutive positions and takes them 32 at a time; a
// position's place is its digit's base plus the equal digits before it.
template <typename I>
__global__ void __launch_bounds__(kSortThreads)
sort_scatter_kernel(uint32_t n, uint32_t v, int shift, const I* __restrict__ in,
                    const uint32_t* __restrict__ pos_in, const uint32_t* __restrict__ base,
                    uint32_t* __restrict__ keys, uint32_t* __restrict__ pos) {
    __shared__ uint32_t count[kSortWarps][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int j = lane; j < 256; j += 32) count[warp][j] = 0;
    __syncwarp();
    const uint32_t first = blockIdx.x * kTile + warp * kPerWarp;
    uint32_t key[kPerWarp / 32];
#pragma unroll
    for (int j = 0; j < kPerWarp / 32; ++j) {
        const uint32_t i = first + j * 32 + lane;
        key[j] = i < n ? key_of(in[i], v) : 0;
        const uint32_t dig = i < n ? key[j] >> shift & 255u : 256u;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, dig);
        if (i < n && (same & ((1u << lane) - 1)) == 0) count[warp][dig] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    {  // digit threadIdx.x: where each warp starts
        uint32_t at = base[threadIdx.x * gridDim.x + blockIdx.x];
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t c = count[w][threadIdx.x];
            count[w][threadIdx.x] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPerWarp / 32; ++j) {
        const uint32_t i = first + j * 32 + lane;
        const uint32_t dig = i < n ? key[j] >> shift & 255u : 256u;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, dig);
        const uint32_t before = same & ((1u << lane) - 1);
        uint32_t at = 0;
        if (i < n) {
            at = count[warp][dig] + __popc(before);
            keys[at] = key[j];
            pos[at] = pos_in ? pos_in[i] : i;
        }
        __syncwarp();
        if (i < n && before == 0) count[warp][dig] += __popc(same);
        __syncwarp();
    }
}

// --------------------------------------------------------------- sums --

// One group of T lanes: the runs of chunk c in the columns of one tile.
template <typename S, int V>
__global__ void __launch_bounds__(256)
embed_sum_kernel(uint32_t n, uint32_t v, int64_t d, int T, uint32_t tiles, uint32_t chunk,
                 uint32_t chunks, const uint32_t* __restrict__ keys,
                 const uint32_t* __restrict__ pos, const S* __restrict__ g, int64_t stride,
                 typename Compute<S>::type scale, S* __restrict__ table,
                 typename Compute<S>::type* __restrict__ partial) {
    using C = typename Compute<S>::type;
    const int64_t w = (int64_t)blockIdx.x * (256 / T) + threadIdx.x / T;
    const uint32_t c = (uint32_t)(w / tiles);
    const int64_t col = (w % tiles * T + threadIdx.x % T) * V;
    if (c >= chunks || col >= d) return;
    const uint32_t first = c * chunk, last = min(first + chunk, n);
    uint32_t cur = keys[first];
    if (cur >= v) return;  // padding sorts last
    bool head = first > 0 && keys[first - 1] == cur;
    C acc[V] = {};
    auto finish = [&](bool tail) {
        if (head || tail) {
            C* p = partial + ((int64_t)c * 2 + (head ? 0 : 1)) * d + col;
#pragma unroll
            for (int k = 0; k < V; ++k) p[k] = acc[k];
        } else {
            Pack<S, V> o;
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] *= scale;
            o.set(acc);
            store_pack(table + (int64_t)cur * d + col, o);
        }
    };
    constexpr int U = 4;  // rows in flight
    for (uint32_t j = first; j < last; j += U) {
        uint32_t key[U];
        Pack<S, V> row[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            key[u] = j + u < last ? keys[j + u] : v;
            if (key[u] < v) row[u] = load_pack<S, V>(g + (int64_t)pos[j + u] * stride + col);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j + u >= last) break;
            if (key[u] != cur) {
                finish(false);
                cur = key[u];
                head = false;
                if (cur >= v) return;
#pragma unroll
                for (int k = 0; k < V; ++k) acc[k] = 0;
            }
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] += row[u].get(k);
        }
    }
    finish(last < n && keys[last] == cur);
}

// The runs that start in chunk c and go on past its end.
template <typename S, int V>
__global__ void __launch_bounds__(256)
embed_join_kernel(uint32_t n, uint32_t v, int64_t d, int T, uint32_t tiles, uint32_t chunk,
                  uint32_t chunks, const uint32_t* __restrict__ keys,
                  typename Compute<S>::type scale, S* __restrict__ table,
                  const typename Compute<S>::type* __restrict__ partial) {
    using C = typename Compute<S>::type;
    const int64_t w = (int64_t)blockIdx.x * (256 / T) + threadIdx.x / T;
    uint32_t c = (uint32_t)(w / tiles);
    const int64_t col = (w % tiles * T + threadIdx.x % T) * V;
    if (c >= chunks || col >= d) return;
    const uint32_t first = c * chunk, last = min(first + chunk, n);
    if (last >= n) return;
    const uint32_t cur = keys[last];
    if (cur >= v || keys[last - 1] != cur) return;
    if (keys[first] == cur && first > 0 && keys[first - 1] == cur) return;  // it starts earlier
    C acc[V];
    const C* p = partial + ((int64_t)c * 2 + 1) * d + col;
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = p[k];
    for (++c;; ++c) {
        p = partial + (int64_t)c * 2 * d + col;
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] += p[k];
        const int64_t end = (int64_t)(c + 1) * chunk;
        if (end >= n || keys[end] != cur) break;
    }
    Pack<S, V> o;
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] *= scale;
    o.set(acc);
    store_pack(table + (int64_t)cur * d + col, o);
}

__global__ void __launch_bounds__(256) embed_zero_kernel(uint8_t* __restrict__ p, int64_t bytes) {
    const int64_t words = bytes / 16, step = (int64_t)gridDim.x * 256;
    const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const bool wide = (uintptr_t)p % 16 == 0;
    if (wide)
        for (int64_t i = i0; i < words; i += step)
            reinterpret_cast<uint4*>(p)[i] = make_uint4(0, 0, 0, 0);
    for (int64_t i = (wide ? words * 16 : 0) + i0; i < bytes; i += step) p[i] = 0;
}

// -------------------------------------------------------------- launching --

int lanes_for(int64_t vecs) {
    int T = 1;
    while (T < 32 && T < vecs) T *= 2;
    return T;
}

uint32_t blocks_for(int64_t groups, int T) {
    return (uint32_t)((groups + 256 / T - 1) / (256 / T));
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

// Positions of a chunk: enough chunks to fill the GPU, few enough that their
// partial rows stay small beside the gradient rows.
uint32_t chunk_of(int64_t n, int64_t d) {
    const int64_t tiles = (d + 127) / 128, want = 152 * 32;
    int64_t c = n * tiles / want;
    c = std::max<int64_t>(16, std::min<int64_t>(c, 256));
    return (uint32_t)c;
}

struct Layout {
    uint32_t chunk, chunks, sort_ctas;
    size_t keys[2], pos[2], hist, partial, total;
};

Layout layout_of(cgtp_dtype type, int64_t n, int64_t d) {
    Layout L;
    L.chunk = chunk_of(n, d);
    L.chunks = (uint32_t)((n + L.chunk - 1) / L.chunk);
    L.sort_ctas = (uint32_t)((n + kTile - 1) / kTile);
    size_t at = 0;
    for (int k = 0; k < 2; ++k) {
        L.keys[k] = at, at += up256((size_t)n * 4);
        L.pos[k] = at, at += up256((size_t)n * 4);
    }
    L.hist = at, at += up256((size_t)L.sort_ctas * 256 * 4);
    L.partial = at;
    at += up256((size_t)L.chunks * 2 * (size_t)d * (type == CGTP_F64 ? 8 : 4));
    L.total = at;
    return L;
}

template <typename I>
cudaError_t sort_pass(const EmbedCall& c, const Layout& L, int shift, const I* in,
                      const uint32_t* pos_in, int to, cudaStream_t s) {
    uint8_t* ws = (uint8_t*)c.ws;
    uint32_t* hist = (uint32_t*)(ws + L.hist);
    const uint32_t n = (uint32_t)c.n, v = (uint32_t)c.v;
    sort_count_kernel<I><<<L.sort_ctas, kSortThreads, 0, s>>>(n, v, shift, in, hist);
    sort_scan_kernel<<<1, 1024, 0, s>>>(L.sort_ctas * 256, hist);
    sort_scatter_kernel<I><<<L.sort_ctas, kSortThreads, 0, s>>>(
        n, v, shift, in, pos_in, hist, (uint32_t*)(ws + L.keys[to]), (uint32_t*)(ws + L.pos[to]));
    for (int k = 0; k < 3; ++k) count_launch();
    return cudaGetLastError();
}

template <typename S, int V>
cudaError_t backward_v(const EmbedCall& c, const Layout& L, int sorted, cudaStream_t s) {
    using C = typename Compute<S>::type;
    uint8_t* ws = (uint8_t*)c.ws;
    const uint32_t* keys = (const uint32_t*)(ws + L.keys[sorted]);
    const uint32_t* pos = (const uint32_t*)(ws + L.pos[sorted]);
    const int T = lanes_for((c.d + V - 1) / V);
    const uint32_t tiles = (uint32_t)((c.d + (int64_t)T * V - 1) / ((int64_t)T * V));
    const uint32_t grid = blocks_for((int64_t)L.chunks * tiles, T);
    embed_sum_kernel<S, V><<<grid, 256, 0, s>>>((uint32_t)c.n, (uint32_t)c.v, c.d, T, tiles,
                                                L.chunk, L.chunks, keys, pos, (const S*)c.in,
                                                c.in_stride, (C)c.scale, (S*)c.out,
                                                (C*)(ws + L.partial));
    embed_join_kernel<S, V><<<grid, 256, 0, s>>>((uint32_t)c.n, (uint32_t)c.v, c.d, T, tiles,
                                                 L.chunk, L.chunks, keys, (C)c.scale, (S*)c.out,
                                                 (const C*)(ws + L.partial));
    count_launch();
    count_launch();
    return cudaGetLastError();
}

// Rows that can move in 16-byte accesses.
template <typename S>
bool wide(const EmbedCall& c) {
    constexpr int V = 16 / sizeof(S);
    return c.d % V == 0 && c.in_stride % V == 0 && c.out_stride % V == 0 &&
           (uintptr_t)c.in % 16 == 0 && (uintptr_t)c.out % 16 == 0;
}

template <typename S>
cudaError_t backward(const EmbedCall& c, cudaStream_t s) {
    const int64_t bytes = c.v * c.d * (int64_t)sizeof(S);
    embed_zero_kernel<<<(unsigned)std::min<int64_t>((bytes / 16 + 255) / 256 + 1, 152 * 16), 256, 0,
                        s>>>((uint8_t*)c.out, bytes);
    count_launch();
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || c.n == 0) return e;
    const Layout L = layout_of(c.type, c.n, c.d);
    uint8_t* ws = (uint8_t*)c.ws;
    int bits = 1;
    while (((int64_t)1 << bits) <= c.v) ++bits;  // keys 0..V
    int to = 0;
    for (int shift = 0; shift < bits; shift += 8, to ^= 1) {
        if (shift == 0)
            e = c.index_bits == 32
                    ? sort_pass(c, L, 0, (const int32_t*)c.index, nullptr, to, s)
                    : sort_pass(c, L, 0, (const int64_t*)c.index, nullptr, to, s);
        else
            e = sort_pass(c, L, shift, (const Sorted*)(ws + L.keys[to ^ 1]),
                          (const uint32_t*)(ws + L.pos[to ^ 1]), to, s);
        if (e != cudaSuccess) return e;
    }
    return wide<S>(c) ? backward_v<S, 16 / sizeof(S)>(c, L, to ^ 1, s)
                      : backward_v<S, 1>(c, L, to ^ 1, s);
}

template <typename S, typename I, int V>
cudaError_t forward_v(const EmbedCall& c, cudaStream_t s) {
    using C = typename Compute<S>::type;
    const int T = lanes_for((c.d + V - 1) / V);
    const int64_t tiles = (c.d + (int64_t)T * V - 1) / ((int64_t)T * V);
    const unsigned grid =
        (unsigned)std::min<int64_t>((c.n * tiles + 256 / T - 1) / (256 / T), 152 * 64);
    embed_forward_kernel<S, I, V><<<grid, 256, 0, s>>>(
        c.n, c.v, c.d, T, tiles, (const I*)c.index, (const S*)c.in, (C)c.scale, (S*)c.out,
        c.out_stride);
    count_launch();
    return cudaGetLastError();
}

template <typename S>
cudaError_t forward(const EmbedCall& c, cudaStream_t s) {
    constexpr int V = 16 / sizeof(S);
    if (c.index_bits == 32)
        return wide<S>(c) ? forward_v<S, int32_t, V>(c, s) : forward_v<S, int32_t, 1>(c, s);
    return wide<S>(c) ? forward_v<S, int64_t, V>(c, s) : forward_v<S, int64_t, 1>(c, s);
}

}  // namespace

cudaError_t launch_embed_forward(const EmbedCall& c, cudaStream_t s) {
    switch (c.type) {
        case CGTP_F64: return forward<double>(c, s);
        case CGTP_BF16: return forward<__nv_bfloat16>(c, s);
        case CGTP_F16: return forward<__half>(c, s);
        default: return forward<float>(c, s);
    }
}

size_t embed_backward_workspace_bytes(cgtp_dtype type, int64_t n, int64_t v, int64_t d) {
    (void)v;
    return n == 0 ? 0 : layout_of(type, n, d).total;
}

cudaError_t launch_embed_backward(const EmbedCall& c, cudaStream_t s) {
    switch (c.type) {
        case CGTP_F64: return backward<double>(c, s);
        case CGTP_BF16: return backward<__nv_bfloat16>(c, s);
        case CGTP_F16: return backward<__half>(c, s);
        default: return backward<float>(c, s);
    }
}

cudaError_t embed_device_status(int* code) {
    const int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, cgtp_embed_error, sizeof(int));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(cgtp_embed_error, &zero, sizeof(int));
    return e;
}

}  // namespace cgtp
