// Per-irrep RMS norm and the gated residual around a block, with gradients
// (sm_103a).  Included by one translation unit per storage type.
//
// A feature row holds irreps one after another, irrep i as [2l+1][mul]; D_i =
// (2l+1) mul.  With one value per (irrep, channel) c for the weights, the
// residual scale and the gate z, and m running over the 2l+1 components,
//   r   = (sum over the irrep of b^2 / D + eps)^(-1/2)
//   h   = x + scale[c] sigmoid(z[c]) weight[c] b r
//   y   = h r' next_weight[c],  r' from h as it is stored
// Leaving x, z and scale out gives the plain norm.  Rotations mix the
// components of a channel only, so every factor commutes with them.
// Gradient, with n = b r, q = h r' and the channel sums P[c] = sum_m gx n,
// Q[c] = sum_m gy q:
//   gx = grad_h + r' (next_weight gy - q (1/D) sum_c next_weight Q)
//   gb = r (a weight gx - n (1/D) sum_c a weight P),   a = scale sigmoid(z)
//   gz = scale weight sigmoid(z) (1 - sigmoid(z)) P
//   gweight += a P,  gscale += weight sigmoid(z) P,  gnext_weight += Q
//
// Work split: one (row, irrep) pair is independent of every other, so a pair is
// the unit of work.  A group of T threads takes a pair; a thread owns K vectors
// of V channels and keeps all their 2l+1 components in registers between the
// two reductions, so every tensor is read once and written once.  A CTA stays
// with one irrep: its threads keep their channels' weights in registers, and in
// the gradient their channels' sums, which leave as one partial row per CTA.
// Both directions are bound by HBM.
#pragma once

#include <algorithm>

#include "internal.hpp"
#include "storage.cuh"

namespace cgtp {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float rsqrt_of(float x) { return rsqrtf(x); }
__device__ __forceinline__ double rsqrt_of(double x) { return 1.0 / sqrt(x); }
__device__ __forceinline__ float sigmoid_of(float z) { return 1.f / (1.f + expf(-z)); }
__device__ __forceinline__ double sigmoid_of(double z) { return 1.0 / (1.0 + exp(-z)); }

// Sums of R <= 3 values over the T threads of a group, the same on all of them
// and in an order that does not depend on timing.  Called by the whole CTA.
// Two sets of slots in turn: a set is written again only after the barrier of
// the call in between, which every thread reaches after its reads.
template <typename C>
struct GroupSum {
    C (*buf)[kThreads / 32];  // [2][3][warps]
    int T, flip = 0;
    template <int R>
    __device__ void operator()(C (&v)[R]) {
        const int width = T < 32 ? T : 32;
        for (int o = width >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int r = 0; r < R; ++r) v[r] += __shfl_xor_sync(0xFFFFFFFFu, v[r], o);
        if (T <= 32) return;
        const int warp = threadIdx.x >> 5, nw = T >> 5, first = warp / nw * nw;
        C (*const side)[kThreads / 32] = buf + flip * 3;
        flip ^= 1;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int r = 0; r < R; ++r) side[r][warp] = v[r];
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            C s = 0;
            for (int w = 0; w < nw; ++w) s += side[r][first + w];
            v[r] = s;
        }
    }
};

template <typename C, int V>
__device__ __forceinline__ void load_param(C (&out)[V], const C* p, int at, C missing) {
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = p ? p[at + i] : missing;
}

// ------------------------------------------------------------- forward --

template <typename S, int V, int L, int K>
__device__ __forceinline__ void forward_body(const NormIrrep& ir, int cta, const NormForward& a,
                                             typename Compute<S>::type (*sums)[kThreads / 32]) {
    using C = typename Compute<S>::type;
    constexpr int M = 2 * L + 1;
    const int T = ir.T, t = threadIdx.x % T, G = kThreads / T;
    const int U = ir.mul / V;
    const C inv_d = (C)1 / (C)(M * ir.mul), eps = (C)a.eps;
    const C *w = (const C*)a.weight, *sc = (const C*)a.scale, *w2 = (const C*)a.next_weight;
    C coef[K][V], next[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = ir.ch + (t + k * T < U ? t + k * T : 0) * V;
        load_param(coef[k], w, c, (C)1);
        load_param(next[k], w2, c, (C)1);
#pragma unroll
        for (int i = 0; i < V; ++i) coef[k][i] *= sc ? sc[c + i] : (C)1;
    }
    GroupSum<C> sum{sums, T};
    for (int64_t base = (int64_t)cta * G; base < a.n; base += (int64_t)ir.ctas * G) {
        const int64_t row = base + threadIdx.x / T;
        const bool in = row < a.n;
        const S* b = (const S*)a.b.data + row * a.b.stride + ir.off;
        const S* x = a.x.data ? (const S*)a.x.data + row * a.x.stride + ir.off : nullptr;
        const S* z = a.gate.data ? (const S*)a.gate.data + row * a.gate.stride + ir.ch : nullptr;
        Pack<S, V> bp[K][M], xp[K][M], zp[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const bool on = in && t + k * T < U;
            const int u = (t + k * T) * V;
#pragma unroll
            for (int m = 0; m < M; ++m) {
                if (on) {
                    bp[k][m] = load_pack<S, V>(b + m * ir.mul + u);
                    if (x) xp[k][m] = load_pack<S, V>(x + m * ir.mul + u);
                }
            }
            if (on && z) zp[k] = load_pack<S, V>(z + u);
        }
        C s[1] = {0};
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (in && t + k * T < U)
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const C v = widen(bp[k][m].v[i]);
                        s[0] += v * v;
                    }
        sum(s);
        const C r = rsqrt_of(s[0] * inv_d + eps);
        s[0] = 0;
        S* h = (S*)a.h.data + row * a.h.stride + ir.off;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (in && t + k * T < U) {
                C f[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    f[i] = r * coef[k][i];
                    if (z) f[i] *= sigmoid_of(widen(zp[k].v[i]));
                }
#pragma unroll
                for (int m = 0; m < M; ++m) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        C v = f[i] * widen(bp[k][m].v[i]);
                        if (x) v += widen(xp[k][m].v[i]);
                        bp[k][m].v[i] = narrow<S>(v);
                        v = widen(bp[k][m].v[i]);
                        s[0] += v * v;
                    }
                    store_pack(h + m * ir.mul + (t + k * T) * V, bp[k][m]);
                }
            }
        if (a.y.data) {
            sum(s);
            const C r2 = rsqrt_of(s[0] * inv_d + eps);
            S* y = (S*)a.y.data + row * a.y.stride + ir.off;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (in && t + k * T < U)
#pragma unroll
                    for (int m = 0; m < M; ++m) {
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            bp[k][m].v[i] = narrow<S>(widen(bp[k][m].v[i]) * r2 * next[k][i]);
                        store_pack(y + m * ir.mul + (t + k * T) * V, bp[k][m]);
                    }
        }
    }
}

// Irreps with more channels than a CTA's registers hold: the CTA takes a row at
// a time and reads b (and the h it wrote) again instead of keeping them; the
// second read comes from L2.
template <typename S, int V>
__device__ void forward_wide(const NormIrrep& ir, int cta, const NormForward& a,
                             typename Compute<S>::type (*sums)[kThreads / 32]) {
    using C = typename Compute<S>::type;
    const int M = 2 * ir.l + 1, U = ir.mul / V;
    const C inv_d = (C)1 / ((C)M * (C)ir.mul), eps = (C)a.eps;
    const C *w = (const C*)a.weight, *sc = (const C*)a.scale, *w2 = (const C*)a.next_weight;
    GroupSum<C> sum{sums, kThreads};
    for (int64_t row = cta; row < a.n; row += ir.ctas) {
        const S* b = (const S*)a.b.data + row * a.b.stride + ir.off;
        const S* x = a.x.data ? (const S*)a.x.data + row * a.x.stride + ir.off : nullptr;
        const S* z = a.gate.data ? (const S*)a.gate.data + row * a.gate.stride + ir.ch : nullptr;
        S* h = (S*)a.h.data + row * a.h.stride + ir.off;
        C s[1] = {0};
        for (int64_t e = threadIdx.x; e < (int64_t)M * U; e += kThreads) {
            const Pack<S, V> p = load_pack<S, V>(b + e * V);
#pragma unroll
            for (int i = 0; i < V; ++i) s[0] += widen(p.v[i]) * widen(p.v[i]);
        }
        sum(s);
        const C r = rsqrt_of(s[0] * inv_d + eps);
        s[0] = 0;
        for (int u = threadIdx.x; u < U; u += kThreads) {
            const int c = ir.ch + u * V;
            C f[V];
            load_param(f, w, c, (C)1);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                f[i] *= r * (sc ? sc[c + i] : (C)1);
                if (z) f[i] *= sigmoid_of(widen(z[u * V + i]));
            }
            for (int m = 0; m < M; ++m) {
                const int64_t at = (int64_t)m * ir.mul + (int64_t)u * V;
                Pack<S, V> p = load_pack<S, V>(b + at), q;
                if (x) q = load_pack<S, V>(x + at);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    C v = f[i] * widen(p.v[i]);
                    if (x) v += widen(q.v[i]);
                    p.v[i] = narrow<S>(v);
                    s[0] += widen(p.v[i]) * widen(p.v[i]);
                }
                store_pack(h + at, p);
            }
        }
        if (a.y.data) {
            sum(s);
            const C r2 = rsqrt_of(s[0] * inv_d + eps);
            S* y = (S*)a.y.data + row * a.y.stride + ir.off;
            for (int u = threadIdx.x; u < U; u += kThreads) {
                C f[V];
                load_param(f, w2, ir.ch + u * V, (C)1);
                for (int m = 0; m < M; ++m) {  // the thread's own stores to h
                    const int64_t at = (int64_t)m * ir.mul + (int64_t)u * V;
                    Pack<S, V> p = load_pack<S, V>(h + at);
#pragma unroll
                    for (int i = 0; i < V; ++i) p.v[i] = narrow<S>(widen(p.v[i]) * r2 * f[i]);
                    store_pack(y + at, p);
                }
            }
        }
    }
}

// LC: the largest l a launch holds, in classes (0, 3 or 6), so that plain rows
// do not carry the registers of 13 components.
#define CGTP_NORM_BODIES(LC, CALL, WIDE)                          \
    if (ir.K == 0) {                                              \
        WIDE;                                                     \
    } else if (ir.l == 0) {                                       \
        if (ir.K == 1) { CALL(0, 1); }                            \
        else if (ir.K == 2) { CALL(0, 2); }                       \
        else if (ir.K == 4) { CALL(0, 4); }                       \
        else { CALL(0, 8); }                                      \
    }                                                             \
    if constexpr (LC >= 3) {                                      \
        if (ir.K != 0 && ir.l == 1) {                             \
            if (ir.K == 1) { CALL(1, 1); } else { CALL(1, 2); }   \
        }                                                         \
        if (ir.K != 0 && ir.l == 2) { CALL(2, 1); }               \
        if (ir.K != 0 && ir.l == 3) { CALL(3, 1); }               \
    }                                                             \
    if constexpr (LC >= 6) {                                      \
        if (ir.K != 0 && ir.l == 4) { CALL(4, 1); }               \
        if (ir.K != 0 && ir.l == 5) { CALL(5, 1); }               \
        if (ir.K != 0 && ir.l == 6) { CALL(6, 1); }               \
    }

template <typename S, int V, int LC>
__global__ void __launch_bounds__(kThreads)
norm_forward_kernel(const __grid_constant__ NormTable tab, const __grid_constant__ NormForward a) {
    __shared__ typename Compute<S>::type sums[6][kThreads / 32];
    int i = 0;
    while (i + 1 < tab.n && (int)blockIdx.x >= tab.ir[i + 1].cta0) ++i;
    const NormIrrep& ir = tab.ir[i];
    const int cta = blockIdx.x - ir.cta0;
#define CALL(L, K) forward_body<S, V, L, K>(ir, cta, a, sums)
    CGTP_NORM_BODIES(LC, CALL, (forward_wide<S, V>(ir, cta, a, sums)))
#undef CALL
}

// ------------------------------------------------------------ gradient --

// The three channel sums of a CTA, [3][mul] at its place in the partial rows.
template <typename C>
__device__ __forceinline__ C* partial_row(const NormIrrep& ir, int cta, const NormBackward& a) {
    return (C*)a.partial + ir.part0 + (int64_t)cta * 3 * ir.mul;
}

template <typename S, int V, int L, int K>
__device__ __forceinline__ void backward_body(const NormIrrep& ir, int cta, const NormBackward& a,
                                              typename Compute<S>::type (*sums)[kThreads / 32],
                                              typename Compute<S>::type* rows) {
    using C = typename Compute<S>::type;
    constexpr int M = 2 * L + 1;
    const int T = ir.T, t = threadIdx.x % T, G = kThreads / T;
    const int U = ir.mul / V;
    const C inv_d = (C)1 / (C)(M * ir.mul), eps = (C)a.eps;
    C w[K][V], sc[K][V], w2[K][V], acc_w[K][V], acc_s[K][V], acc_n[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = ir.ch + (t + k * T < U ? t + k * T : 0) * V;
        load_param(w[k], (const C*)a.weight, c, (C)1);
        load_param(sc[k], (const C*)a.scale, c, (C)1);
        load_param(w2[k], (const C*)a.next_weight, c, (C)1);
#pragma unroll
        for (int i = 0; i < V; ++i) acc_w[k][i] = acc_s[k][i] = acc_n[k][i] = 0;
    }
    GroupSum<C> sum{sums, T};
    for (int64_t base = (int64_t)cta * G; base < a.n; base += (int64_t)ir.ctas * G) {
        const int64_t row = base + threadIdx.x / T;
        const bool in = row < a.n;
        auto at = [&](const cgtp_rows& q) {
            return q.data ? (const S*)q.data + row * q.stride + ir.off : nullptr;
        };
        const S *b = at(a.b), *h = at(a.h), *gh = at(a.grad_h), *gy = at(a.grad_y);
        const S* z = a.gate.data ? (const S*)a.gate.data + row * a.gate.stride + ir.ch : nullptr;
        Pack<S, V> bp[K][M], hp[K][M], gp[K][M], yp[K][M], zp[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const bool on = in && t + k * T < U;
            const int u = (t + k * T) * V;
#pragma unroll
            for (int m = 0; m < M; ++m) {
                if (on) {
                    bp[k][m] = load_pack<S, V>(b + m * ir.mul + u);
                    if (gh) gp[k][m] = load_pack<S, V>(gh + m * ir.mul + u);
                    if (gy) {
                        hp[k][m] = load_pack<S, V>(h + m * ir.mul + u);
                        yp[k][m] = load_pack<S, V>(gy + m * ir.mul + u);
                    }
                }
            }
            if (on && z) zp[k] = load_pack<S, V>(z + u);
        }
        C s[3] = {0, 0, 0};  // b^2, h^2, next_weight gy h
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (in && t + k * T < U)
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const C v = widen(bp[k][m].v[i]);
                        s[0] += v * v;
                        if (gy) {
                            const C q = widen(hp[k][m].v[i]);
                            s[1] += q * q;
                            s[2] += w2[k][i] * q * widen(yp[k][m].v[i]);
                        }
                    }
        sum(s);
        const C r = rsqrt_of(s[0] * inv_d + eps), r2 = rsqrt_of(s[1] * inv_d + eps);
        const C mean2 = s[2] * inv_d * r2 * r2;  // times h r': the mean's part of gx / r'
        C gx[K][M][V], sig[K][V], P[K][V], dot[1] = {0};
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (in && t + k * T < U) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    sig[k][i] = z ? sigmoid_of(widen(zp[k].v[i])) : (C)1;
                    P[k][i] = 0;
                }
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        C g = gh ? widen(gp[k][m].v[i]) : (C)0;
                        if (gy) {
                            const C q = widen(hp[k][m].v[i]), y = widen(yp[k][m].v[i]);
                            g += r2 * (w2[k][i] * y - q * mean2);
                            acc_n[k][i] += y * q * r2;
                        }
                        gx[k][m][i] = g;
                        P[k][i] += g * widen(bp[k][m].v[i]);
                    }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    P[k][i] *= r;
                    const C aw = sc[k][i] * sig[k][i];
                    dot[0] += aw * w[k][i] * P[k][i];
                    acc_w[k][i] += aw * P[k][i];
                    acc_s[k][i] += w[k][i] * sig[k][i] * P[k][i];
                }
            }
        sum(dot);
        const C mean = dot[0] * inv_d * r;  // times b r: the mean's part of gb / r
        auto to = [&](const cgtp_rows& q) {
            return q.data ? (S*)q.data + row * q.stride + ir.off : nullptr;
        };
        S *ox = to(a.grad_x), *ob = to(a.grad_b);
        S* oz = a.grad_gate.data ? (S*)a.grad_gate.data + row * a.grad_gate.stride + ir.ch
                                 : nullptr;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (in && t + k * T < U) {
                const int u = (t + k * T) * V;
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    if (ox) {
                        Pack<S, V> p;
#pragma unroll
                        for (int i = 0; i < V; ++i) p.v[i] = narrow<S>(gx[k][m][i]);
                        store_pack(ox + m * ir.mul + u, p);
                    }
                    if (ob) {
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            bp[k][m].v[i] = narrow<S>(
                                r * (sc[k][i] * sig[k][i] * w[k][i] * gx[k][m][i] -
                                     widen(bp[k][m].v[i]) * mean));
                        store_pack(ob + m * ir.mul + u, bp[k][m]);
                    }
                }
                if (oz) {
                    Pack<S, V> p;
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        p.v[i] = narrow<S>(sc[k][i] * w[k][i] * sig[k][i] * ((C)1 - sig[k][i]) *
                                           P[k][i]);
                    store_pack(oz + u, p);
                }
            }
    }
    if (!a.partial) return;
    // The groups' sums, added in group order through shared memory.
    C* out = partial_row<C>(ir, cta, a);
    auto flush = [&](C (&acc)[K][V], int which) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) rows[(threadIdx.x * K + k) * V + i] = acc[k][i];
        __syncthreads();
        for (int c = threadIdx.x; c < ir.mul; c += kThreads) {
            const int u = c / V, k = u / T;
            C s = 0;
            for (int g = 0; g < G; ++g) s += rows[((g * T + u % T) * K + k) * V + c % V];
            out[which * ir.mul + c] = s;
        }
    };
    flush(acc_w, 0);
    flush(acc_s, 1);
    flush(acc_n, 2);
}

template <typename S, int V>
__device__ void backward_wide(const NormIrrep& ir, int cta, const NormBackward& a,
                              typename Compute<S>::type (*sums)[kThreads / 32]) {
    using C = typename Compute<S>::type;
    const int M = 2 * ir.l + 1, U = ir.mul / V;
    const C inv_d = (C)1 / ((C)M * (C)ir.mul), eps = (C)a.eps;
    const C *w = (const C*)a.weight, *sc = (const C*)a.scale, *w2 = (const C*)a.next_weight;
    C* part = a.partial ? partial_row<C>(ir, cta, a) : nullptr;
    if (part)  // a thread's channels are the same in every row
        for (int u = threadIdx.x; u < U; u += kThreads)
            for (int i = 0; i < V; ++i)
                for (int which = 0; which < 3; ++which) part[which * ir.mul + u * V + i] = 0;
    GroupSum<C> sum{sums, kThreads};
    for (int64_t row = cta; row < a.n; row += ir.ctas) {
        auto at = [&](const cgtp_rows& q) {
            return q.data ? (S*)q.data + row * q.stride + ir.off : nullptr;
        };
        const S *b = at(a.b), *h = at(a.h), *gh = at(a.grad_h), *gy = at(a.grad_y);
        S *ox = at(a.grad_x), *ob = at(a.grad_b);
        const S* z = a.gate.data ? (const S*)a.gate.data + row * a.gate.stride + ir.ch : nullptr;
        S* oz = a.grad_gate.data ? (S*)a.grad_gate.data + row * a.grad_gate.stride + ir.ch
                                 : nullptr;
        C s[3] = {0, 0, 0};
        for (int u = threadIdx.x; u < U; u += kThreads) {
            C f[V];
            load_param(f, w2, ir.ch + u * V, (C)1);
            for (int m = 0; m < M; ++m) {
                const int64_t e = (int64_t)m * ir.mul + (int64_t)u * V;
                const Pack<S, V> p = load_pack<S, V>(b + e);
#pragma unroll
                for (int i = 0; i < V; ++i) s[0] += widen(p.v[i]) * widen(p.v[i]);
                if (gy) {
                    const Pack<S, V> q = load_pack<S, V>(h + e), y = load_pack<S, V>(gy + e);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        s[1] += widen(q.v[i]) * widen(q.v[i]);
                        s[2] += f[i] * widen(q.v[i]) * widen(y.v[i]);
                    }
                }
            }
        }
        sum(s);
        const C r = rsqrt_of(s[0] * inv_d + eps), r2 = rsqrt_of(s[1] * inv_d + eps);
        const C mean2 = s[2] * inv_d * r2 * r2;
        // gx of element i of pack e, computed the same way in both passes
        auto grad = [&](C g, C q, C y, C f) { return gy ? g + r2 * (f * y - q * mean2) : g; };
        C dot[1] = {0};
        for (int u = threadIdx.x; u < U; u += kThreads) {
            const int c = ir.ch + u * V;
            C f[V], P[V], Q[V];
            load_param(f, w2, c, (C)1);
#pragma unroll
            for (int i = 0; i < V; ++i) P[i] = Q[i] = 0;
            for (int m = 0; m < M; ++m) {
                const int64_t e = (int64_t)m * ir.mul + (int64_t)u * V;
                const Pack<S, V> p = load_pack<S, V>(b + e);
                Pack<S, V> g, q, y;
                if (gh) g = load_pack<S, V>(gh + e);
                if (gy) q = load_pack<S, V>(h + e), y = load_pack<S, V>(gy + e);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const C qv = gy ? widen(q.v[i]) : (C)0, yv = gy ? widen(y.v[i]) : (C)0;
                    P[i] += grad(gh ? widen(g.v[i]) : (C)0, qv, yv, f[i]) * widen(p.v[i]);
                    Q[i] += yv * qv * r2;
                }
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                P[i] *= r;
                const C wi = w ? w[c + i] : (C)1, si = sc ? sc[c + i] : (C)1;
                const C sig = z ? sigmoid_of(widen(z[u * V + i])) : (C)1;
                dot[0] += si * sig * wi * P[i];
                if (oz) oz[u * V + i] = narrow<S>(si * wi * sig * ((C)1 - sig) * P[i]);
                if (part) {
                    part[u * V + i] += si * sig * P[i];
                    part[ir.mul + u * V + i] += wi * sig * P[i];
                    part[2 * ir.mul + u * V + i] += Q[i];
                }
            }
        }
        sum(dot);
        const C mean = dot[0] * inv_d * r;
        if (ox || ob)
            for (int u = threadIdx.x; u < U; u += kThreads) {
                const int c = ir.ch + u * V;
                C f[V], aw[V];
                load_param(f, w2, c, (C)1);
                load_param(aw, w, c, (C)1);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    aw[i] *= (sc ? sc[c + i] : (C)1) *
                             (z ? sigmoid_of(widen(z[u * V + i])) : (C)1);
                for (int m = 0; m < M; ++m) {
                    const int64_t e = (int64_t)m * ir.mul + (int64_t)u * V;
                    Pack<S, V> p = load_pack<S, V>(b + e), g, q, y;
                    if (gh) g = load_pack<S, V>(gh + e);
                    if (gy) q = load_pack<S, V>(h + e), y = load_pack<S, V>(gy + e);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const C qv = gy ? widen(q.v[i]) : (C)0, yv = gy ? widen(y.v[i]) : (C)0;
                        const C gx = grad(gh ? widen(g.v[i]) : (C)0, qv, yv, f[i]);
                        g.v[i] = narrow<S>(gx);
                        p.v[i] = narrow<S>(r * (aw[i] * gx - widen(p.v[i]) * mean));
                    }
                    if (ox) store_pack(ox + e, g);
                    if (ob) store_pack(ob + e, p);
                }
            }
    }
}

template <typename S, int V, int LC>
__global__ void __launch_bounds__(kThreads)
norm_backward_kernel(const __grid_constant__ NormTable tab,
                     const __grid_constant__ NormBackward a) {
    using C = typename Compute<S>::type;
    __shared__ C sums[6][kThreads / 32];
    extern __shared__ __align__(16) unsigned char dynamic[];
    C* rows = reinterpret_cast<C*>(dynamic);
    int i = 0;
    while (i + 1 < tab.n && (int)blockIdx.x >= tab.ir[i + 1].cta0) ++i;
    const NormIrrep& ir = tab.ir[i];
    const int cta = blockIdx.x - ir.cta0;
#define CALL(L, K) backward_body<S, V, L, K>(ir, cta, a, sums, rows)
    CGTP_NORM_BODIES(LC, CALL, (backward_wide<S, V>(ir, cta, a, sums)))
#undef CALL
}

// Adds the CTAs' partial rows: 32 sums a CTA, eight threads each walking every
// eighth row, joined in order.
template <typename C>
__global__ void __launch_bounds__(256)
norm_reduce_kernel(const __grid_constant__ NormTable tab, const C* __restrict__ partial,
                   int channels, C* __restrict__ gw, C* __restrict__ gs, C* __restrict__ gn) {
    __shared__ C part[8][32];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), lane = threadIdx.x >> 5;
    const int which = blockIdx.y;
    C* out = which == 0 ? gw : which == 1 ? gs : gn;
    C s = 0;
    if (out && col < channels) {
        int i = 0;
        while (i + 1 < tab.n && col >= tab.ir[i + 1].ch) ++i;
        const NormIrrep& ir = tab.ir[i];
        const C* p = partial + ir.part0 + which * ir.mul + (col - ir.ch);
        for (int r = lane; r < ir.ctas; r += 8) s += p[(int64_t)r * 3 * ir.mul];
    }
    part[lane][threadIdx.x & 31] = s;
    __syncthreads();
    if (lane == 0 && out && col < channels) {
        for (int j = 1; j < 8; ++j) s += part[j][threadIdx.x];
        out[col] = s;
    }
}

// ------------------------------------------------------------ launching --

// T, K and the CTAs of each irrep for vectors of V channels.
template <typename S>
void shape_table(NormTable& tab, int V, int64_t n) {
    int cta0 = 0;
    for (int i = 0; i < tab.n; ++i) {
        NormIrrep& ir = tab.ir[i];
        const int U = ir.mul / V;
        int T = 1;
        while (T < U && T < kThreads) T *= 2;
        const int most = ir.l == 0 ? 8 : ir.l == 1 ? 2 : 1;
        int K = 1;
        while (K * T < U && K <= most) K *= 2;
        if (K > most) K = 0, T = kThreads;  // the body that reads again
        ir.T = T;
        ir.K = K;
        const int64_t G = kThreads / T;
        ir.ctas = (int)std::max<int64_t>(1, std::min<int64_t>(ir.max_ctas, (n + G - 1) / G));
        ir.cta0 = cta0;
        cta0 += ir.ctas;
    }
    tab.ctas = cta0;
}

template <typename S, int V, int LC>
cudaError_t forward_v(const NormTable& tab, const NormForward& a, cudaStream_t s) {
    norm_forward_kernel<S, V, LC><<<tab.ctas, kThreads, 0, s>>>(tab, a);
    count_launch();
    return cudaGetLastError();
}

template <typename S, int V, int LC>
cudaError_t backward_v(const NormTable& tab, const NormBackward& a, cudaStream_t s) {
    using C = typename Compute<S>::type;
    size_t smem = 0;  // one set of channel sums of every thread
    for (int i = 0; i < tab.n; ++i)
        smem = std::max(smem, (size_t)kThreads * std::max(1, tab.ir[i].K) * V * sizeof(C));
    if (!a.partial) smem = 0;
    cudaError_t e = cudaFuncSetAttribute(norm_backward_kernel<S, V, LC>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kThreads * 8 * V * (int)sizeof(C));
    if (e != cudaSuccess) return e;
    norm_backward_kernel<S, V, LC><<<tab.ctas, kThreads, smem, s>>>(tab, a);
    count_launch();
    e = cudaGetLastError();
    if (e != cudaSuccess || !a.partial) return e;
    const dim3 grid((unsigned)((a.channels + 31) / 32), 3);
    norm_reduce_kernel<C><<<grid, 256, 0, s>>>(tab, (const C*)a.partial, a.channels,
                                               (C*)a.grad_weight, (C*)a.grad_scale,
                                               (C*)a.grad_next_weight);
    count_launch();
    return cudaGetLastError();
}

#define CGTP_NORM_LAUNCH(NAME, ARGS)                                            \
    template <typename S>                                                       \
    cudaError_t NAME(NormTable tab, const ARGS& a, bool vectors, cudaStream_t s) { \
        constexpr int W = sizeof(S) == 8 ? 2 : 4;                               \
        shape_table<S>(tab, vectors ? W : 1, a.n);                              \
        int l = 0;                                                              \
        for (int i = 0; i < tab.n; ++i) l = std::max(l, tab.ir[i].l);           \
        if (vectors)                                                            \
            return l == 0   ? NAME##_v<S, W, 0>(tab, a, s)                      \
                   : l <= 3 ? NAME##_v<S, W, 3>(tab, a, s)                      \
                            : NAME##_v<S, W, 6>(tab, a, s);                     \
        return l == 0   ? NAME##_v<S, 1, 0>(tab, a, s)                          \
               : l <= 3 ? NAME##_v<S, 1, 3>(tab, a, s)                          \
                        : NAME##_v<S, 1, 6>(tab, a, s);                         \
    }
CGTP_NORM_LAUNCH(forward, NormForward)
CGTP_NORM_LAUNCH(backward, NormBackward)

}  // namespace

}  // namespace cgtp
