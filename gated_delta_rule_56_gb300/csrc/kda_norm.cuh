// kda_norm.cuh -- what the layer norm and its gradients share (kda_norm.cu, kda_norm_backward.cu): lines held by groups of lanes, in
// register pairs, and their sums.
#pragma once

#include "kda_layers.cuh"

namespace kda {

struct NormParams {
    const void *x, *res, *z, *w, *b, *dy, *d_sum;
    long long xs, rs, zs;  // elements between rows
    long long lines;       // rows * heads
    int heads, width;
    float inv, eps;        // 1 / width
    bool rms, silu;
    void *y, *sum;
    float *dx, *dz, *part;  // part: [blocks, 2, width]
};

// V consecutive values as pairs of fp32; the last half of a single value's pair is nothing.
template <typename T, int V>
__device__ __forceinline__ void to_pairs(const Pack<T, V> &p, f32x2 (&x)[(V + 1) / 2]) {
    if constexpr (V == 1) {
        x[0] = pair(to_float(p.e[0]), 0.f);
    } else {
#pragma unroll
        for (int j = 0; j < V; j += 2) x[j / 2] = pair(to_float(p.e[j]), to_float(p.e[j + 1]));
    }
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> from_pairs(const f32x2 (&x)[(V + 1) / 2]) {
    Pack<T, V> p;
#pragma unroll
    for (int j = 0; j < V; j += 2) {
        float a, b;
        unpair(x[j / 2], a, b);
        p.e[j] = from_float<T>(a);
        if constexpr (V > 1) p.e[j + 1] = from_float<T>(b);
    }
    return p;
}
template <int V>
__device__ __forceinline__ void store_pairs(float *p, const f32x2 (&x)[(V + 1) / 2]) {
    float v[V + 1];
#pragma unroll
    for (int j = 0; j < V; j += 2) unpair(x[j / 2], v[j], v[j + 1]);
    if constexpr (V == 1) {
        *p = v[0];
    } else {
#pragma unroll
        for (int j = 0; j < V; j += 4) *reinterpret_cast<float4 *>(p + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    }
}
__device__ __forceinline__ float total(f32x2 x) {
    float a, b;
    unpair(x, a, b);
    return a + b;
}
__device__ __forceinline__ f32x2 minus(f32x2 x) { return x ^ 0x8000000080000000ull; }

// A line of `width` values in the lanes of a group: V at (i * GROUP + lane) * V for i < K.
template <typename T, int V, int K>
struct Line {
    Pack<T, V> e[K];
};
template <typename T, int V, int K, int GROUP>
__device__ __forceinline__ void load_line(Line<T, V, K> &r, const void *p, long long at, int lane, int width) {
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int e = (i * GROUP + lane) * V;
        if (e < width) {
            r.e[i] = load_pack<T, V>(static_cast<const T *>(p) + at + e);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) r.e[i].e[j] = from_float<T>(0.f);
        }
    }
}
// A weight, or `missing` for all.
template <typename T, int V, int K, int GROUP>
__device__ __forceinline__ void load_weight(Line<T, V, K> &r, const void *p, float missing, int lane, int width) {
    if (p) {
        load_line<T, V, K, GROUP>(r, p, 0, lane, width);
    } else {
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) r.e[i].e[j] = from_float<T>(missing);
    }
}

// Sums over the lanes of a group, N at a time; every lane gets them. Whole blocks go through shared memory, two buffers in turn.
template <int GROUP, int N>
__device__ __forceinline__ void sums(float (&x)[N], float (*buf)[3][32], int &turn) {
    constexpr int IN = GROUP < 32 ? GROUP : 32;
#pragma unroll
    for (int a = 0; a < N; ++a)
#pragma unroll
        for (int m = IN / 2; m > 0; m >>= 1) x[a] += __shfl_xor_sync(0xffffffffu, x[a], m);
    if constexpr (GROUP > 32) {
        constexpr int W = GROUP / 32;
        const int lane = threadIdx.x & 31;
        if (lane == 0)
#pragma unroll
            for (int a = 0; a < N; ++a) buf[turn][a][threadIdx.x >> 5] = x[a];
        __syncthreads();
#pragma unroll
        for (int a = 0; a < N; ++a) {
            x[a] = lane < W ? buf[turn][a][lane] : 0.f;
#pragma unroll
            for (int m = W / 2; m > 0; m >>= 1) x[a] += __shfl_xor_sync(0xffffffffu, x[a], m);
            x[a] = __shfl_sync(0xffffffffu, x[a], 0);
        }
        turn ^= 1;
    }
}

template <int GROUP>
constexpr int kBlock = GROUP <= 32 ? 256 : GROUP;

NormParams norm_params(const kda_layer_norm_args &a);

// All of a call's rows, weights and outputs are 16-byte aligned.
template <typename T>
bool wide_lines(const NormParams &p) {
    constexpr int V = 16 / sizeof(T);
    auto ok = [](const void *x, long long stride) { return aligned16(x) && stride % V == 0; };
    return p.width % V == 0 && ok(p.x, p.xs) && ok(p.res, p.res ? p.rs : 0) && ok(p.z, p.z ? p.zs : 0) && ok(p.w, 0) && ok(p.b, 0) &&
           ok(p.y, 0) && ok(p.sum, 0) && ok(p.dy, 0) && ok(p.d_sum, 0) && ok(p.dx, 0) && ok(p.dz, 0);
}

// Calls f.run<V, K, GROUP>() for a width: up to a warp's lanes with one or two packs of V values each, then blocks of up to 1024 threads;
// single values where something is not aligned.
template <int V, typename F>
cudaError_t by_width(int width, bool wide, const F &f) {
    if (wide) {
        const int packs = width / V;
        if (packs <= 8) return f.template run<V, 1, 8>();
        if (packs <= 16) return f.template run<V, 1, 16>();
        if (packs <= 32) return f.template run<V, 1, 32>();
        if (packs <= 64) return f.template run<V, 2, 32>();
        if (packs <= 128) return f.template run<V, 1, 128>();
        if (packs <= 256) return f.template run<V, 2, 128>();
        if (packs <= 512) return f.template run<V, 2, 256>();
        if (packs <= 1024) return f.template run<V, 2, 512>();
        if (packs <= 2048) return f.template run<V, 2, 1024>();
        if (packs <= 4096) return f.template run<V, 4, 1024>();
        if constexpr (V == 4) return f.template run<V, 8, 1024>();
        return cudaErrorInvalidValue;
    }
    if (width <= 64) return f.template run<1, 2, 32>();
    if (width <= 256) return f.template run<1, 8, 32>();
    if (width <= 1024) return f.template run<1, 4, 256>();
    if (width <= 2048) return f.template run<1, 8, 256>();
    if (width <= 8192) return f.template run<1, 8, 1024>();
    return f.template run<1, 32, 1024>();
}

}  // namespace kda
