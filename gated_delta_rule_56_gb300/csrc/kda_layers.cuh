// kda_layers.cuh -- device helpers shared by the operators around the mixer (kda_conv.cu, kda_scan.cu,
// kda_scan_backward.cu, kda_rotary.cu): element conversion, wide rows, and the sequences that rows belong to.
#pragma once

#include "kda_internal.h"

namespace kda {

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// V consecutive elements. V > 1: 16 bytes or a multiple of it (fp32: 4 per 16 bytes, bf16: 8), 16-byte aligned.
template <typename T, int V>
struct alignas(V == 1 ? sizeof(T) : 16) Pack {
    T e[V];
};

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T *p) {
    Pack<T, V> r;
    if constexpr (V == 1) {
        r.e[0] = *p;
    } else {
        static_assert(V * sizeof(T) % 16 == 0, "whole 16-byte words");
#pragma unroll
        for (int i = 0; i < (int)(V * sizeof(T) / 16); ++i)
            reinterpret_cast<uint4 *>(&r)[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    return r;
}

template <typename T, int V>
__device__ __forceinline__ void store_pack(T *p, const Pack<T, V> &r) {
    if constexpr (V == 1) {
        *p = r.e[0];
    } else {
#pragma unroll
        for (int i = 0; i < (int)(V * sizeof(T) / 16); ++i)
            reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<const uint4 *>(&r)[i];
    }
}

template <int V>
__device__ __forceinline__ void store_floats(float *p, const float (&x)[V]) {
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4 *>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = x[i];
    }
}

// sigmoid(x) from the fast exponential and division: relative error below 2^-21 for the results that
// matter in fp32 (an underflowing result becomes 0).
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// The sequences over the rows: n_seqs of T rows each, or packed ones from cu_seqlens.
struct Seqs {
    const int32_t *cu;
    int n_seqs;
    long long T;     // rows per sequence (cu == nullptr)
    long long rows;  // all rows

    __device__ __forceinline__ long long begin(int n) const { return cu ? (long long)cu[n] : n * T; }
    __device__ __forceinline__ long long end(int n) const { return cu ? (long long)cu[n + 1] : (n + 1) * T; }
    // The last sequence that starts at or before `row`; any cu gives an index in [0, n_seqs).
    __device__ __forceinline__ int at(long long row) const {
        if (!cu) {
            const long long n = T > 0 ? row / T : 0;
            return n < n_seqs ? (int)n : n_seqs - 1;
        }
        int lo = 0, hi = n_seqs;  // cu[lo] <= row < cu[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= row) lo = mid; else hi = mid;
        }
        return lo;
    }
};

// Reports a cu_seqlens that is not a non-decreasing list from 0 to `rows`; called by all threads of one block.
__device__ __forceinline__ void check_seqs(const Seqs &s, unsigned *err) {
    if (!s.cu) return;
    bool bad = false;
    for (int n = threadIdx.x + blockDim.x * threadIdx.y; n <= s.n_seqs; n += blockDim.x * blockDim.y) {
        const long long v = s.cu[n];
        bad |= n == 0 ? v != 0 : v < s.cu[n - 1];
        bad |= n == s.n_seqs && v != s.rows;
    }
    if (bad) atomicOr(err, kErrBadSeqlens);
}

// The slot of sequence n in a state tensor, or -1 when it has none there (see kda_options).
__device__ __forceinline__ long long state_slot(const int32_t *idx, int pool, int n, unsigned *err) {
    if (!idx) return n;
    const int slot = idx[n];
    if (slot >= pool) {
        atomicOr(err, kErrBadIndex);
        return -1;
    }
    return slot < 0 ? -1 : slot;
}

}  // namespace kda
