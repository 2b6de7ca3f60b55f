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

// V consecutive elements, loaded and stored in 16-byte words (one 8-byte word if that is all); aligned to them.
template <typename T, int V>
struct alignas(V == 1 ? sizeof(T) : V * sizeof(T) >= 16 ? 16 : 8) Pack {
    T e[V];
};

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T *p) {
    Pack<T, V> r;
    if constexpr (V == 1) {
        r.e[0] = *p;
    } else if constexpr (V * sizeof(T) == 8) {
        reinterpret_cast<uint2 &>(r) = *reinterpret_cast<const uint2 *>(p);
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
    } else if constexpr (V * sizeof(T) == 8) {
        *reinterpret_cast<uint2 *>(p) = reinterpret_cast<const uint2 &>(r);
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

constexpr float kLog2e = 1.4426950408889634f;

// Two fp32 values in one register pair: sm_103a multiplies and adds both in one instruction.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(f32x2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// 2^x: at most 2^-22.7 off relatively, 2^x < 2^-126 becomes 0.
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// A step's decays exp(dt A), from A log2(e). A state multiplies up as many of them as it remembers tokens, so their mean error
// counts: the instruction rounds results below 1 down, by 5e-9 to 3e-8 on average for exponents above -0.1. The small
// constant takes a half to all of that back (measured: a state with a memory of 500 tokens is 2e-6 off instead of 5e-6); 2^constant is still 1.
__device__ __forceinline__ f32x2 decay2(f32x2 dt, f32x2 A) {
    float a, b;
    unpair(fma2(dt, A, pair(1.2e-8f, 1.2e-8f)), a, b);
    return pair(ex2(a), ex2(b));
}
__device__ __forceinline__ float decay(float dt, float A) { return ex2(fmaf(dt, A, 1.2e-8f)); }
// Over many rows: h exp(time A) + to, the exponential in two factors. With a growing state (A or time steps of the other sign) one factor
// leaves fp32's range where the product is still inside it, and an infinite one would make NaN of a zero. 2^127 twice takes every state but
// zero past the range, so exponents stop there (NaN stays NaN). The constant: as above, for each factor.
__device__ __forceinline__ float ex2_up_to_127(float x) {
    asm("min.NaN.f32 %0, %0, 0f42FE0000;" : "+f"(x));
    return ex2(x);
}
__device__ __forceinline__ float root_decay(float time, float A) { return ex2_up_to_127(fmaf(0.5f * time, A, 1.2e-8f)); }
__device__ __forceinline__ float carried(float root, float h, float to) { return fmaf(root, root * h, to); }
__device__ __forceinline__ f32x2 carried2(f32x2 time, f32x2 A, f32x2 h, f32x2 to) {
    float a, b;
    unpair(fma2(mul2(time, pair(0.5f, 0.5f)), A, pair(1.2e-8f, 1.2e-8f)), a, b);
    const f32x2 s = pair(ex2_up_to_127(a), ex2_up_to_127(b));
    return fma2(s, mul2(s, h), to);
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ f32x2 both(float a) { return pair(a, a); }

// log(1 + exp(x)) without overflow or loss for small results, two at a time: max(x, 0) + log1p(e), e = exp(-|x|) in (0, 1].
// The exponent's product with log2(e) is taken with its rounding error. log1p(e) / e is a polynomial of degree 9, fitted
// to it at the Chebyshev nodes of [0, 1]: 3e-8 off at most, as its coefficients are rounded here. NaN and +inf stay what they are.
__device__ __forceinline__ f32x2 softplus2(f32x2 x) {
    float x0, x1, m0, m1;
    unpair(x, x0, x1);
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(m0) : "f"(x0));
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(m1) : "f"(x1));
    const f32x2 a = pair(fmaxf(-fabsf(x0), -87.f), fmaxf(-fabsf(x1), -87.f));
    const f32x2 minus = mul2(a, both(-kLog2e)), rest = fma2(a, both(kLog2e), minus);
    float t0, t1;
    unpair(minus, t0, t1);
    f32x2 e = pair(ex2(-t0), ex2(-t1));
    e = fma2(mul2(e, rest), both(0.69314718f), e);
    f32x2 q = both(-0x1.aad1eep-9f);
    q = fma2(q, e, both(0x1.4628b0p-6f));
    q = fma2(q, e, both(-0x1.d3784ep-5f));
    q = fma2(q, e, both(0x1.b2c2a2p-4f));
    q = fma2(q, e, both(-0x1.399642p-3f));
    q = fma2(q, e, both(0x1.930202p-3f));
    q = fma2(q, e, both(-0x1.ff11c2p-3f));
    q = fma2(q, e, both(0x1.554c9cp-2f));
    q = fma2(q, e, both(-0x1.ffffc0p-2f));
    q = fma2(q, e, both(1.f));
    return fma2(e, q, pair(m0, m1));
}
// sigmoid(z) and z sigmoid(z), two at a time.
__device__ __forceinline__ f32x2 sigmoid2(f32x2 z) {
    float a, b;
    unpair(mul2(z, both(-kLog2e)), a, b);
    return pair(rcp(1.f + ex2(a)), rcp(1.f + ex2(b)));
}
__device__ __forceinline__ f32x2 silu2(f32x2 z) { return mul2(z, sigmoid2(z)); }

// A sum that keeps its rounding errors: as exact as one in 64 bits, which this GPU adds 64 times slower than one in 32.
struct ExactSum {
    float sum = 0.f, rest = 0.f;
    __device__ __forceinline__ void add(float x) {  // the error of a two-term sum, by D. E. Knuth's branch-free formula
        const float t = __fadd_rn(sum, x), b = __fsub_rn(t, sum);
        rest = __fadd_rn(rest, __fadd_rn(__fsub_rn(sum, __fsub_rn(t, b)), __fsub_rn(x, b)));
        sum = t;
    }
    // Past fp32's range the rest is NaN (inf - inf), and the sum alone what it rounds to.
    __device__ __forceinline__ float value() const { return isfinite(sum) ? sum + rest : sum; }
};

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
