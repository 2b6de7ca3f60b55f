// kda_scan.cuh -- what the selective scan's kernels share: their parameters and the layout of states over lanes.
#pragma once

#include "kda_layers.cuh"
#include "kda_layers.h"

namespace kda {

struct ScanParams {
    const void *x, *dt, *Bm, *Cm, *z;
    long long x_stride, dt_stride, B_stride, C_stride, z_stride;
    const float *A, *D, *dt_bias;
    Seqs seqs;
    int C, N, G;  // channels, states per channel, groups
    bool softplus;
    const float *init;
    const int32_t *init_idx, *fin_idx;
    int pool;
    unsigned *err;
};

inline ScanParams scan_params(const kda_scan_args &a, unsigned *err) {
    ScanParams p{};
    p.x = a.x;
    p.dt = a.dt;
    p.Bm = a.Bm;
    p.Cm = a.Cm;
    p.z = a.z;
    p.x_stride = a.x_stride ? a.x_stride : a.D;
    p.dt_stride = a.dt_stride ? a.dt_stride : a.D;
    p.z_stride = a.z_stride ? a.z_stride : a.D;
    p.B_stride = a.B_stride ? a.B_stride : (long long)a.G * a.N;
    p.C_stride = a.C_stride ? a.C_stride : (long long)a.G * a.N;
    p.A = a.A;
    p.D = a.Dskip;
    p.dt_bias = a.dt_bias;
    p.seqs = Seqs{a.cu_seqlens, a.cu_seqlens ? a.n_seqs : a.B, a.T, (long long)a.B * a.T};
    p.C = a.D;
    p.N = a.N;
    p.G = a.G;
    p.softplus = a.dt_softplus != 0;
    p.init = a.initial_state;
    p.init_idx = a.initial_state_indices;
    p.fin_idx = a.final_state_indices;
    p.pool = a.state_pool_size;
    p.err = err;
    return p;
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
__device__ __forceinline__ float softplus(float x) {
    float a, b;
    unpair(softplus2(both(x)), a, b);
    return a;
}
// sigmoid(z) and z sigmoid(z), two at a time.
__device__ __forceinline__ f32x2 sigmoid2(f32x2 z) {
    float a, b;
    unpair(mul2(z, both(-kLog2e)), a, b);
    return pair(rcp(1.f + ex2(a)), rcp(1.f + ex2(b)));
}
__device__ __forceinline__ f32x2 silu2(f32x2 z) { return mul2(z, sigmoid2(z)); }

// How a call's rows are cut: `chunks` chunks of `rows` rows over all sequences' rows (a chunk may hold several sequences, a
// sequence several chunks). Whole sequences (not packed, enough of them) need no carries between chunks.
struct ScanPlan {
    int chunks;
    long long rows;
    bool carries;
    __host__ __device__ long long windows() const { return (rows + 7) / 8; }  // of kScanWindow rows in a chunk
};
constexpr int kScanWindow = 8;  // rows between the states that the backward pass keeps
enum { kOutputs, kEnds, kStates, kBackEnds };
constexpr int kScanThreads = 128;
ScanPlan scan_plan(const kda_scan_args &a, int sms);
inline int scan_lanes(int N) {  // lanes per channel, 16 states each
    int L = 1;
    while (L * 16 < N) L *= 2;
    return L;
}
inline int scan_blocks(const kda_scan_args &a) {  // channel blocks of all groups, two channels per lane
    const long long per = (long long)a.D / a.G * scan_lanes(a.N);
    return (int)((per + 2 * kScanThreads - 1) / (2 * kScanThreads)) * a.G;
}

// States handed from chunk to chunk, in the workspace.
struct Carries {
    float *state;  // [chunks][C][N]: the chunk's own end state, then the state before the chunk
    float *first;  // [chunks][C][N]: initial state of the sequence that begins in the chunk and goes on after it
    float *time;   // [chunks][C]: sum of the time steps over the chunk's part of its last sequence
    // Backward pass: per window of a chunk, the state before it as the chunk alone gives it, [C][N], and the sum of the time steps
    // since the chunk's first row, [C].
    float *kept, *kept_time;
};

// The states before the windows and the chunks; the gradients at the states after the chunks.
cudaError_t launch_scan_states(const kda_scan_args &a, const ScanPlan &plan, const Carries &carry, unsigned *err, cudaStream_t s);
cudaError_t launch_scan_back_ends(const kda_scan_args &a, const void *dy, const float *d_final, const ScanPlan &plan,
                                  const Carries &carry, unsigned *err, cudaStream_t s);

// Calls f.operator()<T, S, L>() with S states per lane and L lanes per channel, S * L >= N (at most 256).
template <typename F>
cudaError_t scan_by_type(const kda_scan_args &a, F &&f) {
#define KDA_SCAN(S, L)                                                     \
    if (a.N <= S * L) {                                                    \
        if (a.dtype == KDA_BF16)                                           \
            f.template operator()<__nv_bfloat16, S, L>();                  \
        else                                                               \
            f.template operator()<float, S, L>();                          \
        return cudaGetLastError();                                         \
    }
    KDA_SCAN(4, 1)
    KDA_SCAN(8, 1)
    KDA_SCAN(16, 1)
    KDA_SCAN(16, 2)
    KDA_SCAN(16, 4)
    KDA_SCAN(16, 8)
    KDA_SCAN(16, 16)
#undef KDA_SCAN
    return cudaErrorInvalidValue;
}

}  // namespace kda
