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

// log(1 + exp(x)) without overflow or loss for small results: max(x, 0) + log1p(exp(-|x|)).
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }

constexpr float kLog2e = 1.4426950408889634f;

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
