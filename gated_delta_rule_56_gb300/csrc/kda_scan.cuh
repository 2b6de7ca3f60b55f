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

// How a call's rows are cut: `chunks` chunks of `rows` rows over all sequences' rows (a chunk may hold several sequences, a
// sequence several chunks). Whole sequences (not packed, enough of them) need no carries between chunks.
struct ScanPlan {
    int chunks;
    long long rows;
    bool carries;
    // Few chunks: the main kernel's blocks walk over the ones before theirs themselves, and a launch is saved. Measured in a captured
    // graph, itself against the launch: 4 chunks 13.9 us against 15.2 with 128 channels, 16.2 against 20.5 with 8192; 6 chunks 15.6 against
    // 15.6 and 23.2 against 24.7; it is slower from 7 on with 128 to 1024 channels and from 8 on with all (16 chunks: 23.6 against 17.0 with 128 channels, 33.5 against 23.4 with 4096).
    // One eager call after another pays the launch only where the host is the longer side: 16 chunks of 128 channels 49 us against 52.
    __host__ __device__ bool folded() const { return chunks <= 6; }
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
