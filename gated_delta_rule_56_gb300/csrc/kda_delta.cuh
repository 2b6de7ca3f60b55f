// kda_delta.cuh -- what the kernels of the delta rule with one decay per value head share (kda_delta.cu, kda_delta_backward.cu,
// kda_delta_tc.cu).
#pragma once

#include "kda_layers.cuh"

namespace kda {

struct DeltaParams {
    const void *q, *k, *v;
    long long qs, ks, vs;  // elements between rows
    const float *g, *beta;
    Seqs seqs;
    int hk, hv, per;  // key heads, value heads, value heads per key head
    int dk, dv;
    const float *init;
    const int32_t *init_idx, *fin_idx;
    int pool;
    void *o;
    float *fin;
    unsigned *err;
    const int32_t *order;  // tensor-core kernels: null, or the sequences in the order in which their blocks start
};

// The rows of sequence n; false (and an error) if cu_seqlens makes no sense there. Called by whole blocks.
__device__ __forceinline__ bool rows_of(const DeltaParams &p, int n, long long &begin, long long &end) {
    begin = p.seqs.begin(n);
    end = p.seqs.end(n);
    if (begin >= 0 && end >= begin && end <= p.seqs.rows && (n > 0 || begin == 0) && (n < p.seqs.n_seqs - 1 || end == p.seqs.rows))
        return true;
    if (threadIdx.x == 0) atomicOr(p.err, kErrBadSeqlens);
    return false;
}

// Log-decays below this are taken as this (its exponential is 0 in fp32), so that sums of them keep their small terms; NaN stays.
constexpr float kLeastLogDecay = -128.f;
__device__ __forceinline__ float log_decay(float g) { return g < kLeastLogDecay ? kLeastLogDecay : g; }

// Chunks of `rows` rows restart at every sequence: chunk i of sequence n has the number begin / rows + n + i, which no other chunk has, and
// which is below total / rows + n_seqs.
__device__ __forceinline__ long long first_chunk(long long begin, int n, int rows) { return begin / rows + n; }

}  // namespace kda
