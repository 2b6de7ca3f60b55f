// kda_delta_tc.h -- the tensor-core path of the delta rule with one decay per value head.
#pragma once

#include "kda_delta.cuh"

namespace kda {

// bf16 rows, at least `fewest` of them per sequence on average. Workspaces are sized by this alone: where the rows lie is no part of a shape.
bool delta_tc_shape(kda_dtype dtype, const DeltaParams &p, int fewest);
// And TMA can load them (16-byte aligned).
bool delta_tc_supported(kda_dtype dtype, const DeltaParams &p, int fewest);
// The blocks' order of packed sequences: workspace bytes (0: none), and its making (into p.order).
size_t delta_tc_order_bytes(const DeltaParams &p);
cudaError_t launch_delta_tc_order(DeltaParams &p, void *ws, cudaStream_t s);
cudaError_t launch_delta_tc(const DeltaParams &p, cudaStream_t s);

// What the gradients keep of the forward pass, per chunk (number of first_chunk) and value head.
struct DeltaKept {
    uint8_t *tp;  // operands T - I, three bf16 values, and P, two
    float *S;     // the state before the chunk [dk, dv]
    float *U;     // its written values [64, dv]
};
constexpr uint32_t kDeltaP = 24576, kDeltaTpBytes = 40960;  // where P is, and bytes in all
cudaError_t launch_delta_tc_kept(const DeltaParams &p, const DeltaKept &kept, cudaStream_t s);

// Gradients: workspace bytes, and the launches. dq, dk: per value head where value heads share a key head (p.per > 1).
struct DeltaGradients {
    const void *d_o;
    const float *d_fin;
    float *dq, *dk, *dv, *dg, *db, *d_init;
};
size_t delta_tc_backward_bytes(const DeltaParams &p);
cudaError_t launch_delta_tc_backward(const DeltaParams &p, const DeltaGradients &g, void *ws, cudaStream_t s);

}  // namespace kda
