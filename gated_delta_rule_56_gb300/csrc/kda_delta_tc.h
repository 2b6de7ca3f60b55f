// kda_delta_tc.h -- the tensor-core path of the delta rule with one decay per value head.
#pragma once

#include "kda_delta.cuh"

namespace kda {

// bf16 rows that TMA can load (16-byte aligned).
bool delta_tc_supported(kda_dtype dtype, const DeltaParams &p);
cudaError_t launch_delta_tc(const DeltaParams &p, cudaStream_t s);

}  // namespace kda
