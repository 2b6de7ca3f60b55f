// kda_layers.h -- launches of the operators around the mixer; the arguments have passed the host checks.
#pragma once

#include "kda_internal.h"

namespace kda {

cudaError_t launch_conv_prefill(const kda_conv_args &a, void *y, void *final_state, unsigned *err, cudaStream_t s);
cudaError_t launch_conv_decode(const kda_conv_args &a, void *state, void *y, unsigned *err, cudaStream_t s);
size_t conv_backward_workspace_bytes(const kda_conv_args &a);
cudaError_t launch_conv_backward(const kda_conv_args &a, const void *dy, const float *d_final, float *dx, float *dweight,
                                 float *dbias, float *d_init, void *ws, unsigned *err, cudaStream_t s);

size_t scan_prefill_workspace_bytes(const kda_scan_args &a, int sms);
cudaError_t launch_scan_prefill(const kda_scan_args &a, void *y, float *final_state, void *ws, int sms, unsigned *err,
                                cudaStream_t s);
cudaError_t launch_scan_decode(const kda_scan_args &a, float *state, void *y, unsigned *err, cudaStream_t s);
size_t scan_backward_workspace_bytes(const kda_scan_args &a, int sms);
cudaError_t launch_scan_backward(const kda_scan_args &a, const kda_scan_grads &g, void *ws, int sms, unsigned *err,
                                 cudaStream_t s);

cudaError_t launch_rotary(const kda_rotary_args &a, void *q_out, void *k_out, unsigned *err, cudaStream_t s);
size_t rotary_backward_workspace_bytes(const kda_rotary_args &a, int sms);
cudaError_t launch_rotary_backward(const kda_rotary_args &a, const void *dq_out, const void *dk_out, float *dq, float *dk,
                                   float *dq_weight, float *dk_weight, void *ws, int sms, unsigned *err, cudaStream_t s);

}  // namespace kda
