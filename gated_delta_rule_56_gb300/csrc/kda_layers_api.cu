// kda_layers_api.cu -- the C ABI of the operators around the mixer: host-side checks and launches.
//
// As in kda_api.cu, every check that can be made on the host is made before anything is queued.
#include <cmath>
#include <cstring>

#include "kda_layers.cuh"
#include "kda_layers.h"

using namespace kda;

namespace {

__global__ void __launch_bounds__(128) seqs_kernel(Seqs seqs, unsigned *err) { check_seqs(seqs, err); }

// The caller's argument struct, read up to the size it was compiled with.
template <typename A>
kda_status read_args(const A *user, A &a, const char *name) {
    memset(&a, 0, sizeof(a));
    if (!user) return fail(KDA_ERR_INVALID_ARG, "%s is NULL", name);
    if (user->struct_size < sizeof(size_t) || user->struct_size > 4096)
        return fail(KDA_ERR_INVALID_ARG, "%s.struct_size=%zu is not the size of the struct", name, user->struct_size);
    memcpy(&a, user, user->struct_size < sizeof(A) ? user->struct_size : sizeof(A));
    a.struct_size = sizeof(A);
    return KDA_OK;
}

bool aligned_to(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int esize(kda_dtype dt) { return dt == KDA_BF16 ? 2 : 4; }

// An input of `rows` rows that the call reads: present, element-aligned, its rows not overlapping.
kda_status check_rows(const void *p, const char *name, kda_dtype dt, int64_t stride, long long width) {
    if (!p) return fail(KDA_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned_to(p, esize(dt))) return fail(KDA_ERR_INVALID_ARG, "%s is not aligned to its element size", name);
    if (stride != 0 && (stride < width || stride > (int64_t(1) << 31)))
        return fail(KDA_ERR_INVALID_ARG, "%s: a row stride of %lld for rows of %lld elements", name, (long long)stride, width);
    return KDA_OK;
}

kda_status check_optional(const void *p, const char *name, size_t align) {
    if (p && !aligned_to(p, align)) return fail(KDA_ERR_INVALID_ARG, "%s is not aligned to its element size", name);
    return KDA_OK;
}

kda_status check_given(const void *p, const char *name, size_t align) {
    if (!p) return fail(KDA_ERR_INVALID_ARG, "%s is NULL", name);
    return check_optional(p, name, align);
}

kda_status check_workspace(const void *ws, size_t bytes, size_t need) {
    if (need && (!ws || bytes < need || !aligned16(ws)))
        return fail(KDA_ERR_INVALID_ARG, "workspace: %zu bytes at a 16-byte aligned address needed, got %zu", need,
                    ws ? bytes : (size_t)0);
    return KDA_OK;
}

// Sizes, packed sequences and state pools, which the convolution and the scan share.
template <typename A>
kda_status check_sequences(const A &a, bool decode, bool pools) {
    if (a.B < 0 || a.T < 0) return fail(KDA_ERR_INVALID_ARG, "negative size B=%d T=%d", a.B, a.T);
    if ((long long)a.B * a.T > 0x7fffffffLL - 4096) return fail(KDA_ERR_INVALID_ARG, "too many rows: B=%d T=%d", a.B, a.T);
    if (decode) {
        if (a.T != 1) return fail(KDA_ERR_INVALID_ARG, "decode: T=%d must be 1", a.T);
        if (a.cu_seqlens) return fail(KDA_ERR_INVALID_ARG, "decode takes no cu_seqlens");
        if (a.initial_state) return fail(KDA_ERR_INVALID_ARG, "decode takes its state as `state`, not initial_state");
        if (a.final_state_indices && !a.initial_state_indices)
            return fail(KDA_ERR_INVALID_ARG, "decode: final_state_indices needs initial_state_indices");
    }
    if (a.cu_seqlens) {
        if (a.B != 1) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens requires B == 1 (got B=%d)", a.B);
        if (a.n_seqs < 0) return fail(KDA_ERR_INVALID_ARG, "n_seqs=%d is negative", a.n_seqs);
        if (!aligned_to(a.cu_seqlens, 4)) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens is not 4-byte aligned");
    }
    if (a.initial_state_indices || a.final_state_indices) {
        if (!pools) return fail(KDA_ERR_UNSUPPORTED, "the backward pass takes no state pools");
        if (a.state_pool_size <= 0)
            return fail(KDA_ERR_INVALID_ARG, "state_pool_size=%d must be positive when state indices are given",
                        a.state_pool_size);
        if (!aligned_to(a.initial_state_indices, 4) || !aligned_to(a.final_state_indices, 4))
            return fail(KDA_ERR_INVALID_ARG, "state index arrays must be 4-byte aligned");
        if (!decode && a.initial_state_indices && !a.initial_state)
            return fail(KDA_ERR_INVALID_ARG, "initial_state_indices given without initial_state (the pool)");
    }
    return KDA_OK;
}

template <typename A>
long long sequences(const A &a) {
    return a.cu_seqlens ? a.n_seqs : a.B;
}

// Rows that belong to no sequence would be left out.
template <typename A>
kda_status check_some_sequence(const A &a) {
    const long long rows = (long long)a.B * a.T;
    if (sequences(a) == 0 && rows > 0) return fail(KDA_ERR_INVALID_ARG, "no sequences for %lld rows", rows);
    return KDA_OK;
}

kda_status check_conv(const kda_conv_args &a, bool decode, bool pools) {
    kda_status st;
    if ((st = check_dtype(a.dtype)) || (st = check_sequences(a, decode, pools))) return st;
    if (a.C < 0) return fail(KDA_ERR_INVALID_ARG, "negative size C=%d", a.C);
    if (a.W < 1) return fail(KDA_ERR_INVALID_ARG, "W=%d must be positive", a.W);
    if (a.W < 2 || a.W > 4) return fail(KDA_ERR_UNSUPPORTED, "filter width W=%d: supported 2, 3, 4", a.W);
    if (a.C > (1 << 20)) return fail(KDA_ERR_UNSUPPORTED, "C=%d: at most %d channels", a.C, 1 << 20);
    if (a.activation != 0 && a.activation != 1) return fail(KDA_ERR_INVALID_ARG, "unknown activation %d", a.activation);
    if (a.C == 0) return KDA_OK;
    const size_t e = esize(a.dtype);
    if ((long long)a.B * a.T > 0)
        if ((st = check_rows(a.x, "x", a.dtype, a.x_stride, a.C)) || (st = check_given(a.weight, "weight", e))) return st;
    if ((st = check_optional(a.bias, "bias", e)) || (st = check_optional(a.initial_state, "initial_state", e))) return st;
    return KDA_OK;
}

kda_status check_scan(const kda_scan_args &a, bool decode, bool pools) {
    kda_status st;
    if ((st = check_dtype(a.dtype)) || (st = check_sequences(a, decode, pools))) return st;
    if (a.D < 0) return fail(KDA_ERR_INVALID_ARG, "negative size D=%d", a.D);
    if (a.N < 1 || a.G < 1) return fail(KDA_ERR_INVALID_ARG, "N=%d G=%d must be positive", a.N, a.G);
    if (a.N > 256) return fail(KDA_ERR_UNSUPPORTED, "N=%d: at most 256 states per channel", a.N);
    if (a.D > 65536) return fail(KDA_ERR_UNSUPPORTED, "D=%d: at most 65536 channels", a.D);
    if (a.G > 32768) return fail(KDA_ERR_UNSUPPORTED, "G=%d: at most 32768 groups", a.G);
    if (a.D % a.G != 0) return fail(KDA_ERR_INVALID_ARG, "D=%d is not a multiple of G=%d", a.D, a.G);
    if (a.D == 0) return KDA_OK;
    const long long gn = (long long)a.G * a.N;
    if ((long long)a.B * a.T > 0) {
        if ((st = check_rows(a.x, "x", a.dtype, a.x_stride, a.D)) || (st = check_rows(a.dt, "dt", a.dtype, a.dt_stride, a.D)) ||
            (st = check_rows(a.Bm, "B", a.dtype, a.B_stride, gn)) || (st = check_rows(a.Cm, "C", a.dtype, a.C_stride, gn)) ||
            (st = check_given(a.A, "A", 4)))
            return st;
        if (a.z && (st = check_rows(a.z, "z", a.dtype, a.z_stride, a.D))) return st;
    }
    if ((st = check_optional(a.Dskip, "D", 4)) || (st = check_optional(a.dt_bias, "dt_bias", 4)) ||
        (st = check_optional(a.initial_state, "initial_state", 4)))
        return st;
    return KDA_OK;
}

kda_status check_rotary(const kda_rotary_args &a) {
    kda_status st;
    if ((st = check_dtype(a.dtype))) return st;
    if (a.rows < 0 || a.q_heads < 0 || a.k_heads < 0)
        return fail(KDA_ERR_INVALID_ARG, "negative size rows=%lld q_heads=%d k_heads=%d", (long long)a.rows, a.q_heads, a.k_heads);
    if (a.rows > 0x7fffffffLL || a.q_heads > 65536 || a.k_heads > 65536)
        return fail(KDA_ERR_INVALID_ARG, "too many rows or heads");
    if (a.head <= 0) return fail(KDA_ERR_INVALID_ARG, "head=%d must be positive", a.head);
    if (a.head % 8 != 0 || a.head > 256)
        return fail(KDA_ERR_UNSUPPORTED, "head=%d: supported multiples of 8 up to 256", a.head);
    if (a.half < 0 || 2 * (long long)a.half > a.head)
        return fail(KDA_ERR_INVALID_ARG, "half=%d rotated pairs do not fit a head of %d", a.half, a.head);
    if (a.half % (a.interleaved ? 4 : 8) != 0)
        return fail(KDA_ERR_UNSUPPORTED, "half=%d rotated pairs: supported multiples of %d", a.half, a.interleaved ? 4 : 8);
    if (a.norm != 0 && a.norm != 1) return fail(KDA_ERR_INVALID_ARG, "unknown norm %d", a.norm);
    if (!(a.eps >= 0.f) || std::isinf(a.eps)) return fail(KDA_ERR_INVALID_ARG, "eps=%g must be finite and not negative", (double)a.eps);
    if (a.rows == 0) return KDA_OK;
    if (a.q_heads && (st = check_rows(a.q, "q", a.dtype, a.q_stride, (long long)a.q_heads * a.head))) return st;
    if (a.k_heads && (st = check_rows(a.k, "k", a.dtype, a.k_stride, (long long)a.k_heads * a.head))) return st;
    if ((st = check_optional(a.q_weight, "q_weight", esize(a.dtype))) ||
        (st = check_optional(a.k_weight, "k_weight", esize(a.dtype))))
        return st;
    if (a.half) {
        if (a.table_rows < 0) return fail(KDA_ERR_INVALID_ARG, "table_rows=%lld is negative", (long long)a.table_rows);
        if ((st = check_given(a.cos_table, "cos_table", 4)) || (st = check_given(a.sin_table, "sin_table", 4)) ||
            (st = check_given(a.positions, "positions", 4)))
            return st;
    }
    return KDA_OK;
}

// Without rows no kernel goes over them and looks at cu_seqlens: this call does.
template <typename A>
kda_status check_no_rows(const A &a, unsigned *err, cudaStream_t s) {
    if (!a.cu_seqlens || a.T > 0) return KDA_OK;
    seqs_kernel<<<1, 128, 0, s>>>(Seqs{a.cu_seqlens, a.n_seqs, 0, 0}, err);
    return launched(cudaGetLastError(), "cu_seqlens");
}

kda_status no_error_word() { return fail(KDA_ERR_CUDA, "cannot reach the device error word: %s", cudaGetErrorString(cudaGetLastError())); }

cudaStream_t as_stream(kda_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

extern "C" {

kda_status kda_conv_prefill(const kda_conv_args *args, void *y, void *final_state, kda_stream_t stream) {
    kda_conv_args a;
    kda_status st;
    if ((st = read_args(args, a, "kda_conv_args")) || (st = check_conv(a, false, true))) return st;
    const size_t e = esize(a.dtype);
    if (a.final_state_indices && !final_state)
        return fail(KDA_ERR_INVALID_ARG, "final_state_indices given without final_state (the pool)");
    if ((st = check_optional(final_state, "final_state", e))) return st;
    if (a.C == 0) return ok();
    if ((st = check_some_sequence(a))) return st;
    if (sequences(a) == 0 && !a.cu_seqlens) return ok();
    if ((long long)a.B * a.T > 0 && (st = check_given(y, "y", e))) return st;
    unsigned *err = device_error_word();
    if (!err) return no_error_word();
    if ((st = check_no_rows(a, err, as_stream(stream))) || sequences(a) == 0) return st;
    return launched(launch_conv_prefill(a, y, final_state, err, as_stream(stream)), "convolution");
}

kda_status kda_conv_decode_step(const kda_conv_args *args, void *state, void *y, kda_stream_t stream) {
    kda_conv_args a;
    kda_status st;
    if ((st = read_args(args, a, "kda_conv_args")) || (st = check_conv(a, true, true))) return st;
    if (a.C == 0 || a.B == 0) return ok();
    const size_t e = esize(a.dtype);
    if ((st = check_given(state, "state", e)) || (st = check_given(y, "y", e))) return st;
    unsigned *err = device_error_word();
    if (!err) return no_error_word();
    return launched(launch_conv_decode(a, state, y, err, as_stream(stream)), "convolution decode step");
}

size_t kda_conv_backward_workspace_size(const kda_conv_args *args) {
    kda_conv_args a;
    if (read_args(args, a, "kda_conv_args") || check_conv(a, false, false)) return 0;
    return conv_backward_workspace_bytes(a);
}

kda_status kda_conv_backward(const kda_conv_args *args, const void *dy, const float *d_final_state, float *dx, float *dweight,
                             float *dbias, float *d_initial_state, void *workspace, size_t workspace_bytes,
                             kda_stream_t stream) {
    kda_conv_args a;
    kda_status st;
    if ((st = read_args(args, a, "kda_conv_args")) || (st = check_conv(a, false, false))) return st;
    if (a.C == 0) return ok();
    const long long rows = (long long)a.B * a.T;
    if (rows > 0 && ((st = check_given(dy, "dy", esize(a.dtype))) || (st = check_given(dx, "dx", 4)))) return st;
    if ((st = check_given(dweight, "dweight", 4)) || (st = check_optional(dbias, "dbias", 4)) ||
        (st = check_optional(d_final_state, "d_final_state", 4)) || (st = check_optional(d_initial_state, "d_initial_state", 4)) ||
        (st = check_workspace(workspace, workspace_bytes, conv_backward_workspace_bytes(a))))
        return st;
    if ((st = check_some_sequence(a))) return st;
    unsigned *err = device_error_word();
    if (!err) return no_error_word();
    if ((st = check_no_rows(a, err, as_stream(stream)))) return st;
    return launched(launch_conv_backward(a, dy, d_final_state, dx, dweight, dbias, sequences(a) ? d_initial_state : nullptr,
                                         workspace, err, as_stream(stream)),
                    "convolution backward");
}

size_t kda_scan_prefill_workspace_size(const kda_scan_args *args) {
    kda_scan_args a;
    if (read_args(args, a, "kda_scan_args") || check_scan(a, false, true)) return 0;
    return scan_prefill_workspace_bytes(a, current_sms());
}

kda_status kda_scan_prefill(const kda_scan_args *args, void *y, float *final_state, void *workspace, size_t workspace_bytes,
                            kda_stream_t stream) {
    kda_scan_args a;
    kda_status st;
    if ((st = read_args(args, a, "kda_scan_args")) || (st = check_scan(a, false, true))) return st;
    if (a.final_state_indices && !final_state)
        return fail(KDA_ERR_INVALID_ARG, "final_state_indices given without final_state (the pool)");
    if ((st = check_optional(final_state, "final_state", 4))) return st;
    if (a.D == 0) return ok();
    if ((st = check_some_sequence(a))) return st;
    if (sequences(a) == 0 && !a.cu_seqlens) return ok();
    if ((long long)a.B * a.T > 0 && (st = check_given(y, "y", esize(a.dtype)))) return st;
    const int sms = current_sms();
    if ((st = check_workspace(workspace, workspace_bytes, scan_prefill_workspace_bytes(a, sms)))) return st;
    unsigned *err = device_error_word();
    if (!err) return no_error_word();
    if ((st = check_no_rows(a, err, as_stream(stream))) || sequences(a) == 0) return st;
    return launched(launch_scan_prefill(a, y, final_state, workspace, sms, err, as_stream(stream)), "scan");
}

kda_status kda_scan_decode_step(const kda_scan_args *args, float *state, void *y, kda_stream_t stream) {
    kda_scan_args a;
    kda_status st;
    if ((st = read_args(args, a, "kda_scan_args")) || (st = check_scan(a, true, true))) return st;
    if (a.D == 0 || a.B == 0) return ok();
    if ((st = check_given(state, "state", 4)) || (st = check_given(y, "y", esize(a.dtype)))) return st;
    unsigned *err = device_error_word();
    if (!err) return no_error_word();
    return launched(launch_scan_decode(a, state, y, err, as_stream(stream)), "scan decode step");
}

size_t kda_scan_backward_workspace_size(const kda_scan_args *args) {
    kda_scan_args a;
    if (read_args(args, a, "kda_scan_args") || check_scan(a, false, false)) return 0;
    return scan_backward_workspace_bytes(a, current_sms());
}

kda_status kda_scan_backward(const kda_scan_args *args, const kda_scan_grads *grads, void *workspace, size_t workspace_bytes,
                             kda_stream_t stream) {
    kda_scan_args a;
    kda_scan_grads g;
    kda_status st;
    if ((st = read_args(args, a, "kda_scan_args")) || (st = read_args(grads, g, "kda_scan_grads")) ||
        (st = check_scan(a, false, false)))
        return st;
    if (a.D == 0) return ok();
    const long long rows = (long long)a.B * a.T;
    if (rows > 0) {
        if ((st = check_given(g.dy, "dy", esize(a.dtype))) || (st = check_given(g.dx, "dx", 4)) ||
            (st = check_given(g.ddt, "ddt", 4)) || (st = check_given(g.dB, "dB", 4)) || (st = check_given(g.dC, "dC", 4)))
            return st;
        if (a.z && (st = check_given(g.dz, "dz", 4))) return st;
    }
    if ((st = check_given(g.dA, "dA", 4)) || (a.Dskip && (st = check_given(g.dDskip, "dD", 4))) ||
        (a.dt_bias && (st = check_given(g.ddt_bias, "ddt_bias", 4))))
        return st;
    if ((!a.z && g.dz) || (!a.Dskip && g.dDskip) || (!a.dt_bias && g.ddt_bias))
        return fail(KDA_ERR_INVALID_ARG, "a gradient is asked for an input that is not given");
    if ((st = check_optional(g.d_final_state, "d_final_state", 4)) || (st = check_optional(g.d_initial_state, "d_initial_state", 4)))
        return st;
    if ((st = check_some_sequence(a))) return st;
    const int sms = current_sms();
    if ((st = check_workspace(workspace, workspace_bytes, scan_backward_workspace_bytes(a, sms)))) return st;
    unsigned *err = device_error_word();
    if (!err) return no_error_word();
    if ((st = check_no_rows(a, err, as_stream(stream)))) return st;
    return launched(launch_scan_backward(a, g, workspace, sms, err, as_stream(stream)), "scan backward");
}

kda_status kda_qk_norm_rotary(const kda_rotary_args *args, void *q_out, void *k_out, kda_stream_t stream) {
    kda_rotary_args a;
    kda_status st;
    if ((st = read_args(args, a, "kda_rotary_args")) || (st = check_rotary(a))) return st;
    if (a.rows == 0 || (!a.q_heads && !a.k_heads)) return ok();
    if ((a.q_heads && (st = check_ptr(q_out, "q_out", true))) || (a.k_heads && (st = check_ptr(k_out, "k_out", true)))) return st;
    unsigned *err = device_error_word();
    if (!err) return no_error_word();
    return launched(launch_rotary(a, q_out, k_out, err, as_stream(stream)), "norm and rotation");
}

size_t kda_qk_norm_rotary_backward_workspace_size(const kda_rotary_args *args) {
    kda_rotary_args a;
    if (read_args(args, a, "kda_rotary_args") || check_rotary(a)) return 0;
    return rotary_backward_workspace_bytes(a, current_sms());
}

kda_status kda_qk_norm_rotary_backward(const kda_rotary_args *args, const void *dq_out, const void *dk_out, float *dq, float *dk,
                                       float *dq_weight, float *dk_weight, void *workspace, size_t workspace_bytes,
                                       kda_stream_t stream) {
    kda_rotary_args a;
    kda_status st;
    if ((st = read_args(args, a, "kda_rotary_args")) || (st = check_rotary(a))) return st;
    if (a.rows > 0) {
        if (a.q_heads && ((st = check_ptr(dq_out, "dq_out", true)) || (st = check_ptr(dq, "dq", true)))) return st;
        if (a.k_heads && ((st = check_ptr(dk_out, "dk_out", true)) || (st = check_ptr(dk, "dk", true)))) return st;
    }
    if ((a.q_weight && (st = check_given(dq_weight, "dq_weight", 4))) || (a.k_weight && (st = check_given(dk_weight, "dk_weight", 4))))
        return st;
    if ((!a.q_weight && dq_weight) || (!a.k_weight && dk_weight))
        return fail(KDA_ERR_INVALID_ARG, "a gradient is asked for a weight that is not given");
    const int sms = current_sms();
    if ((st = check_workspace(workspace, workspace_bytes, rotary_backward_workspace_bytes(a, sms)))) return st;
    unsigned *err = device_error_word();
    if (!err) return no_error_word();
    return launched(launch_rotary_backward(a, dq_out, dk_out, dq, dk, dq_weight, dk_weight, workspace, sms, err, as_stream(stream)),
                    "norm and rotation backward");
}

}  // extern "C"
