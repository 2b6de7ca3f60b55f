// kda_conv.cu -- the short causal convolution of a layer's projections: prompts, single tokens, gradients.
//
//     p_t = bias + sum_j w_j x_{t-(W-1)+j},   y_t = p_t or p_t sigmoid(p_t)         (per channel)
//
// Bound by HBM: x is read once and y written once, 2 W + 4 operations per element. A thread owns one
// 16-byte column of channels (8 in bf16, 4 in fp32) and walks down a run of rows with the last W - 1 inputs
// and the filter in registers, so each x row is loaded once per run plus W - 1 rows before it (those hit L2:
// another thread of the same launch streams them). Channels whose rows are not 16-byte aligned go one per thread.
#include "kda_layers.cuh"
#include "kda_layers.h"

namespace kda {
namespace {

constexpr int kLanes = 32;  // threads along the channels
constexpr int kRuns = 8;    // row runs per block

struct ConvParams {
    const void *x, *w, *bias;
    long long x_stride;
    Seqs seqs;
    int C;
    bool silu;
    const void *init;
    const int32_t *init_idx, *fin_idx;
    int pool;
    unsigned *err;
};

template <int W, int V>
struct Filter {
    float w[W][V], b[V];
};

template <typename T, int W, int V>
__device__ __forceinline__ void load_filter(const ConvParams &p, int c, Filter<W, V> &f) {
    const T *pw = static_cast<const T *>(p.w) + (long long)c * W;  // V filters of W values in a row
    T w[V * W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const Pack<T, V> part = load_pack<T, V>(pw + i * V);
#pragma unroll
        for (int v = 0; v < V; ++v) w[i * V + v] = part.e[v];
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < W; ++j) f.w[j][v] = to_float(w[v * W + j]);
    if (p.bias) {
        const Pack<T, V> b = load_pack<T, V>(static_cast<const T *>(p.bias) + c);
#pragma unroll
        for (int v = 0; v < V; ++v) f.b[v] = to_float(b.e[v]);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) f.b[v] = 0.f;
    }
}

// The input of sequence n at row r of the tensor, from the state for the W - 1 rows before `bos`.
template <typename T, int W, int V>
__device__ __forceinline__ Pack<T, V> input_at(const ConvParams &p, long long r, long long bos, long long slot, int c) {
    if (r >= bos) return load_pack<T, V>(static_cast<const T *>(p.x) + r * p.x_stride + c);
    if (slot >= 0)
        return load_pack<T, V>(static_cast<const T *>(p.init) + (slot * (W - 1) + (W - 1) + (r - bos)) * p.C + c);
    Pack<T, V> zero;
#pragma unroll
    for (int v = 0; v < V; ++v) zero.e[v] = from_float<T>(0.f);
    return zero;
}

template <typename T, int W, int V>
__global__ void __launch_bounds__(kLanes *kRuns) conv_prefill_kernel(ConvParams p, T *__restrict__ y, int run_rows) {
    if (blockIdx.x == 0 && blockIdx.y == 0) check_seqs(p.seqs, p.err);
    const int c = (blockIdx.y * kLanes + threadIdx.x) * V;
    if (c >= p.C) return;
    long long r = ((long long)blockIdx.x * kRuns + threadIdx.y) * run_rows;
    const long long stop = min(r + run_rows, p.seqs.rows);
    if (r >= stop) return;
    Filter<W, V> f;
    load_filter<T, W, V>(p, c, f);
    for (int n = p.seqs.at(r); n < p.seqs.n_seqs && r < stop; ++n) {
        const long long bos = p.seqs.begin(n), end = min(p.seqs.end(n), stop);
        if (end <= r || bos > r || bos < 0) continue;  // empty (or a bad cu_seqlens)
        const long long slot = p.init ? state_slot(p.init_idx, p.pool, n, p.err) : -1;
        float x[W][V];  // the last W inputs
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const Pack<T, V> in = input_at<T, W, V>(p, r - (W - 1) + j, bos, slot, c);
#pragma unroll
            for (int v = 0; v < V; ++v) x[j][v] = to_float(in.e[v]);
        }
        const T *px = static_cast<const T *>(p.x) + r * p.x_stride + c;
        T *py = y + r * p.C + c;
        for (; r < end; ++r, px += p.x_stride, py += p.C) {
            const Pack<T, V> in = load_pack<T, V>(px);
            Pack<T, V> out;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                x[W - 1][v] = to_float(in.e[v]);
                float a = f.b[v];
#pragma unroll
                for (int j = 0; j < W; ++j) a = fmaf(f.w[j][v], x[j][v], a);
                out.e[v] = from_float<T>(p.silu ? a * sigmoid(a) : a);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) x[j][v] = x[j + 1][v];
            }
            store_pack<T, V>(py, out);
        }
    }
}

// The state after each sequence: its last W - 1 inputs. All are read before the first is written, so
// that the state may be the one it started from.
template <typename T, int W, int V>
__global__ void conv_state_kernel(ConvParams p, T *fin) {
    const int c = (blockIdx.y * kLanes + threadIdx.x) * V;
    const int n = blockIdx.x;
    if (c >= p.C) return;
    const long long bos = p.seqs.begin(n), eos = p.seqs.end(n);
    if (bos < 0 || eos < bos || eos > p.seqs.rows) return;
    const long long from = p.init ? state_slot(p.init_idx, p.pool, n, p.err) : -1;
    const long long to = state_slot(p.fin_idx, p.pool, n, p.err);
    Pack<T, V> in[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) in[j] = input_at<T, W, V>(p, eos - (W - 1) + j, bos, from, c);
    if (to < 0) return;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_pack<T, V>(fin + (to * (W - 1) + j) * p.C + c, in[j]);
}

template <typename T, int W, int V>
__global__ void conv_decode_kernel(ConvParams p, T *state, T *__restrict__ y) {
    const int c = (blockIdx.y * kLanes + threadIdx.x) * V;
    const int n = blockIdx.x;
    if (c >= p.C) return;
    const long long from = state_slot(p.init_idx, p.pool, n, p.err);
    const long long to = p.fin_idx == p.init_idx ? from : state_slot(p.fin_idx, p.pool, n, p.err);
    p.init = state;
    Pack<T, V> in[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) in[j] = input_at<T, W, V>(p, j - (W - 1), 0, from, c);
    in[W - 1] = load_pack<T, V>(static_cast<const T *>(p.x) + n * p.x_stride + c);
    Filter<W, V> f;
    load_filter<T, W, V>(p, c, f);
    Pack<T, V> out;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float a = f.b[v];
#pragma unroll
        for (int j = 0; j < W; ++j) a = fmaf(f.w[j][v], to_float(in[j].e[v]), a);
        out.e[v] = from_float<T>(p.silu ? a * sigmoid(a) : a);
    }
    store_pack<T, V>(y + (long long)n * p.C + c, out);
    if (to >= 0) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) store_pack<T, V>(state + (to * (W - 1) + j) * p.C + c, in[j + 1]);
    }
}

// Gradients: dp_t = dy_t (SiLU'(p_t)),  dx_t = sum_k w_{W-1-k} dp_{t+k} within the sequence,
// dw_j = sum_t dp_t x_{t-(W-1)+j},  db = sum_t dp_t; the rows before a sequence give its initial state's gradient.
// A thread recomputes p over its run and the W - 1 rows after it. The filter's sums of the block's runs are
// added in shared memory in a fixed order and written to `part` [block][W + 1][C]; conv_reduce_kernel adds those.
template <typename T, int W, int V>
__global__ void __launch_bounds__(kLanes *kRuns) conv_backward_kernel(ConvParams p, const T *__restrict__ dy,
                                                                       const float *__restrict__ d_fin,
                                                                       float *__restrict__ dx, float *__restrict__ d_init,
                                                                       float *__restrict__ part, int run_rows) {
    __shared__ float sums[kRuns][W + 1][kLanes * V];
    if (blockIdx.x == 0 && blockIdx.y == 0) check_seqs(p.seqs, p.err);
    const int c = (blockIdx.y * kLanes + threadIdx.x) * V;
    float dw[W + 1][V];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) dw[j][v] = 0.f;
    long long r = ((long long)blockIdx.x * kRuns + threadIdx.y) * run_rows;
    const long long stop = min(r + run_rows, p.seqs.rows);
    if (c < p.C && r < stop) {
        Filter<W, V> f;
        load_filter<T, W, V>(p, c, f);
        for (int n = p.seqs.at(r); n < p.seqs.n_seqs && r < stop; ++n) {
            const long long bos = p.seqs.begin(n), eos = min(p.seqs.end(n), p.seqs.rows), end = min(eos, stop);
            if (end <= r || bos > r || bos < 0) continue;
            const long long slot = p.init ? n : -1, first = r;
            float x[W][V], dp[W][V];  // the last W inputs and gradients
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                const Pack<T, V> in = input_at<T, W, V>(p, r - (W - 1) + j, bos, slot, c);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    x[j][v] = to_float(in.e[v]);
                    dp[j][v] = 0.f;
                }
            }
            for (; r < end + W - 1; ++r) {
                if (r < eos) {
                    const Pack<T, V> in = load_pack<T, V>(static_cast<const T *>(p.x) + r * p.x_stride + c);
                    const Pack<T, V> d = load_pack<T, V>(dy + r * p.C + c);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        x[W - 1][v] = to_float(in.e[v]);
                        float g = to_float(d.e[v]);
                        if (p.silu) {
                            float a = f.b[v];
#pragma unroll
                            for (int j = 0; j < W; ++j) a = fmaf(f.w[j][v], x[j][v], a);
                            const float sg = sigmoid(a);
                            g *= sg * fmaf(a, 1.f - sg, 1.f);
                        }
                        dp[W - 1][v] = g;
                        if (r < end) {
#pragma unroll
                            for (int j = 0; j < W; ++j) dw[j][v] = fmaf(g, x[j][v], dw[j][v]);
                            dw[W][v] += g;
                        }
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) dp[W - 1][v] = 0.f;
                }
                // Row q of the sequence has all its gradients now; q < bos is a row of the initial state.
                const long long q = r - (W - 1);
                if (q >= first || (first == bos && d_init)) {
                    float g[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        g[v] = 0.f;
#pragma unroll
                        for (int k = 0; k < W; ++k) g[v] = fmaf(f.w[W - 1 - k][v], dp[k][v], g[v]);
                    }
                    if (d_fin && q >= eos - (W - 1)) {
                        const float *df = d_fin + ((long long)n * (W - 1) + (q - (eos - (W - 1)))) * p.C + c;
#pragma unroll
                        for (int v = 0; v < V; ++v) g[v] += df[v];
                    }
                    store_floats<V>(q >= bos ? dx + q * p.C + c : d_init + ((long long)n * (W - 1) + (W - 1) + (q - bos)) * p.C + c,
                                    g);
                }
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) {
                        x[j][v] = x[j + 1][v];
                        dp[j][v] = dp[j + 1][v];
                    }
            }
            r = end;
        }
    }
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) sums[threadIdx.y][j][v * kLanes + threadIdx.x] = dw[j][v];
    __syncthreads();
    for (int i = threadIdx.y * kLanes + threadIdx.x; i < (W + 1) * kLanes * V; i += kLanes * kRuns) {
        const int j = i / (kLanes * V), k = i % (kLanes * V);  // k: channel lane * V + v
        const int ch = blockIdx.y * kLanes * V + k;
        float sum = 0.f;
#pragma unroll
        for (int y = 0; y < kRuns; ++y) sum += sums[y][j][(k % V) * kLanes + k / V];
        if (ch < p.C) part[((long long)blockIdx.x * (W + 1) + j) * p.C + ch] = sum;
    }
}

// dweight and dbias from the blocks' sums, and the initial-state gradient of empty sequences (their final one's).
__global__ void conv_reduce_kernel(const float *__restrict__ part, int blocks, int W, int C, float *__restrict__ dweight,
                                   float *__restrict__ dbias) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x, j = blockIdx.y;
    if (c >= C || (j == W && !dbias)) return;
    double sum = 0.0;
    for (int b = 0; b < blocks; ++b) sum += part[((long long)b * (W + 1) + j) * C + c];
    if (j < W)
        dweight[(long long)c * W + j] = (float)sum;
    else
        dbias[c] = (float)sum;
}

__global__ void conv_empty_kernel(Seqs seqs, int W, int C, const float *__restrict__ d_fin, float *__restrict__ d_init) {
    const int n = blockIdx.x;
    if (seqs.begin(n) != seqs.end(n)) return;
    const long long size = (long long)(W - 1) * C;
    for (long long i = threadIdx.x; i < size; i += blockDim.x) d_init[n * size + i] = d_fin ? d_fin[n * size + i] : 0.f;
}

bool wide_rows(const void *p, long long stride, int esize) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && stride * esize % 16 == 0;
}

// Whether the wide loads fit: every row of every tensor on a 16-byte boundary.
bool conv_wide(const kda_conv_args &a, const void *y, const void *state) {
    const int e = a.dtype == KDA_BF16 ? 2 : 4;
    const long long dense = a.C;
    return wide_rows(a.x, a.x_stride ? a.x_stride : dense, e) && dense * e % 16 == 0 && aligned16(a.weight) &&
           aligned16(a.bias) && aligned16(y) && aligned16(a.initial_state) && aligned16(state);
}

ConvParams conv_params(const kda_conv_args &a, unsigned *err) {
    ConvParams p{};
    p.x = a.x;
    p.w = a.weight;
    p.bias = a.bias;
    p.x_stride = a.x_stride ? a.x_stride : a.C;
    p.seqs = Seqs{a.cu_seqlens, a.cu_seqlens ? a.n_seqs : a.B, a.T, (long long)a.B * a.T};
    p.C = a.C;
    p.silu = a.activation != 0;
    p.init = a.initial_state;
    p.init_idx = a.initial_state_indices;
    p.fin_idx = a.final_state_indices;
    p.pool = a.state_pool_size;
    p.err = err;
    return p;
}

// Rows a thread walks: long runs re-read fewer rows (W - 1 of each), short ones give more threads. 32 where
// that leaves at least 2048 threads per SM's worth of runs on a 152-SM part, down to 4 for short calls.
int run_rows_for(long long rows, int C, int V) {
    const long long cols = (C + V - 1) / V;
    int run = 32;
    while (run > 4 && rows / run * cols < 152 * 2048) run >>= 1;
    return run;
}

template <typename F>
cudaError_t by_type(const kda_conv_args &a, bool wide, F &&f) {
#define KDA_CONV(W)                                                                             \
    case W:                                                                                      \
        if (a.dtype == KDA_BF16)                                                                 \
            wide ? f.template operator()<__nv_bfloat16, W, 8>() : f.template operator()<__nv_bfloat16, W, 1>(); \
        else                                                                                     \
            wide ? f.template operator()<float, W, 4>() : f.template operator()<float, W, 1>();  \
        break;
    switch (a.W) {
        KDA_CONV(2)
        KDA_CONV(3)
        KDA_CONV(4)
        default: return cudaErrorInvalidValue;
    }
#undef KDA_CONV
    return cudaGetLastError();
}

struct PrefillLaunch {
    ConvParams p;
    void *y, *fin;
    cudaStream_t s;
    template <typename T, int W, int V>
    void operator()() {
        const unsigned cols = (unsigned)((p.C + kLanes * V - 1) / (kLanes * V));
        if (p.seqs.rows > 0) {
            const int run = run_rows_for(p.seqs.rows, p.C, V);
            const long long runs = (p.seqs.rows + run - 1) / run;
            conv_prefill_kernel<T, W, V><<<dim3((unsigned)((runs + kRuns - 1) / kRuns), cols), dim3(kLanes, kRuns), 0, s>>>(
                p, static_cast<T *>(y), run);
        }
        if (fin) conv_state_kernel<T, W, V><<<dim3((unsigned)p.seqs.n_seqs, cols), kLanes, 0, s>>>(p, static_cast<T *>(fin));
    }
};

struct DecodeLaunch {
    ConvParams p;
    void *state, *y;
    cudaStream_t s;
    template <typename T, int W, int V>
    void operator()() {
        const unsigned cols = (unsigned)((p.C + kLanes * V - 1) / (kLanes * V));
        conv_decode_kernel<T, W, V><<<dim3((unsigned)p.seqs.n_seqs, cols), kLanes, 0, s>>>(p, static_cast<T *>(state),
                                                                                       static_cast<T *>(y));
    }
};

struct BackwardLaunch {
    ConvParams p;
    const void *dy;
    const float *d_fin;
    float *dx, *d_init, *part;
    int blocks, run;
    cudaStream_t s;
    template <typename T, int W, int V>
    void operator()() {
        const unsigned cols = (unsigned)((p.C + kLanes * V - 1) / (kLanes * V));
        conv_backward_kernel<T, W, V><<<dim3((unsigned)blocks, cols), dim3(kLanes, kRuns), 0, s>>>(
            p, static_cast<const T *>(dy), d_fin, dx, d_init, part, run);
    }
};

constexpr int kBackwardRun = 32;

int backward_blocks(const kda_conv_args &a) {
    const long long rows = (long long)a.B * a.T;
    return (int)((rows + (long long)kBackwardRun * kRuns - 1) / ((long long)kBackwardRun * kRuns));
}

}  // namespace

cudaError_t launch_conv_prefill(const kda_conv_args &a, void *y, void *final_state, unsigned *err, cudaStream_t s) {
    return by_type(a, conv_wide(a, y, final_state), PrefillLaunch{conv_params(a, err), y, final_state, s});
}

cudaError_t launch_conv_decode(const kda_conv_args &a, void *state, void *y, unsigned *err, cudaStream_t s) {
    DecodeLaunch l{conv_params(a, err), state, y, s};
    if (!l.p.fin_idx) l.p.fin_idx = l.p.init_idx;
    return by_type(a, conv_wide(a, y, state), l);
}

size_t conv_backward_workspace_bytes(const kda_conv_args &a) {
    return (size_t)backward_blocks(a) * (a.W + 1) * a.C * sizeof(float);
}

cudaError_t launch_conv_backward(const kda_conv_args &a, const void *dy, const float *d_final, float *dx, float *dweight,
                                 float *dbias, float *d_init, void *ws, unsigned *err, cudaStream_t s) {
    const ConvParams p = conv_params(a, err);
    const int blocks = backward_blocks(a);
    if (blocks > 0) {
        const bool wide = conv_wide(a, dy, d_init) && aligned16(dx) && aligned16(d_final);
        const cudaError_t e = by_type(
            a, wide, BackwardLaunch{p, dy, d_final, dx, d_init, static_cast<float *>(ws), blocks, kBackwardRun, s});
        if (e != cudaSuccess) return e;
    }
    conv_reduce_kernel<<<dim3((unsigned)((a.C + 127) / 128), (unsigned)a.W + 1), 128, 0, s>>>(
        static_cast<const float *>(ws), blocks, a.W, a.C, dweight, dbias);
    if (d_init) conv_empty_kernel<<<(unsigned)p.seqs.n_seqs, 128, 0, s>>>(p.seqs, a.W, a.C, d_final, d_init);
    return cudaGetLastError();
}

}  // namespace kda
