// kda_conv.cu -- the short causal convolution of a layer's projections: prompts, single tokens, gradients.
//
//     p_t = bias + sum_j w_j x_{t-(W-1)+j},   y_t = p_t or p_t sigmoid(p_t)         (per channel)
//
// Bound by HBM: x is read once and y written once, 2 W + 4 operations per element. A thread owns four channels (8 bytes in
// bf16, 16 in fp32; a warp's row is 256 or 512 consecutive bytes) and walks down a run of rows with the last W - 1 inputs
// and the filter in registers, as pairs that one instruction multiplies and adds; the loads of a batch of rows are issued
// together. Eight channels per thread took twice the registers and left half the loads in flight (334 us where four take 265). Only the W - 1
// rows before a run are read twice. Channels whose rows are not 16-byte aligned go one per thread.
// Measured: 32768 rows x 12288 channels in bf16, W = 4, SiLU: 265 us, 6.1 TB/s of x and y (89 % of the measured copy rate).
#include "kda_layers.cuh"
#include "kda_layers.h"

namespace kda {
namespace {

constexpr int kLanes = 32;  // threads along the channels
constexpr int kRuns = 4, kBackRuns = 8;    // row runs per block
constexpr int kBatch = 8, kBackBatch = 6;  // rows loaded together

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

// V channels as pairs (one channel: a pair whose second half is not used).
template <int V>
struct Row {
    static constexpr int P = V == 1 ? 1 : V / 2;
    f32x2 v[P];
};

template <typename T, int V>
__device__ __forceinline__ Row<V> to_row(const Pack<T, V> &in) {
    Row<V> r;
#pragma unroll
    for (int i = 0; i < Row<V>::P; ++i) r.v[i] = pair(to_float(in.e[2 * i]), V == 1 ? 0.f : to_float(in.e[V == 1 ? 0 : 2 * i + 1]));
    return r;
}

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> from_row(const Row<V> &r) {
    Pack<T, V> out;
#pragma unroll
    for (int i = 0; i < Row<V>::P; ++i) {
        float a, b;
        unpair(r.v[i], a, b);
        out.e[2 * i] = from_float<T>(a);
        if constexpr (V > 1) out.e[2 * i + 1] = from_float<T>(b);
    }
    return out;
}

template <int V>
__device__ __forceinline__ Row<V> zero_row() {
    Row<V> r;
#pragma unroll
    for (int i = 0; i < Row<V>::P; ++i) r.v[i] = 0;
    return r;
}

template <int W, int V>
struct Filter {
    Row<V> w[W], b;
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
    for (int j = 0; j < W; ++j) {
        Pack<T, V> column;
#pragma unroll
        for (int v = 0; v < V; ++v) column.e[v] = w[v * W + j];
        f.w[j] = to_row(column);
    }
    f.b = p.bias ? to_row(load_pack<T, V>(static_cast<const T *>(p.bias) + c)) : zero_row<V>();
}

// The filter over W rows, newest last.
template <int W, int V>
__device__ __forceinline__ Row<V> filtered(const Filter<W, V> &f, const Row<V> *x) {
    Row<V> a = f.b;
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
        for (int i = 0; i < Row<V>::P; ++i) a.v[i] = fma2(f.w[j].v[i], x[j].v[i], a.v[i]);
    return a;
}

template <int V>
__device__ __forceinline__ Row<V> activated(Row<V> a, bool silu) {
    if (silu) {
#pragma unroll
        for (int i = 0; i < Row<V>::P; ++i) a.v[i] = silu2(a.v[i]);
    }
    return a;
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

// The state after sequence n: its last W - 1 inputs. All are read before the first is written, so that the state may
// be the one it started from.
template <typename T, int W, int V>
__device__ __forceinline__ void state_after(const ConvParams &p, T *fin, int n, int c) {
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

// The states alone: where the final states lie in the initial ones' memory, they wait for the rows' kernel.
template <typename T, int W, int V>
__global__ void __launch_bounds__(kLanes *kRuns) conv_state_kernel(ConvParams p, T *fin) {
    const int c = (blockIdx.y * kLanes + threadIdx.x) * V, n = blockIdx.x * kRuns + threadIdx.y;
    if (c < p.C && n < p.seqs.n_seqs) state_after<T, W, V>(p, fin, n, c);
}

template <typename T, int W, int V>
__global__ void __launch_bounds__(kLanes *kRuns) conv_prefill_kernel(ConvParams p, T *__restrict__ y, int run_rows, T *fin,
                                                                      int run_blocks) {
    if (blockIdx.x == 0 && blockIdx.y == 0) check_seqs(p.seqs, p.err);
    const int c = (blockIdx.y * kLanes + threadIdx.x) * V;
    if (c >= p.C) return;
    if ((int)blockIdx.x >= run_blocks) {  // the blocks behind those of the rows write the states
        const int n = (blockIdx.x - run_blocks) * kRuns + threadIdx.y;
        if (n < p.seqs.n_seqs) state_after<T, W, V>(p, fin, n, c);
        return;
    }
    long long r = ((long long)blockIdx.x * kRuns + threadIdx.y) * run_rows;
    const long long stop = min(r + run_rows, p.seqs.rows);
    if (r >= stop) return;
    Filter<W, V> f;
    load_filter<T, W, V>(p, c, f);
    for (int n = p.seqs.at(r); n < p.seqs.n_seqs && r < stop; ++n) {
        const long long bos = p.seqs.begin(n), end = min(p.seqs.end(n), stop);
        if (end <= r || bos > r || bos < 0) continue;  // empty (or a bad cu_seqlens)
        const long long slot = p.init ? state_slot(p.init_idx, p.pool, n, p.err) : -1;
        // The last W - 1 inputs, then a batch of kBatch rows whose loads are issued together.
        Row<V> x[W - 1 + kBatch];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) x[j] = to_row(input_at<T, W, V>(p, r - (W - 1) + j, bos, slot, c));
        const T *px = static_cast<const T *>(p.x) + r * p.x_stride + c;
        T *py = y + r * p.C + c;
        for (; r + kBatch <= end; r += kBatch, px += kBatch * p.x_stride, py += kBatch * (long long)p.C) {
            Pack<T, V> in[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) in[u] = load_pack<T, V>(px + u * p.x_stride);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                x[W - 1 + u] = to_row(in[u]);
                store_pack<T, V>(py + u * (long long)p.C, from_row<T, V>(activated<V>(filtered<W, V>(f, x + u), p.silu)));
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j) x[j] = x[kBatch + j];
        }
        for (; r < end; ++r, px += p.x_stride, py += p.C) {
            x[W - 1] = to_row(load_pack<T, V>(px));
            store_pack<T, V>(py, from_row<T, V>(activated<V>(filtered<W, V>(f, x), p.silu)));
#pragma unroll
            for (int j = 0; j < W - 1; ++j) x[j] = x[j + 1];
        }
    }
}

// One token. A thread keeps its filter and takes several sequences, whose loads are issued together.
template <typename T, int W, int V, int SEQS>
__global__ void __launch_bounds__(kLanes *kRuns) conv_decode_kernel(ConvParams p, T *state, T *__restrict__ y) {
    const int c = (blockIdx.y * kLanes * kRuns + threadIdx.y * kLanes + threadIdx.x) * V;
    if (c >= p.C) return;
    p.init = state;
    Pack<T, V> in[SEQS][W];
    long long to[SEQS];
#pragma unroll
    for (int s = 0; s < SEQS; ++s) {
        const int n = blockIdx.x * SEQS + s;
        if (n >= p.seqs.n_seqs) break;
        const long long from = state_slot(p.init_idx, p.pool, n, p.err);
        to[s] = p.fin_idx == p.init_idx ? from : state_slot(p.fin_idx, p.pool, n, p.err);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) in[s][j] = input_at<T, W, V>(p, j - (W - 1), 0, from, c);
        in[s][W - 1] = load_pack<T, V>(static_cast<const T *>(p.x) + n * p.x_stride + c);
    }
    Filter<W, V> f;
    load_filter<T, W, V>(p, c, f);
#pragma unroll
    for (int s = 0; s < SEQS; ++s) {
        const int n = blockIdx.x * SEQS + s;
        if (n >= p.seqs.n_seqs) break;
        Row<V> x[W];
#pragma unroll
        for (int j = 0; j < W; ++j) x[j] = to_row(in[s][j]);
        store_pack<T, V>(y + (long long)n * p.C + c, from_row<T, V>(activated<V>(filtered<W, V>(f, x), p.silu)));
        if (to[s] >= 0) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) store_pack<T, V>(state + (to[s] * (W - 1) + j) * p.C + c, in[s][j + 1]);
        }
    }
}

// Gradients: dp_t = dy_t (SiLU'(p_t)),  dx_t = sum_k w_{W-1-k} dp_{t+k} within the sequence,
// dw_j = sum_t dp_t x_{t-(W-1)+j},  db = sum_t dp_t; the rows before a sequence give its initial state's gradient.
// A thread recomputes p over its run and the W - 1 rows after it. The filter's sums of the block's runs are
// added in shared memory in a fixed order and written to `part` [block][W + 1][C]; conv_reduce_kernel adds those. Plain fp32 within a
// block (up to 256 rows in one accumulator, then 8 of those), which leaves dweight and dbias 3e-7 off 64 bits in the 2-norm over
// 32768 rows, where sums in 64 bits would leave 7e-8; a second value for each sum would take 20 registers.
// Measured: 32768 rows x 4096 channels in bf16: 226 us in all, 4.75 TB/s of x, dy and dx in fp32 (70 % of the copy rate); what
// holds it is the latency of the loads at 16 warps per SM (128 registers for two windows, the filter and its sums). fp32 takes 151,
// which leaves 8 warps: 343 us, 4.7 TB/s.
template <typename T, int W, int V>
__global__ void __launch_bounds__(kLanes *kBackRuns) conv_backward_kernel(ConvParams p, const T *__restrict__ dy,
                                                                       const float *__restrict__ d_fin,
                                                                       float *__restrict__ dx, float *__restrict__ d_init,
                                                                       float *__restrict__ part, int run_rows) {
    constexpr int P = Row<V>::P;
    __shared__ float sums[kBackRuns][kLanes * V];
    if (blockIdx.x == 0 && blockIdx.y == 0) check_seqs(p.seqs, p.err);
    const int c = (blockIdx.y * kLanes + threadIdx.x) * V;
    Row<V> dw[W + 1];
#pragma unroll
    for (int j = 0; j <= W; ++j) dw[j] = zero_row<V>();
    long long r = ((long long)blockIdx.x * kBackRuns + threadIdx.y) * run_rows;
    const long long stop = min(r + run_rows, p.seqs.rows);
    if (c < p.C && r < stop) {
        Filter<W, V> f;
        load_filter<T, W, V>(p, c, f);
        for (int n = p.seqs.at(r); n < p.seqs.n_seqs && r < stop; ++n) {
            const long long bos = p.seqs.begin(n), eos = min(p.seqs.end(n), p.seqs.rows), end = min(eos, stop);
            if (end <= r || bos > r || bos < 0) continue;
            const long long slot = p.init ? n : -1, first = r;
            Row<V> x[W], dp[W];  // the last W inputs and gradients of p
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                x[j] = to_row(input_at<T, W, V>(p, r - (W - 1) + j, bos, slot, c));
                dp[j] = zero_row<V>();
            }
            // One row: its dp into dp[W - 1], its share of the filter's gradient if the row is this run's.
            auto advance = [&](const Pack<T, V> &in, const Pack<T, V> &d, bool mine) {
                x[W - 1] = to_row(in);
                Row<V> g = to_row(d);
                if (p.silu) {
                    const Row<V> a = filtered<W, V>(f, x);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        const f32x2 s = sigmoid2(a.v[i]);
                        g.v[i] = mul2(g.v[i], mul2(s, fma2(a.v[i], fma2(s, both(-1.f), both(1.f)), both(1.f))));
                    }
                }
                dp[W - 1] = g;
                if (mine) {
#pragma unroll
                    for (int i = 0; i < P; ++i) {
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j].v[i] = fma2(g.v[i], x[j].v[i], dw[j].v[i]);
                        dw[W].v[i] = add2(dw[W].v[i], g.v[i]);
                    }
                }
            };
            auto shift = [&]() {
#pragma unroll
                for (int j = 0; j < W - 1; ++j) {
                    x[j] = x[j + 1];
                    dp[j] = dp[j + 1];
                }
            };
            auto gradient = [&](float(&g)[V]) {  // of the row W - 1 before the newest
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    f32x2 a = mul2(f.w[W - 1].v[i], dp[0].v[i]);
#pragma unroll
                    for (int k = 1; k < W; ++k) a = fma2(f.w[W - 1 - k].v[i], dp[k].v[i], a);
                    float lo, hi;
                    unpair(a, lo, hi);
                    g[2 * i] = lo;
                    if constexpr (V > 1) g[2 * i + 1] = hi;
                }
            };
            // Any row: past the sequence's end dp is zero; q < bos is a row of the initial state.
            auto any_row = [&](long long row) {
                if (row < eos) {
                    advance(load_pack<T, V>(static_cast<const T *>(p.x) + row * p.x_stride + c), load_pack<T, V>(dy + row * p.C + c),
                            row < end);
                } else {
                    dp[W - 1] = zero_row<V>();
                }
                const long long q = row - (W - 1);
                if (q >= first || (first == bos && d_init)) {
                    float g[V];
                    gradient(g);
                    if (d_fin && q >= eos - (W - 1)) {
                        const float *df = d_fin + ((long long)n * (W - 1) + (q - (eos - (W - 1)))) * p.C + c;
#pragma unroll
                        for (int v = 0; v < V; ++v) g[v] += df[v];
                    }
                    store_floats<V>(q >= bos ? dx + q * p.C + c : d_init + ((long long)n * (W - 1) + (W - 1) + (q - bos)) * p.C + c,
                                    g);
                }
                shift();
            };
            for (; r < first + W - 1 && r < end + W - 1; ++r) any_row(r);
            // Rows whose gradients go to the run's own rows, below the rows that a final state reaches; loads in batches.
            for (; r + kBackBatch <= end; r += kBackBatch) {
                Pack<T, V> in[kBackBatch], d[kBackBatch];
#pragma unroll
                for (int u = 0; u < kBackBatch; ++u) {
                    in[u] = load_pack<T, V>(static_cast<const T *>(p.x) + (r + u) * p.x_stride + c);
                    d[u] = load_pack<T, V>(dy + (r + u) * p.C + c);
                }
#pragma unroll
                for (int u = 0; u < kBackBatch; ++u) {
                    advance(in[u], d[u], true);
                    float g[V];
                    gradient(g);
                    store_floats<V>(dx + (r + u - (W - 1)) * p.C + c, g);
                    shift();
                }
            }
            for (; r < end + W - 1; ++r) any_row(r);
            r = end;
        }
    }
    // The runs' sums, one of the filter's places at a time.
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        float lo, hi;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            unpair(dw[j].v[i], lo, hi);
            sums[threadIdx.y][2 * i * kLanes + threadIdx.x] = lo;
            if constexpr (V > 1) sums[threadIdx.y][(2 * i + 1) * kLanes + threadIdx.x] = hi;
        }
        __syncthreads();
        for (int k = threadIdx.y * kLanes + threadIdx.x; k < kLanes * V; k += kLanes * kBackRuns) {
            const int ch = blockIdx.y * kLanes * V + k;
            float sum = 0.f;
#pragma unroll
            for (int run = 0; run < kBackRuns; ++run) sum += sums[run][(k % V) * kLanes + k / V];
            if (ch < p.C) part[((long long)blockIdx.x * (W + 1) + j) * p.C + ch] = sum;
        }
        __syncthreads();
    }
}

// dweight and dbias from the blocks' sums, and the initial-state gradient of empty sequences (their final one's).
__global__ void conv_reduce_kernel(const float *__restrict__ part, int blocks, int W, int C, float *__restrict__ dweight,
                                   float *__restrict__ dbias) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x, j = blockIdx.y;
    if (c >= C || (j == W && !dbias)) return;
    ExactSum sum;
#pragma unroll 16
    for (int b = 0; b < blocks; ++b) sum.add(part[((long long)b * (W + 1) + j) * C + c]);
    if (j < W)
        dweight[(long long)c * W + j] = sum.value();
    else
        dbias[c] = sum.value();
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

// Rows a thread walks: long runs re-read fewer rows (W - 1 of each), short ones give more threads. 128 where
// that leaves at least 2048 threads for each of 152 SMs, down to 8 for short calls.
int run_rows_for(long long rows, int C, int V) {
    const long long cols = (C + V - 1) / V;
    int run = 128;
    while (run > 8 && rows / run * cols < 152 * 2048) run >>= 1;
    return run;
}

template <typename F>
cudaError_t by_type(const kda_conv_args &a, bool wide, F &&f) {
#define KDA_CONV(W)                                                                             \
    case W:                                                                                      \
        if (a.dtype == KDA_BF16)                                                                 \
            wide ? f.template operator()<__nv_bfloat16, W, 4>() : f.template operator()<__nv_bfloat16, W, 1>(); \
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
        const int run = run_rows_for(p.seqs.rows, p.C, V);
        const long long runs = (p.seqs.rows + run - 1) / run;
        const unsigned run_blocks = (unsigned)((runs + kRuns - 1) / kRuns);
        const unsigned state_blocks = fin ? (unsigned)((p.seqs.n_seqs + kRuns - 1) / kRuns) : 0;
        // In one launch unless a row's block might read an initial state that is already overwritten.
        const size_t bytes = (size_t)(p.pool > p.seqs.n_seqs ? p.pool : p.seqs.n_seqs) * (W - 1) * p.C * sizeof(T);
        const char *a = static_cast<const char *>(p.init), *b = static_cast<const char *>(fin);
        const bool apart = !p.init || !fin || a + bytes <= b || b + bytes <= a;
        const unsigned first = run_blocks + (apart ? state_blocks : 0);
        const dim3 block(kLanes, kRuns);
        if (first)
            conv_prefill_kernel<T, W, V><<<dim3(first, cols), block, 0, s>>>(p, static_cast<T *>(y), run, static_cast<T *>(fin),
                                                                            (int)run_blocks);
        if (!apart && state_blocks) conv_state_kernel<T, W, V><<<dim3(state_blocks, cols), block, 0, s>>>(p, static_cast<T *>(fin));
    }
};

struct DecodeLaunch {
    ConvParams p;
    void *state, *y;
    cudaStream_t s;
    template <typename T, int W, int V>
    void operator()() {
        // Four sequences per thread where that still gives every SM two blocks: the filter is loaded once for them.
        const unsigned cols = (unsigned)((p.C + kLanes * kRuns * V - 1) / (kLanes * kRuns * V));
        const dim3 block(kLanes, kRuns);
        T *st = static_cast<T *>(state), *out = static_cast<T *>(y);
        const unsigned fours = (unsigned)(p.seqs.n_seqs + 3) / 4;
        if ((long long)fours * cols >= 304)
            conv_decode_kernel<T, W, V, 4><<<dim3(fours, cols), block, 0, s>>>(p, st, out);
        else
            conv_decode_kernel<T, W, V, 1><<<dim3((unsigned)p.seqs.n_seqs, cols), block, 0, s>>>(p, st, out);
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
        conv_backward_kernel<T, W, V><<<dim3((unsigned)blocks, cols), dim3(kLanes, kBackRuns), 0, s>>>(
            p, static_cast<const T *>(dy), d_fin, dx, d_init, part, run);
    }
};

// Rows a thread walks in the backward pass: long runs leave fewer partial sums; 256 (225 us against 240 us with 128 on 32768 rows of
// 4096 channels) while that gives every one of 152 SMs two blocks, down to 32.
int backward_run(const kda_conv_args &a) {
    const long long rows = (long long)a.B * a.T, cols = (a.C + 4 * kLanes - 1) / (4 * kLanes);
    int run = 256;
    while (run > 32 && rows / (run * kBackRuns) * cols < 2 * 152) run >>= 1;
    return run;
}

int backward_blocks(const kda_conv_args &a) {
    const long long rows = (long long)a.B * a.T, per = (long long)backward_run(a) * kBackRuns;
    return (int)((rows + per - 1) / per);
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
            a, wide, BackwardLaunch{p, dy, d_final, dx, d_init, static_cast<float *>(ws), blocks, backward_run(a), s});
        if (e != cudaSuccess) return e;
    }
    conv_reduce_kernel<<<dim3((unsigned)((a.C + 127) / 128), (unsigned)a.W + 1), 128, 0, s>>>(
        static_cast<const float *>(ws), blocks, a.W, a.C, dweight, dbias);
    if (d_init) conv_empty_kernel<<<(unsigned)p.seqs.n_seqs, 128, 0, s>>>(p.seqs, a.W, a.C, d_final, d_init);
    return cudaGetLastError();
}

}  // namespace kda
