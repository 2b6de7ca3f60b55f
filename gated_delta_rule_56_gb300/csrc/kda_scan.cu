// kda_scan.cu -- the selective state space scan: prompts and single tokens.
//
//     h_t[c, n] = exp(dt_t[c] A[c, n]) h_{t-1}[c, n] + dt_t[c] x_t[c] B_t[n],   y_t[c] = sum_n C_t[n] h_t[c, n] + D[c] x_t[c]
//
// Prompts: one lane per channel holds up to 16 states in registers (more states: 2 to 16 lanes per channel,
// their parts of y added by shuffles) and walks down its sequence.
#include "kda_scan.cuh"

namespace kda {
namespace {

template <typename T, int S, int L>
__global__ void __launch_bounds__(32) scan_prefill_kernel(ScanParams p, T *__restrict__ y, float *fin) {
    if (blockIdx.x == 0 && blockIdx.y == 0) check_seqs(p.seqs, p.err);
    const int per = p.C / p.G;  // channels per group
    const int blocks = (per * L + 31) / 32;
    const int g = blockIdx.y / blocks;
    const int k = (blockIdx.y % blocks) * (32 / L) + threadIdx.x / L, n0 = (threadIdx.x % L) * S;
    const bool live = k < per;
    const int c = g * per + (live ? k : 0), n = blockIdx.x;
    const long long bos = p.seqs.begin(n), eos = p.seqs.end(n);
    if (bos < 0 || eos < bos || eos > p.seqs.rows) return;
    const long long from = p.init ? state_slot(p.init_idx, p.pool, n, p.err) : -1;
    float h[S], A[S];
#pragma unroll
    for (int i = 0; i < S; ++i) {
        const bool in = n0 + i < p.N;
        A[i] = in ? p.A[(long long)c * p.N + n0 + i] * kLog2e : 0.f;
        h[i] = in && from >= 0 ? p.init[(from * p.C + c) * p.N + n0 + i] : 0.f;
    }
    const float bias = p.dt_bias ? p.dt_bias[c] : 0.f, skip = p.D ? p.D[c] : 0.f;
    const T *X = static_cast<const T *>(p.x), *DT = static_cast<const T *>(p.dt), *Z = static_cast<const T *>(p.z);
    const T *B = static_cast<const T *>(p.Bm) + g * p.N + n0, *Cm = static_cast<const T *>(p.Cm) + g * p.N + n0;
    for (long long r = bos; r < eos; ++r) {
        const float x = to_float(X[r * p.x_stride + c]);
        float dt = to_float(DT[r * p.dt_stride + c]) + bias;
        if (p.softplus) dt = softplus(dt);
        const float u = dt * x;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            if (n0 + i < p.N) {
                h[i] = fmaf(exp2f(dt * A[i]), h[i], u * to_float(B[r * p.B_stride + i]));
                sum = fmaf(to_float(Cm[r * p.C_stride + i]), h[i], sum);
            }
        }
#pragma unroll
        for (int m = L / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        sum = fmaf(skip, x, sum);
        if (Z) {
            const float z = to_float(Z[r * p.z_stride + c]);
            sum *= z * sigmoid(z);
        }
        if (live && n0 == 0) y[r * p.C + c] = from_float<T>(sum);
    }
    if (!fin || !live) return;
    const long long to = state_slot(p.fin_idx, p.pool, n, p.err);
    if (to < 0) return;
#pragma unroll
    for (int i = 0; i < S; ++i)
        if (n0 + i < p.N) fin[(to * p.C + c) * p.N + n0 + i] = h[i];
}

struct PrefillLaunch {
    ScanParams p;
    void *y;
    float *fin;
    cudaStream_t s;
    template <typename T, int S, int L>
    void operator()() {
        const int per = p.C / p.G;
        scan_prefill_kernel<T, S, L><<<dim3((unsigned)p.seqs.n_seqs, (unsigned)(((per * L + 31) / 32) * p.G)), 32, 0, s>>>(
            p, static_cast<T *>(y), fin);
    }
};

// One token: bound by HBM, the state is read and written once. LP lanes hold a channel's states, V consecutive
// ones each (16 bytes where N and the state's address allow it), so that a warp streams whole
// 512-byte runs of the state; the parts of y are added by shuffles.
template <typename T, int LP, int V>
__global__ void __launch_bounds__(128) scan_decode_kernel(ScanParams p, float *state, T *__restrict__ y) {
    const int k = blockIdx.y * (128 / LP) + threadIdx.x / LP, l = threadIdx.x % LP;
    const int n = blockIdx.x;
    const bool live = k < p.C;
    const int c = live ? k : p.C - 1;
    const int g = c / (p.C / p.G);
    const long long from = state_slot(p.init_idx, p.pool, n, p.err);
    const long long to = p.fin_idx == p.init_idx ? from : state_slot(p.fin_idx, p.pool, n, p.err);
    const float x = to_float(static_cast<const T *>(p.x)[n * p.x_stride + c]);
    float dt = to_float(static_cast<const T *>(p.dt)[n * p.dt_stride + c]) + (p.dt_bias ? p.dt_bias[c] : 0.f);
    if (p.softplus) dt = softplus(dt);
    const float u = dt * x;
    const T *B = static_cast<const T *>(p.Bm) + n * p.B_stride + g * p.N;
    const T *Cm = static_cast<const T *>(p.Cm) + n * p.C_stride + g * p.N;
    float sum = 0.f;
    for (int n0 = l * V; n0 < p.N; n0 += LP * V) {
        Pack<float, V> a = load_pack<float, V>(p.A + (long long)c * p.N + n0), h;
        if (from >= 0) {
            h = load_pack<float, V>(state + (from * p.C + c) * p.N + n0);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) h.e[v] = 0.f;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h.e[v] = fmaf(exp2f(dt * (a.e[v] * kLog2e)), h.e[v], u * to_float(B[n0 + v]));
            sum = fmaf(to_float(Cm[n0 + v]), h.e[v], sum);
        }
        if (to >= 0 && live) store_pack<float, V>(state + (to * p.C + c) * p.N + n0, h);
    }
#pragma unroll
    for (int m = LP / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (!live || l != 0) return;
    if (p.D) sum = fmaf(p.D[c], x, sum);
    if (p.z) {
        const float z = to_float(static_cast<const T *>(p.z)[n * p.z_stride + c]);
        sum *= z * sigmoid(z);
    }
    y[(long long)n * p.C + c] = from_float<T>(sum);
}

template <typename T, int V>
void launch_decode(const ScanParams &p, float *state, void *y, cudaStream_t s) {
    const int words = (p.N + V - 1) / V;
    T *out = static_cast<T *>(y);
#define KDA_DECODE(LP)                                                                                              \
    scan_decode_kernel<T, LP, V><<<dim3((unsigned)p.seqs.n_seqs, (unsigned)((p.C + 128 / LP - 1) / (128 / LP))), 128, 0, s>>>( \
        p, state, out)
    if (words <= 1)
        KDA_DECODE(1);
    else if (words <= 2)
        KDA_DECODE(2);
    else if (words <= 4)
        KDA_DECODE(4);
    else if (words <= 8)
        KDA_DECODE(8);
    else
        KDA_DECODE(16);
#undef KDA_DECODE
}

}  // namespace

size_t scan_prefill_workspace_bytes(const kda_scan_args &, int) { return 0; }

cudaError_t launch_scan_prefill(const kda_scan_args &a, void *y, float *final_state, void *, int, unsigned *err,
                                cudaStream_t s) {
    return scan_by_type(a, PrefillLaunch{scan_params(a, err), y, final_state, s});
}

cudaError_t launch_scan_decode(const kda_scan_args &a, float *state, void *y, unsigned *err, cudaStream_t s) {
    ScanParams p = scan_params(a, err);
    if (!p.fin_idx) p.fin_idx = p.init_idx;
    const bool wide = p.N % 4 == 0 && aligned16(state) && aligned16(p.A);
    if (a.dtype == KDA_BF16)
        wide ? launch_decode<__nv_bfloat16, 4>(p, state, y, s) : launch_decode<__nv_bfloat16, 1>(p, state, y, s);
    else
        wide ? launch_decode<float, 4>(p, state, y, s) : launch_decode<float, 1>(p, state, y, s);
    return cudaGetLastError();
}

}  // namespace kda
