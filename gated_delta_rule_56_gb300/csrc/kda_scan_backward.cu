// kda_scan_backward.cu -- gradients of the selective scan.
//
// With dy' = dy z sigmoid(z) (or dy), g_t = dL/dh_t and a_t = exp(dt_t A):
//     g_t = C_t dy'_t + a_{t+1} g_{t+1}                 (at a sequence's end: + the final state's gradient)
//     dC_t[n] = sum_c dy'_t h_t,    dB_t[n] = sum_c g_t dt_t x_t          (over the channels of the group)
//     dx_t = D dy'_t + dt_t sum_n g_t B_t,   ddt'_t = sum_n g_t (A a_t h_{t-1} + B_t x_t)
//     dA = sum_t g_t dt_t a_t h_{t-1},  dD = sum_t dy'_t x_t,  the initial state's gradient: a_first g_first.
// The states of all tokens are kept in the workspace by a forward walk; a second walk goes back.
#include "kda_scan.cuh"

namespace kda {
namespace {

struct GradParams {
    const void *dy;
    const float *d_fin;
    float *dx, *ddt, *dz, *d_init;
    float *states;         // [rows][C][N]
    float *part_B, *part_C;  // [blocks per group][rows][G][N]
    float *part_A;         // [n_seqs][C][N]
    float *part_D, *part_bias;  // [n_seqs][C]
    int blocks;            // channel blocks per group
};

__device__ __forceinline__ float warp_sum_from(float x, int first) {  // over the lanes that differ by multiples of `first`
    for (int m = 16; m >= first; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

template <typename T, int S, int L>
__global__ void __launch_bounds__(32) scan_backward_kernel(ScanParams p, GradParams q) {
    if (blockIdx.x == 0 && blockIdx.y == 0) check_seqs(p.seqs, p.err);
    const int per = p.C / p.G;
    const int g = blockIdx.y / q.blocks, blk = blockIdx.y % q.blocks;
    const int k = blk * (32 / L) + threadIdx.x / L, n0 = (threadIdx.x % L) * S;
    const bool live = k < per;
    const int c = g * per + (live ? k : 0), n = blockIdx.x;
    const long long bos = p.seqs.begin(n), eos = p.seqs.end(n);
    if (bos < 0 || eos < bos || eos > p.seqs.rows) return;
    float h[S], A[S], A2[S], dA[S], gr[S];
#pragma unroll
    for (int i = 0; i < S; ++i) {
        const bool in = n0 + i < p.N;
        const long long at = ((long long)n * p.C + c) * p.N + n0 + i;
        A[i] = in ? p.A[(long long)c * p.N + n0 + i] : 0.f;
        A2[i] = A[i] * kLog2e;
        h[i] = in && p.init ? p.init[at] : 0.f;
        gr[i] = in && q.d_fin && live ? q.d_fin[at] : 0.f;
        dA[i] = 0.f;
    }
    const float bias = p.dt_bias ? p.dt_bias[c] : 0.f, skip = p.D ? p.D[c] : 0.f;
    const T *X = static_cast<const T *>(p.x), *DT = static_cast<const T *>(p.dt), *Z = static_cast<const T *>(p.z);
    const T *B = static_cast<const T *>(p.Bm) + g * p.N + n0, *Cm = static_cast<const T *>(p.Cm) + g * p.N + n0;
    const T *DY = static_cast<const T *>(q.dy);
    for (long long r = bos; r < eos; ++r) {
        const float x = to_float(X[r * p.x_stride + c]);
        float dt = to_float(DT[r * p.dt_stride + c]) + bias;
        if (p.softplus) dt = softplus(dt);
#pragma unroll
        for (int i = 0; i < S; ++i)
            if (n0 + i < p.N) {
                h[i] = fmaf(exp2f(dt * A2[i]), h[i], dt * x * to_float(B[r * p.B_stride + i]));
                if (live) q.states[(r * p.C + c) * p.N + n0 + i] = h[i];
            }
    }
    float dD = 0.f, dbias = 0.f;
    for (long long r = eos - 1; r >= bos; --r) {
        const float x = to_float(X[r * p.x_stride + c]), raw = to_float(DT[r * p.dt_stride + c]) + bias;
        const float dt = p.softplus ? softplus(raw) : raw;
        const float dy0 = live ? to_float(DY[r * p.C + c]) : 0.f;
        float z = 0.f, sz = 1.f, dy = dy0;
        if (Z) {
            z = to_float(Z[r * p.z_stride + c]);
            sz = sigmoid(z);
            dy = dy0 * (z * sz);
        }
        float out = 0.f, gB = 0.f, gA = 0.f;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const bool in = n0 + i < p.N;
            const float Bv = in ? to_float(B[r * p.B_stride + i]) : 0.f, Cv = in ? to_float(Cm[r * p.C_stride + i]) : 0.f;
            const float before = !in ? 0.f : r > bos ? (live ? q.states[((r - 1) * p.C + c) * p.N + n0 + i] : 0.f)
                                                    : (p.init ? p.init[((long long)n * p.C + c) * p.N + n0 + i] : 0.f);
            gr[i] = fmaf(Cv, dy, gr[i]);
            out = fmaf(Cv, h[i], out);
            const float sB = warp_sum_from(gr[i] * (dt * x), L), sC = warp_sum_from(dy * h[i], L);
            if (in && threadIdx.x < L) {
                const long long at = (((long long)blk * p.seqs.rows + r) * p.G + g) * p.N + n0 + i;
                q.part_B[at] = sB;
                q.part_C[at] = sC;
            }
            gB = fmaf(gr[i], Bv, gB);
            gr[i] *= exp2f(dt * A2[i]);
            const float w = gr[i] * before;
            gA = fmaf(w, A[i], gA);
            dA[i] = fmaf(w, dt, dA[i]);
            h[i] = before;
        }
#pragma unroll
        for (int m = L / 2; m > 0; m >>= 1) {
            out += __shfl_xor_sync(0xffffffffu, out, m);
            gB += __shfl_xor_sync(0xffffffffu, gB, m);
            gA += __shfl_xor_sync(0xffffffffu, gA, m);
        }
        float ddt = fmaf(gB, x, gA);
        if (p.softplus) ddt *= sigmoid(raw);
        dD = fmaf(dy, x, dD);
        dbias += ddt;
        if (live && n0 == 0) {
            q.dx[r * p.C + c] = fmaf(gB, dt, dy * skip);
            q.ddt[r * p.C + c] = ddt;
            if (Z) q.dz[r * p.C + c] = dy0 * fmaf(skip, x, out) * (sz * fmaf(z, 1.f - sz, 1.f));
        }
    }
    if (!live) return;
#pragma unroll
    for (int i = 0; i < S; ++i)
        if (n0 + i < p.N) {
            const long long at = ((long long)n * p.C + c) * p.N + n0 + i;
            if (q.d_init) q.d_init[at] = gr[i];
            q.part_A[at] = dA[i];
        }
    if (n0 == 0) {
        q.part_D[(long long)n * p.C + c] = dD;
        q.part_bias[(long long)n * p.C + c] = dbias;
    }
}

// out[i] = sum over j < count of in[j][i], in order.
__global__ void scan_reduce_kernel(const float *__restrict__ in, long long size, int count, float *__restrict__ out) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= size) return;
    double sum = 0.0;
    for (int j = 0; j < count; ++j) sum += in[j * size + i];
    out[i] = (float)sum;
}

struct BackwardLaunch {
    ScanParams p;
    GradParams q;
    cudaStream_t s;
    template <typename T, int S, int L>
    void operator()() {
        scan_backward_kernel<T, S, L><<<dim3((unsigned)p.seqs.n_seqs, (unsigned)(q.blocks * p.G)), 32, 0, s>>>(p, q);
    }
};

size_t layout(const kda_scan_args &a, GradParams *q, char *ws) {
    const long long rows = (long long)a.B * a.T, n = a.cu_seqlens ? a.n_seqs : a.B;
    const int blocks = (a.D / a.G * scan_lanes(a.N) + 31) / 32;
    size_t at = 0;
    auto take = [&](size_t count) {
        float *r = reinterpret_cast<float *>(ws + at);
        at += (count * sizeof(float) + 255) / 256 * 256;
        return r;
    };
    GradParams t{};
    t.blocks = blocks;
    t.states = take((size_t)rows * a.D * a.N);
    t.part_B = take((size_t)blocks * rows * a.G * a.N);
    t.part_C = take((size_t)blocks * rows * a.G * a.N);
    t.part_A = take((size_t)n * a.D * a.N);
    t.part_D = take((size_t)n * a.D);
    t.part_bias = take((size_t)n * a.D);
    if (q) *q = t;
    return at;
}

void reduce(const float *in, long long size, int count, float *out, cudaStream_t s) {
    if (out && size) scan_reduce_kernel<<<(unsigned)((size + 255) / 256), 256, 0, s>>>(in, size, count, out);
}

}  // namespace

size_t scan_backward_workspace_bytes(const kda_scan_args &a, int) { return layout(a, nullptr, nullptr); }

cudaError_t launch_scan_backward(const kda_scan_args &a, const kda_scan_grads &g, void *ws, int, unsigned *err,
                                 cudaStream_t s) {
    BackwardLaunch l{scan_params(a, err), {}, s};
    layout(a, &l.q, static_cast<char *>(ws));
    l.q.dy = g.dy;
    l.q.d_fin = g.d_final_state;
    l.q.dx = g.dx;
    l.q.ddt = g.ddt;
    l.q.dz = g.dz;
    l.q.d_init = g.d_initial_state;
    const cudaError_t e = scan_by_type(a, l);
    if (e != cudaSuccess) return e;
    const long long rows = l.p.seqs.rows;
    const int n = l.p.seqs.n_seqs;
    reduce(l.q.part_B, rows * a.G * a.N, l.q.blocks, g.dB, s);
    reduce(l.q.part_C, rows * a.G * a.N, l.q.blocks, g.dC, s);
    reduce(l.q.part_A, (long long)a.D * a.N, n, g.dA, s);
    reduce(l.q.part_D, a.D, n, g.dDskip, s);
    reduce(l.q.part_bias, a.D, n, g.ddt_bias, s);
    return cudaGetLastError();
}

}  // namespace kda
