// kda_norm.cu -- layer norm and RMS norm with the residual sum before them and the gate behind them, and their gradients.
//
//     s = x + residual;  h = s - mean (layer) or s (RMS);  r = 1 / sqrt(mean h^2 + eps);  n = h r w + b;  y = n act(z)
// Gradients, with d = dy act(z) and t = d w:
//     dx = r (t - mean(t) - h r^2 mean(t h)) + d_sum   (without mean(t) for RMS);   dz = dy n act'(z)
//     dweight = sum d h r,  dbias = sum d   over all lines
//
// A line (`width` values) is held in registers by a group of lanes (8 to 32 of a warp, or a whole block), so every input is read once:
// bound by HBM. The mean is taken first and the squares of the differences after it, both from registers: no cancellation. The gradients need
// two rounds of sums (one for RMS): sum t and sum t h come with the squares. Weights stay in registers while a group goes over its lines, and so do
// its sums of the weights' gradients; a second kernel adds the blocks' parts in a fixed order (no atomics).
#include "kda_layers.cuh"
#include "kda_layers.h"

namespace kda {
namespace {

struct NormParams {
    const void *x, *res, *z, *w, *b, *dy, *d_sum;
    long long xs, rs, zs;  // elements between rows
    long long lines;       // rows * heads
    int heads, width;
    float inv, eps;        // 1 / width
    bool rms, silu;
    void *y, *sum;
    float *dx, *dz, *part;  // part: [blocks, 2, width]
};

template <typename T, int V, int K>
struct Line {
    Pack<T, V> e[K];
};

// V values at (i * GROUP + lane) * V for i < K.
template <typename T, int V, int K, int GROUP>
__device__ __forceinline__ void load_line(Line<T, V, K> &r, const void *p, long long at, int lane, int width) {
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int e = (i * GROUP + lane) * V;
        if (e < width) {
            r.e[i] = load_pack<T, V>(static_cast<const T *>(p) + at + e);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) r.e[i].e[j] = from_float<T>(0.f);
        }
    }
}

template <int V>
__device__ __forceinline__ void store_line(float *p, const float *x) {
    float v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = x[j];
    store_floats<V>(p, v);
}

// Sums over the lanes of a group, N at a time; every lane gets them. Whole blocks go through shared memory, two buffers in turn.
template <int GROUP, int N>
__device__ __forceinline__ void sums(float (&x)[N], float (*buf)[3][32], int &turn) {
    constexpr int IN = GROUP < 32 ? GROUP : 32;
#pragma unroll
    for (int a = 0; a < N; ++a)
#pragma unroll
        for (int m = IN / 2; m > 0; m >>= 1) x[a] += __shfl_xor_sync(0xffffffffu, x[a], m);
    if constexpr (GROUP > 32) {
        constexpr int W = GROUP / 32;
        const int lane = threadIdx.x & 31;
        if (lane == 0)
#pragma unroll
            for (int a = 0; a < N; ++a) buf[turn][a][threadIdx.x >> 5] = x[a];
        __syncthreads();
#pragma unroll
        for (int a = 0; a < N; ++a) {
            x[a] = lane < W ? buf[turn][a][lane] : 0.f;
#pragma unroll
            for (int m = W / 2; m > 0; m >>= 1) x[a] += __shfl_xor_sync(0xffffffffu, x[a], m);
            x[a] = __shfl_sync(0xffffffffu, x[a], 0);
        }
        turn ^= 1;
    }
}

__device__ __forceinline__ float sigmoid(float z) { return rcp(1.f + ex2(-kLog2e * z)); }

template <int GROUP>
constexpr int kBlock = GROUP < 256 ? 256 : GROUP;

template <typename T, int V, int K, int GROUP>
__global__ void __launch_bounds__(kBlock<GROUP>) norm_kernel(NormParams p) {
    constexpr int LINES = kBlock<GROUP> / GROUP;  // of a block at a time
    static_assert(GROUP <= 32 || LINES == 1, "one line per block");
    __shared__ float buf[2][3][32];
    int turn = 0;
    const int lane = threadIdx.x % GROUP, grp = threadIdx.x / GROUP;
    Line<T, V, K> w, b;
    if (p.w) load_line<T, V, K, GROUP>(w, p.w, 0, lane, p.width);
    if (p.b) load_line<T, V, K, GROUP>(b, p.b, 0, lane, p.width);
    for (long long first = (long long)blockIdx.x * LINES; first < p.lines; first += (long long)gridDim.x * LINES) {
        const long long line = min(first + grp, p.lines - 1);
        const bool live = first + grp < p.lines;
        const long long row = line / p.heads, in = (line - row * p.heads) * p.width, out = line * p.width;
        Line<T, V, K> x, o, z;
        load_line<T, V, K, GROUP>(x, p.x, row * p.xs + in, lane, p.width);
        if (p.res) load_line<T, V, K, GROUP>(o, p.res, row * p.rs + in, lane, p.width);
        if (p.z) load_line<T, V, K, GROUP>(z, p.z, row * p.zs + in, lane, p.width);
        float h[K][V], q[1] = {0.f};
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                h[i][j] = to_float(x.e[i].e[j]);
                if (p.res) h[i][j] += to_float(o.e[i].e[j]);
                q[0] += h[i][j];
            }
        if (p.sum && live)
#pragma unroll
            for (int i = 0; i < K; ++i) {
                const int e = (i * GROUP + lane) * V;
                Pack<T, V> t;
#pragma unroll
                for (int j = 0; j < V; ++j) t.e[j] = from_float<T>(h[i][j]);
                if (e < p.width) store_pack<T, V>(static_cast<T *>(p.sum) + out + e, t);
            }
        float mean = 0.f;
        if (!p.rms) {
            sums<GROUP>(q, buf, turn);
            mean = q[0] * p.inv;
        }
        q[0] = 0.f;
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                h[i][j] = (i * GROUP + lane) * V < p.width ? h[i][j] - mean : 0.f;
                q[0] = fmaf(h[i][j], h[i][j], q[0]);
            }
        sums<GROUP>(q, buf, turn);
        const float r = 1.f / sqrtf(fmaf(q[0], p.inv, p.eps));
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int e = (i * GROUP + lane) * V;
            Pack<T, V> t;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float y = h[i][j] * r;
                if (p.w) y *= to_float(w.e[i].e[j]);
                if (p.b) y += to_float(b.e[i].e[j]);
                if (p.z) {
                    const float zv = to_float(z.e[i].e[j]), s = sigmoid(zv);
                    y *= p.silu ? zv * s : s;
                }
                t.e[j] = from_float<T>(y);
            }
            if (live && e < p.width) store_pack<T, V>(static_cast<T *>(p.y) + out + e, t);
        }
    }
}

template <typename T, int V, int K, int GROUP>
__global__ void __launch_bounds__(kBlock<GROUP>) norm_back_kernel(NormParams p) {
    constexpr int LINES = kBlock<GROUP> / GROUP;
    __shared__ float buf[2][3][32];
    extern __shared__ float gathered[];  // groups of a block: [LINES][K * GROUP * V]
    int turn = 0;
    const int lane = threadIdx.x % GROUP, grp = threadIdx.x / GROUP;
    Line<T, V, K> w, b;
    if (p.w) load_line<T, V, K, GROUP>(w, p.w, 0, lane, p.width);
    if (p.b) load_line<T, V, K, GROUP>(b, p.b, 0, lane, p.width);
    float dw[K][V], db[K][V];
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) dw[i][j] = db[i][j] = 0.f;
    for (long long first = (long long)blockIdx.x * LINES; first < p.lines; first += (long long)gridDim.x * LINES) {
        const long long line = min(first + grp, p.lines - 1);
        const bool live = first + grp < p.lines;
        const long long row = line / p.heads, in = (line - row * p.heads) * p.width, out = line * p.width;
        Line<T, V, K> x, d, z, ds;
        load_line<T, V, K, GROUP>(x, p.x, row * p.xs + in, lane, p.width);
        load_line<T, V, K, GROUP>(d, p.dy, out, lane, p.width);
        if (p.z) load_line<T, V, K, GROUP>(z, p.z, row * p.zs + in, lane, p.width);
        if (p.d_sum) load_line<T, V, K, GROUP>(ds, p.d_sum, out, lane, p.width);
        float mean = 0.f;
        if (!p.rms) {
            float q[1] = {0.f};
#pragma unroll
            for (int i = 0; i < K; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) q[0] += to_float(x.e[i].e[j]);
            sums<GROUP>(q, buf, turn);
            mean = q[0] * p.inv;
        }
        float t[K][V], q[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float h = (i * GROUP + lane) * V < p.width ? to_float(x.e[i].e[j]) - mean : 0.f;
                float v = to_float(d.e[i].e[j]);
                if (p.z) {
                    const float zv = to_float(z.e[i].e[j]), s = sigmoid(zv);
                    v *= p.silu ? zv * s : s;
                }
                if (live) db[i][j] += v;
                if (p.w) v *= to_float(w.e[i].e[j]);
                t[i][j] = v;
                q[0] = fmaf(h, h, q[0]);
                q[1] = fmaf(v, h, q[1]);
                q[2] += v;
            }
        sums<GROUP>(q, buf, turn);
        const float r = 1.f / sqrtf(fmaf(q[0], p.inv, p.eps));
        const float c1 = q[1] * p.inv * r * r, c0 = p.rms ? 0.f : q[2] * p.inv;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int e = (i * GROUP + lane) * V;
            float o[V], g[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float h = to_float(x.e[i].e[j]) - mean;
                o[j] = r * (t[i][j] - c0 - h * c1);
                if (p.d_sum) o[j] += to_float(ds.e[i].e[j]);
                float dv = to_float(d.e[i].e[j]);
                if (p.z) {
                    const float zv = to_float(z.e[i].e[j]), s = sigmoid(zv);
                    float n = h * r;
                    if (p.w) n *= to_float(w.e[i].e[j]);
                    if (p.b) n += to_float(b.e[i].e[j]);
                    g[j] = dv * n * (p.silu ? s * fmaf(zv, 1.f - s, 1.f) : s * (1.f - s));
                    dv *= p.silu ? zv * s : s;
                }
                if (live) dw[i][j] = fmaf(dv, h * r, dw[i][j]);
            }
            if (live && e < p.width) {
                store_line<V>(p.dx + out + e, o);
                if (p.z) store_line<V>(p.dz + out + e, g);
            }
        }
    }
    if (!p.part) return;
    float *part = p.part + (size_t)blockIdx.x * 2 * p.width;
    for (int a = 0; a < 2; ++a) {
        if (a == 0 ? !p.w : !p.b) continue;
        if constexpr (LINES == 1) {
#pragma unroll
            for (int i = 0; i < K; ++i) {
                const int e = (i * GROUP + lane) * V;
                if (e < p.width)
#pragma unroll
                    for (int j = 0; j < V; ++j) part[a * p.width + e + j] = a ? db[i][j] : dw[i][j];
            }
        } else {
            constexpr int WIDTH = K * GROUP * V;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < K; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) gathered[grp * WIDTH + (i * GROUP + lane) * V + j] = a ? db[i][j] : dw[i][j];
            __syncthreads();
            for (int e = threadIdx.x; e < p.width; e += kBlock<GROUP>) {
                float x = 0.f;
                for (int l = 0; l < LINES; ++l) x += gathered[l * WIDTH + e];
                part[a * p.width + e] = x;
            }
        }
    }
}

// Sums of the blocks' parts: 32 columns of one of the two per block, 8 rows at a time.
__global__ void __launch_bounds__(256) norm_parts_kernel(const float *part, int blocks, int width, float *dweight, float *dbias) {
    __shared__ float sum[8][33], rest[8][33];
    float *out = blockIdx.y ? dbias : dweight;
    if (!out) return;
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
    ExactSum s;
    if (c < width)
        for (int i = g; i < blocks; i += 8) s.add(part[((size_t)i * 2 + blockIdx.y) * width + c]);
    sum[g][threadIdx.x & 31] = s.sum;
    rest[g][threadIdx.x & 31] = s.rest;
    __syncthreads();
    if (g == 0 && c < width) {
        for (int i = 1; i < 8; ++i) {
            s.add(sum[i][threadIdx.x]);
            s.rest += rest[i][threadIdx.x];
        }
        out[c] = s.value();
    }
}

constexpr int kBackBlocks = 2;  // blocks of 256 threads per SM of the gradients

NormParams norm_params(const kda_layer_norm_args &a) {
    NormParams p{};
    p.x = a.x;
    p.res = a.residual;
    p.z = a.z;
    p.w = a.weight;
    p.b = a.bias;
    const long long dense = (long long)a.heads * a.width;
    p.xs = a.x_stride ? a.x_stride : dense;
    p.rs = a.residual_stride ? a.residual_stride : dense;
    p.zs = a.z_stride ? a.z_stride : dense;
    p.lines = a.rows * a.heads;
    p.heads = a.heads;
    p.width = a.width;
    p.inv = 1.f / (float)a.width;
    p.eps = a.eps;
    p.rms = a.norm == 1;
    p.silu = a.activation == 0;
    return p;
}

// Blocks of the gradients' first kernel, by the width alone (the workspace is sized before the alignment is known).
int back_blocks(long long lines, int sms) { return (int)(lines < (long long)kBackBlocks * sms ? (lines > 0 ? lines : 1) : (long long)kBackBlocks * sms); }

template <typename T, int V, int K, int GROUP, bool BACK>
cudaError_t launch_norm(const NormParams &p, int blocks, cudaStream_t s) {
    constexpr int LINES = kBlock<GROUP> / GROUP;
    const long long all = (p.lines + LINES - 1) / LINES;
    if constexpr (BACK) {
        constexpr int bytes = LINES == 1 ? 0 : LINES * K * GROUP * V * 4;
        static_assert(bytes <= 48 * 1024 - 1024, "shared memory of the weights' sums");
        norm_back_kernel<T, V, K, GROUP><<<blocks, kBlock<GROUP>, bytes, s>>>(p);
    } else {
        norm_kernel<T, V, K, GROUP><<<(unsigned)(all < blocks ? all : blocks), kBlock<GROUP>, 0, s>>>(p);
    }
    return cudaGetLastError();
}

// The group for a width: one warp or less while a lane holds at most 32 values, then blocks.
template <typename T, bool BACK>
cudaError_t norm_by_width(const NormParams &p, bool wide, int blocks, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    if (wide) {
        const int packs = p.width / V;
        if (packs <= 8) return launch_norm<T, V, 1, 8, BACK>(p, blocks, s);
        if (packs <= 16) return launch_norm<T, V, 1, 16, BACK>(p, blocks, s);
        if (packs <= 32) return launch_norm<T, V, 1, 32, BACK>(p, blocks, s);
        if (packs <= 64) return launch_norm<T, V, 2, 32, BACK>(p, blocks, s);
        if (packs <= 128) return launch_norm<T, V, 4, 32, BACK>(p, blocks, s);
        if (packs <= 256) return launch_norm<T, V, 1, 256, BACK>(p, blocks, s);
        if (packs <= 512) return launch_norm<T, V, 2, 256, BACK>(p, blocks, s);
        if (packs <= 1024) return launch_norm<T, V, 2, 512, BACK>(p, blocks, s);
        if (packs <= 2048) return launch_norm<T, V, 2, 1024, BACK>(p, blocks, s);
        if (packs <= 4096) return launch_norm<T, V, 4, 1024, BACK>(p, blocks, s);
        if constexpr (V == 4) return launch_norm<T, V, 8, 1024, BACK>(p, blocks, s);
        return cudaErrorInvalidValue;
    }
    if (p.width <= 64) return launch_norm<T, 1, 2, 32, BACK>(p, blocks, s);
    if (p.width <= 256) return launch_norm<T, 1, 8, 32, BACK>(p, blocks, s);
    if (p.width <= 1024) return launch_norm<T, 1, 4, 256, BACK>(p, blocks, s);
    if (p.width <= 2048) return launch_norm<T, 1, 8, 256, BACK>(p, blocks, s);
    if (p.width <= 8192) return launch_norm<T, 1, 8, 1024, BACK>(p, blocks, s);
    return launch_norm<T, 1, 32, 1024, BACK>(p, blocks, s);
}

template <typename T>
bool wide_lines(const NormParams &p) {
    constexpr int V = 16 / sizeof(T);
    auto ok = [](const void *x, long long stride) { return aligned16(x) && stride % V == 0; };
    return p.width % V == 0 && ok(p.x, p.xs) && ok(p.res, p.res ? p.rs : 0) && ok(p.z, p.z ? p.zs : 0) && ok(p.w, 0) && ok(p.b, 0) &&
           ok(p.y, 0) && ok(p.sum, 0) && ok(p.dy, 0) && ok(p.d_sum, 0) && ok(p.dx, 0) && ok(p.dz, 0);
}

}  // namespace

cudaError_t launch_layer_norm(const kda_layer_norm_args &a, void *y, void *sum, int sms, cudaStream_t s) {
    NormParams p = norm_params(a);
    p.y = y;
    p.sum = sum;
    const int blocks = sms * 16;
    return a.dtype == KDA_BF16 ? norm_by_width<__nv_bfloat16, false>(p, wide_lines<__nv_bfloat16>(p), blocks, s)
                               : norm_by_width<float, false>(p, wide_lines<float>(p), blocks, s);
}

size_t layer_norm_backward_workspace_bytes(const kda_layer_norm_args &a, int sms) {
    return a.weight || a.bias ? (size_t)back_blocks(a.rows * a.heads, sms) * 2 * a.width * 4 : 0;
}

cudaError_t launch_layer_norm_backward(const kda_layer_norm_args &a, const void *dy, const void *d_sum, float *dx, float *dz,
                                       float *dweight, float *dbias, void *ws, int sms, cudaStream_t s) {
    NormParams p = norm_params(a);
    p.dy = dy;
    p.d_sum = d_sum;
    p.dx = dx;
    p.dz = dz;
    p.part = a.weight || a.bias ? static_cast<float *>(ws) : nullptr;
    const int blocks = back_blocks(p.lines, sms);
    const cudaError_t e = a.dtype == KDA_BF16 ? norm_by_width<__nv_bfloat16, true>(p, wide_lines<__nv_bfloat16>(p), blocks, s)
                                              : norm_by_width<float, true>(p, wide_lines<float>(p), blocks, s);
    if (e != cudaSuccess || !p.part) return e;
    norm_parts_kernel<<<dim3((unsigned)((a.width + 31) / 32), 2), 256, 0, s>>>(p.part, blocks, a.width, dweight, dbias);
    return cudaGetLastError();
}

}  // namespace kda
