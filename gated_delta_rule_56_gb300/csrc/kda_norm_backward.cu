// kda_norm_backward.cu -- gradients of the layer norm and RMS norm with their gate.
//
// With h = x - mean (or x), r = 1 / sqrt(mean h^2 + eps), d = dy act(z), t = d w:
//     dx = r (t - mean(t) - h r^2 mean(t h)) + d_sum   (without mean(t) for RMS);   dz = dy (h r w + b) act'(z)
//     dweight = sum d h r,  dbias = sum d   over all lines
//
// A line is held in registers as in the forward pass (above 4096 values, 2048 that are not aligned, part of it spills): every
// input is read from HBM once, two rounds of sums (one for RMS): sum t and sum t h come with
// the squares. A group keeps its sums of the weights' gradients in registers while it goes over its lines; a second kernel adds the
// blocks' parts in a fixed order with their rounding errors (no atomics). Bound by the latency of the loads: 8 accumulators and 8 inputs per pair
// leave two blocks of 256 threads per SM. Measured: 8192 tokens x 32 heads of 128 with a gate in bf16 109 us, 4.3 TB/s (64 % of the copy rate);
// 4101 lines of 1531 in fp32, which take single values, 44 us, 2.3 TB/s. 2^28 values with weight and bias: width 4096 933 us, 8192 771 us, 16384 1.0 ms,
// 32768 2.3 ms, 32767 6.4 ms; 2^27 in fp32 483, 382, 534 us, 1.1 and 2.4 ms.
#include "kda_layers.h"
#include "kda_norm.cuh"

namespace kda {
namespace {

// sigmoid(z) and 1 - sigmoid(z) = sigmoid(-z), two at a time. With e = exp(-z) the second is e sigmoid(z) where the first is near 1: a
// difference would leave 24 bits of 1, and behind z = 17 nothing (a sigmoid gate's gradient is their product).
__device__ __forceinline__ void sigmoids2(f32x2 z, f32x2 &s, f32x2 &other) {
    float z0, z1, t0, t1;
    unpair(z, z0, z1);
    unpair(mul2(z, both(-kLog2e)), t0, t1);
    const float e0 = ex2(t0), e1 = ex2(t1), s0 = rcp(1.f + e0), s1 = rcp(1.f + e1);
    s = pair(s0, s1);
    other = pair(z0 < 0.f ? 1.f - s0 : e0 * s0, z1 < 0.f ? 1.f - s1 : e1 * s1);
}

template <typename T, int V, int K, int GROUP, bool GATE>
__global__ void __launch_bounds__(kBlock<GROUP>) norm_back_kernel(NormParams p) {
    constexpr int LINES = kBlock<GROUP> / GROUP, P = (V + 1) / 2;
    __shared__ float buf[2][3][32];
    extern __shared__ float gathered[];  // groups of a block: [LINES][K * GROUP * V]
    int turn = 0;
    const int lane = threadIdx.x % GROUP, grp = threadIdx.x / GROUP;
    Line<T, V, K> w, b;
    load_weight<T, V, K, GROUP>(w, p.w, 1.f, lane, p.width);
    if constexpr (GATE) load_weight<T, V, K, GROUP>(b, p.b, 0.f, lane, p.width);
    f32x2 dw[K][P], db[K][P];
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
        for (int j = 0; j < P; ++j) dw[i][j] = db[i][j] = 0ull;
    for (long long first = (long long)blockIdx.x * LINES; first < p.lines; first += (long long)gridDim.x * LINES) {
        const uint32_t line = (uint32_t)min(first + grp, p.lines - 1), row = line / (uint32_t)p.heads;
        const bool live = first + grp < p.lines;
        const long long in = (long long)(line - row * (uint32_t)p.heads) * p.width, out = (long long)line * p.width;
        Line<T, V, K> x, d, z, ds;
        load_line<T, V, K, GROUP>(x, p.x, row * p.xs + in, lane, p.width);
        load_line<T, V, K, GROUP>(d, p.dy, out, lane, p.width);
        if constexpr (GATE) load_line<T, V, K, GROUP>(z, p.z, row * p.zs + in, lane, p.width);
        if (p.d_sum) load_line<T, V, K, GROUP>(ds, p.d_sum, out, lane, p.width);
        f32x2 h[K][P], t[K][P], g[GATE ? K : 1][P];
#pragma unroll
        for (int i = 0; i < K; ++i) to_pairs<T, V>(x.e[i], h[i]);
        if (!p.rms) {
            f32x2 q2 = 0ull;
#pragma unroll
            for (int i = 0; i < K; ++i)
#pragma unroll
                for (int j = 0; j < P; ++j) q2 = add2(q2, h[i][j]);
            float q[1] = {total(q2)};
            sums<GROUP>(q, buf, turn);
            const float mean = q[0] * p.inv;
            const f32x2 less = pair(-mean, V == 1 ? 0.f : -mean);
#pragma unroll
            for (int i = 0; i < K; ++i)
                if ((i * GROUP + lane) * V < p.width)
#pragma unroll
                    for (int j = 0; j < P; ++j) h[i][j] = add2(h[i][j], less);
        }
        f32x2 s0 = 0ull, s1 = 0ull, s2 = 0ull;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            f32x2 wi[P], zi[P];
            to_pairs<T, V>(d.e[i], t[i]);
            to_pairs<T, V>(w.e[i], wi);
            if constexpr (GATE) to_pairs<T, V>(z.e[i], zi);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                f32x2 v = t[i][j];
                if constexpr (GATE) {  // silu' = s (1 + z (1 - s)), sigmoid' = s (1 - s)
                    f32x2 s, other;
                    sigmoids2(zi[j], s, other);
                    const f32x2 vs = mul2(v, s);
                    g[i][j] = mul2(vs, p.silu ? fma2(zi[j], other, both(1.f)) : other);
                    v = p.silu ? mul2(vs, zi[j]) : vs;
                }
                if (live) db[i][j] = add2(db[i][j], v);
                t[i][j] = v;
                v = mul2(v, wi[j]);
                s0 = fma2(h[i][j], h[i][j], s0);
                s1 = fma2(v, h[i][j], s1);
                s2 = add2(s2, v);
            }
        }
        float q[3] = {total(s0), total(s1), total(s2)};
        sums<GROUP>(q, buf, turn);
        const float rf = 1.f / sqrtf(fmaf(q[0], p.inv, p.eps));
        const f32x2 r = both(rf), c1 = both(-q[1] * p.inv * rf * rf), c0 = both(p.rms ? 0.f : -q[2] * p.inv);
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int e = (i * GROUP + lane) * V;
            f32x2 wi[P], o[P], more[P];
            to_pairs<T, V>(w.e[i], wi);
            if (p.d_sum) to_pairs<T, V>(ds.e[i], more);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const f32x2 u = fma2(h[i][j], c1, fma2(t[i][j], wi[j], c0)), hr = mul2(h[i][j], r);
                o[j] = p.d_sum ? fma2(u, r, more[j]) : mul2(u, r);
                if (live) dw[i][j] = fma2(t[i][j], hr, dw[i][j]);
                h[i][j] = hr;
            }
            if (live && e < p.width) {
                store_pairs<V>(p.dx + out + e, o);
                if constexpr (GATE) {
                    f32x2 bi[P];
                    to_pairs<T, V>(b.e[i], bi);
#pragma unroll
                    for (int j = 0; j < P; ++j) o[j] = mul2(g[i][j], fma2(h[i][j], wi[j], bi[j]));
                    store_pairs<V>(p.dz + out + e, o);
                }
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
                    for (int j = 0; j < V; j += 2) {
                        float x, y;
                        unpair(a ? db[i][j / 2] : dw[i][j / 2], x, y);
                        part[a * p.width + e + j] = x;
                        if (V > 1) part[a * p.width + e + j + 1] = y;
                    }
            }
        } else {
            constexpr int WIDTH = K * GROUP * V;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < K; ++i)
#pragma unroll
                for (int j = 0; j < V; j += 2) {
                    float x, y;
                    unpair(a ? db[i][j / 2] : dw[i][j / 2], x, y);
                    gathered[grp * WIDTH + (i * GROUP + lane) * V + j] = x;
                    if (V > 1) gathered[grp * WIDTH + (i * GROUP + lane) * V + j + 1] = y;
                }
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

// Blocks of the first kernel: four per SM, two where they have 512 threads and more, and no more than there are lines (by the width alone: the
// workspace is sized before the alignment is known). 8192 tokens x 32 heads of 128 with a gate, bf16: 108 us with four, 143 with two, 121 with
// eight, whose parts cost more to add up.
int back_blocks(long long lines, int width, int sms) {
    const long long most = (long long)sms * (width <= 2048 ? 4 : 2);
    return (int)(lines < 1 ? 1 : lines < most ? lines : most);
}

template <typename T, bool GATE>
struct Backward {
    const NormParams &p;
    int blocks;
    cudaStream_t s;
    template <int V, int K, int GROUP>
    cudaError_t run() const {
        constexpr int LINES = kBlock<GROUP> / GROUP, bytes = LINES == 1 ? 0 : LINES * K * GROUP * V * 4;
        static_assert(bytes <= 48 * 1024 - 1024, "shared memory of the weights' sums");
        norm_back_kernel<T, V, K, GROUP, GATE><<<blocks, kBlock<GROUP>, bytes, s>>>(p);
        return cudaGetLastError();
    }
};

template <typename T>
cudaError_t backward(const NormParams &p, int blocks, cudaStream_t s) {
    const bool wide = wide_lines<T>(p);
    constexpr int V = 16 / sizeof(T);
    return p.z ? by_width<V>(p.width, wide, Backward<T, true>{p, blocks, s}) : by_width<V>(p.width, wide, Backward<T, false>{p, blocks, s});
}

}  // namespace

size_t layer_norm_backward_workspace_bytes(const kda_layer_norm_args &a, int sms) {
    return a.weight || a.bias ? (size_t)back_blocks(a.rows * a.heads, a.width, sms) * 2 * a.width * 4 : 0;
}

cudaError_t launch_layer_norm_backward(const kda_layer_norm_args &a, const void *dy, const void *d_sum, float *dx, float *dz,
                                       float *dweight, float *dbias, void *ws, int sms, cudaStream_t s) {
    NormParams p = norm_params(a);
    p.dy = dy;
    p.d_sum = d_sum;
    p.dx = dx;
    p.dz = dz;
    p.part = a.weight || a.bias ? static_cast<float *>(ws) : nullptr;
    const int blocks = back_blocks(p.lines, p.width, sms);
    const cudaError_t e = a.dtype == KDA_BF16 ? backward<__nv_bfloat16>(p, blocks, s) : backward<float>(p, blocks, s);
    if (e != cudaSuccess || !p.part) return e;
    norm_parts_kernel<<<dim3((unsigned)((a.width + 31) / 32), 2), 256, 0, s>>>(p.part, blocks, a.width, dweight, dbias);
    return cudaGetLastError();
}

}  // namespace kda
