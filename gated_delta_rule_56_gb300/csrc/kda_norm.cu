// kda_norm.cu -- layer norm and RMS norm with the residual sum before them and the gate behind them.
//
//     s = x + residual;  h = s - mean (layer) or s (RMS);  r = 1 / sqrt(mean h^2 + eps);  y = (h r w + b) act(z)
//
// A line (`width` values) is held in registers by a group of lanes (8 to 32 of a warp, or a whole block), so every input is read from HBM once:
// bound by it as long as the instructions fit, which they do in register pairs with the options known to the compiler. Lines above 16384 values
// (8192 with a gate, or where they are not 16-byte aligned) take more registers than a thread of such blocks has, and part of them spills. The mean is taken
// first and the squares of the differences after it, both from registers: no cancellation. Weights stay in registers while a group goes over its lines.
// Measured (bf16): 32768 tokens x 32 heads of 128 with a SiLU gate 151 us, 5.3 TB/s (79 % of the copy rate); 8192 rows of 4096 with residual and bias
// 52 us, 5.2 TB/s (77 %); 16 rows 4.1 us in a captured graph, a launch. 2^28 values with weight
// and bias: width 4096 235 us, 8192 269 us, 16384 321 us, 32768 294 us; width 32767, value by value, 750 us; 2^27 in fp32 190, 290, 219, 302 and 389 us. One element at a time with the options looked up per element it took 203
// and 82 us; the next line's loads ahead of the work took registers and with them blocks: 269 to 404 us.
#include "kda_layers.h"
#include "kda_norm.cuh"

namespace kda {
namespace {

template <typename T, int V, int K, int GROUP, bool RES, bool GATE>
__global__ void __launch_bounds__(kBlock<GROUP>) norm_kernel(NormParams p) {
    constexpr int LINES = kBlock<GROUP> / GROUP, P = (V + 1) / 2;  // lines of a block at a time, pairs of a pack
    static_assert(GROUP <= 32 || LINES == 1, "one line per block");
    __shared__ float buf[2][3][32];
    int turn = 0;
    const int lane = threadIdx.x % GROUP, grp = threadIdx.x / GROUP;
    Line<T, V, K> w, b;
    load_weight<T, V, K, GROUP>(w, p.w, 1.f, lane, p.width);
    load_weight<T, V, K, GROUP>(b, p.b, 0.f, lane, p.width);
    for (long long first = (long long)blockIdx.x * LINES; first < p.lines; first += (long long)gridDim.x * LINES) {
        const uint32_t line = (uint32_t)min(first + grp, p.lines - 1), row = line / (uint32_t)p.heads;
        const bool live = first + grp < p.lines;
        const long long in = (long long)(line - row * (uint32_t)p.heads) * p.width, out = (long long)line * p.width;
        Line<T, V, K> x, o, z;
        load_line<T, V, K, GROUP>(x, p.x, row * p.xs + in, lane, p.width);
        if constexpr (RES) load_line<T, V, K, GROUP>(o, p.res, row * p.rs + in, lane, p.width);
        if constexpr (GATE) load_line<T, V, K, GROUP>(z, p.z, row * p.zs + in, lane, p.width);
        f32x2 h[K][P], q2 = 0ull;
        float q[1];
#pragma unroll
        for (int i = 0; i < K; ++i) {
            to_pairs<T, V>(x.e[i], h[i]);
            if constexpr (RES) {
                f32x2 r[P];
                to_pairs<T, V>(o.e[i], r);
#pragma unroll
                for (int j = 0; j < P; ++j) h[i][j] = add2(h[i][j], r[j]);
                const int e = (i * GROUP + lane) * V;
                if (p.sum && live && e < p.width) store_pack<T, V>(static_cast<T *>(p.sum) + out + e, from_pairs<T, V>(h[i]));
            }
        }
        if (!p.rms) {
#pragma unroll
            for (int i = 0; i < K; ++i)
#pragma unroll
                for (int j = 0; j < P; ++j) q2 = add2(q2, h[i][j]);
            q[0] = total(q2);
            sums<GROUP>(q, buf, turn);
            const float mean = q[0] * p.inv;
            const f32x2 less = pair(-mean, V == 1 ? 0.f : -mean);
#pragma unroll
            for (int i = 0; i < K; ++i)
                if ((i * GROUP + lane) * V < p.width)
#pragma unroll
                    for (int j = 0; j < P; ++j) h[i][j] = add2(h[i][j], less);
        }
        q2 = 0ull;
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
            for (int j = 0; j < P; ++j) q2 = fma2(h[i][j], h[i][j], q2);
        q[0] = total(q2);
        sums<GROUP>(q, buf, turn);
        const f32x2 r = both(1.f / sqrtf(fmaf(q[0], p.inv, p.eps)));
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int e = (i * GROUP + lane) * V;
            f32x2 wi[P], bi[P], zi[P];
            to_pairs<T, V>(w.e[i], wi);
            to_pairs<T, V>(b.e[i], bi);
            if constexpr (GATE) to_pairs<T, V>(z.e[i], zi);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                h[i][j] = fma2(mul2(h[i][j], r), wi[j], bi[j]);
                if constexpr (GATE) {
                    const f32x2 s = sigmoid2(zi[j]);
                    h[i][j] = mul2(p.silu ? mul2(h[i][j], zi[j]) : h[i][j], s);
                }
            }
            if (live && e < p.width) store_pack<T, V>(static_cast<T *>(p.y) + out + e, from_pairs<T, V>(h[i]));
        }
    }
}

template <typename T, bool RES, bool GATE>
struct Forward {
    const NormParams &p;
    int sms;
    cudaStream_t s;
    template <int V, int K, int GROUP>
    cudaError_t run() const {
        constexpr int LINES = kBlock<GROUP> / GROUP;
        static const int per_sm = [] {
            int n = 0;
            return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, norm_kernel<T, V, K, GROUP, RES, GATE>, kBlock<GROUP>, 0) == cudaSuccess &&
                           n > 0
                       ? n
                       : 1;
        }();
        const long long all = (p.lines + LINES - 1) / LINES, resident = (long long)sms * per_sm;
        norm_kernel<T, V, K, GROUP, RES, GATE><<<(unsigned)(all < resident ? all : resident), kBlock<GROUP>, 0, s>>>(p);
        return cudaGetLastError();
    }
};

template <typename T>
cudaError_t forward(const NormParams &p, int sms, cudaStream_t s) {
    const bool wide = wide_lines<T>(p);
    constexpr int V = 16 / sizeof(T);
    if (p.res) return p.z ? by_width<V>(p.width, wide, Forward<T, true, true>{p, sms, s}) : by_width<V>(p.width, wide, Forward<T, true, false>{p, sms, s});
    return p.z ? by_width<V>(p.width, wide, Forward<T, false, true>{p, sms, s}) : by_width<V>(p.width, wide, Forward<T, false, false>{p, sms, s});
}

}  // namespace

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

cudaError_t launch_layer_norm(const kda_layer_norm_args &a, void *y, void *sum, int sms, cudaStream_t s) {
    NormParams p = norm_params(a);
    p.y = y;
    p.sum = sum;
    return a.dtype == KDA_BF16 ? forward<__nv_bfloat16>(p, sms, s) : forward<float>(p, sms, s);
}

}  // namespace kda
