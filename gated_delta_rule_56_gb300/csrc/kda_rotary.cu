// kda_rotary.cu -- the norm of every head's row of q and k and the position rotation, in one pass.
//
//     u = x w r,  r = 1 / sqrt(sum x^2 / size + eps)  (size: the head for RMS, 1 for L2);  pairs of u rotated
//
// Bound by HBM: q and k are read once and written once. A row of a head is held by a group of lanes, 8 values
// each (one 16-byte load in bf16); the sum of squares goes through the group's shuffles. The lane's cosines and
// sines stay in registers while its warp goes over the heads of one token, so the tables are read once per
// token and not once per head. Four heads' loads are issued together and kept as they were loaded until used: converted at
// once they took twice the registers and the kernel 238 us where it takes 172 (32768 tokens x 64 heads of 128 in bf16: 6.2 TB/s
// of q and k read and written, 92 % of the measured copy rate). The 64 registers of four blocks per SM hold that but for 12 to 24 bytes; in fp32,
// and for rows that are not 16-byte aligned, 110 to 200 bytes per thread spill (fp32: 339 us, 6.3 TB/s all the same). The backward pass (8192 tokens x 40 heads):
// 70 us, 4.8 TB/s; its two inputs, the gradient and the weights' sums leave room for 16 warps per SM (fp32: up to 147 registers, 8 warps, 101 us,
// 5.0 TB/s).
#include "kda_layers.cuh"
#include "kda_layers.h"

namespace kda {
namespace {

constexpr int kWarps = 8;
constexpr int kBatch = 4, kBackBatch = 4;  // heads of a lane group whose loads are issued together

struct RotaryParams {
    const void *q, *k, *qw, *kw;
    long long q_stride, k_stride, rows, table_rows;
    int q_heads, k_heads, head, half;
    bool interleaved;
    float inv_size, eps;  // sum x^2 * inv_size + eps
    const float *cos, *sin;
    const int32_t *pos;
    unsigned *err;
};

// The 8 cosines and sines of a lane's values. Every value x becomes x * cs + partner * sn, with the sign of its
// place in the pair in sn; values past the rotated ones keep cs = 1, sn = 0.
struct Turn {
    float cs[8], sn[8];
};

__device__ __forceinline__ void load_turn(const RotaryParams &p, long long row, int e0, Turn &t) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        t.cs[i] = 1.f;
        t.sn[i] = 0.f;
    }
    if (e0 >= 2 * p.half) return;
    const long long at = p.pos[row];
    if (at < 0 || at >= p.table_rows) {
        atomicOr(p.err, kErrBadPosition);
        return;
    }
    const float *c = p.cos + at * p.half, *s = p.sin + at * p.half;
    if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float cv = c[e0 / 2 + i], sv = s[e0 / 2 + i];
            t.cs[2 * i] = t.cs[2 * i + 1] = cv;
            t.sn[2 * i] = -sv;
            t.sn[2 * i + 1] = sv;
        }
    } else {
        const bool second = e0 >= p.half;
        const int at0 = second ? e0 - p.half : e0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            t.cs[i] = c[at0 + i];
            t.sn[i] = second ? s[at0 + i] : -s[at0 + i];
        }
    }
}

// x * cs + sign * partner * sn: sign 1 rotates, -1 rotates back. `partner`: the lane that holds the other halves.
__device__ __forceinline__ void rotate(float (&x)[8], const Turn &t, float sign, bool interleaved, int partner) {
    float o[8];
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = x[i ^ 1];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, x[i], partner);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], t.cs[i], sign * t.sn[i] * o[i]);
}

template <typename T, bool WIDE>
__device__ __forceinline__ Pack<T, 8> load8(const T *p) {
    if constexpr (WIDE) return load_pack<T, 8>(p);
    Pack<T, 8> r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.e[i] = p[i];
    return r;
}
template <typename T>
__device__ __forceinline__ void to_floats(const Pack<T, 8> &v, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_float(v.e[i]);
}

template <int LANES>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int m = LANES / 2; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// One warp per (token, part of its heads): LANES lanes per head, 32 / LANES heads at a time.
template <typename T, int LANES, bool WIDE>
__global__ void __launch_bounds__(kWarps * 32, 4) rotary_kernel(RotaryParams p, T *__restrict__ q_out, T *__restrict__ k_out,
                                                             int parts) {
    constexpr int GROUPS = 32 / LANES;
    const int lane = threadIdx.x & 31, l = lane % LANES, grp = lane / LANES;
    const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const long long row = w / parts;
    const int part = (int)(w % parts);
    if (row >= p.rows) return;
    const int e0 = l * 8;
    const bool live = e0 < p.head;
    Turn t;
    load_turn(p, row, e0, t);
    const int hv = p.half / 8;  // lanes per half
    const int partner = p.interleaved || e0 >= 2 * p.half ? lane : (l < hv ? lane + hv : lane - hv);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const int heads = side ? p.k_heads : p.q_heads;
        const T *in = static_cast<const T *>(side ? p.k : p.q) + row * (side ? p.k_stride : p.q_stride) + e0;
        T *out = (side ? k_out : q_out) + row * heads * p.head + e0;
        const T *wt = static_cast<const T *>(side ? p.kw : p.qw);
        float g[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = wt && live ? to_float(wt[e0 + i]) : 1.f;
        const int step = parts * GROUPS;
        for (int h0 = part * GROUPS; h0 < heads; h0 += kBatch * step) {
            Pack<T, 8> raw[kBatch];  // a head that is not there takes another's place and is not stored
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int h = min(h0 + b * step + grp, heads - 1);
                raw[b] = load8<T, WIDE>(in + (live ? 0 : -e0) + (long long)h * p.head);
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (h0 + b * step >= heads) break;
                const int h = h0 + b * step + grp;
                float x[8], ss = 0.f;
                to_floats(raw[b], x);
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
                if (!live) ss = 0.f;
                const float r = rsqrtf(fmaf(group_sum<LANES>(ss), p.inv_size, p.eps));
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= r * g[i];
                rotate(x, t, 1.f, p.interleaved, partner);
                if (live && h < heads) {
                    Pack<T, 8> o;
#pragma unroll
                    for (int i = 0; i < 8; ++i) o.e[i] = from_float<T>(x[i]);
                    store_pack<T, 8>(out + (long long)h * p.head, o);
                }
            }
        }
    }
}

// Gradients: d = the output's gradient rotated back;  dw = sum d x r;  dx = r (d w - x r^2 sum(d w x) / size).
// A warp goes over tokens with a stride; the weights' sums of a block's warps are added in a fixed
// order and written to `part` [block][2][head], which rotary_reduce_kernel adds. Plain fp32 within a block (a thread's tokens and heads in one
// accumulator): 2e-7 off 64 bits in the 2-norm for 8192 tokens x 32 heads, where sums in 64 bits would leave 7e-8.
template <typename T, int LANES, bool WIDE>
__global__ void __launch_bounds__(kWarps * 32) rotary_backward_kernel(RotaryParams p, const T *__restrict__ dq_out,
                                                                      const T *__restrict__ dk_out, float *__restrict__ dq,
                                                                      float *__restrict__ dk, float *__restrict__ part) {
    constexpr int GROUPS = 32 / LANES;
    __shared__ float sums[2][kWarps * GROUPS][LANES * 8];
    const int lane = threadIdx.x & 31, l = lane % LANES, grp = lane / LANES, warp = threadIdx.x >> 5;
    const int e0 = l * 8;
    const bool live = e0 < p.head;
    const int hv = p.half / 8;
    const int partner = p.interleaved || e0 >= 2 * p.half ? lane : (l < hv ? lane + hv : lane - hv);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const int heads = side ? p.k_heads : p.q_heads;
        const T *wt = static_cast<const T *>(side ? p.kw : p.qw);
        const T *dout = side ? dk_out : dq_out;
        float *din = side ? dk : dq;
        float g[8], dw[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            g[i] = wt && live ? to_float(wt[e0 + i]) : 1.f;
            dw[i] = 0.f;
        }
        for (long long row = (long long)blockIdx.x * kWarps + warp; row < p.rows && heads > 0; row += (long long)gridDim.x * kWarps) {
            Turn t;
            load_turn(p, row, e0, t);
            const T *in = static_cast<const T *>(side ? p.k : p.q) + row * (side ? p.k_stride : p.q_stride) + e0;
            const long long at = row * heads * p.head + e0;
            for (int h0 = 0; h0 < heads; h0 += kBackBatch * GROUPS) {
                Pack<T, 8> raw[kBackBatch], raw_d[kBackBatch];
#pragma unroll
                for (int b = 0; b < kBackBatch; ++b) {
                    const long long h = (long long)min(h0 + b * GROUPS + grp, heads - 1) * p.head - (live ? 0 : e0);
                    raw[b] = load8<T, WIDE>(in + h);
                    raw_d[b] = load8<T, WIDE>(dout + at + h);
                }
#pragma unroll
                for (int b = 0; b < kBackBatch; ++b) {
                    if (h0 + b * GROUPS >= heads) break;
                    const int h = h0 + b * GROUPS + grp;
                    float x[8], d[8];
                    to_floats(raw[b], x);
                    to_floats(raw_d[b], d);
                    if (!live || h >= heads) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = d[i] = 0.f;
                    }
                    rotate(d, t, -1.f, p.interleaved, partner);
                    float ss = 0.f, dot = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        ss = fmaf(x[i], x[i], ss);
                        dot = fmaf(d[i] * g[i], x[i], dot);
                    }
                    ss = group_sum<LANES>(ss);
                    dot = group_sum<LANES>(dot);
                    const float r = rsqrtf(fmaf(ss, p.inv_size, p.eps)), k = r * r * dot * p.inv_size;
                    float o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        dw[i] = fmaf(d[i], x[i] * r, dw[i]);
                        o[i] = r * (d[i] * g[i] - x[i] * k);
                    }
                    if (live && h < heads) store_floats<8>(din + at + (long long)h * p.head, o);
                }
            }
        }
        if (part) {
#pragma unroll
            for (int i = 0; i < 8; ++i) sums[side][warp * GROUPS + grp][e0 + i] = dw[i];
        }
    }
    if (!part) return;
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.head; i += kWarps * 32) {
        float sum = 0.f;
        for (int w = 0; w < kWarps * GROUPS; ++w) sum += sums[i / p.head][w][i % p.head];
        part[(long long)blockIdx.x * 2 * p.head + i] = sum;
    }
}

__global__ void rotary_reduce_kernel(const float *__restrict__ part, int blocks, int head, float *__restrict__ dqw,
                                     float *__restrict__ dkw) {
    // One warp per value of one weight: the lanes' sums, then the warp's.
    const int i = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32, lane = threadIdx.x & 31;
    if (i >= 2 * head) return;
    ExactSum lanes;
#pragma unroll 4
    for (int b = lane; b < blocks; b += 32) lanes.add(part[(long long)b * 2 * head + i]);
    float sum = lanes.value();
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    float *out = i < head ? dqw : dkw;
    if (lane == 0 && out) out[i % head] = sum;
}

RotaryParams rotary_params(const kda_rotary_args &a, unsigned *err) {
    RotaryParams p{};
    p.q = a.q;
    p.k = a.k;
    p.qw = a.q_weight;
    p.kw = a.k_weight;
    p.q_stride = a.q_stride ? a.q_stride : (long long)a.q_heads * a.head;
    p.k_stride = a.k_stride ? a.k_stride : (long long)a.k_heads * a.head;
    p.rows = a.rows;
    p.table_rows = a.table_rows;
    p.q_heads = a.q_heads;
    p.k_heads = a.k_heads;
    p.head = a.head;
    p.half = a.half;
    p.interleaved = a.interleaved != 0;
    p.inv_size = a.norm == 0 ? 1.f / (float)a.head : 1.f;
    p.eps = a.eps;
    p.cos = a.cos_table;
    p.sin = a.sin_table;
    p.pos = a.positions;
    p.err = err;
    return p;
}

bool rotary_wide(const RotaryParams &p, int e) {
    return (!p.q_heads || (aligned16(p.q) && p.q_stride * e % 16 == 0)) &&
           (!p.k_heads || (aligned16(p.k) && p.k_stride * e % 16 == 0));
}

template <typename T, bool WIDE, typename F>
void by_lanes(int head, F &&f) {
    const int lanes = head / 8;  // 8 values per lane
    if (lanes <= 1)
        f.template operator()<T, 1, WIDE>();
    else if (lanes <= 2)
        f.template operator()<T, 2, WIDE>();
    else if (lanes <= 4)
        f.template operator()<T, 4, WIDE>();
    else if (lanes <= 8)
        f.template operator()<T, 8, WIDE>();
    else if (lanes <= 16)
        f.template operator()<T, 16, WIDE>();
    else
        f.template operator()<T, 32, WIDE>();
}

template <typename F>
cudaError_t by_type(kda_dtype dtype, const RotaryParams &p, F &&f) {
    if (dtype == KDA_BF16)
        rotary_wide(p, 2) ? by_lanes<__nv_bfloat16, true>(p.head, f) : by_lanes<__nv_bfloat16, false>(p.head, f);
    else
        rotary_wide(p, 4) ? by_lanes<float, true>(p.head, f) : by_lanes<float, false>(p.head, f);
    return cudaGetLastError();
}

struct Forward {
    RotaryParams p;
    void *q_out, *k_out;
    cudaStream_t s;
    template <typename T, int LANES, bool WIDE>
    void operator()() {
        // Warps per token: one while the tokens alone give every SM 32 warps, more for few tokens.
        const int most = ((p.q_heads > p.k_heads ? p.q_heads : p.k_heads) * LANES + 31) / 32;
        int parts = 1;
        while (parts < most && p.rows * parts < 152 * 32) parts *= 2;
        const long long warps = p.rows * parts;
        rotary_kernel<T, LANES, WIDE><<<(unsigned)((warps + kWarps - 1) / kWarps), kWarps * 32, 0, s>>>(
            p, static_cast<T *>(q_out), static_cast<T *>(k_out), parts);
    }
};

struct Backward {
    RotaryParams p;
    const void *dq_out, *dk_out;
    float *dq, *dk, *part;
    int blocks;
    cudaStream_t s;
    template <typename T, int LANES, bool WIDE>
    void operator()() {
        rotary_backward_kernel<T, LANES, WIDE><<<blocks, kWarps * 32, 0, s>>>(
            p, static_cast<const T *>(dq_out), static_cast<const T *>(dk_out), dq, dk, part);
    }
};

int backward_blocks(const kda_rotary_args &a, int sms) {
    // Two blocks per SM are resident in bf16 (one in fp32, for most heads: the others follow it); with four times as many the weights' sums
    // cost 8 us more on 8192 tokens x 40 heads.
    const long long need = (a.rows + kWarps - 1) / kWarps, most = 2LL * (sms > 0 ? sms : 152);
    return (int)(need < most ? need : most);
}

}  // namespace

cudaError_t launch_rotary(const kda_rotary_args &a, void *q_out, void *k_out, unsigned *err, cudaStream_t s) {
    const RotaryParams p = rotary_params(a, err);
    return by_type(a.dtype, p, Forward{p, q_out, k_out, s});
}

size_t rotary_backward_workspace_bytes(const kda_rotary_args &a, int sms) {
    return (size_t)backward_blocks(a, sms) * 2 * a.head * sizeof(float);
}

cudaError_t launch_rotary_backward(const kda_rotary_args &a, const void *dq_out, const void *dk_out, float *dq, float *dk,
                                   float *dq_weight, float *dk_weight, void *ws, int sms, unsigned *err, cudaStream_t s) {
    const RotaryParams p = rotary_params(a, err);
    const int blocks = backward_blocks(a, sms);
    float *part = dq_weight || dk_weight ? static_cast<float *>(ws) : nullptr;
    if (blocks > 0) {
        const cudaError_t e = by_type(a.dtype, p, Backward{p, dq_out, dk_out, dq, dk, part, blocks, s});
        if (e != cudaSuccess) return e;
    }
    if (dq_weight || dk_weight)  // over no rows too: the sums are zeros
        rotary_reduce_kernel<<<(unsigned)((2 * a.head + 7) / 8), 256, 0, s>>>(part, blocks, a.head, dq_weight, dk_weight);
    return cudaGetLastError();
}

}  // namespace kda
