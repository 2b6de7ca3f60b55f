// kda_delta_tc.cuh -- what the tensor-core kernels of the delta rule with one decay per value head share (kda_delta_tc.cu,
// kda_delta_tc_backward.cu): operands in several bf16 values, waits, decays of a chunk, tensor maps.
#pragma once

#include <cudaTypedefs.h>

#include "kda_delta.cuh"
#include "kda_delta_tc.h"
#include "kda_tc.cuh"

namespace kda {
namespace delta_tc {

using namespace tc;

constexpr int C = 64;                        // rows of a chunk
constexpr uint64_t kWaitNs = 1000000000ull;  // 1 s per wait

struct Vec {
    float E[C], F[C], b[C], be[C];  // exp(G_i), exp(G_C - G_i), beta_i, beta_i exp(G_i)
    float whole, pad[3];            // exp(G_C)
};

// a, b as hi + lo, each a pair of bf16 values: 2^-16 at most is left.
__device__ __forceinline__ void rest_of(float a, float b, uint32_t hi, float &c, float &d) {
    c = a - __uint_as_float(hi << 16);
    d = b - __uint_as_float(hi & 0xffff0000u);
}
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    float c, d;
    hi = pack_bf16(a, b);
    rest_of(a, b, hi, c, d);
    lo = pack_bf16(c, d);
}
__device__ __forceinline__ void split3(float a, float b, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    float c, d, e, f;
    hi = pack_bf16(a, b);
    rest_of(a, b, hi, c, d);
    mid = pack_bf16(c, d);
    rest_of(c, d, mid, e, f);
    lo = pack_bf16(e, f);
}

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, kWaitNs));
}
// One arrival per warp, behind everything its lanes did.
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// K step st (16 channels) of a K-major operand in 128-byte swizzled tiles of 64 channels, `tile` bytes apart.
__device__ __forceinline__ uint64_t kstep(int st, uint32_t tile) {
    return (uint64_t)(((uint32_t)(st >> 2) * tile + (uint32_t)(st & 3) * 32u) >> 4);
}

// x[j] = D_ij x[j] (times `scale`) for the 16 columns from c0, a block: decays of row i against the rows of its own and earlier blocks
// of 16; zero behind the diagonal (on it unless `diagonal`). Only products of decays, so nothing cancels and nothing overflows. a: decay of a
// row; pre: within its block, up to the row; f: from the row to its block's end.
__device__ __forceinline__ void decay_block(float *x, const float *a, const float *pre, const float *f, int i, int c0, bool diagonal, float scale) {
    const int bi = i >> 4, in = i & 15;
    if (c0 < 16 * bi) {  // row -> end of the block, the blocks between, start of this block -> row
        float e = scale * pre[i];
        for (int m = (c0 >> 4) + 1; m < bi; ++m) e *= pre[16 * m + 15];
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            const ulonglong2 f4 = *reinterpret_cast<const ulonglong2 *>(f + c0 + j);
            unpair(mul2(pair(x[j], x[j + 1]), mul2(both(e), f4.x)), x[j], x[j + 1]);
            unpair(mul2(pair(x[j + 2], x[j + 3]), mul2(both(e), f4.y)), x[j + 2], x[j + 3]);
        }
    } else if (c0 == 16 * bi) {
        float D = scale;
#pragma unroll
        for (int j = 12; j >= 0; j -= 4) {
            const float4 a4 = *reinterpret_cast<const float4 *>(a + c0 + j);
            const float av[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
            for (int m = 3; m >= 0; --m) {
                const int at = j + m;  // D is that of column `at` when its turn comes
                x[at] = at < in || (diagonal && at == in) ? D * x[at] : 0.f;
                D = at <= in ? D * av[m] : D;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = 0.f;
    }
}

// A chunk's decays, by one warp: lane = rows lane and lane + 32 with log-decays own and beta b. Each is the exponential of a sum of its own
// log-decays alone (prefix or suffix sums, never differences): neighbours behind a strong decay keep their small ones. `wait` is called
// between the sums and the first store.
template <typename Wait>
__device__ __forceinline__ bool chunk_decays(Vec &v, float *a, float *pre, float *f, int lane, const float (&own)[2], const float (&b)[2],
                                             Wait wait) {
    const bool second = lane & 16, last = (lane & 15) == 15;
    float up[2] = {own[0], own[1]}, down[2] = {own[0], own[1]}, total[4];
#pragma unroll
    for (int d = 1; d < 16; d *= 2)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float x = __shfl_up_sync(0xffffffffu, up[half], d, 16), y = __shfl_down_sync(0xffffffffu, down[half], d, 16);
            if ((lane & 15) >= d) up[half] += x;
            if ((lane & 15) + d < 16) down[half] += y;
        }
#pragma unroll
    for (int e = 0; e < 4; ++e) total[e] = __shfl_sync(0xffffffffu, up[e >> 1], 16 * (e & 1) + 15);
    if (!wait()) return false;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const float next = __shfl_down_sync(0xffffffffu, down[half], 1, 16), behind = last ? 0.f : next;
        const int i = lane + 32 * half;
        float before = half ? total[0] + total[1] : 0.f, after = half ? 0.f : total[2] + total[3];
        if (second) before += total[2 * half]; else after += total[2 * half + 1];
        const float E = expf(up[half] + before);
        if (a) {
            a[i] = expf(own[half]);
            pre[i] = expf(up[half]);
            f[i] = expf(behind);
        }
        v.E[i] = E;
        v.F[i] = expf(behind + after);
        v.b[i] = b[half];
        v.be[i] = b[half] * E;
    }
    if (lane == 0) v.whole = expf((total[0] + total[1]) + (total[2] + total[3]));
    return true;
}

// 8 values of row i, channels 8 chunk .. 8 chunk + 7, as two bf16 operands of 64 x 64 (128-byte swizzle).
__device__ __forceinline__ void store_operand(uint8_t *hi, uint8_t *lo, int i, int chunk, const float *x) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split2(x[2 * e], x[2 * e + 1], h[e], l[e]);
    const uint32_t at = (uint32_t)i * 128u + (uint32_t)((chunk ^ (i & 7)) << 4);
    *reinterpret_cast<uint4 *>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4 *>(lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
}

// The state's operands from its fp32 values, N of a thread.
template <int N>
__device__ __forceinline__ void publish_state(const float (&S)[N], uint32_t at) {
#pragma unroll
    for (int g = 0; g < N; g += 16) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) split2(S[g + 2 * e], S[g + 2 * e + 1], hi[e], lo[e]);
        tmem_st(at + g / 2, hi);
        tmem_st(at + 64 + g / 2, lo);
    }
    tmem_st_wait();
    tc_fence_before();
}

// 16 values times 16 of shared memory.
__device__ __forceinline__ void scale16(float (&x)[16], const float *by) {
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
        const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(by + e);
        unpair(mul2(pair(x[e], x[e + 1]), f.x), x[e], x[e + 1]);
        unpair(mul2(pair(x[e + 2], x[e + 3]), f.y), x[e + 2], x[e + 3]);
    }
}

// Rows of `heads` heads of d channels, `stride` elements apart, in boxes of 64 rows x 64 channels (128-byte swizzle); what lies past the
// channels and the rows reads as zeros. False if the driver's encoder is unavailable or rejects it.
bool encode(CUtensorMap *map, const void *base, long long rows, int heads, int d, long long stride);

}  // namespace delta_tc
}  // namespace kda
