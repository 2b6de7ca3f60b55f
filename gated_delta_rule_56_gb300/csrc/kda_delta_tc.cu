// kda_delta_tc.cu -- the delta rule with one decay per value head over bf16 prompts, on the sm_103a tensor cores (tcgen05 + TMA + TMEM).
//
// Chunks of C = 64 rows of one (sequence, value head), S the state before the chunk, G_i the sum of the log-decays up to row i:
//     A_ij = b_i exp(G_i - G_j) k_i.k_j (j < i),  P_ij = exp(G_i - G_j) q_i.k_j (j <= i),  T = (I + A)^-1
//     R_i = b_i v_i - b_i exp(G_i) S^T k_i,  U = T R,  o_i = exp(G_i) S^T q_i + sum_j P_ij u_j
//     S <- exp(G_C) S + sum_j k_j (exp(G_C - G_j) u_j)^T
// With one decay per head every decay is a scalar of a row pair: exponents are differences (<= 0) and no product needs a decayed
// operand, so K and Q go into every MMA as they are in memory, exact in bf16.
//
// Everything of the chain is transposed: TMEM lane = value column, so S^T, R^T, U^T are A operands in TMEM, K and Q (and T, P) are B operands
// in shared memory, read K-major or MN-major from the same 128-byte swizzled tile, and all work between two MMAs is within a lane:
//     KS = S^T K^T  ->  R  ->  (T - I) R  ->  U  ->  S^T += U^T K        (o: QS and P U, beside the chain)
//
// Precision. The state is kept in fp32 registers, its final value is an fp32 output, and a bf16 operand has 8 bits. So what is not exact goes in
// as several bf16 values: S and R as two (their rounding, 2^-17, meets products that are smaller than the sums they go into), U with its
// decay as three in the state's update, where its rounding would be the state's. U = R + (T - I) R adds R itself in fp32. T and P as two each.
//
// Roles (16 warps, one block per SM): warps 0-7 the chain (two per lane quarter, half of the columns each), 8 issues the MMAs, 9 the TMA
// loads, 12-15 prepare the next chunk: decays, A and P from the K K^T and Q K^T accumulators (thread = TMEM lane = row), the inverse of I + A by
// 16 x 16 blocks in fp32, T - I and P as operands. Tiles of K and Q have three stages, V, T and P two.
//
// Bound by the chain's latency (three dependent MMA groups and the conversions between them), not by HBM.
#include <cudaTypedefs.h>

#include <mutex>

#include "kda_delta.cuh"
#include "kda_delta_tc.h"
#include "kda_tc.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int C = 64;
constexpr int kThreads = 512;
constexpr uint64_t kWaitNs = 1000000000ull;  // 1 s per wait
constexpr int kPrep = 128;

// TMEM columns
constexpr uint32_t TM_S = 0;      // S^T: first bf16 values in 0..63, second in 64..127; then U with its decay, three times 32
constexpr uint32_t TM_KS = 128;   // KS, then (T - I) R
constexpr uint32_t TM_R = 192;    // R, then U: two times 32
constexpr uint32_t TM_DS = 256;   // QS, then the update of the state
constexpr uint32_t TM_PU = 384;
constexpr uint32_t TM_KK = 448;   // [K; Q] K^T

constexpr int kKqStages = 3, kVStages = 2, kTpStages = 2;
constexpr uint32_t kKqBytes = 32768, kVBytes = 16384, kTpBytes = 32768;

struct Vec {
    float E[C], F[C], b[C], be[C];  // exp(G_i), exp(G_C - G_i), beta_i, beta_i exp(G_i)
    float whole, pad[3];            // exp(G_C)
};

struct Shared {
    uint8_t kq[kKqStages][kKqBytes];  // per 64 key channels: 64 rows of K, 64 rows of Q
    uint8_t v[kVStages][kVBytes];     // per 64 value channels: 64 rows
    uint8_t tp[kTpStages][kTpBytes];  // T - I (two bf16 values), P (two)
    float A[C][C + 4];
    float Y[32][36];
    Vec vec[kTpStages];
    float Gh[C], Gl[C], f[C];
    uint64_t full_kq[kKqStages], free_kq[kKqStages], ready_kq[kKqStages];
    uint64_t full_v[kVStages], free_v[kVStages], ready_v[kVStages];
    uint64_t free_tp[kTpStages], ready_tp[kTpStages];
    uint64_t kk, kk_free, s, ks, qs, r, u, u2, up, ds, pu, drain;
    uint32_t tmem;
};

struct Maps {
    CUtensorMap q, k, v;
};

__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(a, b);
    lo = pack_bf16(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
}
__device__ __forceinline__ void split3(float a, float b, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    hi = pack_bf16(a, b);
    const float c = a - __uint_as_float(hi << 16), d = b - __uint_as_float(hi & 0xffff0000u);
    mid = pack_bf16(c, d);
    lo = pack_bf16(c - __uint_as_float(mid << 16), d - __uint_as_float(mid & 0xffff0000u));
}

__device__ __forceinline__ void prep_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// All prep threads wait, and leave together when a wait runs out.
__device__ __forceinline__ bool prep_wait(uint64_t *bar, uint32_t parity) {
    const uint32_t bad = mbar_wait(bar, parity, kWaitNs) ? 0u : 1u;
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(bad)
        : "memory");
    return any == 0;
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

// ------------------------------------------------------------------------ prep -----------

// x[j] = D_ij x[j] (times b): decays of row i against the rows of its own and earlier blocks of 16; zero behind the diagonal.
__device__ __forceinline__ void decay_row(float (&x)[C], const Shared &s, int i, bool q_row, float Gh, float Gl, float scale) {
    const int bi = i >> 4;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        if (b < bi) {  // through the block's last row: both exponents are differences, at most 0
            const float e = scale * expf(__fadd_rn(__fsub_rn(Gh, s.Gh[16 * b + 15]), __fsub_rn(Gl, s.Gl[16 * b + 15])));
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(&s.f[16 * b + j]);
                x[16 * b + j] *= e * f.x;
                x[16 * b + j + 1] *= e * f.y;
                x[16 * b + j + 2] *= e * f.z;
                x[16 * b + j + 3] *= e * f.w;
            }
        } else if (b == bi) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int at = 16 * b + j;
                const float D = expf(__fadd_rn(__fsub_rn(Gh, s.Gh[at]), __fsub_rn(Gl, s.Gl[at])));
                x[at] = at < i || (q_row && at == i) ? scale * D * x[at] : 0.f;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) x[16 * b + j] = 0.f;
        }
    }
}

// (I + A)^-1 in place of A (strictly lower, zeros above), 128 threads: 16 x 16 blocks by substitution, then joined twice.
__device__ __forceinline__ void invert(Shared &s, int pt) {
    const int w = pt >> 5, lane = pt & 31;
    {
        const int j = lane & 15, o = 16 * w;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float a = i == j ? 1.f : 0.f;
#pragma unroll
            for (int m = 0; m < i; ++m) a = fmaf(-s.A[o + i][o + m], x[m], a);
            x[i] = a;
        }
        __syncwarp();
        if (lane < 16)
#pragma unroll
            for (int i = 0; i < 16; ++i) s.A[o + i][o + j] = x[i];
    }
    prep_sync();
    {
        const int o = 32 * (pt >> 6), t = pt & 63, r = t >> 2, c = (t & 3) * 4;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float a = s.A[o + 16 + r][o + j];
            const float4 x = *reinterpret_cast<const float4 *>(&s.A[o + j][o + c]);
            y = make_float4(fmaf(a, x.x, y.x), fmaf(a, x.y, y.y), fmaf(a, x.z, y.z), fmaf(a, x.w, y.w));
        }
        *reinterpret_cast<float4 *>(&s.Y[(o >> 1) + r][c]) = y;
        prep_sync();
        y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float a = -s.A[o + 16 + r][o + 16 + j];
            const float4 x = *reinterpret_cast<const float4 *>(&s.Y[(o >> 1) + j][c]);
            y = make_float4(fmaf(a, x.x, y.x), fmaf(a, x.y, y.y), fmaf(a, x.z, y.z), fmaf(a, x.w, y.w));
        }
        *reinterpret_cast<float4 *>(&s.A[o + 16 + r][o + c]) = y;
    }
    prep_sync();
    {
        const int r = pt >> 2, c = (pt & 3) * 8;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = 0.f;
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(half ? &s.A[32 + r][32 + j] : &s.A[32 + r][j]);
                const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float *line = half ? &s.Y[j + m][c] : &s.A[j + m][c];
                    const float4 lo = *reinterpret_cast<const float4 *>(line), hi = *reinterpret_cast<const float4 *>(line + 4);
                    y[0] = fmaf(av[m], lo.x, y[0]);
                    y[1] = fmaf(av[m], lo.y, y[1]);
                    y[2] = fmaf(av[m], lo.z, y[2]);
                    y[3] = fmaf(av[m], lo.w, y[3]);
                    y[4] = fmaf(av[m], hi.x, y[4]);
                    y[5] = fmaf(av[m], hi.y, y[5]);
                    y[6] = fmaf(av[m], hi.z, y[6]);
                    y[7] = fmaf(av[m], hi.w, y[7]);
                }
            }
            float *to = half ? &s.A[32 + r][c] : &s.Y[r][c];
            const float sign = half ? -1.f : 1.f;
            *reinterpret_cast<float4 *>(to) = make_float4(sign * y[0], sign * y[1], sign * y[2], sign * y[3]);
            *reinterpret_cast<float4 *>(to + 4) = make_float4(sign * y[4], sign * y[5], sign * y[6], sign * y[7]);
            prep_sync();
        }
    }
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

template <int DK>
__device__ __forceinline__ bool prep(Shared &s, const DeltaParams &p, int h, long long begin, long long end, int chunks, uint32_t tmem) {
    const int pt = threadIdx.x - (kThreads - kPrep), lane = pt & 31, w = pt >> 5;
    const int i = pt & 63;  // this thread's row
    const bool q_row = pt >= 64;
    const uint32_t tq = (uint32_t)(32 * w) << 16;
    const int vtiles = p.dv > 64 ? 2 : 1;
    for (int c = 0; c < chunks; ++c) {
        const int ks = c % kKqStages, vs = c % kVStages, ts = c % kTpStages;
        const long long row0 = begin + (long long)c * C;
        const int m = (int)min((long long)C, end - row0);
        // Both halves of the rows, for the sums.
        float g0 = lane < m ? log_decay(p.g[(row0 + lane) * p.hv + h]) : 0.f;
        float g1 = lane + 32 < m ? log_decay(p.g[(row0 + lane + 32) * p.hv + h]) : 0.f;
        const float beta = i < m ? p.beta[(row0 + i) * p.hv + h] : 0.f;
        if (!prep_wait(&s.full_kq[ks], (uint32_t)(c / kKqStages) & 1u) || !prep_wait(&s.full_v[vs], (uint32_t)(c / kVStages) & 1u)) return false;
        if (m < C) {  // the rows behind the sequence are another one's: zeros, so that nothing of theirs meets a product
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            for (int e = pt; e < (C - m) * 8; e += kPrep) {
                const uint32_t at = (uint32_t)m * 128u + (uint32_t)e * 16u;
#pragma unroll
                for (int a = 0; a < DK / 32; ++a) *reinterpret_cast<uint4 *>(&s.kq[ks][a * 8192 + at]) = zero;
                for (int a = 0; a < vtiles; ++a) *reinterpret_cast<uint4 *>(&s.v[vs][a * 8192 + at]) = zero;
            }
            fence_async_smem();
        }
        warp_arrive(&s.ready_kq[ks]);
        warp_arrive(&s.ready_v[vs]);
        if (c >= kTpStages && !prep_wait(&s.free_tp[ts], (uint32_t)(c / kTpStages - 1) & 1u)) return false;
        // Sums of up to 64 decays in two fp32 values, so that differences of neighbours behind strong decays stay exact (the error of a
        // two-term sum, by D. E. Knuth's branch-free formula).
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const float x0 = __shfl_up_sync(0xffffffffu, g0, d), y0 = __shfl_up_sync(0xffffffffu, l0, d);
            const float x1 = __shfl_up_sync(0xffffffffu, g1, d), y1 = __shfl_up_sync(0xffffffffu, l1, d);
            if (lane >= d) {
                float t = __fadd_rn(g0, x0), z = __fsub_rn(t, g0);
                l0 = __fadd_rn(__fadd_rn(l0, y0), __fadd_rn(__fsub_rn(g0, __fsub_rn(t, z)), __fsub_rn(x0, z)));
                g0 = t;
                t = __fadd_rn(g1, x1), z = __fsub_rn(t, g1);
                l1 = __fadd_rn(__fadd_rn(l1, y1), __fadd_rn(__fsub_rn(g1, __fsub_rn(t, z)), __fsub_rn(x1, z)));
                g1 = t;
            }
        }
        {
            const float x = __shfl_sync(0xffffffffu, g0, 31), y = __shfl_sync(0xffffffffu, l0, 31);
            const float t = __fadd_rn(g1, x), z = __fsub_rn(t, g1);
            l1 = __fadd_rn(__fadd_rn(l1, y), __fadd_rn(__fsub_rn(g1, __fsub_rn(t, z)), __fsub_rn(x, z)));
            g1 = t;
        }
        const float Gc = __shfl_sync(0xffffffffu, g1, 31), Lc = __shfl_sync(0xffffffffu, l1, 31);
        const float Gh = w & 1 ? g1 : g0, Gl = w & 1 ? l1 : l0;  // of row i
        {
            const float eh = __shfl_sync(0xffffffffu, Gh, lane | 15), el = __shfl_sync(0xffffffffu, Gl, lane | 15);
            if (!q_row) {
                Vec &v = s.vec[ts];
                const float E = expf(__fadd_rn(Gh, Gl));
                s.Gh[i] = Gh;
                s.Gl[i] = Gl;
                s.f[i] = expf(__fadd_rn(__fsub_rn(eh, Gh), __fsub_rn(el, Gl)));
                v.E[i] = E;
                v.F[i] = expf(__fadd_rn(__fsub_rn(Gc, Gh), __fsub_rn(Lc, Gl)));
                v.b[i] = beta;
                v.be[i] = beta * E;
                if (i == 0) v.whole = expf(__fadd_rn(Gc, Lc));
            }
        }
        if (!prep_wait(&s.kk, (uint32_t)c & 1u)) return false;  // also: the sums are in shared memory
        tc_fence_after();
        float x[C];
        {
            float a[32], b[32];
            tmem_ld32(tmem + tq + TM_KK, a);
            tmem_ld32(tmem + tq + TM_KK + 32, b);
            tmem_ld_wait();
            tc_fence_before();
            warp_arrive(&s.kk_free);
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = a[e], x[32 + e] = b[e];
        }
        decay_row(x, s, i, q_row, Gh, Gl, q_row ? 1.f : beta);
        uint8_t *tp = s.tp[ts];
        if (q_row) {
#pragma unroll
            for (int e = 0; e < 8; ++e) store_operand(tp + 16384, tp + 24576, i, e, &x[8 * e]);
        } else {
#pragma unroll
            for (int e = 0; e < C; e += 4) *reinterpret_cast<float4 *>(&s.A[i][e]) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        }
        prep_sync();
        invert(s, pt);
        {
            const int r = pt >> 1, c0 = (pt & 1) * 32;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    const int at = c0 + 8 * e + j;
                    const float4 t = *reinterpret_cast<const float4 *>(&s.A[r][at]);
                    y[j] = at < r ? t.x : 0.f;
                    y[j + 1] = at + 1 < r ? t.y : 0.f;
                    y[j + 2] = at + 2 < r ? t.z : 0.f;
                    y[j + 3] = at + 3 < r ? t.w : 0.f;
                }
                store_operand(tp, tp + 8192, r, c0 / 8 + e, y);
            }
        }
        fence_async_smem();
        warp_arrive(&s.ready_tp[ts]);
        prep_sync();  // A is read out before the next chunk's
    }
    return true;
}

// ------------------------------------------------------------------------ issuer ---------

template <int DK>
__device__ __forceinline__ bool issue(Shared &s, int chunks) {
    const uint32_t tmem = __shfl_sync(0xffffffffu, s.tmem, 0);
    const uint32_t kq = smem_u32(s.kq[0]), tp = smem_u32(s.tp[0]);
    auto gram = [&](int c) -> bool {  // [K; Q] K^T
        const int ks = c % kKqStages;
        if (!warp_wait(&s.ready_kq[ks], (uint32_t)(c / kKqStages) & 1u)) return false;
        if (c > 0 && !warp_wait(&s.kk_free, (uint32_t)(c - 1) & 1u)) return false;
        tc_fence_after();
        const uint64_t d = sdesc_sw128(kq + ks * kKqBytes, 16u, 1024u);
#pragma unroll
        for (int st = 0; st < DK / 16; ++st)
            mma_bf16_warp(tmem + TM_KK, d + kstep(st, 16384u), d + kstep(st, 16384u), idesc_bf16(128, 64), st > 0);
        mma_commit_warp(&s.kk);
        return true;
    };
    if (chunks > 0 && !gram(0)) return false;
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
        const uint32_t par = (uint32_t)c & 1u;
        const uint32_t kqc = kq + (uint32_t)(c % kKqStages) * kKqBytes, tpc = tp + (uint32_t)(c % kTpStages) * kTpBytes;
        const uint64_t d_k = sdesc_sw128(kqc, 16u, 1024u), d_q = sdesc_sw128(kqc + 8192u, 16u, 1024u);
        const uint64_t d_kn = sdesc_sw128(kqc, 16384u, 1024u);  // MN-major: the two tiles of 64 channels lie 16384 bytes apart
        if (!warp_wait(&s.s, par)) return false;
        tc_fence_after();
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int st = 0; st < DK / 16; ++st)
                mma_bf16_tmem_a_warp(tmem + TM_KS, tmem + TM_S + 64 * e + 8 * st, d_k + kstep(st, 16384u), idesc_bf16(128, 64), e + st > 0);
        mma_commit_warp(&s.ks);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int st = 0; st < DK / 16; ++st)
                mma_bf16_tmem_a_warp(tmem + TM_DS, tmem + TM_S + 64 * e + 8 * st, d_q + kstep(st, 16384u), idesc_bf16(128, 64), e + st > 0);
        mma_commit_warp(&s.qs);
        if (c + 1 < chunks && !gram(c + 1)) return false;
        if (!warp_wait(&s.ready_tp[c % kTpStages], (uint32_t)(c / kTpStages) & 1u) || !warp_wait(&s.r, par)) return false;
        tc_fence_after();
        const uint64_t d_t = sdesc_sw128(tpc, 16u, 1024u), d_p = sdesc_sw128(tpc + 16384u, 16u, 1024u);
#pragma unroll
        for (int e = 0; e < 3; ++e)  // first x first, first x second, second x first
#pragma unroll
            for (int st = 0; st < C / 16; ++st)
                mma_bf16_tmem_a_warp(tmem + TM_KS, tmem + TM_R + (e == 2 ? 32 : 0) + 8 * st, d_t + (e == 1 ? 512u : 0u) + kstep(st, 0u),
                                     idesc_bf16(128, 64), e + st > 0);
        mma_commit_warp(&s.u);
        if (!warp_wait(&s.u2, par)) return false;
        tc_fence_after();
#pragma unroll
        for (int e = 0; e < 3; ++e)
#pragma unroll
            for (int st = 0; st < C / 16; ++st)
                mma_bf16_tmem_a_warp(tmem + TM_DS, tmem + TM_S + 32 * e + 8 * st, d_kn + kDescStepMN128 * st,
                                     idesc_bf16(128, DK) | kIdescBMajorMN, e + st > 0);
        mma_commit_warp(&s.ds);
        if (!warp_wait(&s.up, par)) return false;
        tc_fence_after();
#pragma unroll
        for (int e = 0; e < 3; ++e)
#pragma unroll
            for (int st = 0; st < C / 16; ++st)
                mma_bf16_tmem_a_warp(tmem + TM_PU, tmem + TM_R + (e == 2 ? 32 : 0) + 8 * st, d_p + (e == 1 ? 512u : 0u) + kstep(st, 0u),
                                     idesc_bf16(128, 64), e + st > 0);
        mma_commit_warp(&s.pu);
        mma_commit_warp(&s.free_tp[c % kTpStages]);
        mma_commit_warp(&s.free_kq[c % kKqStages]);
    }
    return true;
}

// ------------------------------------------------------------------------ loads ----------

template <int DK>
__device__ __forceinline__ bool load(Shared &s, const Maps &maps, const DeltaParams &p, int h, long long begin, int chunks) {
    const int hk = h / p.per, vtiles = p.dv > 64 ? 2 : 1;
    int c = 0;
    bool ok = true;
    for (; c < chunks; ++c) {
        const int ks = c % kKqStages, vs = c % kVStages, row = (int)(begin + (long long)c * C);
        if (c >= kKqStages && !(ok = warp_wait(&s.free_kq[ks], (uint32_t)(c / kKqStages - 1) & 1u))) break;
        if (elect_one()) {
            mbar_arrive_expect_tx(&s.full_kq[ks], DK / 64 * 16384);
            for (int a = 0; a < DK / 64; ++a) {
                tma_load_3d(s.kq[ks] + a * 16384, &maps.k, &s.full_kq[ks], 64 * a, hk, row);
                tma_load_3d(s.kq[ks] + a * 16384 + 8192, &maps.q, &s.full_kq[ks], 64 * a, hk, row);
            }
        }
        __syncwarp();
        if (c >= kVStages && !(ok = warp_wait(&s.free_v[vs], (uint32_t)(c / kVStages - 1) & 1u))) {
            ++c;
            break;
        }
        if (elect_one()) {
            mbar_arrive_expect_tx(&s.full_v[vs], vtiles * 8192);
            for (int a = 0; a < vtiles; ++a) tma_load_3d(s.v[vs] + a * 8192, &maps.v, &s.full_v[vs], 64 * a, h, row);
        }
        __syncwarp();
    }
    if (!ok)  // the latest copies of every stage, before the block's shared memory goes
        for (int b = c > kKqStages ? c - kKqStages : 0; b < c; ++b) {
            (void)mbar_wait(&s.full_kq[b % kKqStages], (uint32_t)(b / kKqStages) & 1u, kWaitNs);
            if (b + kVStages >= c) (void)mbar_wait(&s.full_v[b % kVStages], (uint32_t)(b / kVStages) & 1u, kWaitNs / 10);
        }
    return ok;
}

// ------------------------------------------------------------------------ chain ----------

template <int DK>
__device__ __forceinline__ void publish_state(const float (&S)[DK / 2], uint32_t at) {
#pragma unroll
    for (int g = 0; g < DK / 64; ++g) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) split2(S[32 * g + 2 * e], S[32 * g + 2 * e + 1], hi[e], lo[e]);
        tmem_st16(at + 16 * g, hi);
        tmem_st16(at + 64 + 16 * g, lo);
    }
    tmem_st_wait();
    tc_fence_before();
}

template <int DK>
__device__ __forceinline__ bool chain(Shared &s, const DeltaParams &p, int n, int h, long long begin, long long end, int chunks, uint32_t tmem) {
    constexpr int H = DK / 2;  // key channels of a thread
    const int wg = threadIdx.x >> 7, col = threadIdx.x & 127;  // half, value column
    const uint32_t at = tmem + ((uint32_t)(col & 96) << 16);
    const bool live = col < p.dv;
    const size_t one = (size_t)p.hv * p.dk * p.dv, in = (size_t)h * p.dk * p.dv + (size_t)wg * H * p.dv + col;
    const int keys = min(max(p.dk - wg * H, 0), H);  // of this half that the state has
    const long long from = p.init ? state_slot(p.init_idx, p.pool, n, p.err) : -1;
    float S[H];
#pragma unroll
    for (int e = 0; e < H; ++e) S[e] = from >= 0 && live && e < keys ? p.init[from * one + in + (size_t)e * p.dv] : 0.f;
    // This column's place in a row of a V tile: 16-byte piece ^ (row % 8).
    const uint32_t v_in = (uint32_t)(col >> 6) * 8192u + (uint32_t)(col & 7) * 2u, piece = (uint32_t)(col & 63) >> 3;
    const bool loaded = col < (p.dv > 64 ? 128 : 64);
    if (chunks > 0) {
        publish_state<DK>(S, at + TM_S + wg * (H / 2));
        warp_arrive(&s.s);
    }
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.o) + (begin * p.hv + h) * p.dv + col;
    const long long o_row = (long long)p.hv * p.dv;
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
        const uint32_t par = (uint32_t)c & 1u;
        const int vs = c % kVStages, t0 = 32 * wg;
        const Vec &vec = s.vec[c % kTpStages];
        float R[32], acc[32];
        // R = b v - b E KS
        if (!warp_wait(&s.ready_v[vs], (uint32_t)(c / kVStages) & 1u) ||
            !warp_wait(&s.ready_tp[c % kTpStages], (uint32_t)(c / kTpStages) & 1u))
            return false;
        const uint8_t *v = s.v[vs] + v_in + (size_t)t0 * 128;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            const uint32_t x = loaded ? *reinterpret_cast<const uint16_t *>(v + e * 128 + ((piece ^ (uint32_t)(e & 7)) << 4)) : 0u;
            R[e] = vec.b[t0 + e] * __uint_as_float(x << 16);
        }
        warp_arrive(&s.free_v[vs]);
        if (!warp_wait(&s.ks, par)) return false;
        tc_fence_after();
        tmem_ld32(at + TM_KS + t0, acc);
        tmem_ld_wait();
        {
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                R[e] = fmaf(-vec.be[t0 + e], acc[e], R[e]);
                R[e + 1] = fmaf(-vec.be[t0 + e + 1], acc[e + 1], R[e + 1]);
                split2(R[e], R[e + 1], hi[e / 2], lo[e / 2]);
            }
            tmem_st16(at + TM_R + 16 * wg, hi);
            tmem_st16(at + TM_R + 32 + 16 * wg, lo);
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&s.r);
        }
        // Beside (T - I) R: the reading of the state
        if (!warp_wait(&s.qs, par)) return false;
        tc_fence_after();
        tmem_ld32(at + TM_DS + t0, acc);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e) acc[e] *= vec.E[t0 + e];
        if (!warp_wait(&s.u, par)) return false;
        tc_fence_after();
        {
            float x[32];
            tmem_ld32(at + TM_KS + t0, x);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) R[e] += x[e];  // U
            uint32_t hi[16], mid[16], lo[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2)
                split3(vec.F[t0 + e] * R[e], vec.F[t0 + e + 1] * R[e + 1], hi[e / 2], mid[e / 2], lo[e / 2]);
            tmem_st16(at + TM_S + 16 * wg, hi);
            tmem_st16(at + TM_S + 32 + 16 * wg, mid);
            tmem_st16(at + TM_S + 64 + 16 * wg, lo);
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&s.u2);
#pragma unroll
            for (int e = 0; e < 32; e += 2) split2(R[e], R[e + 1], hi[e / 2], lo[e / 2]);
            tmem_st16(at + TM_R + 16 * wg, hi);
            tmem_st16(at + TM_R + 32 + 16 * wg, lo);
        }
        const float whole = vec.whole;
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&s.up);
        if (!warp_wait(&s.ds, par)) return false;
        tc_fence_after();
#pragma unroll
        for (int g = 0; g < H / 32; ++g) {
            float x[32];
            tmem_ld32(at + TM_DS + wg * H + 32 * g, x);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) S[32 * g + e] = fmaf(whole, S[32 * g + e], x[e]);
        }
        if (c + 1 < chunks) {
            publish_state<DK>(S, at + TM_S + wg * (H / 2));
            warp_arrive(&s.s);
        }
        // Beside the next chunk's KS: the outputs
        if (!warp_wait(&s.pu, par)) return false;
        tc_fence_after();
        {
            float x[32];
            tmem_ld32(at + TM_PU + t0, x);
            tmem_ld_wait();
            const int m = (int)min((long long)32, end - (begin + (long long)c * C + t0));
            __nv_bfloat16 *to = o + ((long long)c * C + t0) * o_row;
            if (live) {
                if (m == 32) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) to[e * o_row] = __float2bfloat16_rn(acc[e] + x[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (e < m) to[e * o_row] = __float2bfloat16_rn(acc[e] + x[e]);
                }
            }
        }
    }
    const long long to = p.fin ? state_slot(p.fin_idx, p.pool, n, p.err) : -1;
    if (to >= 0 && live)
#pragma unroll
        for (int e = 0; e < H; ++e)
            if (e < keys) p.fin[to * one + in + (size_t)e * p.dv] = S[e];
    return true;
}

template <int DK>
__global__ void __launch_bounds__(kThreads, 1) delta_tc_kernel(const __grid_constant__ Maps maps, const __grid_constant__ DeltaParams p) {
    extern __shared__ uint8_t raw[];
    Shared &s = *reinterpret_cast<Shared *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5;
    const int h = blockIdx.x % p.hv, n = blockIdx.x / p.hv;
    long long begin, end;
    if (!rows_of(p, n, begin, end)) return;
    const int chunks = (int)((end - begin + C - 1) / C);
    if (warp == 0) {
        tmem_alloc(&s.tmem, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < kKqStages; ++i) {
            mbar_init(&s.full_kq[i], 1);
            mbar_init(&s.free_kq[i], 1);
            mbar_init(&s.ready_kq[i], 4);
        }
        for (int i = 0; i < kVStages; ++i) {
            mbar_init(&s.full_v[i], 1);
            mbar_init(&s.free_v[i], 8);
            mbar_init(&s.ready_v[i], 4);
        }
        for (int i = 0; i < kTpStages; ++i) {
            mbar_init(&s.free_tp[i], 1);
            mbar_init(&s.ready_tp[i], 4);
        }
        mbar_init(&s.kk_free, 4);
        for (uint64_t *b : {&s.s, &s.r, &s.u2, &s.up}) mbar_init(b, 8);
        for (uint64_t *b : {&s.kk, &s.ks, &s.qs, &s.u, &s.ds, &s.pu, &s.drain}) mbar_init(b, 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 64) {
        prefetch_tensormap(&maps.q);
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    bool ok = true;
    // 2 x 128 x 176 + 128 x 40 + 128 x 120 = 512 x 128 registers, what the block was launched with.
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        ok = chain<DK>(s, p, n, h, begin, end, chunks, tmem);
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 8) {
            ok = issue<DK>(s, chunks);
            if (!ok) {  // nothing may be in flight at the end
                mma_commit_warp(&s.drain);
                (void)mbar_wait(&s.drain, 0, kWaitNs);
            }
            __syncwarp();
        } else if (warp == 9) {
            ok = load<DK>(s, maps, p, h, begin, chunks);
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
        ok = prep<DK>(s, p, h, begin, end, chunks, tmem);
    }
    if (!ok) atomicOr(p.err, kErrTimeout);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// Rows of `heads` heads of d channels, `stride` elements apart, in boxes of 64 rows x 64 channels (128-byte swizzle); what lies past the
// channels and the rows reads as zeros.
bool encode(CUtensorMap *map, const void *base, long long rows, int heads, int d, long long stride) {
    auto enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)C}, es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kSharedBytes = sizeof(Shared) + 1024;

template <int DK>
cudaError_t launch(const Maps &maps, const DeltaParams &p, cudaStream_t s) {
    auto *f = &delta_tc_kernel<DK>;
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSharedBytes);
    if (e != cudaSuccess) return e;
    f<<<(unsigned)((long long)p.seqs.n_seqs * p.hv), kThreads, kSharedBytes, s>>>(maps, p);
    return cudaGetLastError();
}

}  // namespace

bool delta_tc_supported(kda_dtype dtype, const DeltaParams &p) {
    auto ok = [](const void *x, long long stride) { return aligned16(x) && stride % 8 == 0; };
    return dtype == KDA_BF16 && p.seqs.rows > 0 && ok(p.q, p.qs) && ok(p.k, p.ks) && ok(p.v, p.vs) && encoder();
}

cudaError_t launch_delta_tc(const DeltaParams &p, cudaStream_t s) {
    Maps maps;
    if (!encode(&maps.q, p.q, p.seqs.rows, p.hk, p.dk, p.qs) || !encode(&maps.k, p.k, p.seqs.rows, p.hk, p.dk, p.ks) ||
        !encode(&maps.v, p.v, p.seqs.rows, p.hv, p.dv, p.vs))
        return cudaErrorInvalidValue;
    return p.dk == 128 ? launch<128>(maps, p, s) : launch<64>(maps, p, s);
}

}  // namespace kda
