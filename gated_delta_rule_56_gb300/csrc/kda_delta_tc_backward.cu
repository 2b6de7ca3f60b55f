// kda_delta_tc_backward.cu -- gradients of the delta rule with one decay per value head on the sm_103a tensor cores (bf16 inputs).
//
// The formulas are those of kda_delta_backward.cu, on chunks of 64 rows, in three launches:
//   1. the forward kernel (kda_delta_tc.cu) without its outputs: it keeps, per chunk, the state S0 before it, the values U, and T - I and P as
//      the operands that they are;
//   2. the chain of the state's gradient, chunks from the last to the first. One block per (sequence, value head), all transposed
//      (TMEM lane = value column) as in the forward chain, the same three dependent MMA groups per chunk:
//          dS^T K^T -> dU^T = F (dS^T K^T) + dO^T P -> dR^T = dU^T + dU^T (T - I) -> dS^T <- e^{G_C} dS^T + (E dO)^T Q - (b E dR)^T K
//      T - I, P, K and Q are the operands of the forward pass read with the other index as the long one. It keeps dS and dR per chunk;
//   3. everything else, which needs no other chunk: one block per (chunk, value head), [dO; dR] as the 128 rows of the accumulators:
//          [dO; dR] U^T -> Gp, Ga;   [dO; dR] S0^T, scaled by +-E, + [Gp; Ga] K = [dq; row];   F (U dS^T) + Gp^T Q + (b Ga)^T K = col.
//      dg is made of the pairs' products with [Q; K] K^T and of the parts of dq, row and col that come from the states.
// Where value heads share key heads, dq and dk go per value head to the workspace and are added up in a fixed order.
//
// Operands that are not exact in bf16 go in as two values (2^-18 of them is left, the products of both rests are left out), T - I and those that
// are added to the gradient of the state as three; sums, states and outputs are fp32.
//
// Gradients are 2e-6 to 6e-6 off 64 bits in the 2-norm (the plain fp32 form 0.3e-6).
//
// Measured at 2 x 2048 rows, 32 value heads, 16 key heads of 128 (642 us in all): the kept forward pass 215 us, the chain 160, the chunks 229, the sums
// over shared heads 29; with 4 x 2048 rows 227, 162, 442 and 58. The chains are bound by latency, as the forward one (9 000 cycles per chunk, a
// quarter of them the stores of dS, which the chain's warps make themselves); the third kernel by its phases, which load (280 KB per
// chunk and head: S0, dS, U, dR), compute and store one after the other with one block per SM: 3.5 TB/s, 27 % of the issue slots. L2 prefetches for a
// later block made it slower (480 for 440), bulk copies of single rows out of shared memory too (550); 32 lanes that write to 32 rows took 470.
#include <cstddef>

#include "kda_delta_tc.cuh"

namespace kda {
namespace {

using namespace delta_tc;

// ------------------------------------------------------------------ the chain backward ---

constexpr int kChainWarps = 16, kIssuer = 16, kLoader = 17, kDecays = 18;
constexpr int kThreads = 20 * 32;
constexpr int kStages = 2, kVecs = 3;

// TMEM columns
constexpr uint32_t TM_D = 0;      // dS^T: first bf16 values in 0..63, second in 64..127; then b E dR, three times 32
constexpr uint32_t TM_KD = 128;   // dS^T K^T, then dU^T (T - I)
constexpr uint32_t TM_U = 192;    // dU: two times 32
constexpr uint32_t TM_DF = 256;   // dS^T in fp32
constexpr uint32_t TM_O = 384;    // dO^T (exact), 32; then E dO, three times 32
constexpr uint32_t TM_PD = 416;   // dO^T P

struct ChainShared {
    uint8_t kq[kStages][32768];  // as in the forward kernel: per 64 key channels, 64 rows of K, 64 rows of Q
    uint8_t d_o[kStages][16384];
    uint8_t tp[kStages][kDeltaTpBytes];
    Vec vec[kVecs];
    uint64_t full[kStages], free[kStages], ready;
    uint64_t ready_vec[kVecs], free_vec[kVecs];
    uint64_t s, o, pd, pd_read, kd, r, u, h, u2, ds, drain;
    uint32_t tmem;
};

struct ChainMaps {
    CUtensorMap q, k, d_o;
};
struct ChainParams {
    DeltaParams f;
    const uint8_t *tp;
    const float *d_fin;
    float *dS, *dR, *d_init;  // dS: of the state behind a chunk [chunk, value head, dk, dv]; dR [chunk, value head, 64, dv]
};

template <int DK>
__device__ __forceinline__ bool chain_issue(ChainShared &s, int chunks) {
    const uint32_t tmem = __shfl_sync(0xffffffffu, s.tmem, 0);
#pragma unroll 1
    for (int k = 0; k < chunks; ++k) {
        const uint32_t par = (uint32_t)k & 1u;
        const int st = k % kStages;
        const uint32_t kq = smem_u32(s.kq[st]), tp = smem_u32(s.tp[st]);
        const uint64_t d_k = sdesc_sw128(kq, 16u, 1024u), d_kn = sdesc_sw128(kq, 16384u, 1024u), d_qn = sdesc_sw128(kq + 8192u, 16384u, 1024u);
        const uint64_t d_t = sdesc_sw128(tp, 8192u, 1024u), d_p = sdesc_sw128(tp + kDeltaP, 8192u, 1024u);  // MN-major: the column is the N index
        // The last chunk's rows behind the sequence are cleared first; the others are there as soon as they are loaded.
        if (!warp_wait(k == 0 ? &s.ready : &s.full[st], (uint32_t)(k / kStages) & 1u) || !warp_wait(&s.s, par)) return false;
        tc_fence_after();
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < DK / 16; ++i)
                mma_bf16_tmem_a_warp(tmem + TM_KD, tmem + TM_D + 64 * e + 8 * i, d_k + kstep(i, 16384u), idesc_bf16(128, 64), e + i > 0);
        mma_commit_warp(&s.kd);
        if (!warp_wait(&s.o, par)) return false;
        tc_fence_after();
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < C / 16; ++i)
                mma_bf16_tmem_a_warp(tmem + TM_PD, tmem + TM_O + 8 * i, d_p + 512u * e + kDescStepMN128 * i, idesc_bf16(128, 64) | kIdescBMajorMN,
                                     e + i > 0);
        mma_commit_warp(&s.pd);
        if (!warp_wait(&s.r, par)) return false;
        tc_fence_after();
#pragma unroll
        for (int e = 0; e < 5; ++e)  // dU's first value by T's first, second and third, dU's second by T's first and second
#pragma unroll
            for (int i = 0; i < C / 16; ++i)
                mma_bf16_tmem_a_warp(tmem + TM_KD, tmem + TM_U + (e > 2 ? 32 : 0) + 8 * i, d_t + 512u * (e > 2 ? e - 3 : e) + kDescStepMN128 * i,
                                     idesc_bf16(128, 64) | kIdescBMajorMN, e + i > 0);
        mma_commit_warp(&s.u);
        if (!warp_wait(&s.h, par)) return false;
        tc_fence_after();
#pragma unroll
        for (int e = 0; e < 3; ++e)
#pragma unroll
            for (int i = 0; i < C / 16; ++i)
                mma_bf16_tmem_a_warp(tmem + TM_DF, tmem + TM_O + 32 * e + 8 * i, d_qn + kDescStepMN128 * i, idesc_bf16(128, DK) | kIdescBMajorMN, 1u);
        if (!warp_wait(&s.u2, par)) return false;
        tc_fence_after();
#pragma unroll
        for (int e = 0; e < 3; ++e)
#pragma unroll
            for (int i = 0; i < C / 16; ++i)
                mma_bf16_tmem_a_warp(tmem + TM_DF, tmem + TM_D + 32 * e + 8 * i, d_kn + kDescStepMN128 * i, idesc_bf16(128, DK) | kIdescBMajorMN, 1u);
        mma_commit_warp(&s.ds);
        mma_commit_warp(&s.free[st]);
        mma_commit_warp(&s.free_vec[k % kVecs]);
    }
    return true;
}

template <int DK>
__device__ __forceinline__ bool chain_load(ChainShared &s, const ChainMaps &maps, const ChainParams &p, int n, int h, long long begin, int chunks) {
    const int hk = h / p.f.per, vtiles = p.f.dv > 64 ? 2 : 1;
    int k = 0;
    bool ok = true;
    for (; k < chunks; ++k) {
        const int st = k % kStages, c = chunks - 1 - k, row = (int)(begin + (long long)c * C);
        if (k >= kStages && !(ok = warp_wait(&s.free[st], (uint32_t)(k / kStages - 1) & 1u))) break;
        if (elect_one()) {
            mbar_arrive_expect_tx(&s.full[st], DK / 64 * 16384 + vtiles * 8192 + kDeltaTpBytes);
            for (int a = 0; a < DK / 64; ++a) {
                tma_load_3d(s.kq[st] + a * 16384, &maps.k, &s.full[st], 64 * a, hk, row);
                tma_load_3d(s.kq[st] + a * 16384 + 8192, &maps.q, &s.full[st], 64 * a, hk, row);
            }
            for (int a = 0; a < vtiles; ++a) tma_load_3d(s.d_o[st] + a * 8192, &maps.d_o, &s.full[st], 64 * a, h, row);
            bulk_load(s.tp[st], p.tp + ((size_t)(first_chunk(begin, n, C) + c) * p.f.hv + h) * kDeltaTpBytes, kDeltaTpBytes, &s.full[st]);
        }
        __syncwarp();
    }
    if (!ok)  // the copies in flight, before the block's shared memory goes
        for (int b = k > kStages ? k - kStages : 0; b < k; ++b) (void)mbar_wait(&s.full[b % kStages], (uint32_t)(b / kStages) & 1u, kWaitNs);
    return ok;
}

__device__ __forceinline__ bool chain_decays(ChainShared &s, const ChainParams &p, int h, long long begin, long long end, int chunks) {
    const int lane = threadIdx.x & 31;
    for (int k = 0; k < chunks; ++k) {
        const long long row = begin + (long long)(chunks - 1 - k) * C + lane;
        float own[2], b[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const long long r = row + 32 * half;
            own[half] = r < end ? log_decay(p.f.g[r * p.f.hv + h]) : 0.f;
            b[half] = r < end ? p.f.beta[r * p.f.hv + h] : 0.f;
        }
        const bool ok = chunk_decays(s.vec[k % kVecs], nullptr, nullptr, nullptr, lane, own, b, [&] {
            return k < kVecs || warp_wait(&s.free_vec[k % kVecs], (uint32_t)(k / kVecs - 1) & 1u);
        });
        if (!ok) return false;
        warp_arrive(&s.ready_vec[k % kVecs]);
    }
    return true;
}

template <int DK>
__device__ __forceinline__ bool chain(ChainShared &s, const ChainParams &p, int n, int h, long long begin, long long end, int chunks, uint32_t tmem) {
    constexpr int H = DK / 4;  // key channels of a thread
    const int part = threadIdx.x >> 7, col = threadIdx.x & 127;  // quarter of the rows and of the key channels; value column
    const int t0 = 16 * part, dk = p.f.dk, dv = p.f.dv;
    const uint32_t at = tmem + ((uint32_t)(col & 96) << 16);
    const bool live = col < dv;
    const size_t one = (size_t)p.f.hv * dk * dv, in = (size_t)h * dk * dv + (size_t)part * H * dv + col;
    const int keys = min(max(dk - part * H, 0), H);
    const uint32_t o_in = (uint32_t)(col >> 6) * 8192u + (uint32_t)(col & 7) * 2u + (uint32_t)t0 * 128u, piece = (uint32_t)(col & 63) >> 3;
    const long long chunk0 = first_chunk(begin, n, C);
    auto scaled = [&](const float (&S)[H], int k) -> bool {
        if (!warp_wait(&s.ready_vec[k % kVecs], (uint32_t)(k / kVecs) & 1u)) return false;
        const float whole = s.vec[k % kVecs].whole;
        float x[H];
#pragma unroll
        for (int e = 0; e < H; ++e) x[e] = whole * S[e];
        tmem_st(at + TM_DF + part * H, x);
        return true;
    };
    float S[H];
    auto store = [&](float *to) {
        if (live)
#pragma unroll
            for (int e = 0; e < H; ++e)
                if (e < keys) to[in + (size_t)e * dv] = S[e];
    };
    {
#pragma unroll
        for (int e = 0; e < H; ++e) S[e] = p.d_fin && live && e < keys ? p.d_fin[(size_t)n * one + in + (size_t)e * dv] : 0.f;
        if (chunks == 0) {
            if (p.d_init) store(p.d_init + (size_t)n * one);
            return true;
        }
        publish_state(S, at + TM_D + part * (H / 2));
        warp_arrive(&s.s);
        store(p.dS + (size_t)(chunk0 + chunks - 1) * one);
        if (!scaled(S, 0)) return false;
    }
#pragma unroll 1
    for (int k = 0; k < chunks; ++k) {
        const uint32_t par = (uint32_t)k & 1u;
        const int st = k % kStages, c = chunks - 1 - k, m = (int)min((long long)C, end - begin - (long long)c * C);
        const Vec &vec = s.vec[k % kVecs];
        if (!warp_wait(&s.full[st], (uint32_t)(k / kStages) & 1u)) return false;
        if (m < C) {  // K and Q behind the sequence are another one's: zeros
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            for (int e = threadIdx.x; e < (C - m) * 8; e += kChainWarps * 32)
#pragma unroll
                for (int a = 0; a < DK / 32; ++a) *reinterpret_cast<uint4 *>(&s.kq[st][a * 8192 + m * 128 + e * 16]) = zero;
            fence_async_smem();
        }
        if (k == 0) warp_arrive(&s.ready);
        // dO^T: exact for P, with its decay for Q
        float d_o[16];
        {
            const uint8_t *v = s.d_o[st] + o_in;
            uint32_t word[8];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                uint32_t x = *reinterpret_cast<const uint16_t *>(v + e * 128 + ((piece ^ (uint32_t)(e & 7)) << 4));
                if (t0 + e >= m) x = 0u;
                d_o[e] = __uint_as_float(x << 16);
                word[e / 2] = e & 1 ? word[e / 2] | (x << 16) : x;
            }
            tmem_st(at + TM_O + 8 * part, word);
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&s.o);
        }
        float dU[16];
        if (!warp_wait(&s.pd, par)) return false;
        tc_fence_after();
        tmem_ld(at + TM_PD + t0, dU);
        tmem_ld_wait();
        tc_fence_before();
        warp_arrive(&s.pd_read);
        if (!warp_wait(&s.kd, par)) return false;
        tc_fence_after();
        {
            float x[16];
            tmem_ld(at + TM_KD + t0, x);
            tmem_ld_wait();
            scale16(x, vec.F + t0);
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int e = 0; e < 16; ++e) dU[e] += x[e];
#pragma unroll
            for (int e = 0; e < 8; ++e) split2(dU[2 * e], dU[2 * e + 1], hi[e], lo[e]);
            tmem_st(at + TM_U + 8 * part, hi);
            tmem_st(at + TM_U + 32 + 8 * part, lo);
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&s.r);
        }
        // Beside dU (T - I): E dO, in the place of dO and of dO^T P, which everyone has read
        if (!warp_wait(&s.pd_read, par)) return false;
        tc_fence_after();
        {
            scale16(d_o, vec.E + t0);
            uint32_t hi[8], mid[8], lo[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) split3(d_o[2 * e], d_o[2 * e + 1], hi[e], mid[e], lo[e]);
            tmem_st(at + TM_O + 8 * part, hi);
            tmem_st(at + TM_O + 32 + 8 * part, mid);
            tmem_st(at + TM_O + 64 + 8 * part, lo);
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&s.h);
        }
        if (!warp_wait(&s.u, par)) return false;
        tc_fence_after();
        {
            float x[16];
            tmem_ld(at + TM_KD + t0, x);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = dU[e] += x[e];  // dR
            scale16(x, vec.be + t0);
            uint32_t hi[8], mid[8], lo[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) split3(-x[2 * e], -x[2 * e + 1], hi[e], mid[e], lo[e]);
            tmem_st(at + TM_D + 8 * part, hi);
            tmem_st(at + TM_D + 32 + 8 * part, mid);
            tmem_st(at + TM_D + 64 + 8 * part, lo);
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&s.u2);
            if (live) {
                float *to = p.dR + (((size_t)(chunk0 + c) * p.f.hv + h) * C + t0) * dv + col;
#pragma unroll
                for (int e = 0; e < 16; ++e) to[(size_t)e * dv] = dU[e];
            }
        }
        if (!warp_wait(&s.ds, par)) return false;
        tc_fence_after();
        tmem_ld(at + TM_DF + part * H, S);
        tmem_ld_wait();
        if (k + 1 < chunks) {
            publish_state(S, at + TM_D + part * (H / 2));
            warp_arrive(&s.s);
            store(p.dS + (size_t)(chunk0 + c - 1) * one);
            if (!scaled(S, k + 1)) return false;
        } else if (p.d_init) {
            store(p.d_init + (size_t)n * one);
        }
    }
    return true;
}

template <int DK>
__global__ void __launch_bounds__(kThreads, 1) delta_chain_back_kernel(const __grid_constant__ ChainMaps maps, const __grid_constant__ ChainParams p) {
    extern __shared__ uint8_t raw[];
    ChainShared &s = *reinterpret_cast<ChainShared *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5;
    const int h = blockIdx.x % p.f.hv, n = p.f.order ? p.f.order[blockIdx.x / p.f.hv] : blockIdx.x / p.f.hv;
    long long begin, end;
    if (!rows_of(p.f, n, begin, end)) return;
    const int chunks = (int)((end - begin + C - 1) / C);
    if (warp == 0) {
        tmem_alloc(&s.tmem, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.free[i], 1);
        }
        mbar_init(&s.ready, kChainWarps);
        for (int i = 0; i < kVecs; ++i) {
            mbar_init(&s.ready_vec[i], 1);
            mbar_init(&s.free_vec[i], 1);
        }
        for (uint64_t *b : {&s.s, &s.o, &s.pd_read, &s.r, &s.h, &s.u2}) mbar_init(b, kChainWarps);
        for (uint64_t *b : {&s.pd, &s.kd, &s.u, &s.ds, &s.drain}) mbar_init(b, 1);
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    bool ok = true;
    if (warp < kChainWarps) {
        ok = chain<DK>(s, p, n, h, begin, end, chunks, tmem);
    } else if (warp == kIssuer) {
        ok = chain_issue<DK>(s, chunks);
        if (!ok) {  // nothing may be in flight at the end
            mma_commit_warp(&s.drain);
            (void)mbar_wait(&s.drain, 0, kWaitNs);
        }
    } else if (warp == kLoader) {
        ok = chain_load<DK>(s, maps, p, n, h, begin, chunks);
    } else if (warp == kDecays) {
        ok = chain_decays(s, p, h, begin, end, chunks);
    }
    __syncwarp();
    if (!ok) atomicOr(p.f.err, kErrTimeout);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------- everything of a chunk -----

constexpr int kGradThreads = 512;
constexpr uint32_t TG_1 = 0;     // [dO; dR] S0^T, scaled, then with [Gp; Ga] K: [dq; row]
constexpr uint32_t TG_2 = 128;   // U dS^T, scaled, then with Gp^T Q + (b Ga)^T K: col in lanes 0..63
constexpr uint32_t TG_P = 256;   // [dO; dR] U^T
constexpr uint32_t TG_A = 320;   // [dO; dR]: two times 64
constexpr uint32_t TG_G = 448;   // [Q; K] K^T

// The MMAs that take 64 rows (U) or 64 columns (Gp, b Ga) as 128 read what lies behind them as well, into lanes that nobody reads: the order here
// keeps that inside the block's memory.
struct GradShared {
    uint8_t qk[32768];                   // per 64 key channels, 64 rows of Q, 64 rows of K
    uint8_t g_hi[16384], g_lo[16384];    // [Gp; Ga], 128 rows
    uint8_t bg_hi[8192], bg_lo[8192];    // b Ga
    uint8_t u_hi[16384], u_lo[16384];    // U, per 64 value channels 64 rows
    uint8_t s_hi[32768], s_lo[32768];    // S0, then dS, per 64 value channels 128 rows (key channels)
    Vec vec;
    float a[C], pre[C], f[C];
    float sums[4][5][C];                 // per quarter of the columns: q.(the part of dq from S0), k.row, k.(the part of row from S0),
                                         // k.(the part of col from dS), dR.v
    float cross[4][C], pairs[4][2 * C];  // dg_t from the pairs in t's quarter of the columns, per 32 lanes; a quarter's pairs of a lane
    float joined[kGradThreads / 32];
    uint64_t full, b0, b1, b2, b3, b4;
    uint32_t tmem;
};
static_assert(offsetof(GradShared, bg_lo) + 16384 <= offsetof(GradShared, vec) && offsetof(GradShared, u_lo) + 24576 <= offsetof(GradShared, vec),
              "128 rows or columns from every operand of 64");
struct GradMaps {
    CUtensorMap q, k;
};
struct GradParams {
    DeltaParams f;
    const void *d_o;
    const float *S, *U, *dS, *dR;
    float *dq, *dk, *dv, *dg, *db;  // dq, dk [rows, value heads, dk]
};

// N consecutive fp32 values from column c of a row of `width`, zeros past it (width is a multiple of 32, c of 8).
template <int N>
__device__ __forceinline__ void load_row(float (&x)[N], const float *row, int c, int width) {
#pragma unroll
    for (int e = 0; e < N; e += 4) {
        const float4 v = c + e < width ? *reinterpret_cast<const float4 *>(row + c + e) : make_float4(0.f, 0.f, 0.f, 0.f);
        x[e] = v.x, x[e + 1] = v.y, x[e + 2] = v.z, x[e + 3] = v.w;
    }
}
__device__ __forceinline__ void bf16_pairs(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) x[2 * e] = __uint_as_float(w[e] << 16), x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
}

// A state [dk, dv]: thread = half a line's 16-byte words, so a warp reads two lines; N = DK / 32 pieces of 8 values.
template <int N>
__device__ __forceinline__ void load_state(float (&x)[N][8], const float *S, int dk, int dv) {
    const int c = (threadIdx.x & 15) * 8;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const int r = (threadIdx.x >> 4) + 32 * e;
        load_row(x[e], S + (size_t)r * dv, c, r < dk ? dv : 0);
    }
}
// The same as the operand of s_hi, s_lo.
template <int N>
__device__ __forceinline__ void state_operand(GradShared &s, const float (&x)[N][8]) {
    const int c = (threadIdx.x & 15) * 8;
#pragma unroll
    for (int e = 0; e < N; ++e)
        store_operand(s.s_hi + (c >> 6) * 16384, s.s_lo + (c >> 6) * 16384, (threadIdx.x >> 4) + 32 * e, (c & 63) >> 3, x[e]);
}

static_assert(2 * 16384 + 2 * 32768 >= 2 * C * 132 * 4 && 2 * 16384 + 2 * 8192 >= C * 132 * 4, "rows in the operands' places");

// A chunk's fp32 outputs leave through shared memory: a thread holds a part of a row, and 32 lanes that write to 32 rows at a time take four
// times as long.
constexpr int kPitch = 132;  // floats between rows there
template <int N>
__device__ __forceinline__ void put_row(float *rows, int i, int c, const float (&x)[N]) {
#pragma unroll
    for (int e = 0; e < N; e += 4) *reinterpret_cast<float4 *>(rows + i * kPitch + c + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
}
// All threads, behind a barrier: rows 0 .. m - 1 of `width` values (a multiple of 32), `stride` apart in `to`.
__device__ __forceinline__ void rows_out(float *to, size_t stride, const float *rows, int m, int width) {
    const int c = (threadIdx.x & 31) * 4;
    if (c < width)
#pragma unroll
        for (int r = threadIdx.x >> 5; r < C; r += kGradThreads / 32)
            if (r < m) *reinterpret_cast<float4 *>(to + r * stride + c) = *reinterpret_cast<const float4 *>(rows + r * kPitch + c);
}

template <int DK>
__global__ void __launch_bounds__(kGradThreads, 1) delta_chunk_back_kernel(const __grid_constant__ GradMaps maps, const __grid_constant__ GradParams p) {
    extern __shared__ uint8_t raw[];
    GradShared &s = *reinterpret_cast<GradShared *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    constexpr int W = DK / 4;  // key columns of a thread
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hv = p.f.hv, dk = p.f.dk, dv = p.f.dv;
    const int h = blockIdx.x % hv;
    const long long slot = blockIdx.x / hv;
    // The sequence whose chunk has this number, if any: the last one that starts at or before it.
    int n = 0;
    for (int hi = p.f.seqs.n_seqs; hi - n > 1;) {
        const int mid = (n + hi) >> 1;
        if (first_chunk(p.f.seqs.begin(mid), mid, C) <= slot) n = mid; else hi = mid;
    }
    const long long begin = p.f.seqs.begin(n), end = p.f.seqs.end(n), c = slot - first_chunk(begin, n, C);
    if (begin < 0 || end < begin || end > p.f.seqs.rows || c < 0 || c * C >= end - begin) return;
    const long long row0 = begin + c * C;
    const int m = (int)min((long long)C, end - row0);
    const size_t at_chunk = (size_t)slot * hv + h;
    const int L = tid & 127, part = tid >> 7, i = L & 63;  // TMEM lane, quarter of the columns, row of the chunk
    const bool second = L >= 64;                           // a row of dR
    // The loads of the first products, all in flight together.
    constexpr int N = DK / 32;
    const float *S0 = p.S + at_chunk * dk * dv, *dS = p.dS + at_chunk * dk * dv;
    float state[N][8], u_row[16], dR[32], beta_row = 0.f;
    uint4 words[4];  // of dO's row, or v's
    {
        const bool there = i < m && 32 * part < dv;
        const __nv_bfloat16 *from = second ? static_cast<const __nv_bfloat16 *>(p.f.v) + (row0 + i) * p.f.vs + (size_t)h * dv
                                           : static_cast<const __nv_bfloat16 *>(p.d_o) + ((row0 + i) * hv + h) * dv;
#pragma unroll
        for (int e = 0; e < 4; ++e) words[e] = there ? *reinterpret_cast<const uint4 *>(from + 32 * part + 8 * e) : make_uint4(0u, 0u, 0u, 0u);
        if (second) {
            load_row(dR, p.dR + (at_chunk * C + i) * dv, 32 * part, dv);
            if (there) beta_row = p.f.beta[(row0 + i) * hv + h];
        }
    }
    load_row(u_row, p.U + (at_chunk * C + (tid >> 3)) * dv, (tid & 7) * 16, dv);
    load_state(state, S0, dk, dv);

    if (warp == 0) {
        tmem_alloc(&s.tmem, 512);
        tmem_relinquish();
    }
    if (tid == 32) {
        for (uint64_t *b : {&s.full, &s.b0, &s.b1, &s.b2, &s.b3, &s.b4}) mbar_init(b, 1);
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s.tmem, 0);
    const uint32_t at = tmem + ((uint32_t)(L & 96) << 16);
    bool ok = true;
    if (tid == 0) {
        mbar_arrive_expect_tx(&s.full, DK / 64 * 16384);
        for (int a = 0; a < DK / 64; ++a) {
            tma_load_3d(s.qk + a * 16384, &maps.q, &s.full, 64 * a, h / p.f.per, (int)row0);
            tma_load_3d(s.qk + a * 16384 + 8192, &maps.k, &s.full, 64 * a, h / p.f.per, (int)row0);
        }
    }
    if (warp == 1) {
        float own[2], b[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = lane + 32 * half;
            own[half] = r < m ? log_decay(p.f.g[(row0 + r) * hv + h]) : 0.f;
            b[half] = r < m ? p.f.beta[(row0 + r) * hv + h] : 0.f;
        }
        chunk_decays(s.vec, s.a, s.pre, s.f, lane, own, b, [] { return true; });
    }
    __syncwarp();
    {  // [dO; dR], and dv, dR.v on the way
        const int c0 = 32 * part;
        uint32_t hi[16], lo[16];
        if (!second) {
#pragma unroll
            for (int e = 0; e < 4; ++e) hi[4 * e] = words[e].x, hi[4 * e + 1] = words[e].y, hi[4 * e + 2] = words[e].z, hi[4 * e + 3] = words[e].w;
#pragma unroll
            for (int e = 0; e < 16; ++e) lo[e] = 0u;
        } else {
            float dot = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) split2(dR[2 * e], dR[2 * e + 1], hi[e], lo[e]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float y[8];
                bf16_pairs(words[e], y);
#pragma unroll
                for (int j = 0; j < 8; ++j) dot = fmaf(dR[8 * e + j], y[j], dot);
            }
            s.sums[part][4][i] = dot;
#pragma unroll
            for (int e = 0; e < 32; ++e) dR[e] *= beta_row;
            put_row(reinterpret_cast<float *>(s.g_hi), i, c0, dR);  // dv, in the place of Gp and Ga, which come later
        }
        tmem_st(at + TG_A + 16 * part, hi);
        tmem_st(at + TG_A + 64 + 16 * part, lo);
    }
    {
        const int r = tid >> 3, c0 = (tid & 7) * 16;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            store_operand(s.u_hi + (c0 >> 6) * 8192, s.u_lo + (c0 >> 6) * 8192, r, ((c0 & 63) >> 3) + e, u_row + 8 * e);
    }
    state_operand(s, state);
    ok = mbar_wait(&s.full, 0, kWaitNs);
    if (m < C) {  // the rows behind the sequence are another one's
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        for (int e = tid; e < (C - m) * 8; e += kGradThreads)
#pragma unroll
            for (int a = 0; a < DK / 32; ++a) *reinterpret_cast<uint4 *>(&s.qk[a * 8192 + m * 128 + e * 16]) = zero;
    }
    tmem_st_wait();
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint64_t u_hi = sdesc_sw128(smem_u32(s.u_hi), 16u, 1024u), s_hi = sdesc_sw128(smem_u32(s.s_hi), 16u, 1024u);
    constexpr uint64_t kULo = sizeof(s.u_hi) >> 4, kSLo = sizeof(s.s_hi) >> 4, kGLo = sizeof(s.g_hi) >> 4, kBLo = sizeof(s.bg_hi) >> 4;
    const uint32_t qk = smem_u32(s.qk);
    if (warp == 0) {
        const uint64_t d_qk = sdesc_sw128(qk, 16u, 1024u), d_k = sdesc_sw128(qk + 8192u, 16u, 1024u);
#pragma unroll
        for (int st = 0; st < DK / 16; ++st)
            mma_bf16_warp(tmem + TG_G, d_qk + kstep(st, 16384u), d_k + kstep(st, 16384u), idesc_bf16(128, 64), st > 0);
#pragma unroll
        for (int e = 0; e < 3; ++e)  // first x first, first x second, second x first
#pragma unroll
            for (int st = 0; st < 8; ++st)
                mma_bf16_tmem_a_warp(tmem + TG_P, tmem + TG_A + (e == 2 ? 64 : 0) + 8 * st, u_hi + (e == 1 ? kULo : 0) + kstep(st, 8192u),
                                     idesc_bf16(128, 64), e + st > 0);
        mma_commit_warp(&s.b0);
#pragma unroll
        for (int e = 0; e < 3; ++e)
#pragma unroll
            for (int st = 0; st < 8; ++st)
                mma_bf16_tmem_a_warp(tmem + TG_1, tmem + TG_A + (e == 2 ? 64 : 0) + 8 * st, s_hi + (e == 1 ? kSLo : 0) + kstep(st, 16384u),
                                     idesc_bf16(128, DK), e + st > 0);
        mma_commit_warp(&s.b1);
    }
    __syncwarp();
    rows_out(p.dv + (row0 * hv + h) * dv, (size_t)hv * dv, reinterpret_cast<const float *>(s.g_hi), m, dv);
    float joined = 0.f;  // <S0, dS>
    {
        float d[N][8];
        load_state(d, dS, dk, dv);
#pragma unroll
        for (int e = 0; e < N; ++e)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                joined = fmaf(state[e][j], d[e][j], joined);
                state[e][j] = d[e][j];
            }
    }
    ok = mbar_wait(&s.b0, 0, kWaitNs) && ok;
    tc_fence_after();
    __syncthreads();  // dv is out of the place
    const float b_row = s.vec.b[i];
    // Row i of Q (0) or K (1), this thread's columns.
    auto dot_row = [&](const float (&x)[W], uint32_t k) {
        float sum = 0.f;
        const int c0 = W * part;
#pragma unroll
        for (int e = 0; e < W / 8; ++e) {
            const int cc = c0 + 8 * e;
            float y[8];
            bf16_pairs(*reinterpret_cast<const uint4 *>(&s.qk[(cc >> 6) * 16384 + k * 8192 + i * 128 + ((((cc & 63) >> 3) ^ (i & 7)) << 4)]), y);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(x[8 * e + j], y[j], sum);
        }
        return sum;
    };
    {  // Gp, Ga (without b) and b Ga
        float x[16];
        tmem_ld(at + TG_P + 16 * part, x);
        tmem_ld_wait();
        decay_block(x, s.a, s.pre, s.f, i, 16 * part, !second, second ? -1.f : 1.f);
#pragma unroll
        for (int e = 0; e < 2; ++e) store_operand(s.g_hi, s.g_lo, L, 2 * part + e, x + 8 * e);
        if (second) {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] *= b_row;
#pragma unroll
            for (int e = 0; e < 2; ++e) store_operand(s.bg_hi, s.bg_lo, i, 2 * part + e, x + 8 * e);
        }
        // dg_t has the pairs j < t <= i. For this quarter's t, from those j < t that are in the quarter: the lane's sums up to t, then the sum
        // over the lanes i >= t, which leaves lane l with t = its quarter's l & 15. The earlier quarters' pairs come at the end.
        float y[16], sum = 0.f;
        tmem_ld(at + TG_G + 16 * part, y);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int t = 16 * part + e;
            const float pair = t < i ? x[e] * y[e] : 0.f;
            y[e] = t <= i ? sum : 0.f;
            sum += pair;
        }
        s.pairs[part][L] = sum;
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) {
            const bool up = lane & d;
#pragma unroll
            for (int e = 0; e < d; ++e) {
                const float other = __shfl_xor_sync(0xffffffffu, up ? y[e] : y[e + d], d);
                y[e] = (up ? y[e + d] : y[e]) + other;
            }
        }
        y[0] += __shfl_xor_sync(0xffffffffu, y[0], 16);
        if (lane < 16) s.cross[L >> 5][16 * part + lane] = y[0];
    }
    ok = mbar_wait(&s.b1, 0, kWaitNs) && ok;
    tc_fence_after();
    {
        float x[W];
        const float E = second ? -s.vec.E[i] : s.vec.E[i];
        tmem_ld(at + TG_1 + W * part, x);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < W; ++e) x[e] *= E;
        tmem_st(at + TG_1 + W * part, x);
        s.sums[part][second ? 2 : 0][i] = dot_row(x, second ? 1u : 0u);
    }
    state_operand(s, state);  // S0's operand is read: dS in its place
    tmem_st_wait();
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint64_t q_n = sdesc_sw128(qk, 16384u, 1024u), k_n = sdesc_sw128(qk + 8192u, 16384u, 1024u);
    if (warp == 0) {
        const uint64_t g = sdesc_sw128(smem_u32(s.g_hi), 16u, 1024u);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int st = 0; st < C / 16; ++st)
                mma_bf16_warp(tmem + TG_1, g + (e ? kGLo : 0) + kstep(st, 0u), k_n + kDescStepMN128 * st, idesc_bf16(128, DK) | kIdescBMajorMN, 1u);
        mma_commit_warp(&s.b2);
        // A: the 64 rows of U; what lies behind them fills lanes 64..127, which are not read.
#pragma unroll
        for (int e = 0; e < 3; ++e)
#pragma unroll
            for (int st = 0; st < 8; ++st)
                mma_bf16_warp(tmem + TG_2, u_hi + (e == 2 ? kULo : 0) + kstep(st, 8192u), s_hi + (e == 1 ? kSLo : 0) + kstep(st, 16384u),
                              idesc_bf16(128, DK), e + st > 0);
        mma_commit_warp(&s.b3);
    }
    __syncwarp();
    const int kc = W * part;  // this thread's first key column
    float x[W];
    ok = mbar_wait(&s.b3, 0, kWaitNs) && ok;  // also: U's and dS's operands are read
    tc_fence_after();
    if (!second) {
        const float F = s.vec.F[i];
        tmem_ld(at + TG_2 + kc, x);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < W; ++e) x[e] *= F;
        s.sums[part][3][i] = dot_row(x, 1u);
        tmem_st(at + TG_2 + kc, x);
        tmem_st_wait();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) {
        // A MN-major: the columns of Gp and of b Ga in lanes 0..63; the next 64 are not read.
        const uint64_t g = sdesc_sw128(smem_u32(s.g_hi), 8192u, 1024u), bg = sdesc_sw128(smem_u32(s.bg_hi), 8192u, 1024u);
        constexpr uint32_t kind = idesc_bf16(128, DK) | kIdescAMajorMN | kIdescBMajorMN;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int st = 0; st < C / 16; ++st) {
                mma_bf16_warp(tmem + TG_2, g + (e ? kGLo : 0) + kDescStepMN128 * st, q_n + kDescStepMN128 * st, kind, 1u);
                mma_bf16_warp(tmem + TG_2, bg + (e ? kBLo : 0) + kDescStepMN128 * st, k_n + kDescStepMN128 * st, kind, 1u);
            }
        mma_commit_warp(&s.b4);
    }
    __syncwarp();
    // dq and b row in the place of the operands of U and dS
    float *dq_rows = reinterpret_cast<float *>(s.u_hi), *row_rows = dq_rows + C * kPitch;
    ok = mbar_wait(&s.b2, 0, kWaitNs) && ok;
    tc_fence_after();
    tmem_ld(at + TG_1 + kc, x);
    tmem_ld_wait();
    if (second) {
        s.sums[part][1][i] = dot_row(x, 1u);
#pragma unroll
        for (int e = 0; e < W; ++e) x[e] *= b_row;
    }
    put_row(second ? row_rows : dq_rows, i, kc, x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) joined += __shfl_xor_sync(0xffffffffu, joined, d);
    if (lane == 0) s.joined[warp] = joined;
    __syncthreads();
    rows_out(p.dq + (row0 * hv + h) * dk, (size_t)hv * dk, dq_rows, m, dk);
    ok = mbar_wait(&s.b4, 0, kWaitNs) && ok;
    tc_fence_after();
    if (!second) {
        tmem_ld(at + TG_2 + kc, x);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < W; e += 4) {
            const float4 r = *reinterpret_cast<const float4 *>(row_rows + i * kPitch + kc + e);
            x[e] += r.x, x[e + 1] += r.y, x[e + 2] += r.z, x[e + 3] += r.w;
        }
        put_row(row_rows, i, kc, x);  // dk
    }
    if (!ok) atomicOr(p.f.err, kErrTimeout);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
    rows_out(p.dk + (row0 * hv + h) * dk, (size_t)hv * dk, row_rows, m, dk);
    if (warp == 1) {
        // dg_t: the pairs across t, the rows i >= t that read S0, the rows j < t whose values dS reads, and whole <S0, dS>. Only terms that t's
        // own decay is in, so a strong one leaves no rest of terms of size 1.
        float dg[2], from[2], before[2], krow[2], dRv[2], inner = lane < kGradThreads / 32 ? s.joined[lane] : 0.f;
        float earlier[2][3];  // of row r: its pairs with the quarters before quarter 1, 2, 3
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = lane + 32 * half;
            float v[5];
#pragma unroll
            for (int e = 0; e < 5; ++e) v[e] = (s.sums[0][e][r] + s.sums[1][e][r]) + (s.sums[2][e][r] + s.sums[3][e][r]);
            from[half] = fmaf(s.vec.b[r], v[2], v[0]);
            before[half] = v[3];
            krow[half] = v[1];
            dRv[half] = v[4];
            dg[half] = (s.cross[0][r] + s.cross[1][r]) + (s.cross[2][r] + s.cross[3][r]);
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 3; ++e) earlier[half][e] = sum += s.pairs[e][r] + s.pairs[e][C + r];
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, d);
        {  // the pairs of t with the quarters before its own: over the rows from t to its quarter's end, and the quarters behind it
            const bool upper = lane & 16;
            float own[2] = {upper ? earlier[0][0] : 0.f, upper ? earlier[1][2] : earlier[1][1]};
#pragma unroll
            for (int d = 1; d < 16; d *= 2)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float y = __shfl_down_sync(0xffffffffu, own[half], d, 16);
                    if ((lane & 15) + d < 16) own[half] += y;
                }
            float first = earlier[1][0], second = upper ? earlier[1][1] : 0.f;  // rows 32..63 for quarter 1, 48..63 for quarter 2
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                first += __shfl_xor_sync(0xffffffffu, first, d);
                second += __shfl_xor_sync(0xffffffffu, second, d);
            }
            dg[0] += upper ? own[0] + first : 0.f;
            dg[1] += upper ? own[1] : own[1] + second;
        }
#pragma unroll
        for (int d = 1; d < 32; d *= 2)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float y = __shfl_down_sync(0xffffffffu, from[half], d), z = __shfl_up_sync(0xffffffffu, before[half], d);
                if (lane + d < 32) from[half] += y;
                if (lane >= d) before[half] += z;
            }
        from[0] += __shfl_sync(0xffffffffu, from[1], 0);
        const float lower = __shfl_sync(0xffffffffu, before[0], 31);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float y = __shfl_up_sync(0xffffffffu, before[half], 1);
            before[half] = (lane > 0 ? y : 0.f) + (half ? lower : 0.f);
            dg[half] += (from[half] + before[half]) + s.vec.whole * inner;
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = lane + 32 * half;
            if (r < m) {
                p.dg[(row0 + r) * hv + h] = dg[half];
                p.db[(row0 + r) * hv + h] = dRv[half] + krow[half];
            }
        }
    }
}

// ---------------------------------------------------------------------------- launches ---

long long chunk_slots(const DeltaParams &p) { return p.seqs.rows / C + p.seqs.n_seqs; }

struct Parts {
    DeltaKept kept;
    float *dS, *dR;
    size_t bytes;
};
Parts parts_of(const DeltaParams &p, void *ws) {
    const size_t n = (size_t)chunk_slots(p) * p.hv, state = n * p.dk * p.dv * 4, rows = n * C * p.dv * 4;
    uint8_t *at = static_cast<uint8_t *>(ws);
    Parts r;
    r.kept = DeltaKept{at, reinterpret_cast<float *>(at + n * kDeltaTpBytes), reinterpret_cast<float *>(at + n * kDeltaTpBytes + state)};
    r.dS = reinterpret_cast<float *>(at + n * kDeltaTpBytes + state + rows);
    r.dR = reinterpret_cast<float *>(at + n * kDeltaTpBytes + 2 * state + rows);
    r.bytes = n * kDeltaTpBytes + 2 * state + 2 * rows;
    return r;
}

template <typename F>
cudaError_t more_shared(F *f, size_t bytes) {
    return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int DK>
cudaError_t launch(const DeltaParams &p, const DeltaGradients &g, const Parts &w, cudaStream_t s) {
    ChainMaps maps;
    GradMaps grad_maps;
    if (!encode(&maps.q, p.q, p.seqs.rows, p.hk, p.dk, p.qs) || !encode(&maps.k, p.k, p.seqs.rows, p.hk, p.dk, p.ks) ||
        !encode(&maps.d_o, g.d_o, p.seqs.rows, p.hv, p.dv, (long long)p.hv * p.dv))
        return cudaErrorInvalidValue;
    grad_maps.q = maps.q;
    grad_maps.k = maps.k;
    cudaError_t e = launch_delta_tc_kept(p, w.kept, s);
    if (e != cudaSuccess) return e;
    constexpr size_t chain_bytes = sizeof(ChainShared) + 1024, grad_bytes = sizeof(GradShared) + 1024;
    static_assert(chain_bytes <= 227 * 1024 && grad_bytes <= 227 * 1024, "shared memory of a block");
    if ((e = more_shared(&delta_chain_back_kernel<DK>, chain_bytes)) != cudaSuccess) return e;
    const ChainParams cp{p, w.kept.tp, g.d_fin, w.dS, w.dR, g.d_init};
    delta_chain_back_kernel<DK><<<(unsigned)((long long)p.seqs.n_seqs * p.hv), kThreads, chain_bytes, s>>>(maps, cp);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = more_shared(&delta_chunk_back_kernel<DK>, grad_bytes)) != cudaSuccess) return e;
    const GradParams gp{p, g.d_o, w.kept.S, w.kept.U, w.dS, w.dR, g.dq, g.dk, g.dv, g.dg, g.db};
    delta_chunk_back_kernel<DK><<<(unsigned)(chunk_slots(p) * p.hv), kGradThreads, grad_bytes, s>>>(grad_maps, gp);
    return cudaGetLastError();
}

}  // namespace

size_t delta_tc_backward_bytes(const DeltaParams &p) { return parts_of(p, nullptr).bytes + delta_tc_order_bytes(p); }

cudaError_t launch_delta_tc_backward(const DeltaParams &params, const DeltaGradients &g, void *ws, cudaStream_t s) {
    DeltaParams p = params;
    const Parts w = parts_of(p, ws);
    const cudaError_t e = launch_delta_tc_order(p, static_cast<uint8_t *>(ws) + w.bytes, s);
    if (e != cudaSuccess) return e;
    return p.dk == 128 ? launch<128>(p, g, w, s) : launch<64>(p, g, w, s);
}

}  // namespace kda
