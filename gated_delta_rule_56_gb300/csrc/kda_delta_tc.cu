// kda_delta_tc.cu -- the delta rule with one decay per value head over bf16 prompts, on the sm_103a tensor cores (tcgen05 + TMA + TMEM).
//
// Chunks of C = 64 rows of one (sequence, value head), S the state before the chunk, G_i the sum of the log-decays up to row i:
//     A_ij = b_i exp(G_i - G_j) k_i.k_j (j < i),  P_ij = exp(G_i - G_j) q_i.k_j (j <= i),  T = (I + A)^-1
//     R_i = b_i v_i - b_i exp(G_i) S^T k_i,  U = T R,  o_i = exp(G_i) S^T q_i + sum_j P_ij u_j
//     S <- exp(G_C) S + sum_j k_j (exp(G_C - G_j) u_j)^T
// With one decay per head every decay is a scalar of a row pair, the exponential of the log-decays between the two rows (<= 0), and no product
// needs a decayed operand, so K and Q go into every MMA as they are in memory, exact in bf16.
//
// Everything of the chain is transposed: TMEM lane = value column, so S^T, R^T, U^T are A operands in TMEM, K and Q (and T, P) are B operands
// in shared memory, read K-major or MN-major from the same 128-byte swizzled tile, and all work between two MMAs is within a lane:
//     KS = S^T K^T  ->  R  ->  (T - I) R  ->  U  ->  S^T += U^T K        (o: QS and P U, beside the chain)
//
// Precision. The state is accumulated in fp32, its final value is an fp32 output, and a bf16 operand has 8 bits. So what is not exact goes in
// as several bf16 values: S, R and P as two (2^-18 of them is left), T - I as three (of its products with R, those of 2^-25 and less are left
// out), U with its decay as three in the state's update, where its rounding would be the state's. U = R + (T - I) R adds R itself in fp32. The inverse
// is made in fp32 with joins of two tf32 values: an error there is multiplied by |A| |T|. The final state of 8192 rows is 1.3e-6 off 64
// bits in the 2-norm (the plain fp32 form 0.2e-6); one bf16 value for S and U would leave 2e-3. With T - I and the joins in two bf16 values it was
// 1.9e-6, but 2e-2 with equal keys and beta = 2, where it is 7e-4 now (fp32 row by row: 1e-4), and the prompt below took 661 us. The outputs are
// as near as their one rounding.
//
// Roles (one block per SM): warps 0-15 the chain (four per lane quarter, a quarter of the rows and key channels each), 16-23 prepare the next
// chunk: A and P from the K K^T and Q K^T accumulators (thread = TMEM lane = row), the inverse of I + A, T - I and P as operands; 24
// issues the MMAs, 25 the TMA loads, 26 makes the decays, 27 hands T and P out for the gradients. Tiles of K and Q have three stages, V, T and
// P two: 218 KB of shared memory, and all 512 columns of TMEM.
//
// Measured: 4 x 8192 rows, 32 value heads, 16 key heads of 128: 0.70 ms, 10 600 cycles per chunk on 128 of 152 SMs; 37 packed sequences of 20 011
// rows, 16 heads: 0.24 ms. Bound by the latency of the chain (three dependent MMA groups and the conversions between them, some 7 000 cycles) and of
// the preparation beside it, which sets the pace: substitution and joins have six barriers between them. Kept out by measurement: 8 chain and 4 prep
// warps (1.02 ms: each waits for its own latencies), the joins' last block through shared memory (0.72 ms), substitution and first joins on
// the four warps that hold K's rows while the others make P (0.77 ms: those four sit on two of the SM's schedulers), conversions by truncation or on
// register pairs (the same time), waits that sleep longer (the same).
#include <atomic>
#include <mutex>

#include "kda_delta_tc.cuh"

namespace kda {
namespace {

using namespace delta_tc;

constexpr int kChainWarps = 16, kPrepWarps = 8, kIssuer = 24, kLoader = 25, kDecays = 26, kKeeper = 27;
constexpr int kThreads = 28 * 32, kPrep = kPrepWarps * 32;

// Registers of a thread: the preparing warps take what the last four give, the chain keeps what the block was launched with. More than that
// in all waits forever, and a move in the wrong direction is an illegal instruction; the count is the compiler's (72 as built: 896 x 72 = 512 x
// 72 + 256 x 80 + 128 x 56), so launch() asks for it first.
constexpr int kPrepRegisters = 80, kOtherRegisters = 56;
constexpr bool registers_suffice(int launched) {
    return kOtherRegisters <= launched && launched <= kPrepRegisters &&
           kPrep * (kPrepRegisters - launched) <= (kThreads - kPrep - kChainWarps * 32) * (launched - kOtherRegisters);
}
static_assert(registers_suffice(72) && registers_suffice(80) && !registers_suffice(64) && !registers_suffice(48) && !registers_suffice(88),
              "enough to give, and moves in their directions");

// TMEM columns
constexpr uint32_t TM_S = 0;      // S^T: first bf16 values in 0..63, second in 64..127; then U with its decay, three times 32
constexpr uint32_t TM_KS = 128;   // KS, then (T - I) R
constexpr uint32_t TM_R = 192;    // R, then U: two times 32
constexpr uint32_t TM_SF = 256;   // S^T in fp32: scaled by a chunk's decay before the MMAs add the chunk's rows
constexpr uint32_t TM_O = 384;    // QS, scaled, then with P U added
constexpr uint32_t TM_KK = 448;   // [K; Q] K^T

constexpr int kKqStages = 3, kVStages = 2, kTpStages = 2, kVecs = 3;
constexpr uint32_t kKqBytes = 32768, kVBytes = 16384, kTpBytes = kDeltaTpBytes;

struct Shared {
    uint8_t kq[kKqStages][kKqBytes];  // per 64 key channels: 64 rows of K, 64 rows of Q
    uint8_t v[kVStages][kVBytes];     // per 64 value channels: 64 rows
    uint8_t tp[kTpStages][kTpBytes];  // T - I (three bf16 values; before that A and its inverse in fp32), P (two)
    Vec vec[kVecs];
    float a[2][C], pre[2][C], f[2][C];  // decays: of a row; within its block of 16, up to the row; from the row to the block's end
    uint64_t full_kq[kKqStages], free_kq[kKqStages], ready_kq;
    uint64_t full_v[kVStages], free_v[kVStages], ready_v[kVStages];
    uint64_t free_tp[kTpStages], ready_tp[kTpStages];
    uint64_t free_vec[kVecs], ready_decays[2];
    uint64_t kk, kk_free, s, ks, qs, r, u, u2, up, ds, pu, o_free, drain;
    uint32_t tmem;
};

struct Maps {
    CUtensorMap q, k, v;
};

__device__ __forceinline__ void prep_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// prep_sync; true if `ok` in all of them, so that they leave together when a wait runs out.
__device__ __forceinline__ bool prep_all(bool ok) {
    const uint32_t bad = ok ? 0u : 1u;
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, 256, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(bad)
        : "memory");
    return any == 0;
}
// ------------------------------------------------------------------------ prep -----------

// ---- the inverse of I + A, in fp32 in A's place, which the operand takes afterwards. Right of the diagonal's blocks of 32 lies what the joins
// hold in between. Blocks of 16 by substitution, then joined twice through X21 = -X22 (A21 X11). An error of A or of a
// join is multiplied by |A| |(I + A)^-1|, a hundred where keys resemble one another and thousands with b near 2, so the joins' operands are
// two tf32 values each, 2^-21 of a product is left (two bf16 values, 2^-17: final states 20 to 100 times as far off there).
__device__ __forceinline__ void two_tf32(float x, uint32_t &hi, uint32_t &lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
constexpr int kPitch = C + 4;  // floats between rows
static_assert(C * kPitch * 4 == 16384 + 8 * 128, "in the place of T - I: its first and second values, and 8 rows of the third");
// d = A (16 x K) B (K x 8), by one warp: lane 4 g + t has columns 2 t, 2 t + 1 of rows g and g + 8.
template <int K>
__device__ __forceinline__ void join(float (&d)[4], const float *A, const float *B, int lane) {
    const int g = lane >> 2, t = lane & 3;
    float more[2][4] = {};  // three chains of MMAs
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = 0.f;
#pragma unroll
    for (int k = 0; k < K; k += 8) {
        uint32_t ah[4], al[4], bh[2], bl[2];
#pragma unroll
        for (int e = 0; e < 4; ++e) two_tf32(A[(g + 8 * (e & 1)) * kPitch + k + t + 4 * (e >> 1)], ah[e], al[e]);
#pragma unroll
        for (int e = 0; e < 2; ++e) two_tf32(B[(k + t + 4 * e) * kPitch + g], bh[e], bl[e]);
        mma_tf32(d, ah, bh);
        mma_tf32(more[0], ah, bl);
        mma_tf32(more[1], al, bh);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] += more[0][e] + more[1][e];
}
__device__ __forceinline__ void put_join(float *to, float sign, const float (&d)[4], int lane) {
    const int g = lane >> 2, t = lane & 3;
    *reinterpret_cast<float2 *>(to + g * kPitch + 2 * t) = make_float2(sign * d[0], sign * d[1]);
    *reinterpret_cast<float2 *>(to + (g + 8) * kPitch + 2 * t) = make_float2(sign * d[2], sign * d[3]);
}

// 8 values of row i as three bf16 operands of 64 x 64.
__device__ __forceinline__ void store_operand3(uint8_t *to, int i, int chunk, const float *x) {
    uint32_t h[4], m[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split3(x[2 * e], x[2 * e + 1], h[e], m[e], l[e]);
    const uint32_t at = (uint32_t)i * 128u + (uint32_t)((chunk ^ (i & 7)) << 4);
    *reinterpret_cast<uint4 *>(to + at) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4 *>(to + 8192 + at) = make_uint4(m[0], m[1], m[2], m[3]);
    *reinterpret_cast<uint4 *>(to + 16384 + at) = make_uint4(l[0], l[1], l[2], l[3]);
}

// A in the operand's place -> the operand.
__device__ __forceinline__ void invert(uint8_t *tp, int pt) {
    float *A = reinterpret_cast<float *>(tp);
    auto at = [A](int r, int c) { return A + r * kPitch + c; };
    const int w = pt >> 5, lane = pt & 31;
    if (w < 4) {  // by substitution, lane = column
        const int j = lane & 15, o = 16 * w;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i == j ? 1.f : 0.f;
#pragma unroll
        for (int m = 0; m < 16; m += 4) {  // four columns of A at a time
            float4 own[4];
#pragma unroll
            for (int i = 1; i < 4; ++i) own[i] = *reinterpret_cast<const float4 *>(at(o + m + i, o + m));
            x[m + 1] = fmaf(-own[1].x, x[m], x[m + 1]);
            x[m + 2] = fmaf(-own[2].y, x[m + 1], fmaf(-own[2].x, x[m], x[m + 2]));
            x[m + 3] = fmaf(-own[3].z, x[m + 2], fmaf(-own[3].y, x[m + 1], fmaf(-own[3].x, x[m], x[m + 3])));
#pragma unroll
            for (int i = m + 4; i < 16; ++i) {
                const float4 a = *reinterpret_cast<const float4 *>(at(o + i, o + m));
                x[i] = fmaf(-a.w, x[m + 3], fmaf(-a.z, x[m + 2], fmaf(-a.y, x[m + 1], fmaf(-a.x, x[m], x[i]))));
            }
        }
        __syncwarp();
        if (lane < 16)
#pragma unroll
            for (int i = 0; i < 16; ++i) *at(o + i, o + j) = x[i];
    }
    prep_sync();
    float d[4];
    {  // two pairs of blocks
        const int o = 32 * ((w >> 1) & 1), n = 8 * (w & 1);
        if (w < 4) {
            join<16>(d, at(o + 16, o), at(o, o + n), lane);
            put_join(at(o >> 1, 32 + n), 1.f, d, lane);
        }
        prep_sync();
        if (w < 4) {
            join<16>(d, at(o + 16, o + 16), at(o >> 1, 32 + n), lane);
            put_join(at(o + 16, o + n), -1.f, d, lane);
        }
    }
    prep_sync();
    const int o = 16 * (w & 1), n = 8 * (w >> 1);
    join<32>(d, at(32 + o, 0), at(0, n), lane);
    put_join(at(o, 32 + n), 1.f, d, lane);
    prep_sync();
    join<32>(d, at(32 + o, 32), at(0, 32 + n), lane);
    // T - I from here: the last join's block from the registers, the blocks of 32 on the diagonal, zeros behind them.
    const int r = pt >> 2, c = (r & 32) + 8 * (pt & 3);
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(at(r, c + j));
        y[j] = x.x, y[j + 1] = x.y, y[j + 2] = x.z, y[j + 3] = x.w;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = c + j < r ? y[j] : 0.f;
    prep_sync();  // everyone has read
    store_operand3(tp, r, c >> 3, y);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int row = 32 + o + (lane >> 2) + 8 * half;
        uint32_t v[3];
        split3(-d[2 * half], -d[2 * half + 1], v[0], v[1], v[2]);
#pragma unroll
        for (int e = 0; e < 3; ++e)
            *reinterpret_cast<uint32_t *>(tp + 8192 * e + row * 128 + (((n >> 3) ^ (row & 7)) << 4) + (lane & 3) * 4) = v[e];
    }
    const int zero = (pt >> 2 & 31) * 128 + (((4 + (pt & 3)) ^ (pt >> 2 & 7)) << 4);
    *reinterpret_cast<uint4 *>(tp + 8192 * (pt >> 7) + zero) = make_uint4(0u, 0u, 0u, 0u);
    if (pt < 32) *reinterpret_cast<uint4 *>(tp + 16384 + zero) = make_uint4(0u, 0u, 0u, 0u);  // A ends in its row 7
}

// The chunks' decays, by one warp, up to two chunks ahead of the chain.
__device__ __forceinline__ bool decays(Shared &s, const DeltaParams &p, int h, long long begin, long long end, int chunks) {
    const int lane = threadIdx.x & 31;
    const float *g = p.g + (begin + lane) * p.hv + h, *beta = p.beta + (begin + lane) * p.hv + h;
    const long long half_rows = 32ll * p.hv;
    for (int c = 0; c < chunks; ++c) {
        const long long left = end - begin - (long long)c * C - lane;
        float own[2], b[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            own[half] = left > 32 * half ? log_decay(g[half * half_rows]) : 0.f;
            b[half] = left > 32 * half ? beta[half * half_rows] : 0.f;
        }
        g += 2 * half_rows;
        beta += 2 * half_rows;
        const bool ok = chunk_decays(s.vec[c % kVecs], s.a[c & 1], s.pre[c & 1], s.f[c & 1], lane, own, b, [&] {
            if (c >= kVecs && !warp_wait(&s.free_vec[c % kVecs], (uint32_t)(c / kVecs - 1) & 1u)) return false;
            return c < 2 || warp_wait(&s.ready_tp[c & 1], (uint32_t)(c / 2 - 1) & 1u);  // chunk c - 2 is prepared
        });
        if (!ok) return false;
        warp_arrive(&s.ready_decays[c & 1]);
    }
    return true;
}

template <int DK>
__device__ __forceinline__ bool prep(Shared &s, const DeltaParams &p, int h, long long begin, long long end, int chunks, uint32_t tmem) {
    const int pt = threadIdx.x - kChainWarps * 32, w = pt >> 5;
    // A warp's rows: quarter w % 4 of [K; Q], columns of half w / 4. Rows 0..31 have nothing in the second half.
    const int i = pt & 63, c0 = 32 * (w >> 2);
    const bool q_row = w & 2, live = (w & 1) || w < 4;
    const uint32_t tq = (uint32_t)(32 * (w & 3)) << 16;
    const int vtiles = p.dv > 64 ? 2 : 1;
    // What the operands have right of the diagonal blocks is never written again.
    for (int e = pt; e < kTpStages * (int)kTpBytes / 16; e += kPrep) reinterpret_cast<uint4 *>(s.tp[0])[e] = make_uint4(0u, 0u, 0u, 0u);
    prep_sync();
    for (int c = 0; c < chunks; ++c) {
        const int ks = c % kKqStages, vs = c % kVStages, ts = c % kTpStages;
        const int m = (int)min((long long)C, end - begin - (long long)c * C);
        bool ok = mbar_wait(&s.full_kq[ks], (uint32_t)(c / kKqStages) & 1u, kWaitNs) && mbar_wait(&s.full_v[vs], (uint32_t)(c / kVStages) & 1u, kWaitNs);
        if (ok && m < C) {  // the rows behind the sequence are another one's: zeros, so that nothing of theirs meets a product
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            for (int e = pt; e < (C - m) * 8; e += kPrep) {
                const uint32_t at = (uint32_t)m * 128u + (uint32_t)e * 16u;
#pragma unroll
                for (int a = 0; a < DK / 32; ++a) *reinterpret_cast<uint4 *>(&s.kq[ks][a * 8192 + at]) = zero;
                for (int a = 0; a < vtiles; ++a) *reinterpret_cast<uint4 *>(&s.v[vs][a * 8192 + at]) = zero;
            }
            fence_async_smem();
        }
        if (c == chunks - 1) warp_arrive(&s.ready_kq);
        warp_arrive(&s.ready_v[vs]);
        if (c >= kTpStages) ok = ok && mbar_wait(&s.free_tp[ts], (uint32_t)(c / kTpStages - 1) & 1u, kWaitNs);
        if (!prep_all(ok && mbar_wait(&s.ready_decays[c & 1], (uint32_t)(c >> 1) & 1u, kWaitNs) && mbar_wait(&s.kk, (uint32_t)c & 1u, kWaitNs)))
            return false;
        tc_fence_after();
        uint8_t *tp = s.tp[ts];
        float *A = reinterpret_cast<float *>(tp);
        if (live) {
            float x[32];
            tmem_ld32(tmem + tq + TM_KK + c0, x);
            tmem_ld_wait();
            tc_fence_before();
            warp_arrive(&s.kk_free);
            const float scale = q_row ? 1.f : s.vec[c % kVecs].b[i];
#pragma unroll
            for (int b = 0; b < 2; ++b) decay_block(x + 16 * b, s.a[c & 1], s.pre[c & 1], s.f[c & 1], i, c0 + 16 * b, q_row, scale);
            if (q_row) {
#pragma unroll
                for (int e = 0; e < 4; ++e) store_operand(tp + kDeltaP, tp + kDeltaP + 8192, i, c0 / 8 + e, &x[8 * e]);
            } else {
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<float4 *>(A + i * kPitch + c0 + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
            }
        }
        prep_sync();
        invert(tp, pt);
        fence_async_smem();
        warp_arrive(&s.ready_tp[ts]);
    }
    return true;
}

// ------------------------------------------------------------------------ issuer ---------

template <int DK, bool KEEP>
__device__ __forceinline__ bool issue(Shared &s, int chunks) {
    const uint32_t tmem = __shfl_sync(0xffffffffu, s.tmem, 0);
    const uint32_t kq = smem_u32(s.kq[0]), tp = smem_u32(s.tp[0]);
    auto gram = [&](int c) -> bool {  // [K; Q] K^T
        const int ks = c % kKqStages;
        // The last chunk's rows behind the sequence are cleared first; the others are there as soon as they are loaded.
        if (!warp_wait(c == chunks - 1 ? &s.ready_kq : &s.full_kq[ks], c == chunks - 1 ? 0u : (uint32_t)(c / kKqStages) & 1u)) return false;
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
        if (c + 1 < chunks && !gram(c + 1)) return false;
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
        if constexpr (!KEEP) {
            if (c > 0 && !warp_wait(&s.o_free, par ^ 1u)) return false;
            tc_fence_after();
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int st = 0; st < DK / 16; ++st)
                    mma_bf16_tmem_a_warp(tmem + TM_O, tmem + TM_S + 64 * e + 8 * st, d_q + kstep(st, 16384u), idesc_bf16(128, 64), e + st > 0);
            mma_commit_warp(&s.qs);
        }
        if (!warp_wait(&s.ready_tp[c % kTpStages], (uint32_t)(c / kTpStages) & 1u) || !warp_wait(&s.r, par)) return false;
        tc_fence_after();
        const uint64_t d_t = sdesc_sw128(tpc, 16u, 1024u), d_p = sdesc_sw128(tpc + kDeltaP, 16u, 1024u);
#pragma unroll
        for (int e = 0; e < 5; ++e)  // R's first value by T's first, second and third, R's second by T's first and second
#pragma unroll
            for (int st = 0; st < C / 16; ++st)
                mma_bf16_tmem_a_warp(tmem + TM_KS, tmem + TM_R + (e > 2 ? 32 : 0) + 8 * st, d_t + 512u * (e > 2 ? e - 3 : e) + kstep(st, 0u),
                                     idesc_bf16(128, 64), e + st > 0);
        mma_commit_warp(&s.u);
        if (!warp_wait(&s.u2, par)) return false;
        tc_fence_after();
#pragma unroll
        for (int e = 0; e < 3; ++e)
#pragma unroll
            for (int st = 0; st < C / 16; ++st)
                mma_bf16_tmem_a_warp(tmem + TM_SF, tmem + TM_S + 32 * e + 8 * st, d_kn + kDescStepMN128 * st,
                                     idesc_bf16(128, DK) | kIdescBMajorMN, 1u);
        mma_commit_warp(&s.ds);
        if constexpr (!KEEP) {
            if (!warp_wait(&s.up, par)) return false;
            tc_fence_after();
#pragma unroll
            for (int e = 0; e < 3; ++e)
#pragma unroll
                for (int st = 0; st < C / 16; ++st)
                    mma_bf16_tmem_a_warp(tmem + TM_O, tmem + TM_R + (e == 2 ? 32 : 0) + 8 * st, d_p + (e == 1 ? 512u : 0u) + kstep(st, 0u),
                                         idesc_bf16(128, 64), 1u);
            mma_commit_warp(&s.pu);
        }
        mma_commit_warp(&s.free_tp[c % kTpStages]);
        mma_commit_warp(&s.free_kq[c % kKqStages]);
        mma_commit_warp(&s.free_vec[c % kVecs]);
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

template <int DK, bool KEEP>
__device__ __forceinline__ bool chain(Shared &s, const DeltaParams &p, const DeltaKept &kept, int n, int h, long long begin, long long end, int chunks, uint32_t tmem) {
    constexpr int H = DK / 4;  // key channels of a thread
    const int part = threadIdx.x >> 7, col = threadIdx.x & 127;  // quarter of the rows and of the key channels; value column
    const int t0 = 16 * part;
    const uint32_t at = tmem + ((uint32_t)(col & 96) << 16);
    const bool live = col < p.dv;
    const size_t one = (size_t)p.hv * p.dk * p.dv, in = (size_t)h * p.dk * p.dv + (size_t)part * H * p.dv + col;
    const int keys = min(max(p.dk - part * H, 0), H);  // of this quarter that the state has
    // This column's place in a row of a V tile: 16-byte piece ^ (row % 8). Columns past dv read what is there; lanes do not meet, and those are
    // not stored.
    const uint32_t v_in = (uint32_t)(col >> 6) * 8192u + (uint32_t)(col & 7) * 2u + (uint32_t)t0 * 128u, piece = (uint32_t)(col & 63) >> 3;
    // Scaled by the next chunk's decay, the state goes back for the MMAs to add to.
    auto scaled = [&](float (&S)[H], int c) -> bool {
        if (!warp_wait(&s.ready_tp[c % kTpStages], (uint32_t)(c / kTpStages) & 1u)) return false;
        const float whole = s.vec[c % kVecs].whole;
#pragma unroll
        for (int e = 0; e < H; ++e) S[e] *= whole;
        tmem_st(at + TM_SF + part * H, S);
        return true;
    };
    // Kept for the gradients: the state before chunk c.
    float *kept_S = KEEP ? kept.S + (size_t)first_chunk(begin, n, C) * one + in : nullptr;
    auto keep = [&](const float (&S)[H], int c) {
        if constexpr (KEEP) {
            if (live) {
#pragma unroll
                for (int e = 0; e < H; ++e)
                    if (e < keys) kept_S[(size_t)c * one + (size_t)e * p.dv] = S[e];
            }
        }
    };
    auto finish = [&](const float (&S)[H]) {
        const long long to = p.fin ? state_slot(p.fin_idx, p.pool, n, p.err) : -1;
        if (to >= 0 && live)
#pragma unroll
            for (int e = 0; e < H; ++e)
                if (e < keys) p.fin[to * one + in + (size_t)e * p.dv] = S[e];
    };
    {
        const long long from = p.init ? state_slot(p.init_idx, p.pool, n, p.err) : -1;
        float S[H];
#pragma unroll
        for (int e = 0; e < H; ++e) S[e] = from >= 0 && live && e < keys ? p.init[from * one + in + (size_t)e * p.dv] : 0.f;
        if (chunks > 0) {
            publish_state(S, at + TM_S + part * (H / 2));
            warp_arrive(&s.s);
            keep(S, 0);
            if (!scaled(S, 0)) return false;
        } else {
            finish(S);
        }
    }
    // A chunk's values, for R = b v - b E KS
    float R[16];
    auto values = [&](int c) -> bool {
        const int vs = c % kVStages;
        if (!warp_wait(&s.ready_v[vs], (uint32_t)(c / kVStages) & 1u)) return false;
        const uint8_t *v = s.v[vs] + v_in;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const uint32_t x = *reinterpret_cast<const uint16_t *>(v + e * 128 + ((piece ^ (uint32_t)(e & 7)) << 4));
            R[e] = __uint_as_float(x << 16);
        }
        warp_arrive(&s.free_v[vs]);
        return true;
    };
    if (chunks > 0 && !values(0)) return false;
    const uint32_t o_step = (uint32_t)p.hv * p.dv * 2;  // bytes between rows of o
    char *o = reinterpret_cast<char *>(static_cast<__nv_bfloat16 *>(p.o) + (begin * p.hv + h) * p.dv);
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
        const uint32_t par = (uint32_t)c & 1u;
        const Vec &vec = s.vec[c % kVecs];  // there: the state was scaled by it
        scale16(R, vec.b + t0);
        if (!warp_wait(&s.ks, par)) return false;
        tc_fence_after();
        {
            float x[16];
            tmem_ld(at + TM_KS + t0, x);
            tmem_ld_wait();
            scale16(x, vec.be + t0);
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                R[e] -= x[e];
                R[e + 1] -= x[e + 1];
                split2(R[e], R[e + 1], hi[e / 2], lo[e / 2]);
            }
            tmem_st(at + TM_R + 8 * part, hi);
            tmem_st(at + TM_R + 32 + 8 * part, lo);
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&s.r);
        }
        if constexpr (!KEEP) {
            // Beside (T - I) R: the reading of the state, with its decay
            if (!warp_wait(&s.qs, par)) return false;
            tc_fence_after();
            {
                float x[16];
                tmem_ld(at + TM_O + t0, x);
                tmem_ld_wait();
                scale16(x, vec.E + t0);
                tmem_st(at + TM_O + t0, x);
            }
        }
        if (!warp_wait(&s.u, par)) return false;
        tc_fence_after();
        {
            float x[16];
            tmem_ld(at + TM_KS + t0, x);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = R[e] += x[e];  // U
            scale16(x, vec.F + t0);
            uint32_t hi[8], lo[8];
            {
                uint32_t mid[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) split3(x[2 * e], x[2 * e + 1], hi[e], mid[e], lo[e]);
                tmem_st(at + TM_S + 8 * part, hi);
                tmem_st(at + TM_S + 32 + 8 * part, mid);
                tmem_st(at + TM_S + 64 + 8 * part, lo);
            }
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&s.u2);
            if constexpr (KEEP) {
                if (live) {
                    float *to = kept.U + (((size_t)(first_chunk(begin, n, C) + c) * p.hv + h) * C + t0) * p.dv + col;
#pragma unroll
                    for (int e = 0; e < 16; ++e) to[(size_t)e * p.dv] = R[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) split2(R[2 * e], R[2 * e + 1], hi[e], lo[e]);
                tmem_st(at + TM_R + 8 * part, hi);
                tmem_st(at + TM_R + 32 + 8 * part, lo);
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(&s.up);
            }
        }
        if (c + 1 < chunks && !values(c + 1)) return false;  // beside the state's update
        if (!warp_wait(&s.ds, par)) return false;
        tc_fence_after();
        {
            float S[H];
            tmem_ld(at + TM_SF + part * H, S);
            tmem_ld_wait();
            if (c + 1 < chunks) {
                publish_state(S, at + TM_S + part * (H / 2));
                warp_arrive(&s.s);
                keep(S, c + 1);
                if (!scaled(S, c + 1)) return false;
            } else {
                finish(S);
            }
        }
        if constexpr (KEEP) continue;
        // Beside the next chunk's KS: the outputs
        if (!warp_wait(&s.pu, par)) return false;
        tc_fence_after();
        {
            float x[16];
            tmem_ld(at + TM_O + t0, x);
            tmem_ld_wait();
            tc_fence_before();
            warp_arrive(&s.o_free);
            const int m = (int)min((long long)16, end - (begin + (long long)c * C + t0));
            char *to = o + (size_t)((long long)c * C + t0) * o_step;
            const uint32_t off = (uint32_t)col * 2u;
            if (live && m == 16) {
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const uint32_t two = pack_bf16(x[e], x[e + 1]);
                    *reinterpret_cast<uint16_t *>(to + (off + e * o_step)) = (uint16_t)two;
                    *reinterpret_cast<uint16_t *>(to + (off + (e + 1) * o_step)) = (uint16_t)(two >> 16);
                }
            } else if (live) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (e < m) *reinterpret_cast<__nv_bfloat16 *>(to + (off + e * o_step)) = __float2bfloat16_rn(x[e]);
            }
        }
    }
    return true;
}

// For the gradients: T and P of every chunk go out as they are, from shared memory.
__device__ __forceinline__ bool keep_operands(Shared &s, uint8_t *to, long long step, int chunks) {
    for (int c = 0; c < chunks; ++c) {
        if (!warp_wait(&s.ready_tp[c % kTpStages], (uint32_t)(c / kTpStages) & 1u)) return false;
        if ((threadIdx.x & 31) == 0) {
            bulk_store(to + c * step, s.tp[c % kTpStages], kTpBytes);
            bulk_commit();
            bulk_wait_read_all();
            mbar_arrive(&s.free_tp[c % kTpStages]);
        }
        __syncwarp();
    }
    if ((threadIdx.x & 31) == 0) bulk_wait_all();
    __syncwarp();
    return true;
}

template <int DK, bool KEEP>
__global__ void __launch_bounds__(kThreads, 1)
    delta_tc_kernel(const __grid_constant__ Maps maps, const __grid_constant__ DeltaParams p, const __grid_constant__ DeltaKept kept) {
    extern __shared__ uint8_t raw[];
    Shared &s = *reinterpret_cast<Shared *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5;
    const int h = blockIdx.x % p.hv, n = p.order ? p.order[blockIdx.x / p.hv] : blockIdx.x / p.hv;
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
        }
        mbar_init(&s.ready_kq, kPrepWarps);
        for (int i = 0; i < kVStages; ++i) {
            mbar_init(&s.full_v[i], 1);
            mbar_init(&s.free_v[i], kChainWarps);
            mbar_init(&s.ready_v[i], kPrepWarps);
        }
        for (int i = 0; i < kTpStages; ++i) {
            mbar_init(&s.free_tp[i], KEEP ? 2 : 1);
            mbar_init(&s.ready_tp[i], kPrepWarps);
        }
        for (int i = 0; i < kVecs; ++i) mbar_init(&s.free_vec[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&s.ready_decays[i], 1);
        mbar_init(&s.kk_free, 6);  // the warps that have rows there
        for (uint64_t *b : {&s.s, &s.r, &s.u2, &s.up, &s.o_free}) mbar_init(b, kChainWarps);
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
    if (warp < kChainWarps) {
        ok = chain<DK, KEEP>(s, p, kept, n, h, begin, end, chunks, tmem);
    } else if (warp < kChainWarps + kPrepWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPrepRegisters));
        ok = prep<DK>(s, p, h, begin, end, chunks, tmem);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegisters));
        if (warp == kIssuer) {
            ok = issue<DK, KEEP>(s, chunks);
            if (!ok) {  // nothing may be in flight at the end
                mma_commit_warp(&s.drain);
                (void)mbar_wait(&s.drain, 0, kWaitNs);
            }
            __syncwarp();
        } else if (warp == kLoader) {
            ok = load<DK>(s, maps, p, h, begin, chunks);
            __syncwarp();
        } else if (warp == kDecays) {
            ok = decays(s, p, h, begin, end, chunks);
        } else if (KEEP && warp == kKeeper) {
            ok = keep_operands(s, kept.tp + ((size_t)first_chunk(begin, n, C) * p.hv + h) * kTpBytes, (long long)p.hv * kTpBytes, chunks);
        }
    }
    if (!ok) atomicOr(p.err, kErrTimeout);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

constexpr size_t kSharedBytes = sizeof(Shared) + 1024;
static_assert(kSharedBytes <= 227 * 1024, "shared memory of a block");

template <int DK, bool KEEP>
cudaError_t launch(const Maps &maps, const DeltaParams &p, const DeltaKept &kept, cudaStream_t s) {
    auto *f = &delta_tc_kernel<DK, KEEP>;
    static std::atomic<int> registers{0};  // of a thread, in the units of 8 that they are given in
    cudaError_t e;
    if (registers == 0) {
        cudaFuncAttributes compiled;
        if ((e = cudaFuncGetAttributes(&compiled, f)) != cudaSuccess) return e;
        registers = (compiled.numRegs + 7) / 8 * 8;
    }
    if (!registers_suffice(registers)) return cudaErrorLaunchOutOfResources;
    if ((e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSharedBytes)) != cudaSuccess) return e;
    f<<<(unsigned)((long long)p.seqs.n_seqs * p.hv), kThreads, kSharedBytes, s>>>(maps, p, kept);
    return cudaGetLastError();
}

template <bool KEEP>
cudaError_t launch_any(const DeltaParams &p, const DeltaKept &kept, cudaStream_t s) {
    Maps maps;
    if (!encode(&maps.q, p.q, p.seqs.rows, p.hk, p.dk, p.qs) || !encode(&maps.k, p.k, p.seqs.rows, p.hk, p.dk, p.ks) ||
        !encode(&maps.v, p.v, p.seqs.rows, p.hv, p.dv, p.vs))
        return cudaErrorInvalidValue;
    return p.dk == 128 ? launch<128, KEEP>(maps, p, kept, s) : launch<64, KEEP>(maps, p, kept, s);
}

}  // namespace

namespace delta_tc {

static PFN_cuTensorMapEncodeTiled_v12000 encoder() {
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

bool encode(CUtensorMap *map, const void *base, long long rows, int heads, int d, long long stride) {
    auto enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)C}, es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace delta_tc

bool delta_tc_shape(kda_dtype dtype, const DeltaParams &p, int fewest) {
    return dtype == KDA_BF16 && p.seqs.rows > 0 && p.seqs.rows >= (long long)fewest * p.seqs.n_seqs;
}
bool delta_tc_supported(kda_dtype dtype, const DeltaParams &p, int fewest) {
    auto ok = [](const void *x, long long stride) { return aligned16(x) && stride % 8 == 0; };
    return delta_tc_shape(dtype, p, fewest) && ok(p.q, p.qs) && ok(p.k, p.ks) && ok(p.v, p.vs) && delta_tc::encoder();
}

// Packed sequences start longest first, so that no long one is left for the end.
size_t delta_tc_order_bytes(const DeltaParams &p) {
    return p.seqs.cu && p.seqs.n_seqs >= 2 && p.seqs.n_seqs <= kMaxOrderedSeqs ? ((size_t)p.seqs.n_seqs * 4 + 255) / 256 * 256 : 0;
}
cudaError_t launch_delta_tc_order(DeltaParams &p, void *ws, cudaStream_t s) {
    if (!delta_tc_order_bytes(p)) return cudaSuccess;
    int32_t *order = static_cast<int32_t *>(ws);
    p.order = order;
    return launch_order_by_length(p.seqs.cu, p.seqs.n_seqs, order, s);
}

cudaError_t launch_delta_tc(const DeltaParams &p, cudaStream_t s) { return launch_any<false>(p, DeltaKept{}, s); }
cudaError_t launch_delta_tc_kept(const DeltaParams &p, const DeltaKept &kept, cudaStream_t s) { return launch_any<true>(p, kept, s); }

}  // namespace kda
