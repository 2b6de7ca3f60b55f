// kda_delta.cu -- the delta rule with one decay per value head in fp32 on the CUDA cores: the step of a single token, prompts in fp32 and short
// prompts, row by row and (below) in chunks of 16 rows.
//
// Per value head and token, with a = exp(g): u = b (v - a S^T k), S <- a S + k u^T, o = a S^T q + (q.k) u, where S is the state before
// the token: both products read the old state, so one pass over it serves them and the update follows in registers.
//
// Columns of the state do not meet: a warp owns 16 of them, 8 groups of lanes the rows of 16 (dk = 128) each, a lane 4 columns.
// Row pairs sit in register pairs, so decay, update and both products are two elements per instruction. The 8 partial sums of a lane (4
// columns, k and q) meet in 7 shuffles that leave every lane one finished sum.
//
// Single token: bound by HBM, the fp32 state is read once and written once (16-byte accesses, all of a lane's loads in flight together): 256
// sequences x 32 heads of 128 x 128 take 158 us, 6.85 TB/s (what is above the copy rate of 6.7 comes out of L2); one sequence 4.8 us.
// Prompts row by row: bound by a token's latency where warps are few (the sums' shuffles between two dependent passes over the registers): 0.35 us
// per token with heads of 64, 0.43 us with 128; with 4 warps per scheduler by the instructions.
#include "kda_delta.cuh"
#include "kda_delta_tc.h"
#include "kda_layers.h"

namespace kda {
namespace {

constexpr int kCols = 16;   // columns of a warp
constexpr int kStage = 8;   // tokens of a stage (and lanes that hold their decays)
constexpr int kStages = 4;
constexpr int kC = 16;      // rows of a chunk

__device__ __forceinline__ f32x2 dup(float a) { return pair(a, a); }

// One warp's part of a state: rows [r0, r0 + R) in pairs, 4 columns.
template <int R>
struct Tile {
    f32x2 s[R / 2][4];

    __device__ __forceinline__ void load(const float *p, int dv) {
#pragma unroll
        for (int r = 0; r < R; r += 2) {
            const float4 a = __ldcs(reinterpret_cast<const float4 *>(p + (size_t)r * dv));
            const float4 b = __ldcs(reinterpret_cast<const float4 *>(p + (size_t)(r + 1) * dv));
            s[r / 2][0] = pair(a.x, b.x);
            s[r / 2][1] = pair(a.y, b.y);
            s[r / 2][2] = pair(a.z, b.z);
            s[r / 2][3] = pair(a.w, b.w);
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int r = 0; r < R / 2; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[r][c] = 0ull;
    }
    __device__ __forceinline__ void store(float *p, int dv) const {
#pragma unroll
        for (int r = 0; r < R; r += 2) {
            float4 a, b;
            unpair(s[r / 2][0], a.x, b.x);
            unpair(s[r / 2][1], a.y, b.y);
            unpair(s[r / 2][2], a.z, b.z);
            unpair(s[r / 2][3], a.w, b.w);
            __stcs(reinterpret_cast<float4 *>(p + (size_t)r * dv), a);
            __stcs(reinterpret_cast<float4 *>(p + (size_t)(r + 1) * dv), b);
        }
    }

    // One token: k, q the lane's rows; v the value of column (lane / 4) % 4 of the lane's four. Returns o of that column in lanes 16 to 31.
    __device__ __forceinline__ float step(const f32x2 (&k)[R / 2], const f32x2 (&q)[R / 2], float v, float a, float b, int lane) {
        f32x2 ks[4], qs[4], kq = 0ull;
#pragma unroll
        for (int c = 0; c < 4; ++c) ks[c] = qs[c] = 0ull;
#pragma unroll
        for (int r = 0; r < R / 2; ++r) {
            kq = fma2(k[r], q[r], kq);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                ks[c] = fma2(k[r], s[r][c], ks[c]);
                qs[c] = fma2(q[r], s[r][c], qs[c]);
            }
        }
        float x[8], lo, hi;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            unpair(ks[c], lo, hi);
            x[c] = lo + hi;
            unpair(qs[c], lo, hi);
            x[4 + c] = lo + hi;
        }
        unpair(kq, lo, hi);
        float dot = lo + hi;
#pragma unroll
        for (int m = 4; m < 32; m *= 2) dot += __shfl_xor_sync(0xffffffffu, dot, m);
        // Lane group rl = lane / 4 ends with the whole sum x[rl].
        const bool up4 = lane & 16, up2 = lane & 8, up1 = lane & 4;
        float y[4], z[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = (up4 ? x[4 + i] : x[i]) + __shfl_xor_sync(0xffffffffu, up4 ? x[i] : x[4 + i], 16);
#pragma unroll
        for (int i = 0; i < 2; ++i) z[i] = (up2 ? y[2 + i] : y[i]) + __shfl_xor_sync(0xffffffffu, up2 ? y[i] : y[2 + i], 8);
        const float sum = (up1 ? z[1] : z[0]) + __shfl_xor_sync(0xffffffffu, up1 ? z[0] : z[1], 4);
        float u = b * (v - a * sum);  // in lanes 0 to 15
        u = __shfl_sync(0xffffffffu, u, lane & 15);
        const float o = fmaf(a, sum, dot * u);
        const f32x2 a2 = dup(a);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const f32x2 uc = dup(__shfl_sync(0xffffffffu, u, c * 4 + (lane & 3)));
#pragma unroll
            for (int r = 0; r < R / 2; ++r) s[r][c] = fma2(k[r], uc, mul2(a2, s[r][c]));
        }
        return o;
    }
};

// R consecutive values of a row as pairs of fp32.
template <typename T, int R, bool WIDE>
__device__ __forceinline__ void load_pairs(const T *p, f32x2 (&x)[R / 2]) {
    if constexpr (WIDE) {
        constexpr int V = R * sizeof(T) >= 16 ? 16 / sizeof(T) : R;
#pragma unroll
        for (int i = 0; i < R; i += V) {
            const Pack<T, V> w = load_pack<T, V>(p + i);
#pragma unroll
            for (int j = 0; j < V; j += 2) x[(i + j) / 2] = pair(to_float(w.e[j]), to_float(w.e[j + 1]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < R; i += 2) x[i / 2] = pair(to_float(p[i]), to_float(p[i + 1]));
    }
}

// One token of every sequence. A block: one value head of one sequence, or part of its columns.
template <typename T, int DK, bool WIDE>
__global__ void __launch_bounds__(64) delta_token_kernel(DeltaParams p) {
    constexpr int R = DK / 8;
    const int lane = threadIdx.x & 31, rl = lane >> 2;
    const int warps = p.dv / kCols;
    const long long w = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int slice = (int)(w % warps);
    const long long nh = w / warps;
    const int h = (int)(nh % p.hv);
    const long long n = nh / p.hv;
    if (n >= p.seqs.n_seqs) return;
    const int c0 = slice * kCols + (lane & 3) * 4, hk = h / p.per;
    const long long from = p.init_idx ? state_slot(p.init_idx, p.pool, (int)n, p.err) : n;
    const long long to = p.fin_idx ? state_slot(p.fin_idx, p.pool, (int)n, p.err) : from;
    const size_t at = ((size_t)h * DK + rl * R) * p.dv + c0, one = (size_t)p.hv * DK * p.dv;
    Tile<R> S;
    if (from >= 0) S.load(p.init + from * one + at, p.dv); else S.clear();
    f32x2 k[R / 2], q[R / 2];
    load_pairs<T, R, WIDE>(static_cast<const T *>(p.k) + n * p.ks + hk * DK + rl * R, k);
    load_pairs<T, R, WIDE>(static_cast<const T *>(p.q) + n * p.qs + hk * DK + rl * R, q);
    const int col = c0 + (rl & 3);
    const float v = to_float(static_cast<const T *>(p.v)[n * p.vs + (size_t)h * p.dv + col]);
    const float a = expf(log_decay(p.g[n * p.hv + h])), b = p.beta[n * p.hv + h];
    const float o = S.step(k, q, v, a, b, lane);
    if (lane >= 16) static_cast<T *>(p.o)[(n * p.hv + h) * p.dv + col] = from_float<T>(o);
    if (to >= 0) S.store(p.fin + to * one + at, p.dv);
}

__device__ __forceinline__ void copy_async(void *to, const void *from, int bytes) {
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    if (bytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// ---- whole sequences, row by row. A block of W warps: one value head of one sequence, 16 W of its columns. The rows come through a ring of stages of 8
// tokens in shared memory, so a token's latency holds none of HBM's.
template <typename T, int DK, int W>
struct Stage {
    T k[kStage][DK], q[kStage][DK], v[kStage][W * kCols];
    float g[kStage], b[kStage];
};

template <typename T, int DK, int W, bool WIDE>
__device__ __forceinline__ void fill(Stage<T, DK, W> &s, const DeltaParams &p, long long row, int m, int h, int c0) {
    const int hk = h / p.per, tid = threadIdx.x;
    const T *k = static_cast<const T *>(p.k) + hk * DK, *q = static_cast<const T *>(p.q) + hk * DK;
    const T *v = static_cast<const T *>(p.v) + (size_t)h * p.dv + c0;
    constexpr int V = WIDE ? 16 / sizeof(T) : 1, KV = DK / V, VV = W * kCols / V;
    for (int i = tid; i < m * (2 * KV + VV); i += W * 32) {
        const int t = i / (2 * KV + VV), j = i % (2 * KV + VV);
        const T *from = j < KV ? k + (row + t) * p.ks + j * V : j < 2 * KV ? q + (row + t) * p.qs + (j - KV) * V
                                                                       : v + (row + t) * p.vs + (j - 2 * KV) * V;
        T *to = j < KV ? &s.k[t][j * V] : j < 2 * KV ? &s.q[t][(j - KV) * V] : &s.v[t][(j - 2 * KV) * V];
        if constexpr (WIDE) copy_async(to, from, 16); else *to = *from;
    }
    if (tid < 2 * m) {
        const int t = tid >> 1;
        copy_async(tid & 1 ? &s.b[t] : &s.g[t], (tid & 1 ? p.beta : p.g) + (row + t) * p.hv + h, 4);
    }
}

// `kept` non-null: the state before every chunk of 16 rows goes there (number of first_chunk).
template <typename T, int DK, int W, bool WIDE>
__global__ void __launch_bounds__(W * 32) delta_rows_kernel(DeltaParams p, float *kept) {
    constexpr int R = DK / 8;
    extern __shared__ __align__(16) unsigned char raw[];
    Stage<T, DK, W> *ring = reinterpret_cast<Stage<T, DK, W> *>(raw);
    const int lane = threadIdx.x & 31, rl = lane >> 2, warp = threadIdx.x >> 5;
    const int slices = p.dv / (W * kCols);
    const int slice = blockIdx.x % slices, h = (blockIdx.x / slices) % p.hv, n = blockIdx.x / slices / p.hv;
    const int c0 = slice * W * kCols;
    long long begin, end;
    if (!rows_of(p, n, begin, end)) return;
    const long long from = p.init ? state_slot(p.init_idx, p.pool, n, p.err) : -1;
    const size_t at = ((size_t)h * DK + rl * R) * p.dv + c0 + warp * kCols + (lane & 3) * 4, one = (size_t)p.hv * DK * p.dv;
    Tile<R> S;
    if (from >= 0) S.load(p.init + from * one + at, p.dv); else S.clear();

    const int stages = (int)((end - begin + kStage - 1) / kStage);
    auto tokens = [&](int i) { return (int)min((long long)kStage, end - begin - (long long)i * kStage); };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        if (i < stages) fill<T, DK, W, WIDE>(ring[i], p, begin + (long long)i * kStage, tokens(i), h, c0);
        copies_commit();
    }
    const int col = warp * kCols + (lane & 3) * 4 + (rl & 3);
    for (int i = 0; i < stages; ++i) {
        copies_wait<kStages - 2>();
        __syncthreads();  // stage i is here, and everyone is done with stage i - 1
        const int ahead = i + kStages - 1;
        if (ahead < stages) fill<T, DK, W, WIDE>(ring[ahead % kStages], p, begin + (long long)ahead * kStage, tokens(ahead), h, c0);
        copies_commit();
        if (kept && i * kStage % kC == 0) S.store(kept + (first_chunk(begin, n, kC) + i * kStage / kC) * one + at, p.dv);
        const Stage<T, DK, W> &s = ring[i % kStages];
        const int m = tokens(i);
        const float a8 = expf(log_decay(s.g[lane & 7])), b8 = s.b[lane & 7];  // of the stage's tokens, those behind its end unused
        for (int t = 0; t < m; ++t) {
            f32x2 k[R / 2], q[R / 2];
            load_pairs<T, R, true>(&s.k[t][rl * R], k);
            load_pairs<T, R, true>(&s.q[t][rl * R], q);
            const float a = __shfl_sync(0xffffffffu, a8, t), b = __shfl_sync(0xffffffffu, b8, t);
            const float o = S.step(k, q, to_float(s.v[t][col]), a, b, lane);
            if (p.o && lane >= 16)
                static_cast<T *>(p.o)[((begin + (long long)i * kStage + t) * p.hv + h) * p.dv + c0 + col] = from_float<T>(o);
        }
    }
    const long long to = p.fin ? state_slot(p.fin_idx, p.pool, n, p.err) : -1;
    if (to >= 0) S.store(p.fin + to * one + at, p.dv);
}

// ---- whole sequences, in chunks of 16 rows. With G the sum of the log-decays up to a row in the chunk, D_ij = exp(G_i - G_j), E_i = exp(G_i),
// F_i = exp(G_C - G_i), S the state before the chunk and A_ij = b_i D_ij k_i.k_j (j < i), P_ij = D_ij q_i.k_j (j <= i):
//     (I + A) U = b (V - E K S),   O = E Q S + P U,   S <- exp(G_C) S + (F K)^T U
// A block: 32 columns of one (sequence, value head). Warps 0-3 hold the state, a lane 4 columns of a sixteenth of the rows, and solve for U by
// substitution, lane = column, each warp for itself; warps 4-7 load the chunks and make the next one's A, P and decays. Bound by
// latency, one warp per scheduler that goes from the products over sums and substitution to the update: 2.6 us per chunk with heads of 64, 3.5 us
// with 128 (16 rows one by one: 5.6 and 6.9). With one column and a quarter of the rows per lane heads of 128 took 3.8 us.
constexpr int kSlice = 32, kHalf = 128;

template <int DK>
struct ChunkShared {
    float k[2][kC][DK + 4], q[2][kC][DK + 4], v[2][kC][kSlice];
    float A[2][kC][kC];  // [j][i]: columns
    float P[2][kC][kC];
    float b[2][kC], E[2][kC], F[2][kC];
    float G[kC], rest[kC];  // sums of the log-decays in two fp32 values
    float part[2][4][kC][kSlice];
    float fu[4][kC][kSlice];  // per warp: F U
};

__device__ __forceinline__ void half_sync(int which) { asm volatile("bar.sync %0, 128;" ::"r"(which + 1) : "memory"); }

// A chunk's rows on their way, in the registers of 128 threads.
template <typename T, int DK, bool WIDE>
struct ChunkRows {
    static constexpr int V = WIDE ? 16 / (int)sizeof(T) : 1, KP = kC * DK / V, VP = kC * kSlice / V;
    static constexpr int KN = (KP + kHalf - 1) / kHalf, VN = (VP + kHalf - 1) / kHalf;
    Pack<T, V> k[KN], q[KN], v[VN];
    float g, b;

    // Rows [row, row + m) of key head hk and of 32 value columns from `col` of a row; zeros behind them.
    __device__ __forceinline__ void load(const DeltaParams &p, long long row, int m, int h, int c0, int t) {
        const T *kp = static_cast<const T *>(p.k) + h / p.per * DK, *qp = static_cast<const T *>(p.q) + h / p.per * DK;
        const T *vp = static_cast<const T *>(p.v) + (size_t)h * p.dv + c0;
        Pack<T, V> zero;
#pragma unroll
        for (int j = 0; j < V; ++j) zero.e[j] = from_float<T>(0.f);
#pragma unroll
        for (int e = 0; e < KN; ++e) {
            const int at = t + kHalf * e, r = at / (DK / V), x = at % (DK / V) * V;
            const bool there = at < KP && r < m;
            k[e] = there ? load_pack<T, V>(kp + (row + r) * p.ks + x) : zero;
            q[e] = there ? load_pack<T, V>(qp + (row + r) * p.qs + x) : zero;
        }
#pragma unroll
        for (int e = 0; e < VN; ++e) {
            const int at = t + kHalf * e, r = at / (kSlice / V), x = at % (kSlice / V) * V;
            v[e] = at < VP && r < m ? load_pack<T, V>(vp + (row + r) * p.vs + x) : zero;
        }
        g = t < m ? log_decay(p.g[(row + t) * p.hv + h]) : 0.f;  // m <= 16
        b = t < m ? p.beta[(row + t) * p.hv + h] : 0.f;
    }
    __device__ __forceinline__ static void put(float *to, const Pack<T, V> &x) {
        float f[V];
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = to_float(x.e[j]);
        store_floats<V>(to, f);
    }
    __device__ __forceinline__ void store(ChunkShared<DK> &s, int buf, int t) const {
#pragma unroll
        for (int e = 0; e < KN; ++e) {
            const int at = t + kHalf * e, r = at / (DK / V), x = at % (DK / V) * V;
            if (at < KP) {
                put(&s.k[buf][r][x], k[e]);
                put(&s.q[buf][r][x], q[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < VN; ++e) {
            const int at = t + kHalf * e, r = at / (kSlice / V), x = at % (kSlice / V) * V;
            if (at < VP) put(&s.v[buf][r][x], v[e]);
        }
        if (t < 32) {
            // Sums of up to 16 decays in two fp32 values, so that differences of neighbours behind strong decays stay exact.
            float G = g, r = 0.f;
#pragma unroll
            for (int d = 1; d < kC; d *= 2) {
                const float x = __shfl_up_sync(0xffffffffu, G, d, kC), y = __shfl_up_sync(0xffffffffu, r, d, kC);
                if ((t & 15) >= d) {
                    const float sum = __fadd_rn(G, x), w = __fsub_rn(sum, G);
                    r = __fadd_rn(__fadd_rn(r, y), __fadd_rn(__fsub_rn(G, __fsub_rn(sum, w)), __fsub_rn(x, w)));
                    G = sum;
                }
            }
            const float Gc = __shfl_sync(0xffffffffu, G, kC - 1, kC), rc = __shfl_sync(0xffffffffu, r, kC - 1, kC);
            if (t < kC) {
                s.G[t] = G;
                s.rest[t] = r;
                s.b[buf][t] = b;
                s.E[buf][t] = expf(G + r);
                s.F[buf][t] = expf(__fadd_rn(__fsub_rn(Gc, G), __fsub_rn(rc, r)));
            }
        }
    }
};

__device__ __forceinline__ float dot4(const float4 a, const float4 b, float c) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}
// A and P of the chunk in `buf`: thread (i, j), for j and j + 8.
template <int DK>
__device__ __forceinline__ void chunk_pairs(ChunkShared<DK> &s, int buf, int t) {
    const int i = t >> 3, j = t & 7;
    float kk[2] = {0.f, 0.f}, qk[2] = {0.f, 0.f};
#pragma unroll 4
    for (int x = 0; x < DK; x += 4) {
        const float4 ki = *reinterpret_cast<const float4 *>(&s.k[buf][i][x]), qi = *reinterpret_cast<const float4 *>(&s.q[buf][i][x]);
        const float4 kj = *reinterpret_cast<const float4 *>(&s.k[buf][j][x]);
        kk[0] = dot4(ki, kj, kk[0]);
        qk[0] = dot4(qi, kj, qk[0]);
        if (i >= 8) {  // whole warps
            const float4 kj8 = *reinterpret_cast<const float4 *>(&s.k[buf][j + 8][x]);
            kk[1] = dot4(ki, kj8, kk[1]);
            qk[1] = dot4(qi, kj8, qk[1]);
        }
    }
    const float G = s.G[i], r = s.rest[i], b = s.b[buf][i];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int c = j + 8 * e;
        const float D = c <= i ? expf(__fadd_rn(__fsub_rn(G, s.G[c]), __fsub_rn(r, s.rest[c]))) : 0.f;
        s.A[buf][c][i] = c < i ? b * D * kk[e] : 0.f;
        s.P[buf][i][c] = c <= i ? D * qk[e] : 0.f;
    }
}

// KEEP: no outputs, but the state before every chunk goes to `kept` (number of first_chunk).
template <typename T, int DK, bool WIDE, bool KEEP>
__global__ void __launch_bounds__(2 * kHalf, 2) delta_chunks_kernel(DeltaParams p, float *kept) {
    constexpr int R = DK / 16;  // rows of a lane
    extern __shared__ __align__(16) unsigned char raw[];
    auto &s = *reinterpret_cast<ChunkShared<DK> *>(raw);
    const int slices = p.dv / kSlice;
    const int slice = blockIdx.x % slices, h = (blockIdx.x / slices) % p.hv, n = blockIdx.x / slices / p.hv;
    const int c0 = slice * kSlice;
    long long begin, end;
    if (!rows_of(p, n, begin, end)) return;
    const int chunks = (int)((end - begin + kC - 1) / kC);
    auto rows_in = [&](int c) { return (int)min((long long)kC, end - begin - (long long)c * kC); };
    if (threadIdx.x >= kHalf) {
        const int t = threadIdx.x - kHalf;
        ChunkRows<T, DK, WIDE> next;
        if (chunks > 0) next.load(p, begin, rows_in(0), h, c0, t);
        for (int c = 0; c <= chunks; ++c) {  // makes chunk c beside the work on chunk c - 1
            if (c < chunks) {
                next.store(s, c & 1, t);
                if (c + 1 < chunks) next.load(p, begin + (long long)(c + 1) * kC, rows_in(c + 1), h, c0, t);
                half_sync(1);
                chunk_pairs<DK>(s, c & 1, t);
            }
            __syncthreads();
        }
        return;
    }
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, rg = lane >> 3, c4 = (lane & 7) * 4, r0 = (4 * w + rg) * R;
    const long long from = p.init ? state_slot(p.init_idx, p.pool, n, p.err) : -1;
    const size_t at = ((size_t)h * DK + r0) * p.dv + c0 + c4, one = (size_t)p.hv * DK * p.dv;
    Tile<R> S;
    if (from >= 0) S.load(p.init + from * one + at, p.dv); else S.clear();
    // This lane's rows of a row of K or Q.
    auto row = [&](const float *from, f32x2 (&x)[R / 2]) {
        if constexpr (R == 2) {
            x[0] = *reinterpret_cast<const f32x2 *>(from + r0);
        } else {
#pragma unroll
            for (int e = 0; e < R / 2; e += 2) {
                const ulonglong2 two = *reinterpret_cast<const ulonglong2 *>(from + r0 + 2 * e);
                x[e] = two.x;
                x[e + 1] = two.y;
            }
        }
    };
    // Sums over the lanes' row groups of four rows of products, which leave row rg with this lane.
    const bool up = lane & 16, odd = lane & 8;
    auto join = [&](const float (&x)[4][4]) {
        float y[2][4], z[4];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int j = 0; j < 4; ++j) y[e][j] = (up ? x[2 + e][j] : x[e][j]) + __shfl_xor_sync(0xffffffffu, up ? x[e][j] : x[2 + e][j], 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = (odd ? y[1][j] : y[0][j]) + __shfl_xor_sync(0xffffffffu, odd ? y[0][j] : y[1][j], 8);
        return make_float4(z[0], z[1], z[2], z[3]);
    };
    __syncthreads();  // chunk 0 is made
    for (int c = 0; c < chunks; ++c) {
        const int buf = c & 1, m = rows_in(c);
        if constexpr (KEEP) S.store(kept + (size_t)(first_chunk(begin, n, kC) + c) * one + at, p.dv);
        // K S and Q S over this lane's rows of S, then over the warp's
#pragma unroll
        for (int r = 0; r < kC; r += 4) {
#pragma unroll
            for (int which = 0; which < (KEEP ? 1 : 2); ++which) {
                float sums[4][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f32x2 x[R / 2];
                    row(which ? s.q[buf][r + e] : s.k[buf][r + e], x);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        f32x2 sum = mul2(x[0], S.s[0][j]);
#pragma unroll
                        for (int i = 1; i < R / 2; ++i) sum = fma2(x[i], S.s[i][j], sum);
                        float lo, hi;
                        unpair(sum, lo, hi);
                        sums[e][j] = lo + hi;
                    }
                }
                *reinterpret_cast<float4 *>(&s.part[which][w][r + rg][c4]) = join(sums);
            }
        }
        half_sync(0);
        float u[kC];
#pragma unroll
        for (int i = 0; i < kC; ++i) {
            const float ks = (s.part[0][0][i][lane] + s.part[0][1][i][lane]) + (s.part[0][2][i][lane] + s.part[0][3][i][lane]);
            u[i] = s.b[buf][i] * (s.v[buf][i][lane] - s.E[buf][i] * ks);
        }
#pragma unroll
        for (int j = 0; j < kC - 1; ++j)
#pragma unroll
            for (int i4 = (j + 1) & ~3; i4 < kC; i4 += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(&s.A[buf][j][i4]);
                const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (i4 + e > j) u[i4 + e] = fmaf(-av[e], u[j], u[i4 + e]);
            }
        if constexpr (!KEEP) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // rows w, w + 4, ...: about the same work in every warp
                const int i = 4 * e + w;
                const float qs = (s.part[1][0][i][lane] + s.part[1][1][i][lane]) + (s.part[1][2][i][lane] + s.part[1][3][i][lane]);
                float o = s.E[buf][i] * qs;
#pragma unroll
                for (int j = 0; j < 4 * e + 4; ++j)
                    if (j <= i) o = fmaf(s.P[buf][i][j], u[j], o);
                if (i < m) static_cast<T *>(p.o)[((begin + (long long)c * kC + i) * p.hv + h) * p.dv + c0 + lane] = from_float<T>(o);
            }
        }
#pragma unroll
        for (int j = 0; j < kC; ++j)  // rows behind the sequence leave even a state that is not finite as it is
            s.fu[w][j][lane] = j < m ? s.F[buf][j] * u[j] : 0.f;
        __syncwarp();
        const f32x2 whole = dup(s.E[buf][kC - 1]);
#pragma unroll
        for (int i = 0; i < R / 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) S.s[i][j] = mul2(whole, S.s[i][j]);
#pragma unroll
        for (int t = 0; t < kC; ++t) {
            f32x2 k[R / 2];
            row(s.k[buf][t], k);
            const float4 f = *reinterpret_cast<const float4 *>(&s.fu[w][t][c4]);
            const f32x2 fu[4] = {dup(f.x), dup(f.y), dup(f.z), dup(f.w)};
#pragma unroll
            for (int i = 0; i < R / 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) S.s[i][j] = fma2(k[i], fu[j], S.s[i][j]);
        }
        __syncthreads();  // chunk c + 1 is made, and everyone is done with chunk c
    }
    const long long to = p.fin ? state_slot(p.fin_idx, p.pool, n, p.err) : -1;
    if (to >= 0) S.store(p.fin + to * one + at, p.dv);
}

template <typename T, int DK, bool WIDE>
cudaError_t launch_token(const DeltaParams &p, cudaStream_t s) {
    const long long warps = (long long)p.seqs.n_seqs * p.hv * (p.dv / kCols);
    // Two warps per block: 256 sequences of 32 heads of 128 take 158 us (171 with eight), one takes 4.8 us (6.2).
    delta_token_kernel<T, DK, WIDE><<<(unsigned)((warps + 1) / 2), 64, 0, s>>>(p);
    return cudaGetLastError();
}

// Blocks of `columns` columns.
template <typename F>
cudaError_t launch_sequences(F *f, const DeltaParams &p, float *kept, int columns, int threads, size_t bytes, cudaStream_t s) {
    if (bytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e != cudaSuccess) return e;
    }
    f<<<(unsigned)((long long)p.seqs.n_seqs * p.hv * (p.dv / columns)), threads, bytes, s>>>(p, kept);
    return cudaGetLastError();
}

// Chunks of 16 rows where their blocks are few and a token's latency is what counts, else row by row, whose many warps hide it. fp32, heads of 128 (of
// 64), row by row and in chunks: 256 rows in 8 blocks 113 and 60 us (92 and 43), in 304 115 and 90 (92 and 66), in 608 162 and 174 (115 and 125), in
// 2432 561 and 690; 16 rows in 304 blocks 12.3 and 12.3 (10.3 and 10.3), 32 rows 20.5 and 16.8, 8 rows 8.2 and 12.3.
constexpr int kChunkBlocks = 2;  // per SM

template <typename T, int DK, bool WIDE>
cudaError_t launch_rows(const DeltaParams &p, float *kept, int sms, cudaStream_t s) {
    const long long blocks = (long long)p.seqs.n_seqs * p.hv * (p.dv / kSlice);
    if (blocks > (long long)kChunkBlocks * sms || p.seqs.rows < (long long)kC * p.seqs.n_seqs)
        return launch_sequences(&delta_rows_kernel<T, DK, 2, WIDE>, p, kept, 2 * kCols, 64, sizeof(Stage<T, DK, 2>) * kStages, s);
    auto *f = kept ? &delta_chunks_kernel<T, DK, WIDE, true> : &delta_chunks_kernel<T, DK, WIDE, false>;
    return launch_sequences(f, p, kept, kSlice, 2 * kHalf, sizeof(ChunkShared<DK>), s);
}

template <typename T>
bool wide_rows(const DeltaParams &p) {
    auto ok = [](const void *x, long long stride) { return aligned16(x) && stride * (long long)sizeof(T) % 16 == 0; };
    return ok(p.q, p.qs) && ok(p.k, p.ks) && ok(p.v, p.vs);
}

template <typename T, typename F>
cudaError_t by_size(const DeltaParams &p, F f) {
    const bool wide = wide_rows<T>(p);
    switch (p.dk) {
        case 32: return wide ? f.template operator()<T, 32, true>() : f.template operator()<T, 32, false>();
        case 64: return wide ? f.template operator()<T, 64, true>() : f.template operator()<T, 64, false>();
        case 128: return wide ? f.template operator()<T, 128, true>() : f.template operator()<T, 128, false>();
        default: return cudaErrorInvalidValue;
    }
}

struct Token {
    const DeltaParams &p;
    cudaStream_t s;
    template <typename T, int DK, bool WIDE>
    cudaError_t operator()() const { return launch_token<T, DK, WIDE>(p, s); }
};
struct Rows {
    const DeltaParams &p;
    float *kept;
    int sms;
    cudaStream_t s;
    template <typename T, int DK, bool WIDE>
    cudaError_t operator()() const { return launch_rows<T, DK, WIDE>(p, kept, sms, s); }
};

}  // namespace

DeltaParams delta_params(const kda_delta_args &a, void *o, float *final_state, unsigned *err) {
    DeltaParams p{};
    p.q = a.q;
    p.k = a.k;
    p.v = a.v;
    p.qs = a.q_stride ? a.q_stride : (long long)a.k_heads * a.dk;
    p.ks = a.k_stride ? a.k_stride : (long long)a.k_heads * a.dk;
    p.vs = a.v_stride ? a.v_stride : (long long)a.v_heads * a.dv;
    p.g = a.g;
    p.beta = a.beta;
    p.seqs = Seqs{a.cu_seqlens, a.cu_seqlens ? a.n_seqs : a.B, a.T, (long long)a.B * a.T};
    p.hk = a.k_heads;
    p.hv = a.v_heads;
    p.per = a.v_heads / a.k_heads;
    p.dk = a.dk;
    p.dv = a.dv;
    p.init = a.initial_state;
    p.init_idx = a.initial_state_indices;
    p.fin_idx = a.final_state_indices;
    p.pool = a.state_pool_size;
    p.o = o;
    p.fin = final_state;
    p.err = err;
    return p;
}

cudaError_t launch_delta_rows(kda_dtype dtype, const DeltaParams &p, float *kept, int sms, cudaStream_t s) {
    const Rows f{p, kept, sms, s};
    return dtype == KDA_BF16 ? by_size<__nv_bfloat16>(p, f) : by_size<float>(p, f);
}

cudaError_t launch_delta_decode(const kda_delta_args &a, float *state, void *o, unsigned *err, cudaStream_t s) {
    DeltaParams p = delta_params(a, o, state, err);
    p.init = state;
    const Token f{p, s};
    return a.dtype == KDA_BF16 ? by_size<__nv_bfloat16>(p, f) : by_size<float>(p, f);
}

// bf16 prompts of fewer rows than this on average are computed in fp32 here: a chunk of 64 rows takes the tensor-core kernel the same time whatever it
// holds. 32 heads of 128, sequences of 16 rows: 10.3 us here and 14.4 there for one, 131 and 160 for 64; of 32 rows: 14.4 and 14.4, 252 and 162. The
// average does not see a long sequence among many short ones, which then goes row by row: a prompt of 4096 rows packed with 255 single tokens
// takes 2.0 ms, the two apart 0.35 and 0.10 ms.
constexpr int kFewestRows = 20;

size_t delta_prefill_workspace_bytes(const kda_delta_args &a, int) {
    const DeltaParams p = delta_params(a, nullptr, nullptr, nullptr);
    return delta_tc_shape(a.dtype, p, kFewestRows) ? delta_tc_order_bytes(p) : 0;
}

cudaError_t launch_delta_prefill(const kda_delta_args &a, void *o, float *final_state, void *ws, int sms, unsigned *err, cudaStream_t s) {
    DeltaParams p = delta_params(a, o, final_state, err);
    if (!delta_tc_supported(a.dtype, p, kFewestRows)) return launch_delta_rows(a.dtype, p, nullptr, sms, s);
    const cudaError_t e = launch_delta_tc_order(p, ws, s);
    return e != cudaSuccess ? e : launch_delta_tc(p, s);
}

}  // namespace kda
