// kda_delta_backward.cu -- gradients of the delta rule with one decay per value head: the kernel for every size and type.
//
// Chunks of C = 16 rows of a sequence, S0 the state before the chunk and dS the gradient of the state behind it. With G the sum of the
// log-decays up to a row in the chunk, D_ij = exp(G_i - G_j), E_i = exp(G_i), F_i = exp(G_C - G_i):
//     A_ij = b_i D_ij k_i.k_j (j < i),  P_ij = D_ij q_i.k_j (j <= i)
//     (I + A) U = R,  R_i = b_i (v_i - E_i S0^T k_i)            the values that the chunk writes
//     dU = P^T dO + F K dS,   (I + A)^T dR = dU,   dv = b dR
//     Gp = D lower(dO U^T),   Ga = -D strict(dR U^T)
//     dq = E dO S0^T + Gp K
//     dk = b row + col,  row = Ga K - E dR S0^T (through k_i of the row itself),  col = F U dS^T + Gp^T Q + Ga^T (b K)
//     db_i = dR_i.v_i + k_i.row_i
//     dg_t = sum over the pairs j < t <= i of (dO_i.u_j) P_ij - (dR_i.u_j) A_ij, + sum_{i >= t} E_i (q_i.(S0 dO_i) - b_i k_i.(S0 dR_i))
//            + sum_{j < t} F_j k_j.(dS u_j) + exp(G_C) <S0, dS>
//     dS <- exp(G_C) dS + sum_i E_i (q_i dO_i^T - b_i k_i dR_i^T)
// dg_t is a sum of those terms alone whose decay has row t's in it, so behind a strong decay it is as small as they are. (As a sum of
// q.dq + b k.row - k.col over the rows from t on it would be the rest of terms of size 1: at g = -12 a tenth of it lost in fp32, at -20 all.)
// No division, so b = 0 and decays of 0 are ordinary values. All of it is fp32; the states before the chunks come from a run of the
// recurrence before this kernel (kda_delta.cu).
//
// One block per (sequence, value head), the chunks from the last to the first with S0 and dS in shared memory. Bound by the
// latency of its phases (ten barriers per chunk; 6 products of 16 rows with a state, whose operands come out of shared memory), a path for fp32 and
// for short sequences: 1501 rows in 9 sequences, 8 heads of 64, fp32: 253 us in a captured graph where the longest
// sequence has 252 rows, 468 us where it has 490 (15 us per chunk of it, a sixth of that for the states before the chunks).
#include "kda_delta.cuh"
#include "kda_delta_tc.h"
#include "kda_layers.h"

namespace kda {

DeltaParams delta_params(const kda_delta_args &a, void *o, float *final_state, unsigned *err);
cudaError_t launch_delta_rows(kda_dtype dtype, const DeltaParams &p, float *kept, int sms, cudaStream_t s);

namespace {

constexpr int kC = 16;
constexpr int kThreads = 256;

struct BackParams {
    DeltaParams f;
    const void *d_o;
    const float *d_fin, *kept;
    float *dq, *dk, *dv, *dg, *db, *d_init;  // dq, dk: [rows, value heads, dk]
};

__device__ __forceinline__ float dot4(const float4 a, const float4 b, float c) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}

template <int DK, int DV>
struct BackShared {
    float S0[DK][DV + 4], dS[DK][DV + 4];
    float k[kC][DK + 4], q[kC][DK + 4];
    float v[kC][DV + 4], d_o[kC][DV + 4], u[kC][DV + 4], dr[kC][DV + 4];
    float A[kC][kC + 1], P[kC][kC + 1], Gp[kC][kC + 1], Ga[kC][kC + 1];
    float cross[kC][kC + 1];  // [i][t]: row i's pairs with the rows before t
    float G[kC], E[kC], F[kC], b[kC], g[kC];
    float sums[8][3][kC];
    float joined[8];
};

// Threads (c, part): column c of 16 / PARTS rows each.
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(kThreads) delta_back_kernel(BackParams p) {
    extern __shared__ __align__(16) unsigned char raw[];
    auto &s = *reinterpret_cast<BackShared<DK, DV> *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.x % p.f.hv, n = blockIdx.x / p.f.hv, hk = h / p.f.per;
    const int hv = p.f.hv;
    long long begin, end;
    if (!rows_of(p.f, n, begin, end)) return;
    constexpr int VR = kC * DV / kThreads, KR = kC * DK / kThreads;  // rows of a thread's value column, of its key column
    const int vc = tid % DV, v0 = tid / DV * VR, kc = tid % DK, k0 = tid / DK * KR;
    const size_t one = (size_t)DK * DV, state = ((size_t)n * hv + h) * one;

    for (int i = tid; i < (int)one; i += kThreads) s.dS[i / DV][i % DV] = p.d_fin ? p.d_fin[state + i] : 0.f;
    const int chunks = (int)((end - begin + kC - 1) / kC);
    const long long chunk0 = first_chunk(begin, n, kC);
    const T *qp = static_cast<const T *>(p.f.q), *kp = static_cast<const T *>(p.f.k), *vp = static_cast<const T *>(p.f.v);
    const T *dop = static_cast<const T *>(p.d_o);
    for (int ch = chunks - 1; ch >= 0; --ch) {
        const long long row0 = begin + (long long)ch * kC;
        const int m = (int)min((long long)kC, end - row0);
        __syncthreads();
        const float *S0 = p.kept + ((size_t)(chunk0 + ch) * hv + h) * one;
        {  // all of a chunk's loads in flight before the first store
            constexpr int NS = DK * DV / 4 / kThreads, NK = kC * DK / kThreads, NV = kC * DV / kThreads;
            float4 st[NS];
            T k[NK], q[NK], v[NV], d[NV];
#pragma unroll
            for (int e = 0; e < NS; ++e) st[e] = reinterpret_cast<const float4 *>(S0)[tid + kThreads * e];
#pragma unroll
            for (int e = 0; e < NK; ++e) {
                const int r = (tid + kThreads * e) / DK, c = (tid + kThreads * e) % DK;
                k[e] = r < m ? kp[(row0 + r) * p.f.ks + hk * DK + c] : from_float<T>(0.f);
                q[e] = r < m ? qp[(row0 + r) * p.f.qs + hk * DK + c] : from_float<T>(0.f);
            }
#pragma unroll
            for (int e = 0; e < NV; ++e) {
                const int r = (tid + kThreads * e) / DV, c = (tid + kThreads * e) % DV;
                v[e] = r < m ? vp[(row0 + r) * p.f.vs + (size_t)h * DV + c] : from_float<T>(0.f);
                d[e] = r < m ? dop[((row0 + r) * hv + h) * DV + c] : from_float<T>(0.f);
            }
#pragma unroll
            for (int e = 0; e < NS; ++e) {
                const int i = (tid + kThreads * e) * 4;
                *reinterpret_cast<float4 *>(&s.S0[i / DV][i % DV]) = st[e];
            }
#pragma unroll
            for (int e = 0; e < NK; ++e) {
                const int r = (tid + kThreads * e) / DK, c = (tid + kThreads * e) % DK;
                s.k[r][c] = to_float(k[e]);
                s.q[r][c] = to_float(q[e]);
            }
#pragma unroll
            for (int e = 0; e < NV; ++e) {
                const int r = (tid + kThreads * e) / DV, c = (tid + kThreads * e) % DV;
                s.v[r][c] = to_float(v[e]);
                s.d_o[r][c] = to_float(d[e]);
            }
        }
        if (warp == 0) {
            const bool live = lane < m;
            s.b[lane & 15] = 0.f;
            __syncwarp();
            if (live) s.b[lane] = p.f.beta[(row0 + lane) * hv + h];
            float G = live ? log_decay(p.f.g[(row0 + lane) * hv + h]) : 0.f;
            // Sums of up to 16 decays in two fp32 values, so that differences of neighbours behind strong decays stay exact.
            float rest = 0.f;
#pragma unroll
            for (int d = 1; d < kC; d *= 2) {
                const float x = __shfl_up_sync(0xffffffffu, G, d), y = __shfl_up_sync(0xffffffffu, rest, d);
                if ((lane & 15) >= d) {
                    const float t = __fadd_rn(G, x), w = __fsub_rn(t, G);
                    rest = __fadd_rn(__fadd_rn(rest, y), __fadd_rn(__fsub_rn(G, __fsub_rn(t, w)), __fsub_rn(x, w)));
                    G = t;
                }
            }
            const float Gc = __shfl_sync(0xffffffffu, G, kC - 1), rc = __shfl_sync(0xffffffffu, rest, kC - 1);
            if (lane < kC) {
                s.G[lane] = G;
                s.g[lane] = rest;
                s.E[lane] = expf(G + rest);
                s.F[lane] = expf(__fadd_rn(__fsub_rn(Gc, G), __fsub_rn(rc, rest)));
            }
        }
        __syncthreads();
        {  // A and P: thread (i, j)
            const int i = tid / kC, j = tid % kC;
            float kk = 0.f, qk = 0.f;
            if (j <= i)
#pragma unroll 4
                for (int x = 0; x < DK; x += 4) {
                    const float4 kj = *reinterpret_cast<const float4 *>(&s.k[j][x]);
                    kk = dot4(*reinterpret_cast<const float4 *>(&s.k[i][x]), kj, kk);
                    qk = dot4(*reinterpret_cast<const float4 *>(&s.q[i][x]), kj, qk);
                }
            const float D = j <= i ? expf(__fadd_rn(__fsub_rn(s.G[i], s.G[j]), __fsub_rn(s.g[i], s.g[j]))) : 0.f;
            s.A[i][j] = j < i ? s.b[i] * D * kk : 0.f;
            s.P[i][j] = j <= i ? D * qk : 0.f;
            s.Gp[i][j] = D;
        }
        {  // R, and F K dS
            float ks[VR], kd[VR];
#pragma unroll
            for (int r = 0; r < VR; ++r) ks[r] = kd[r] = 0.f;
#pragma unroll 2
            for (int x = 0; x < DK; x += 4) {
                const float a0 = s.S0[x][vc], a1 = s.S0[x + 1][vc], a2 = s.S0[x + 2][vc], a3 = s.S0[x + 3][vc];
                const float b0 = s.dS[x][vc], b1 = s.dS[x + 1][vc], b2 = s.dS[x + 2][vc], b3 = s.dS[x + 3][vc];
#pragma unroll
                for (int r = 0; r < VR; ++r) {
                    const float4 k = *reinterpret_cast<const float4 *>(&s.k[v0 + r][x]);
                    ks[r] = dot4(k, make_float4(a0, a1, a2, a3), ks[r]);
                    kd[r] = dot4(k, make_float4(b0, b1, b2, b3), kd[r]);
                }
            }
#pragma unroll
            for (int r = 0; r < VR; ++r) {
                const int i = v0 + r;
                s.u[i][vc] = s.b[i] * (s.v[i][vc] - s.E[i] * ks[r]);
                s.dr[i][vc] = s.F[i] * kd[r];
            }
        }
        __syncthreads();
        if (tid < DV) {  // (I + A) U = R
            float u[kC];
#pragma unroll
            for (int i = 0; i < kC; ++i) {
                float x = s.u[i][tid];
#pragma unroll
                for (int j = 0; j < i; ++j) x = fmaf(-s.A[i][j], u[j], x);
                u[i] = x;
            }
#pragma unroll
            for (int i = 0; i < kC; ++i) s.u[i][tid] = u[i];
        } else if (tid - DV < DV) {  // (I + A)^T dR = P^T dO + F K dS
            const int c = tid - DV;
            float d[kC];
#pragma unroll
            for (int j = kC - 1; j >= 0; --j) {
                float x = s.dr[j][c];
#pragma unroll
                for (int i = j; i < kC; ++i) x = fmaf(s.P[i][j], s.d_o[i][c], x);
#pragma unroll
                for (int i = j + 1; i < kC; ++i) x = fmaf(-s.A[i][j], d[i], x);
                d[j] = x;
            }
#pragma unroll
            for (int j = 0; j < kC; ++j) {
                s.dr[j][c] = d[j];
                if (j < m) p.dv[((row0 + j) * hv + h) * DV + c] = s.b[j] * d[j];
            }
        }
        __syncthreads();
        {  // Gp, Ga (without b): thread (i, j); D is in Gp. The products dR.v by the threads above the diagonal's.
            const int i = tid / kC, j = tid % kC;
            const float D = s.Gp[i][j];
            float gp = 0.f, ga = 0.f;
            if (j <= i)
#pragma unroll 4
                for (int x = 0; x < DV; x += 4) {
                    const float4 u = *reinterpret_cast<const float4 *>(&s.u[j][x]);
                    gp = dot4(*reinterpret_cast<const float4 *>(&s.d_o[i][x]), u, gp);
                    ga = dot4(*reinterpret_cast<const float4 *>(&s.dr[i][x]), u, ga);
                }
            s.Gp[i][j] = j <= i ? D * gp : 0.f;
            s.Ga[i][j] = j < i ? -D * ga : 0.f;
            float pairs = j < i ? fmaf(gp, s.P[i][j], -ga * s.A[i][j]) : 0.f;
#pragma unroll
            for (int d = 1; d < kC; d *= 2) {
                const float y = __shfl_up_sync(0xffffffffu, pairs, d, kC);
                if (j >= d) pairs += y;
            }
            if (j < i) s.cross[i][j + 1] = pairs;
            if (tid < kC) {
                float x = 0.f;
#pragma unroll 4
                for (int c = 0; c < DV; c += 4)
                    x = dot4(*reinterpret_cast<const float4 *>(&s.dr[tid][c]), *reinterpret_cast<const float4 *>(&s.v[tid][c]), x);
                s.g[tid] = x;
            }
        }
        __syncthreads();
        float joined = 0.f;
        {
            float os[KR], rs[KR], us[KR];
#pragma unroll
            for (int r = 0; r < KR; ++r) os[r] = rs[r] = us[r] = 0.f;
#pragma unroll 2
            for (int x = 0; x < DV; x += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(&s.S0[kc][x]), b = *reinterpret_cast<const float4 *>(&s.dS[kc][x]);
                if (k0 == 0) joined = dot4(a, b, joined);
#pragma unroll
                for (int r = 0; r < KR; ++r) {
                    os[r] = dot4(*reinterpret_cast<const float4 *>(&s.d_o[k0 + r][x]), a, os[r]);
                    rs[r] = dot4(*reinterpret_cast<const float4 *>(&s.dr[k0 + r][x]), a, rs[r]);
                    us[r] = dot4(*reinterpret_cast<const float4 *>(&s.u[k0 + r][x]), b, us[r]);
                }
            }
#pragma unroll
            for (int r = 0; r < KR; ++r) {
                const int i = k0 + r;
                const float ki = s.k[i][kc];
                float dq = s.E[i] * os[r], row = -s.E[i] * rs[r], col = s.F[i] * us[r];
                const float from = fmaf(s.q[i][kc], dq, s.b[i] * ki * row), through = ki * col;
                // Pairs beyond the diagonal are left out, not multiplied by zero: a NaN or an infinity stays with the rows that it belongs to. i is
                // the warp's.
                for (int j = 0; j < i; ++j) {
                    const float kj = s.k[j][kc];
                    dq = fmaf(s.Gp[i][j], kj, dq);
                    row = fmaf(s.Ga[i][j], kj, row);
                }
                dq = fmaf(s.Gp[i][i], ki, dq);
                col = fmaf(s.Gp[i][i], s.q[i][kc], col);
                for (int j = i + 1; j < kC; ++j) {
                    col = fmaf(s.Gp[j][i], s.q[j][kc], col);
                    col = fmaf(s.Ga[j][i] * s.b[j], s.k[j][kc], col);
                }
                if (i < m) {
                    const size_t at = ((row0 + i) * hv + h) * DK + kc;
                    p.dq[at] = dq;
                    p.dk[at] = fmaf(s.b[i], row, col);
                }
                float x[3] = {from, through, ki * row};
#pragma unroll
                for (int a = 0; a < 3; ++a) {
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) x[a] += __shfl_xor_sync(0xffffffffu, x[a], d);
                    if (lane == 0) s.sums[warp][a][i] = x[a];
                }
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) joined += __shfl_xor_sync(0xffffffffu, joined, d);
            if (lane == 0) s.joined[warp] = joined;
        }
        __syncthreads();
        const float whole = s.E[kC - 1];
        for (int i = tid; i < (int)one / 4; i += kThreads) {
            const int r = i / (DV / 4), c = i % (DV / 4) * 4;
            float4 d = *reinterpret_cast<const float4 *>(&s.dS[r][c]);
            d = make_float4(whole * d.x, whole * d.y, whole * d.z, whole * d.w);
#pragma unroll 4
            for (int j = 0; j < kC; ++j) {
                const float a = s.E[j] * s.q[j][r], b = -s.b[j] * s.E[j] * s.k[j][r];
                const float4 o = *reinterpret_cast<const float4 *>(&s.d_o[j][c]), x = *reinterpret_cast<const float4 *>(&s.dr[j][c]);
                d.x = fmaf(a, o.x, fmaf(b, x.x, d.x));
                d.y = fmaf(a, o.y, fmaf(b, x.y, d.y));
                d.z = fmaf(a, o.z, fmaf(b, x.z, d.z));
                d.w = fmaf(a, o.w, fmaf(b, x.w, d.w));
            }
            *reinterpret_cast<float4 *>(&s.dS[r][c]) = d;
        }
        if (warp == 0) {  // the sums over the key columns: the warps that hold row i
            const int i = lane & 15, w0 = i / KR * (DK / 32);
            float x[3] = {0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < DK / 32; ++w)
#pragma unroll
                for (int a = 0; a < 3; ++a) x[a] += s.sums[w0 + w][a][i];
            float inner = 0.f;
#pragma unroll
            for (int w = 0; w < DK / 32; ++w) inner += s.joined[w];
            float dg = whole * inner, before = __shfl_up_sync(0xffffffffu, x[1], 1, kC);
            if (i == 0) before = 0.f;
#pragma unroll
            for (int d = 1; d < kC; d *= 2) {  // sums over the rows from i on, and before i
                const float y = __shfl_down_sync(0xffffffffu, x[0], d, kC), z = __shfl_up_sync(0xffffffffu, before, d, kC);
                if (i + d < kC) x[0] += y;
                if (i >= d) before += z;
            }
            float across = 0.f;
            for (int r = i; r < m; ++r)
                if (i > 0) across += s.cross[r][i];
            dg += across + (x[0] + before);
            if (lane < m) {
                p.dg[(row0 + i) * hv + h] = dg;
                p.db[(row0 + i) * hv + h] = s.g[i] + x[2];
            }
        }
    }
    __syncthreads();
    if (p.d_init)
        for (int i = tid; i < (int)one; i += kThreads) p.d_init[state + i] = s.dS[i / DV][i % DV];
}

// Sums over the value heads of every key head, four values per thread.
__global__ void __launch_bounds__(256) delta_shared_kernel(const float4 *dq, const float4 *dk, float4 *dq_out, float4 *dk_out,
                                                           long long n, int line, int per) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const float4 *from = blockIdx.y ? dk : dq;
    const long long head = i / line;
    const int x = (int)(i % line);
    float4 a = from[head * per * line + x];
    for (int j = 1; j < per; ++j) {
        const float4 b = from[(head * per + j) * line + x];
        a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
    }
    (blockIdx.y ? dk_out : dq_out)[i] = a;
}

template <typename T, int DK, int DV>
cudaError_t launch_back(const BackParams &p, cudaStream_t s) {
    auto *f = &delta_back_kernel<T, DK, DV>;
    const int bytes = (int)sizeof(BackShared<DK, DV>);
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    f<<<(unsigned)((long long)p.f.seqs.n_seqs * p.f.hv), kThreads, bytes, s>>>(p);
    return cudaGetLastError();
}

template <typename T, int DK>
cudaError_t launch_back_dv(const BackParams &p, cudaStream_t s) {
    return p.f.dv == 32 ? launch_back<T, DK, 32>(p, s) : p.f.dv == 64 ? launch_back<T, DK, 64>(p, s) : launch_back<T, DK, 128>(p, s);
}

template <typename T>
cudaError_t launch_back_typed(const BackParams &p, cudaStream_t s) {
    return p.f.dk == 32 ? launch_back_dv<T, 32>(p, s) : p.f.dk == 64 ? launch_back_dv<T, 64>(p, s) : launch_back_dv<T, 128>(p, s);
}

size_t kept_floats(const kda_delta_args &a) {
    const long long rows = (long long)a.B * a.T, n = a.cu_seqlens ? a.n_seqs : a.B;
    return (size_t)(rows / kC + n) * a.v_heads * a.dk * a.dv;
}
size_t head_floats(const kda_delta_args &a) {  // one of dq, dk per value head
    return a.v_heads == a.k_heads ? 0 : (size_t)a.B * a.T * a.v_heads * a.dk;
}

}  // namespace

// bf16 sequences of fewer rows than this on average take this file's kernel. 32 heads of 128, sequences of 8 rows: 45 us here and 39 on the
// tensor cores for one, 568 and 488 for 64; 64 sequences of 64 rows: 2391 and 557. Shorter ones do not fill the chunks of 16 either.
constexpr int kFewestRows = 8;

size_t delta_backward_workspace_bytes(const kda_delta_args &a, int) {
    const DeltaParams p = delta_params(a, nullptr, nullptr, nullptr);
    // Rows that TMA cannot load take this file's kernel, which may need more or less.
    const size_t rows = kept_floats(a) * 4, tc = delta_tc_shape(a.dtype, p, kFewestRows) ? delta_tc_backward_bytes(p) : 0;
    return (tc > rows ? tc : rows) + 2 * head_floats(a) * 4;
}

cudaError_t launch_delta_backward(const kda_delta_args &a, const kda_delta_grads &g, void *ws, int sms, unsigned *err, cudaStream_t s) {
    const DeltaParams f = delta_params(a, nullptr, nullptr, err);
    if (f.seqs.n_seqs == 0) return cudaSuccess;
    const bool apart = head_floats(a) > 0, tc = delta_tc_supported(a.dtype, f, kFewestRows);
    float *heads = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + (tc ? delta_tc_backward_bytes(f) : kept_floats(a) * 4));
    float *dq = apart ? heads : g.dq, *dk = apart ? heads + head_floats(a) : g.dk;
    cudaError_t e;
    if (tc) {
        e = launch_delta_tc_backward(f, DeltaGradients{g.d_o, g.d_final_state, dq, dk, g.dv, g.dg, g.dbeta, g.d_initial_state}, ws, s);
    } else {
        float *kept = static_cast<float *>(ws);
        const BackParams p{f, g.d_o, g.d_final_state, kept, dq, dk, g.dv, g.dg, g.dbeta, g.d_initial_state};
        e = launch_delta_rows(a.dtype, f, kept, sms, s);
        if (e != cudaSuccess) return e;
        e = a.dtype == KDA_BF16 ? launch_back_typed<__nv_bfloat16>(p, s) : launch_back_typed<float>(p, s);
    }
    if (e != cudaSuccess || !apart) return e;
    const long long n = f.seqs.rows * a.k_heads * (a.dk / 4);
    if (n == 0) return cudaSuccess;
    delta_shared_kernel<<<dim3((unsigned)((n + 255) / 256), 2), 256, 0, s>>>(
        reinterpret_cast<const float4 *>(dq), reinterpret_cast<const float4 *>(dk), reinterpret_cast<float4 *>(g.dq),
        reinterpret_cast<float4 *>(g.dk), n, a.dk / 4, f.per);
    return cudaGetLastError();
}

}  // namespace kda
