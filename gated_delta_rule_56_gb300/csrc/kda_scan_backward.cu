// kda_scan_backward.cu -- gradients of the selective scan.
//
// With dy' = dy z sigmoid(z) (or dy), g_t = dL/dh_t and a_t = exp(dt_t A):
//     g_t = C_t dy'_t + a_{t+1} g_{t+1}                 (at a sequence's end: + the final state's gradient)
//     dC_t[n] = sum_c dy'_t h_t,    dB_t[n] = sum_c g_t dt_t x_t          (over the channels of the group)
//     dx_t = D dy'_t + dt_t sum_n g_t B_t,   ddt'_t = sum_n g_t (A a_t h_{t-1} + B_t x_t)
//     dA = sum_t g_t dt_t a_t h_{t-1},  dD = sum_t dy'_t x_t,  the initial state's gradient: a_first g_first.
//
// The rows are cut into chunks as for prompts. Kernels: (1) forward over every chunk from zeros, keeping the state before
// every 8th row (4 N / 8 bytes per row and channel; keeping all would be 4 N), and the walk over the chunks' end
// states; (2) the same backwards for the gradients at the states after each chunk, where chunks are joined at all;
// (3) the main kernel, every chunk from its last window of 8 rows to its first; (4) sums over the blocks' parts.
//
// Main kernel: a thread holds a tile of 4 channels x 4 states, a warp N / 4 of those along the states and the rest along
// the channels. The sums over channels (dB, dC) and over states (dx, ddt, y) are both taken in the thread's registers first;
// tiles that are narrow in one direction move 1.3 times as many values between lanes. A window's states are recomputed from
// the kept one, and those before every second row are held in shared memory, each thread its own; the row between is
// recomputed from its decay, which the way back needs anyway. That is 15 multiply-adds and 1.75 exponentials per (row, channel,
// state). With the whole window unrolled and its states in registers the kernel was twice as slow: spills and a
// loop that did not fit the instruction cache.
// Measured: 4 sequences of 2048 rows x 4096 channels x 16 states in bf16 with gate: 1.11 ms (forward 145 us, backward ends 131 us,
// main kernel 793 us, the walks and the sums 36 us). The main kernel issues 436 warp instructions per 32 channels and row at 46 % of the
// issue slots: two blocks per SM hide its latencies no better, and its 234 registers allow no third. A loop that prepares the
// next window beside the passes over this one, with one barrier less, took the same time. In shared memory two blocks fit for 9 to 128
// states in bf16 (114 KB at 16) and 17 to 128 in fp32; the other sizes (130 to 183 KB) run one: fp32 with 16 states 1.65 ms, bf16 with 4 and 8
// states 0.90 and 1.10 ms.
//
// dA, dD and the bias's gradient are plain fp32 within a chunk (dA in one accumulator per thread, the others per window of 8 rows and then
// over the chunk) and compensated over the chunks: 1.0e-6, 1.6e-7 and 3.8e-7 off 64 bits in the 2-norm, with sums in 64 bits (and
// all else in fp32) 0.9e-6, 0.6e-7 and 2.8e-7.
#include <algorithm>

#include "kda_scan.cuh"

namespace kda {
namespace {

constexpr int kWarps = kScanThreads / 32;
constexpr int kRows = kScanWindow;

struct GradParams {
    const void *dy;
    const float *d_fin;
    float *dx, *ddt, *dz, *d_init;
    float *part_B, *part_C;     // [blocks per group][rows][G][N]
    float *part_A;              // [chunks][C][N]
    float *part_D, *part_bias;  // [chunks][C]
    const float *after;         // [chunks][C][N]: gradient at the state after a chunk whose last sequence goes on, or nullptr
};

// EC channels x EN states per thread, NL lanes along the states.
template <int EC, int EN, int NL>
struct Shape {
    static constexpr int EC_ = EC, EN_ = EN;
    static constexpr int NP = EN * NL, CL = 32 / NL, CH = kWarps * CL * EC, PARTS = kWarps * CL;
};

template <typename T, typename SH>
struct Shared {
    alignas(16) T raw[2][4][kRows][SH::CH];       // x, dt, dy, z as they are in memory
    alignas(16) float pre[3][kRows][SH::CH];      // dt', dy', u = dt' x; u's place takes the sum of g B when its row is done
    alignas(16) float sum[2][kRows][SH::CH];      // over the states: g a h A, C h
    alignas(16) float bc[kRows][2][SH::NP][2];    // B and C, every value twice: one for each channel of a pair
    alignas(16) float part[kRows][2][SH::PARTS][SH::NP];  // dB and dC of each thread's channels
    alignas(16) float4 kept[2][SH::EC_ * SH::EN_ / 4][kScanThreads];  // the state before a window, per thread
    alignas(16) ulonglong2 states[2][SH::EC_ * SH::EN_ / 4][kScanThreads];  // the states before rows 2 and 4, per thread
    alignas(16) ulonglong2 first[SH::EC_ * SH::EN_ / 4][kScanThreads];      // the state before the chunk, per thread
    alignas(16) float time[2][SH::CH];                                      // from the chunk's first row to the window's
};

__device__ __forceinline__ void copy16(void *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((unsigned)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}

template <typename T, int EC, int EN, int NL, bool WIDE>
__global__ void __launch_bounds__(kScanThreads, 2) scan_backward_kernel(ScanParams p, GradParams q, ScanPlan plan, Carries carry) {
    using SH = Shape<EC, EN, NL>;
    constexpr int NP = SH::NP, CL = SH::CL, CH = SH::CH, PARTS = SH::PARTS, PAIRS = EC / 2;
    extern __shared__ __align__(16) unsigned char memory[];
    Shared<T, SH> &sm = *reinterpret_cast<Shared<T, SH> *>(memory);
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, nl = lane % NL, cl = lane / NL;
    const int per = p.C / p.G, blocks = (per + CH - 1) / CH;
    const int g = blockIdx.y / blocks, blk = blockIdx.y % blocks;
    const int first_k = blk * CH;                       // the block's first channel in the group
    const int tile_k = (warp * CL + cl) * EC, n0 = nl * EN;  // the thread's first channel in the block, its first state
    const int chunk = blockIdx.x;
    const long long r0 = chunk * plan.rows, stop = min(r0 + plan.rows, p.seqs.rows);
    const long long chunk_states = (long long)p.C * p.N;
    if (r0 >= stop) return;

    // A tensor [C][N] at the thread's tile; pairs run along the channels.
    auto load_tile = [&](const float *from, f32x2(&to)[PAIRS][EN], float scale) {
#pragma unroll
        for (int j = 0; j < PAIRS; ++j)
#pragma unroll
            for (int i = 0; i < EN; ++i) {
                float v[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int k = first_k + tile_k + 2 * j + e;
                    v[e] = k < per && n0 + i < p.N ? from[(long long)(g * per + k) * p.N + n0 + i] * scale : 0.f;
                }
                to[j][i] = pair(v[0], v[1]);
            }
    };
    auto store_tile = [&](float *to, const f32x2(&from)[PAIRS][EN]) {
#pragma unroll
        for (int j = 0; j < PAIRS; ++j)
#pragma unroll
            for (int i = 0; i < EN; ++i) {
                float v[2];
                unpair(from[j][i], v[0], v[1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int k = first_k + tile_k + 2 * j + e;
                    if (k < per && n0 + i < p.N) to[(long long)(g * per + k) * p.N + n0 + i] = v[e];
                }
            }
    };
    f32x2 A[PAIRS][EN], dA[PAIRS][EN], gr[PAIRS][EN], h[PAIRS][EN];
    load_tile(p.A, A, kLog2e);
#pragma unroll
    for (int j = 0; j < PAIRS; ++j)
#pragma unroll
        for (int i = 0; i < EN; ++i) dA[j][i] = gr[j][i] = 0;
    auto tile_or_zero = [&](const float *from, f32x2(&to)[PAIRS][EN]) {
        if (from) {
            load_tile(from, to, 1.f);
        } else {
#pragma unroll
            for (int j = 0; j < PAIRS; ++j)
#pragma unroll
                for (int i = 0; i < EN; ++i) to[j][i] = 0;
        }
    };
    auto of_sequence = [&](const float *all, long long row) {  // a state tensor's part of the sequence of a row
        return all ? all + p.seqs.at(row) * chunk_states : nullptr;
    };
    if (q.after && p.seqs.end(p.seqs.at(stop - 1)) > stop) load_tile(q.after + chunk * chunk_states, gr, 1.f);

    const T *X = static_cast<const T *>(p.x), *DT = static_cast<const T *>(p.dt), *Z = static_cast<const T *>(p.z);
    const T *DY = static_cast<const T *>(q.dy);
    const T *Bm = static_cast<const T *>(p.Bm) + g * p.N, *Cm = static_cast<const T *>(p.Cm) + g * p.N;
    const int c0 = g * per + first_k;
    const bool vectors = p.N % 4 == 0;  // the workspace's states lie on 16-byte boundaries
    auto bring = [&](long long w0, int buf) {  // a window's rows into shared memory
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (t == 3 && !Z) break;
            const T *from = (t == 0 ? X : t == 1 ? DT : t == 2 ? DY : Z) + c0;
            const long long stride = t == 0 ? p.x_stride : t == 1 ? p.dt_stride : t == 2 ? p.C : p.z_stride;
            constexpr int VALUES = WIDE ? 16 / sizeof(T) : 1, WORDS = CH / VALUES;
            for (int i = tid; i < kRows * WORDS; i += kScanThreads) {
                const int u = i / WORDS, k = (i % WORDS) * VALUES;
                if (w0 + u >= stop || first_k + k >= per) continue;
                if constexpr (WIDE)
                    copy16(&sm.raw[buf][t][u][k], from + (w0 + u) * stride + k);
                else
                    sm.raw[buf][t][u][k] = from[(w0 + u) * stride + k];
            }
        }
        // The state that was kept before the window: a thread brings what it will read itself.
        const float *kept = carry.kept + (chunk * plan.windows() + (w0 - r0) / kRows) * chunk_states;
#pragma unroll
        for (int e = 0; e < EC; ++e) {
            const int k = first_k + tile_k + e;
            const float *from = kept + (long long)(g * per + k) * p.N + n0;
#pragma unroll
            for (int i = 0; i < EN; i += 4) {
                float4 *to = &sm.kept[buf][(e * EN + i) / 4][tid];
                if (vectors && k < per && n0 + i + 4 <= p.N) {
                    copy16(to, from + i);
                } else {
                    float v[4];
#pragma unroll
                    for (int o = 0; o < 4; ++o) v[o] = k < per && n0 + i + o < p.N ? from[i + o] : 0.f;
                    *to = make_float4(v[0], v[1], v[2], v[3]);
                }
            }
        }
        if (plan.carries) {
            const float *from = carry.kept_time + (chunk * plan.windows() + (w0 - r0) / kRows) * p.C + c0;
            for (int k = tid; k < CH; k += kScanThreads)
                if (first_k + k < per)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((unsigned)__cvta_generic_to_shared(&sm.time[buf][k])),
                                 "l"(from + k)
                                 : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    // A thread's channels in the passes over (row, channel): one if the block has at most as many channels as threads.
    constexpr int OWN = CH > kScanThreads ? CH / kScanThreads : 1;
    float sum_D[OWN], sum_bias[OWN];
#pragma unroll
    for (int i = 0; i < OWN; ++i) sum_D[i] = sum_bias[i] = 0.f;
    float own_bias[OWN], own_skip[OWN];
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        const int k = (i * kScanThreads + tid) % CH;
        const bool in = first_k + k < per;
        own_bias[i] = in && p.dt_bias ? p.dt_bias[c0 + k] : 0.f;
        own_skip[i] = in && p.D ? p.D[c0 + k] : 0.f;
    }
    for (int k = tid; k < CH; k += kScanThreads)  // channels past the group's: nothing is copied there
        if (first_k + k >= per) sm.time[0][k] = sm.time[1][k] = 0.f;
    const bool joined = plan.carries && p.seqs.begin(p.seqs.at(r0)) < r0;  // the chunk's first sequence came in from before
    if (joined) {
        load_tile(carry.state + chunk * chunk_states, h, 1.f);
#pragma unroll
        for (int i = 0; i < PAIRS * EN / 2; ++i) sm.first[i][tid] = make_ulonglong2((&h[0][0])[2 * i], (&h[0][0])[2 * i + 1]);
    }

    // B and C of a window, fetched one window ahead; rows and states past the end are zeros, which leave states and gradients
    // as they are.
    constexpr int EACH = (kRows * 2 * NP + kScanThreads - 1) / kScanThreads;
    T ahead[EACH];
    auto fetch = [&](long long w0) {
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int v = i * kScanThreads + tid, n = v % NP, side = v / NP % 2;
            const long long row = w0 + v / (2 * NP);
            ahead[i] = v < kRows * 2 * NP && row < stop && n < p.N
                           ? (side ? Cm[row * p.C_stride + n] : Bm[row * p.B_stride + n]) : from_float<T>(0.f);
        }
    };
    long long w = (stop - r0 - 1) / kRows;
    bring(r0 + w * kRows, 0);
    fetch(r0 + w * kRows);
    long long begin = 0, end = -1;  // of the sequence last looked at
    for (int buf = 0; w >= 0; --w, buf ^= 1) {
        const long long w0 = r0 + w * kRows, w1 = min(w0 + kRows, stop);
        const int rows = (int)(w1 - w0);
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int v = i * kScanThreads + tid;
            if (v < kRows * 2 * NP) {
                const float f = to_float(ahead[i]);
                *reinterpret_cast<float2 *>(sm.bc[v / (2 * NP)][v / NP % 2][v % NP]) = make_float2(f, f);
            }
        }
        // Rows of the window that begin or end a sequence, as bits; none where the window lies inside one.
        unsigned begins = 0, ends = 0;
        if (!(begin < w0 && w1 < end)) {
            int n = p.seqs.at(w0);
            begin = p.seqs.begin(n);
            end = p.seqs.end(n);
            if (begin == w0) begins |= 1u;
            for (; n < p.seqs.n_seqs && p.seqs.end(n) < w1; ++n) {
                const long long b = p.seqs.end(n);
                if (b > w0) {
                    begins |= 1u << (int)(b - w0);
                    ends |= 1u << (int)(b - w0 - 1);
                }
            }
            if (n < p.seqs.n_seqs && p.seqs.end(n) == w1) ends |= 1u << (rows - 1);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // the window's rows are there, and the last window's sums are read
        if (w > 0) {
            bring(w0 - kRows, buf ^ 1);
            fetch(w0 - kRows);
        }
        // dt', u and dy' per (row, channel), two at a time.
        constexpr int ITEMS_P = (kRows * CH + kScanThreads - 1) / kScanThreads;
#pragma unroll
        for (int i = 0; i < ITEMS_P; i += 2) {
            float x[2], dt[2], dy[2], z[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int v = (i + e) * kScanThreads + tid, u = v / CH, k = v % CH;
                const bool in = (ITEMS_P > 1 || e == 0) && u < rows && first_k + k < per;
                x[e] = in ? to_float(sm.raw[buf][0][u][k]) : 0.f;
                dt[e] = in ? to_float(sm.raw[buf][1][u][k]) + own_bias[(i + e) % OWN] : 0.f;
                dy[e] = in ? to_float(sm.raw[buf][2][u][k]) : 0.f;
                z[e] = in && Z ? to_float(sm.raw[buf][3][u][k]) : 0.f;
            }
            f32x2 dt2 = pair(dt[0], dt[1]), dy2 = pair(dy[0], dy[1]);
            if (p.softplus) dt2 = softplus2(dt2);
            if (Z) dy2 = mul2(dy2, silu2(pair(z[0], z[1])));
            unpair(dt2, dt[0], dt[1]);
            unpair(dy2, dy[0], dy[1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int v = (i + e) * kScanThreads + tid, u = v / CH, k = v % CH;
                if ((ITEMS_P == 1 && e == 1) || u >= kRows) break;
                const bool in = u < rows && first_k + k < per;
                sm.pre[0][u][k] = in ? dt[e] : 0.f;
                sm.pre[1][u][k] = dy[e];
                sm.pre[2][u][k] = in ? dt[e] * x[e] : 0.f;
            }
        }
        // The state before the window: the kept one, and what the state before the chunk has become by then.
#pragma unroll
        for (int j = 0; j < PAIRS; ++j)
#pragma unroll
            for (int i = 0; i < EN; i += 4) {
                const float4 v = sm.kept[buf][(2 * j * EN + i) / 4][tid], o = sm.kept[buf][((2 * j + 1) * EN + i) / 4][tid];
                h[j][i] = pair(v.x, o.x);
                h[j][i + 1] = pair(v.y, o.y);
                h[j][i + 2] = pair(v.z, o.z);
                h[j][i + 3] = pair(v.w, o.w);
            }
        if (joined && begin < r0) {
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) {
                const f32x2 t2 = *reinterpret_cast<const f32x2 *>(&sm.time[buf][tile_k + 2 * j]);
#pragma unroll
                for (int i = 0; i < EN; i += 2) {
                    const ulonglong2 v = sm.first[(j * EN + i) / 2][tid];
                    h[j][i] = carried2(t2, A[j][i], v.x, h[j][i]);
                    h[j][i + 1] = carried2(t2, A[j][i + 1], v.y, h[j][i + 1]);
                }
            }
        }
        __syncthreads();

        auto row_pairs = [&](int what, int u, f32x2(&to)[PAIRS]) {
#pragma unroll
            for (int j = 0; j < PAIRS; ++j) to[j] = *reinterpret_cast<const f32x2 *>(&sm.pre[what][u][tile_k + 2 * j]);
        };
        auto row_states = [&](int side, int u, f32x2(&to)[EN]) {
#pragma unroll
            for (int i = 0; i < EN; ++i) to[i] = *reinterpret_cast<const f32x2 *>(sm.bc[u][side][n0 + i]);
        };
        // Tiles in the thread's own places of shared memory: before row 0 where the kept state was, then rows 2 and 4.
        auto place = [&](int q2) {
            return q2 == 0 ? reinterpret_cast<ulonglong2 *>(&sm.kept[buf][0][tid]) : &sm.states[q2 - 1][0][tid];
        };
        constexpr int WORDS = PAIRS * EN / 2;
        auto save = [&](int q2) {
            ulonglong2 *to = place(q2);
            f32x2 *flat = &h[0][0];
#pragma unroll
            for (int i = 0; i < WORDS; ++i) to[i * kScanThreads] = make_ulonglong2(flat[2 * i], flat[2 * i + 1]);
        };
        auto restore = [&](int q2) {
            const ulonglong2 *from = place(q2);
            f32x2 *flat = &h[0][0];
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                const ulonglong2 v = from[i * kScanThreads];
                flat[2 * i] = v.x;
                flat[2 * i + 1] = v.y;
            }
        };
        if (begins & 1u) tile_or_zero(of_sequence(p.init, w0), h);
#pragma unroll 1
        for (int u = 0; u < kRows - 2; ++u) {  // up to the state before row 6
            if (u % 2 == 0) save(u / 2);
            f32x2 dt[PAIRS], uu[PAIRS], b[EN];
            row_pairs(0, u, dt);
            row_pairs(2, u, uu);
            row_states(0, u, b);
#pragma unroll
            for (int j = 0; j < PAIRS; ++j)
#pragma unroll
                for (int i = 0; i < EN; ++i) h[j][i] = fma2(decay2(dt[j], A[j][i]), h[j][i], mul2(uu[j], b[i]));
            if (begins >> (u + 1) & 1u) tile_or_zero(of_sequence(p.init, w0 + u + 1), h);
        }
#pragma unroll 1
        for (int q2 = kRows / 2 - 1; q2 >= 0; --q2) {
            if (q2 < kRows / 2 - 1) restore(q2);
            // Row u0's decay and the state after it, which is the one before row u0 + 1 unless a sequence begins there.
            const int u0 = 2 * q2;
            f32x2 a0[PAIRS][EN], mid[PAIRS][EN];
            {
                f32x2 dt[PAIRS], uu[PAIRS], b[EN];
                row_pairs(0, u0, dt);
                row_pairs(2, u0, uu);
                row_states(0, u0, b);
#pragma unroll
                for (int j = 0; j < PAIRS; ++j)
#pragma unroll
                    for (int i = 0; i < EN; ++i) {
                        a0[j][i] = decay2(dt[j], A[j][i]);
                        mid[j][i] = fma2(a0[j][i], h[j][i], mul2(uu[j], b[i]));
                    }
            }
            if (begins >> (u0 + 1) & 1u) tile_or_zero(of_sequence(p.init, w0 + u0 + 1), mid);
#pragma unroll
            for (int e = 1; e >= 0; --e) {
                const int u = u0 + e;
                if (ends >> u & 1u) tile_or_zero(of_sequence(q.d_fin, w0 + u), gr);
                f32x2 dt[PAIRS], uu[PAIRS], b[EN], dy[PAIRS], cc[EN], gB[PAIRS], gA[PAIRS], out[PAIRS], dB[EN], dC[EN];
                row_pairs(0, u, dt);
                row_pairs(2, u, uu);
                row_states(0, u, b);
                row_pairs(1, u, dy);
                row_states(1, u, cc);
#pragma unroll
                for (int j = 0; j < PAIRS; ++j)
#pragma unroll
                    for (int i = 0; i < EN; ++i) {
                        const f32x2 before = e ? mid[j][i] : h[j][i];
                        const f32x2 a = e ? decay2(dt[j], A[j][i]) : a0[j][i];
                        const f32x2 after = fma2(a, before, mul2(uu[j], b[i]));
                        f32x2 gg = fma2(cc[i], dy[j], gr[j][i]);
                        dC[i] = j == 0 ? mul2(dy[j], after) : fma2(dy[j], after, dC[i]);
                        dB[i] = j == 0 ? mul2(gg, uu[j]) : fma2(gg, uu[j], dB[i]);
                        gB[j] = i == 0 ? mul2(gg, b[i]) : fma2(gg, b[i], gB[j]);
                        out[j] = i == 0 ? mul2(cc[i], after) : fma2(cc[i], after, out[j]);
                        gg = mul2(gg, a);
                        gr[j][i] = gg;
                        const f32x2 kept = mul2(gg, before);
                        dA[j][i] = fma2(kept, dt[j], dA[j][i]);
                        gA[j] = i == 0 ? mul2(kept, A[j][i]) : fma2(kept, A[j][i], gA[j]);
                    }
                // Over the thread's channels, to be added over the block's threads below.
                float sB[EN], sC[EN];
#pragma unroll
                for (int i = 0; i < EN; ++i) {
                    float lo, hi;
                    unpair(dB[i], lo, hi);
                    sB[i] = lo + hi;
                    unpair(dC[i], lo, hi);
                    sC[i] = lo + hi;
                }
                store_floats<EN>(&sm.part[u][0][warp * CL + cl][n0], sB);
                store_floats<EN>(&sm.part[u][1][warp * CL + cl][n0], sC);
                // Over the states' lanes: each step halves the channels that a lane keeps.
                float v[3][EC];
#pragma unroll
                for (int j = 0; j < PAIRS; ++j) {
                    unpair(gB[j], v[0][2 * j], v[0][2 * j + 1]);
                    unpair(gA[j], v[1][2 * j], v[1][2 * j + 1]);
                    unpair(out[j], v[2][2 * j], v[2][2 * j + 1]);
                }
                constexpr int FOLD = NL < EC ? NL : EC;  // lanes that share out the channels
                int offset = 0;
#pragma unroll
                for (int t = 0; t < 3; ++t) {
#pragma unroll
                    for (int m = NL / 2; m >= FOLD && m > 0; m >>= 1)
#pragma unroll
                        for (int k = 0; k < EC; ++k) v[t][k] += __shfl_xor_sync(0xffffffffu, v[t][k], m);
                    int count = EC;
                    offset = 0;
#pragma unroll
                    for (int m = FOLD / 2; m > 0; m >>= 1) {
                        count /= 2;
                        const bool upper = nl & m;
#pragma unroll
                        for (int k = 0; k < EC / 2; ++k) {
                            if (k >= count) break;
                            const float keep = upper ? v[t][count + k] : v[t][k], send = upper ? v[t][k] : v[t][count + k];
                            v[t][k] = keep + __shfl_xor_sync(0xffffffffu, send, m);
                        }
                        if (upper) offset += count;
                    }
                    if (nl < FOLD) {
#pragma unroll
                        for (int k = 0; k < EC / FOLD; ++k) (t == 0 ? sm.pre[2] : sm.sum[t - 1])[u][tile_k + offset + k] = v[t][k];
                    }
                }
                if (begins >> u & 1u) {
                    if (q.d_init) store_tile(const_cast<float *>(of_sequence(q.d_init, w0 + u)), gr);
                }
            }
        }
        __syncthreads();

        // Per (row, channel), two at a time. Long sums are taken in two levels, a window's and then the chunk's.
        float part_D[OWN], part_bias[OWN];
#pragma unroll
        for (int i = 0; i < OWN; ++i) part_D[i] = part_bias[i] = 0.f;
        const long long at0 = w0 * p.C + c0;
#pragma unroll
        for (int i = 0; i < ITEMS_P; i += 2) {
            float x[2], dt[2], dy[2], raw[2], gB[2], gA[2];
            bool in[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int v = (i + e) * kScanThreads + tid, u = ITEMS_P == 1 && e == 1 ? kRows : v / CH, k = v % CH;
                in[e] = u < rows && first_k + k < per;
                const int u_ = in[e] ? u : 0, k_ = in[e] ? k : 0;
                x[e] = to_float(sm.raw[buf][0][u_][k_]);
                raw[e] = to_float(sm.raw[buf][1][u_][k_]) + own_bias[(i + e) % OWN];
                dt[e] = sm.pre[0][u_][k_];
                dy[e] = sm.pre[1][u_][k_];
                gB[e] = sm.pre[2][u_][k_];
                gA[e] = sm.sum[0][u_][k_];
            }
            const f32x2 x2 = pair(x[0], x[1]), gB2 = pair(gB[0], gB[1]), dy2 = pair(dy[0], dy[1]);
            const f32x2 skip2 = pair(own_skip[i % OWN], own_skip[(i + 1) % OWN]);
            f32x2 ddt2 = fma2(gB2, x2, mul2(pair(gA[0], gA[1]), both(0.69314718f)));  // A was taken with log2(e)
            if (p.softplus) ddt2 = mul2(ddt2, sigmoid2(pair(raw[0], raw[1])));
            float dx[2], ddt[2];
            unpair(fma2(gB2, pair(dt[0], dt[1]), mul2(dy2, skip2)), dx[0], dx[1]);
            unpair(ddt2, ddt[0], ddt[1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int v = (i + e) * kScanThreads + tid, u = v / CH, k = v % CH;
                if (!in[e]) continue;
                q.dx[at0 + (long long)u * p.C + k] = dx[e];
                q.ddt[at0 + (long long)u * p.C + k] = ddt[e];
                part_D[(i + e) % OWN] = fmaf(dy[e], x[e], part_D[(i + e) % OWN]);
                part_bias[(i + e) % OWN] += ddt[e];
            }
            if (Z) {
                float z[2], dy0[2], out[2], dz[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int v = (i + e) * kScanThreads + tid, u = in[e] ? v / CH : 0, k = in[e] ? v % CH : 0;
                    z[e] = to_float(sm.raw[buf][3][u][k]);
                    dy0[e] = to_float(sm.raw[buf][2][u][k]);
                    out[e] = sm.sum[1][u][k];
                }
                const f32x2 z2 = pair(z[0], z[1]), s2 = sigmoid2(z2), y2 = fma2(skip2, x2, pair(out[0], out[1]));
                const f32x2 slope = mul2(s2, fma2(z2, fma2(s2, both(-1.f), both(1.f)), both(1.f)));  // of z sigmoid(z)
                unpair(mul2(mul2(pair(dy0[0], dy0[1]), y2), slope), dz[0], dz[1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int v = (i + e) * kScanThreads + tid;
                    if (in[e]) q.dz[at0 + (long long)(v / CH) * p.C + v % CH] = dz[e];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            sum_D[i] += part_D[i];
            sum_bias[i] += part_bias[i];
        }
        // dB and dC of the block's channels: four states per thread, the parts shared out over SPLIT lanes.
        constexpr int ITEMS = kRows * 2 * NP / 4, SPLIT = ITEMS < kScanThreads ? kScanThreads / ITEMS : 1;
#pragma unroll
        for (int i = tid; i < ITEMS * SPLIT; i += kScanThreads) {
            const int n = i % (NP / 4) * 4, s = i / (NP / 4) % SPLIT, side = i / (NP / 4 * SPLIT) % 2, u = i / (NP / 4 * SPLIT * 2);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < PARTS / SPLIT; ++k) {
                const float4 o = *reinterpret_cast<const float4 *>(&sm.part[u][side][k * SPLIT + s][n]);
                v.x += o.x;
                v.y += o.y;
                v.z += o.z;
                v.w += o.w;
            }
#pragma unroll
            for (int m = SPLIT / 2; m > 0; m >>= 1) {
                v.x += __shfl_xor_sync(0xffffffffu, v.x, m * (NP / 4));
                v.y += __shfl_xor_sync(0xffffffffu, v.y, m * (NP / 4));
                v.z += __shfl_xor_sync(0xffffffffu, v.z, m * (NP / 4));
                v.w += __shfl_xor_sync(0xffffffffu, v.w, m * (NP / 4));
            }
            if (s != 0 || u >= rows) continue;
            float *to = (side ? q.part_C : q.part_B) + (((long long)blk * p.seqs.rows + w0 + u) * p.G + g) * p.N + n;
            const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (n + k < p.N) to[k] = e[k];
        }
    }
    store_tile(q.part_A + chunk * chunk_states, dA);
    // dD and ddt_bias: the threads that share a channel, in order.
    __syncthreads();
    float *both = &sm.pre[0][0][0];
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        both[i * kScanThreads + tid] = sum_D[i];
        both[(OWN + i) * kScanThreads + tid] = sum_bias[i];
    }
    __syncthreads();
    for (int k = tid; k < CH && first_k + k < per; k += kScanThreads) {
        float d = 0.f, s = 0.f;
        for (int i = k; i < OWN * kScanThreads; i += CH) {
            d += both[i];
            s += both[OWN * kScanThreads + i];
        }
        q.part_D[(long long)chunk * p.C + c0 + k] = d;
        q.part_bias[(long long)chunk * p.C + c0 + k] = s;
    }
}

// out[i] = sum over j < count of in[j][i], in order, for the five tensors of partial sums in one launch.
struct Sums {
    const float *in[5];
    float *out[5];
    long long size[5];
    int count[5];
    unsigned first[6];  // the first block of each
};
__global__ void __launch_bounds__(128) scan_reduce_kernel(Sums s) {
    int t = 0;
    while (t < 4 && blockIdx.x >= s.first[t + 1]) ++t;
    const long long i = (long long)(blockIdx.x - s.first[t]) * 128 + threadIdx.x, size = s.size[t];
    if (i >= size) return;
    const float *in = s.in[t] + i;
    ExactSum sum;
#pragma unroll 16
    for (int j = 0; j < s.count[t]; ++j) sum.add(in[j * size]);
    s.out[t][i] = sum.value();
}

// The initial-state gradients of empty sequences are their final states'.
__global__ void scan_empty_kernel(Seqs seqs, long long size, const float *__restrict__ d_fin, float *__restrict__ d_init) {
    const int n = blockIdx.x;
    if (seqs.begin(n) != seqs.end(n)) return;
    for (long long i = threadIdx.x; i < size; i += blockDim.x) d_init[n * size + i] = d_fin ? d_fin[n * size + i] : 0.f;
}

template <typename F>
cudaError_t by_states(int N, F &&f) {
    if (N <= 4) return f.template operator()<2, 4, 1>();
    if (N <= 8) return f.template operator()<4, 4, 2>();
    if (N <= 16) return f.template operator()<4, 4, 4>();
    if (N <= 32) return f.template operator()<4, 4, 8>();
    if (N <= 64) return f.template operator()<4, 4, 16>();
    if (N <= 128) return f.template operator()<4, 4, 32>();
    return f.template operator()<2, 8, 32>();
}

struct ChannelsOf {
    template <int EC, int EN, int NL>
    cudaError_t operator()() {
        channels = Shape<EC, EN, NL>::CH;
        return cudaSuccess;
    }
    int channels = 0;
};

int blocks_per_group(const kda_scan_args &a) {
    ChannelsOf c;
    by_states(a.N, c);
    return (a.D / a.G + c.channels - 1) / c.channels;
}

struct BackwardLaunch {
    kda_dtype dtype;
    ScanParams p;
    GradParams q;
    ScanPlan plan;
    Carries carry;
    bool wide;
    int blocks;
    cudaStream_t s;
    template <typename T, int EC, int EN, int NL, bool WIDE>
    cudaError_t launch() {
        constexpr int bytes = sizeof(Shared<T, Shape<EC, EN, NL>>);
        auto *kernel = scan_backward_kernel<T, EC, EN, NL, WIDE>;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        kernel<<<dim3((unsigned)plan.chunks, (unsigned)blocks), kScanThreads, bytes, s>>>(p, q, plan, carry);
        return cudaGetLastError();
    }
    template <int EC, int EN, int NL>
    cudaError_t operator()() {
        if (dtype == KDA_BF16)
            return wide ? launch<__nv_bfloat16, EC, EN, NL, true>() : launch<__nv_bfloat16, EC, EN, NL, false>();
        return wide ? launch<float, EC, EN, NL, true>() : launch<float, EC, EN, NL, false>();
    }
};

// Whole sequences where they give every SM three blocks; otherwise chunks that give it four, of at least 64 rows: two full waves where two
// blocks are resident, which is what was measured (16 states in bf16), and four where shared memory holds one.
ScanPlan backward_plan(const kda_scan_args &a, int sms) {
    const long long rows = (long long)a.B * a.T, blocks = (long long)blocks_per_group(a) * a.G;
    if (rows == 0) return ScanPlan{0, 1, false};
    if (sms <= 0) sms = 152;
    if (!a.cu_seqlens && (a.B * blocks >= 3 * sms || a.T <= 64)) return ScanPlan{a.B, a.T, false};
    const long long most = (rows + 63) / 64, chunks = std::max(1LL, std::min(most, 4LL * sms / blocks));
    const long long per = ((rows + chunks - 1) / chunks + kRows - 1) / kRows * kRows;
    const int count = (int)((rows + per - 1) / per);
    return ScanPlan{count, per, count > 1};
}

struct Layout {
    GradParams q{};
    Carries forward{}, back{};
    size_t bytes = 0;
};

Layout layout(const kda_scan_args &a, const ScanPlan &plan, char *ws) {
    const long long rows = (long long)a.B * a.T;
    const size_t states = (size_t)a.D * a.N, chunks = plan.chunks, windows = chunks * plan.windows();
    const int blocks = blocks_per_group(a);
    Layout l;
    auto take = [&](size_t count) {
        float *r = reinterpret_cast<float *>(ws + l.bytes);
        l.bytes += (count * sizeof(float) + 255) / 256 * 256;
        return r;
    };
    l.forward.kept = take(windows * states);
    l.forward.kept_time = take(windows * a.D);
    l.forward.state = take(chunks * states);
    l.forward.time = take(chunks * a.D);
    if (plan.carries) {
        l.back.state = take(chunks * states);
        l.back.time = take(chunks * a.D);
    }
    l.q.part_B = take((size_t)blocks * rows * a.G * a.N);
    l.q.part_C = take((size_t)blocks * rows * a.G * a.N);
    l.q.part_A = take(chunks * states);
    l.q.part_D = take(chunks * a.D);
    l.q.part_bias = take(chunks * a.D);
    return l;
}

}  // namespace

size_t scan_backward_workspace_bytes(const kda_scan_args &a, int sms) {
    return layout(a, backward_plan(a, sms), nullptr).bytes;
}

cudaError_t launch_scan_backward(const kda_scan_args &a, const kda_scan_grads &g, void *ws, int sms, unsigned *err,
                                 cudaStream_t s) {
    const ScanPlan plan = backward_plan(a, sms);
    const Layout l = layout(a, plan, static_cast<char *>(ws));
    const ScanParams p = scan_params(a, err);
    GradParams q = l.q;
    q.dy = g.dy;
    q.d_fin = g.d_final_state;
    q.dx = g.dx;
    q.ddt = g.ddt;
    q.dz = g.dz;
    q.d_init = g.d_initial_state;
    const int blocks = blocks_per_group(a);
    cudaError_t e = cudaSuccess;
    if (plan.chunks > 0) {
        if ((e = launch_scan_states(a, plan, l.forward, err, s)) != cudaSuccess) return e;
        if (plan.carries) {
            if ((e = launch_scan_back_ends(a, g.dy, g.d_final_state, plan, l.back, err, s)) != cudaSuccess) return e;
            q.after = l.back.state;
        }
        const int e16 = a.dtype == KDA_BF16 ? 8 : 4;  // values in 16 bytes
        const bool wide = aligned16(p.x) && aligned16(p.dt) && aligned16(p.z) && aligned16(q.dy) && (a.D / a.G) % e16 == 0 &&
                          p.x_stride % e16 == 0 && p.dt_stride % e16 == 0 && (!p.z || p.z_stride % e16 == 0);
        if ((e = by_states(a.N, BackwardLaunch{a.dtype, p, q, plan, l.forward, wide, blocks * a.G, s})) != cudaSuccess) return e;
    }
    const long long rows = p.seqs.rows;
    const long long states = (long long)a.D * a.N;
    Sums sums{{q.part_B, q.part_C, q.part_A, q.part_D, q.part_bias},
              {g.dB, g.dC, g.dA, g.dDskip, g.ddt_bias},
              {rows * a.G * a.N, rows * a.G * a.N, states, a.D, a.D},
              {blocks, blocks, plan.chunks, plan.chunks, plan.chunks},
              {}};
    for (int t = 0; t < 5; ++t) {
        if (!sums.out[t]) sums.size[t] = 0;
        sums.first[t + 1] = sums.first[t] + (unsigned)((sums.size[t] + 127) / 128);
    }
    scan_reduce_kernel<<<sums.first[5], 128, 0, s>>>(sums);  // dA at least
    if (g.d_initial_state && p.seqs.n_seqs > 0 && (a.cu_seqlens || a.T == 0))
        scan_empty_kernel<<<(unsigned)p.seqs.n_seqs, 256, 0, s>>>(p.seqs, (long long)a.D * a.N, g.d_final_state, g.d_initial_state);
    return cudaGetLastError();
}

}  // namespace kda
