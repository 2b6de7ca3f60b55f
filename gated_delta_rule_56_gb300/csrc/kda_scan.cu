// kda_scan.cu -- the selective state space scan: prompts and single tokens.
//
//     h_t[c, n] = exp(dt_t[c] A[c, n]) h_{t-1}[c, n] + dt_t[c] x_t[c] B_t[n],   y_t[c] = sum_n C_t[n] h_t[c, n] + D[c] x_t[c]
//
// Prompts: one lane per channel holds up to 16 states in registers (more states: 2 to 16 lanes per channel, their parts of y
// added by shuffles) and walks down the rows; a block's B and C rows lie in shared memory in fp32, read as broadcasts. Per
// (token, channel, state) that is 1 exponential and 4 multiply-adds: with 32 exponentials and 128 multiply-adds per SM
// and cycle both units are busy equally long and HBM waits for them.
//
// A sequence has few channels for 152 SMs, so the rows are cut into chunks that run side by side. The state after
// a chunk is linear in the state before it, h_end = exp(A sum dt) h_begin + (the end state from zeros):
// a first kernel computes the end states from zeros and the sums of dt, a second one walks over the chunks to get the
// state before each, and the main kernel runs every chunk from there. That is a second round of exponentials, and it is
// left out where whole sequences fill the GPU.
#include "kda_scan.cuh"

namespace kda {
namespace {

constexpr int kUnroll = 8;  // tokens whose inputs are loaded ahead

template <int NP>
struct Tile {  // tokens of B and C in shared memory at a time: at most 16 KB
    static constexpr int tokens = NP <= 64 ? 32 : 2048 / NP;
};

// ENDS: only the end state of the chunk's last sequence (from zeros, or from its initial state if it begins in the chunk).
template <typename T, int S, int L, bool ENDS>
__global__ void __launch_bounds__(kScanThreads, 4)
    scan_prefill_kernel(ScanParams p, T *__restrict__ y, float *fin, ScanPlan plan, Carries carry) {
    constexpr int NP = S * L, TT = Tile<NP>::tokens, SIDES = ENDS ? 1 : 2;
    constexpr int EACH = TT * SIDES * NP / kScanThreads;  // values of a tile that a thread brings
    static_assert(TT % kUnroll == 0 && TT * SIDES * NP % kScanThreads == 0, "tile");
    __shared__ __align__(16) float tile[2][TT][SIDES][NP];
    if (!ENDS && blockIdx.x == 0 && blockIdx.y == 0) check_seqs(p.seqs, p.err);
    const int per = p.C / p.G;
    const int blocks = (per * L + kScanThreads - 1) / kScanThreads;
    const int g = blockIdx.y / blocks;
    const int k = (blockIdx.y % blocks) * (kScanThreads / L) + threadIdx.x / L, n0 = (threadIdx.x % L) * S;
    const bool live = k < per;
    const int c = g * per + (live ? k : 0);
    const long long at_state = (long long)c * p.N + n0, chunk_states = (long long)p.C * p.N;
    const long long r0 = blockIdx.x * plan.rows, stop = min(r0 + plan.rows, p.seqs.rows);

    f32x2 h[S / 2], A[S / 2];
#pragma unroll
    for (int i = 0; i < S / 2; ++i) {
        const int n = n0 + 2 * i;
        A[i] = pair(n < p.N ? p.A[at_state + 2 * i] * kLog2e : 0.f, n + 1 < p.N ? p.A[at_state + 2 * i + 1] * kLog2e : 0.f);
        h[i] = 0;
    }
    auto load = [&](const float *from) {  // the lane's states of one sequence or chunk
#pragma unroll
        for (int i = 0; i < S / 2; ++i) {
            const int n = n0 + 2 * i;
            h[i] = pair(n < p.N ? from[at_state + 2 * i] : 0.f, n + 1 < p.N ? from[at_state + 2 * i + 1] : 0.f);
        }
    };
    auto store = [&](float *to) {
        if (!live) return;
#pragma unroll
        for (int i = 0; i < S / 2; ++i) {
            const int n = n0 + 2 * i;
            float a, b;
            unpair(h[i], a, b);
            if (n < p.N) to[at_state + 2 * i] = a;
            if (n + 1 < p.N) to[at_state + 2 * i + 1] = b;
        }
    };
    auto initial = [&](int n) {
        const long long slot = p.init ? state_slot(p.init_idx, p.pool, n, p.err) : -1;
        if (slot >= 0) {
            load(p.init + slot * chunk_states);
        } else {
#pragma unroll
            for (int i = 0; i < S / 2; ++i) h[i] = 0;
        }
    };
    auto final_state = [&](int n) {
        if (!fin) return;
        const long long slot = state_slot(p.fin_idx, p.pool, n, p.err);
        if (slot >= 0) store(fin + slot * chunk_states);
    };
    // After the end of sequence n: its final state, and those of the empty sequences behind it.
    auto close_sequence = [&](int n) {
        final_state(n);
        for (++n; n < p.seqs.n_seqs && p.seqs.begin(n) == p.seqs.end(n); ++n) {
            initial(n);
            final_state(n);
        }
        return n;
    };

    long long r = r0;
    int seq = 0;
    if constexpr (ENDS) {
        seq = p.seqs.at(stop - 1);
        const long long bos = p.seqs.begin(seq);
        if (bos >= r0 && bos < stop) {
            r = bos;
            initial(seq);
            store(carry.first + blockIdx.x * chunk_states);
        }
    } else {
        if (blockIdx.x == 0)  // empty sequences before the first row
            for (; seq < p.seqs.n_seqs && p.seqs.begin(seq) == p.seqs.end(seq) && p.seqs.begin(seq) == 0; ++seq) {
                initial(seq);
                final_state(seq);
            }
        if (r0 >= stop) return;
        seq = p.seqs.at(r0);
        if (plan.carries && p.seqs.begin(seq) < r0) load(carry.state + blockIdx.x * chunk_states);
    }
    // The row at which the next sequence begins; the last sequence that begins here and goes on after the chunk
    // takes its initial state from the first kernel's copy, because another block may write its final state there.
    long long end = p.seqs.end(seq);
    auto begin_sequence = [&](int n) {
        end = p.seqs.end(n);
        if (plan.carries && end > stop && blockIdx.x + 1 < plan.chunks)
            load(carry.first + blockIdx.x * chunk_states);
        else
            initial(n);
    };
    if (!ENDS && p.seqs.begin(seq) == r0) begin_sequence(seq);

    const float bias = p.dt_bias ? p.dt_bias[c] : 0.f, skip = p.D ? p.D[c] : 0.f;
    const T *X = static_cast<const T *>(p.x), *DT = static_cast<const T *>(p.dt), *Z = static_cast<const T *>(p.z);
    const T *Bm = static_cast<const T *>(p.Bm) + g * p.N, *Cm = static_cast<const T *>(p.Cm) + g * p.N;

    T ahead[EACH];
    auto fetch = [&](long long first) {  // the next tile's values of this thread
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int v = i * kScanThreads + threadIdx.x, n = v % NP, side = (v / NP) % SIDES;
            const long long row = first + v / (NP * SIDES);
            ahead[i] = row < stop && n < p.N ? (side ? Cm[row * p.C_stride + n] : Bm[row * p.B_stride + n]) : from_float<T>(0.f);
        }
    };
    T rx[kUnroll], rdt[kUnroll], rz[kUnroll];  // the inputs of rows ahead_row .. ahead_row + kUnroll - 1
    long long ahead_row = -1;
    auto fetch_rows = [&](long long first) {
        const T *xr = X + first * p.x_stride, *dtr = DT + first * p.dt_stride, *zr = Z + first * p.z_stride;
        ahead_row = first;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            rx[u] = xr[u * p.x_stride + c];
            rdt[u] = dtr[u * p.dt_stride + c];
            if (!ENDS && Z) rz[u] = zr[u * p.z_stride + c];
        }
    };
    f32x2 total = 0;
    // Two tokens, both of the running sequence, with B and C rows at `bc`; the second only if `two`.
    auto step = [&](float x0, float x1, float dt0, float dt1, float z0, float z1, const float *bc, T *out, bool two) {
        const f32x2 x2 = pair(x0, x1);
        f32x2 dt2 = add2(pair(dt0, dt1), both(bias));
        if (p.softplus) dt2 = softplus2(dt2);
        float dts[2], us[2], sums[2];
        unpair(dt2, dts[0], dts[1]);
        unpair(mul2(dt2, x2), us[0], us[1]);
        if constexpr (ENDS) total = add2(total, two ? dt2 : pair(dts[0], 0.f));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (j == 1 && !two) break;
            const f32x2 *B2 = reinterpret_cast<const f32x2 *>(bc + j * SIDES * NP);
            const f32x2 *C2 = reinterpret_cast<const f32x2 *>(bc + (j * SIDES + SIDES - 1) * NP);
            const f32x2 t2 = both(dts[j]), u2 = both(us[j]);
            f32x2 sum2 = 0;
#pragma unroll
            for (int i = 0; i < S / 2; ++i) {
                h[i] = fma2(ex2_pair(mul2(t2, A[i])), h[i], mul2(u2, B2[i]));
                if constexpr (!ENDS) sum2 = i == 0 ? mul2(C2[i], h[i]) : fma2(C2[i], h[i], sum2);
            }
            if constexpr (!ENDS) {
                float other;
                unpair(sum2, sums[j], other);
                sums[j] += other;
#pragma unroll
                for (int m = L / 2; m > 0; m >>= 1) sums[j] += __shfl_xor_sync(0xffffffffu, sums[j], m);
            }
        }
        if constexpr (!ENDS) {
            f32x2 y2 = fma2(both(skip), x2, pair(sums[0], two ? sums[1] : 0.f));
            if (Z) y2 = mul2(y2, silu2(pair(z0, z1)));
            unpair(y2, sums[0], sums[1]);
            if (live && n0 == 0) {
                out[c] = from_float<T>(sums[0]);
                if (two) out[p.C + c] = from_float<T>(sums[1]);
            }
        }
    };
    fetch(r);
    for (int buf = 0; r < stop; buf ^= 1) {
        float *mine = &tile[buf][0][0][0];
#pragma unroll
        for (int i = 0; i < EACH; ++i) mine[i * kScanThreads + threadIdx.x] = to_float(ahead[i]);
        __syncthreads();  // two buffers: the one written next was last read before this barrier
        fetch(r + TT);
        const float *bc = mine + n0;
        const long long tile_end = min(r + TT, stop);
        while (r < tile_end) {
            if (!ENDS && r == end) {
                seq = close_sequence(seq);
                if (seq >= p.seqs.n_seqs) return;  // rows past the last sequence: a bad cu_seqlens
                begin_sequence(seq);
            }
            const long long until = !ENDS && end > r && end < tile_end ? end : tile_end;
            for (; r + kUnroll <= until; r += kUnroll, bc += kUnroll * SIDES * NP) {
                if (ahead_row != r) fetch_rows(r);
                float xs[kUnroll], dts[kUnroll], zs[kUnroll];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    xs[u] = to_float(rx[u]);
                    dts[u] = to_float(rdt[u]);
                    zs[u] = !ENDS && Z ? to_float(rz[u]) : 0.f;
                }
                if (r + 2 * kUnroll <= stop) fetch_rows(r + kUnroll);
                T *out = y + r * p.C;
#pragma unroll
                for (int u = 0; u < kUnroll; u += 2)
                    step(xs[u], xs[u + 1], dts[u], dts[u + 1], zs[u], zs[u + 1], bc + u * SIDES * NP, out + u * p.C, true);
            }
#pragma unroll 1
            for (; r < until; ++r, bc += SIDES * NP) {  // a few tokens before an end
                const float x0 = to_float(X[r * p.x_stride + c]), dt0 = to_float(DT[r * p.dt_stride + c]);
                const float z0 = !ENDS && Z ? to_float(Z[r * p.z_stride + c]) : 0.f;
                step(x0, 0.f, dt0, 0.f, z0, 0.f, bc, y + r * p.C, false);
            }
        }
    }
    if constexpr (ENDS) {
        store(carry.state + blockIdx.x * chunk_states);
        float even, odd;
        unpair(total, even, odd);
        if (live && n0 == 0) carry.time[(long long)blockIdx.x * p.C + c] = even + odd;
    } else {
        if (stop == end) close_sequence(seq);
    }
}

// From the chunks' end states to the states before them, one thread per (channel, state). A batch of chunks is
// loaded before the walk over it, which is bound by the latency of those loads.
constexpr int kCarryBatch = 16;
__global__ void __launch_bounds__(128) scan_carry_kernel(ScanParams p, ScanPlan plan, Carries carry) {
    extern __shared__ unsigned char fresh[];  // chunk j's last sequence begins in it
    for (int j = threadIdx.x; j < plan.chunks - 1; j += 128) {
        const long long r0 = j * plan.rows;
        fresh[j] = p.seqs.begin(p.seqs.at(r0 + plan.rows - 1)) >= r0;
    }
    __syncthreads();
    const long long size = (long long)p.C * p.N, i = (long long)blockIdx.x * 128 + threadIdx.x;
    if (i >= size) return;
    const float A = p.A[i] * kLog2e;
    const long long c = i / p.N;
    float before = 0.f;
    for (int j0 = 0; j0 < plan.chunks; j0 += kCarryBatch) {
        float local[kCarryBatch], time[kCarryBatch];
#pragma unroll
        for (int b = 0; b < kCarryBatch; ++b) {
            const bool in = j0 + b + 1 < plan.chunks;  // nothing follows the last chunk
            local[b] = in ? carry.state[(j0 + b) * size + i] : 0.f;
            time[b] = in ? carry.time[(long long)(j0 + b) * p.C + c] : 0.f;
        }
#pragma unroll
        for (int b = 0; b < kCarryBatch; ++b) {
            if (j0 + b < plan.chunks) carry.state[(j0 + b) * size + i] = before;
            if (j0 + b + 1 < plan.chunks) before = fresh[j0 + b] ? local[b] : fmaf(ex2(A * time[b]), before, local[b]);
        }
    }
}

Carries carries_in(const kda_scan_args &a, const ScanPlan &plan, void *ws) {
    const size_t states = (size_t)plan.chunks * a.D * a.N;
    float *f = static_cast<float *>(ws);
    return Carries{f, f + states, f + 2 * states};
}

struct PrefillLaunch {
    ScanParams p;
    void *y;
    float *fin;
    ScanPlan plan;
    Carries carry;
    cudaStream_t s;
    template <typename T, int S, int L>
    void operator()() {
        const int per = p.C / p.G;
        const unsigned blocks = (unsigned)(((per * L + kScanThreads - 1) / kScanThreads) * p.G);
        if (plan.carries) {
            scan_prefill_kernel<T, S, L, true><<<dim3((unsigned)plan.chunks - 1, blocks), kScanThreads, 0, s>>>(p, nullptr, nullptr, plan, carry);
            const long long size = (long long)p.C * p.N;
            scan_carry_kernel<<<(unsigned)((size + 127) / 128), 128, (size_t)plan.chunks, s>>>(p, plan, carry);
        }
        scan_prefill_kernel<T, S, L, false><<<dim3((unsigned)plan.chunks, blocks), kScanThreads, 0, s>>>(
            p, static_cast<T *>(y), fin, plan, carry);
    }
};

// One token: bound by HBM, the state is read and written once. LP lanes hold a channel's states, V consecutive
// ones each (16 bytes where N and the state's address allow it), so that a warp streams whole
// 512-byte runs of the state; the parts of y are added by shuffles.
template <typename T, int LP, int V>
__global__ void __launch_bounds__(128) scan_decode_kernel(ScanParams p, float *state, T *__restrict__ y) {
    const int k = blockIdx.y * (128 / LP) + threadIdx.x / LP, l = threadIdx.x % LP;
    const int n = blockIdx.x;
    const bool live = k < p.C;
    const int c = live ? k : p.C - 1;
    const int g = c / (p.C / p.G);
    const long long from = state_slot(p.init_idx, p.pool, n, p.err);
    const long long to = p.fin_idx == p.init_idx ? from : state_slot(p.fin_idx, p.pool, n, p.err);
    const float x = to_float(static_cast<const T *>(p.x)[n * p.x_stride + c]);
    float dt = to_float(static_cast<const T *>(p.dt)[n * p.dt_stride + c]) + (p.dt_bias ? p.dt_bias[c] : 0.f);
    if (p.softplus) dt = softplus(dt);
    const float u = dt * x;
    const T *B = static_cast<const T *>(p.Bm) + n * p.B_stride + g * p.N;
    const T *Cm = static_cast<const T *>(p.Cm) + n * p.C_stride + g * p.N;
    float sum = 0.f;
    for (int n0 = l * V; n0 < p.N; n0 += LP * V) {
        Pack<float, V> a = load_pack<float, V>(p.A + (long long)c * p.N + n0), h;
        if (from >= 0) {
            h = load_pack<float, V>(state + (from * p.C + c) * p.N + n0);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) h.e[v] = 0.f;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h.e[v] = fmaf(exp2f(dt * (a.e[v] * kLog2e)), h.e[v], u * to_float(B[n0 + v]));
            sum = fmaf(to_float(Cm[n0 + v]), h.e[v], sum);
        }
        if (to >= 0 && live) store_pack<float, V>(state + (to * p.C + c) * p.N + n0, h);
    }
#pragma unroll
    for (int m = LP / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (!live || l != 0) return;
    if (p.D) sum = fmaf(p.D[c], x, sum);
    if (p.z) {
        const float z = to_float(static_cast<const T *>(p.z)[n * p.z_stride + c]);
        sum *= z * sigmoid(z);
    }
    y[(long long)n * p.C + c] = from_float<T>(sum);
}

template <typename T, int V>
void launch_decode(const ScanParams &p, float *state, void *y, cudaStream_t s) {
    const int words = (p.N + V - 1) / V;
    T *out = static_cast<T *>(y);
#define KDA_DECODE(LP)                                                                                              \
    scan_decode_kernel<T, LP, V><<<dim3((unsigned)p.seqs.n_seqs, (unsigned)((p.C + 128 / LP - 1) / (128 / LP))), 128, 0, s>>>( \
        p, state, out)
    if (words <= 1)
        KDA_DECODE(1);
    else if (words <= 2)
        KDA_DECODE(2);
    else if (words <= 4)
        KDA_DECODE(4);
    else if (words <= 8)
        KDA_DECODE(8);
    else
        KDA_DECODE(16);
#undef KDA_DECODE
}

}  // namespace

// Whole sequences where they give every SM a block; otherwise chunks that give it four, of at least 64 rows. (Half as many or
// twice as many were slower on one sequence of 16384 rows and 4096 channels.)
ScanPlan scan_plan(const kda_scan_args &a, int sms) {
    const long long rows = (long long)a.B * a.T, blocks = (long long)scan_blocks(a) * a.G;
    if (rows == 0) return ScanPlan{1, 1, false};
    if (sms <= 0) sms = 152;
    if (!a.cu_seqlens && (a.B * blocks >= sms || a.T <= 64)) return ScanPlan{a.B, a.T, false};
    long long chunks = 4LL * sms / blocks, most = (rows + 63) / 64;
    chunks = chunks < 1 ? 1 : chunks > most ? most : chunks;
    long long per = ((rows + chunks - 1) / chunks + 31) / 32 * 32;
    chunks = (rows + per - 1) / per;
    return ScanPlan{(int)chunks, per, chunks > 1};
}

size_t scan_prefill_workspace_bytes(const kda_scan_args &a, int sms) {
    const ScanPlan plan = scan_plan(a, sms);
    return plan.carries ? (size_t)plan.chunks * a.D * (2 * a.N + 1) * sizeof(float) : 0;
}

cudaError_t launch_scan_prefill(const kda_scan_args &a, void *y, float *final_state, void *ws, int sms, unsigned *err,
                                cudaStream_t s) {
    const ScanPlan plan = scan_plan(a, sms);
    return scan_by_type(a, PrefillLaunch{scan_params(a, err), y, final_state, plan, carries_in(a, plan, ws), s});
}

cudaError_t launch_scan_decode(const kda_scan_args &a, float *state, void *y, unsigned *err, cudaStream_t s) {
    ScanParams p = scan_params(a, err);
    if (!p.fin_idx) p.fin_idx = p.init_idx;
    const bool wide = p.N % 4 == 0 && aligned16(state) && aligned16(p.A);
    if (a.dtype == KDA_BF16)
        wide ? launch_decode<__nv_bfloat16, 4>(p, state, y, s) : launch_decode<__nv_bfloat16, 1>(p, state, y, s);
    else
        wide ? launch_decode<float, 4>(p, state, y, s) : launch_decode<float, 1>(p, state, y, s);
    return cudaGetLastError();
}

}  // namespace kda
