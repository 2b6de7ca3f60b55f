// kda_scan.cu -- the selective state space scan: prompts and single tokens.
//
//     h_t[c, n] = exp(dt_t[c] A[c, n]) h_{t-1}[c, n] + dt_t[c] x_t[c] B_t[n],   y_t[c] = sum_n C_t[n] h_t[c, n] + D[c] x_t[c]
//
// Prompts: one lane per two channels holds up to 16 states of each in registers (more states: 2 to 16 lanes, their parts of y
// added by shuffles) and walks down the rows; a block's B and C rows lie in shared memory in fp32, read as broadcasts. Per
// (token, channel, state) that is 1 exponential and 4 multiply-adds: with 32 exponentials and 128 multiply-adds per SM
// and cycle both units are busy equally long and HBM waits for them.
//
// A sequence has few channels for 152 SMs, so the rows are cut into chunks that run side by side. The state after
// a chunk is linear in the state before it, h_end = exp(A sum dt) h_begin + (the end state from zeros):
// a first kernel computes the end states from zeros and the sums of dt, a second one walks over the chunks to get the
// state before each, and the main kernel runs every chunk from there. That is a second round of exponentials, and it is
// left out where whole sequences fill the GPU.
// Measured: one sequence of 16384 rows x 4096 channels x 16 states in bf16 with gate: 482 us (190 us the end states, 290 us
// the rows; the exponentials alone are 112 us in each). Issue slots are half used: per 32 channels and row 100 warp instructions, of which 43
// are paired multiply-adds at 2.4 cycles each and 19 are exponentials or reciprocals at 4 cycles, so both units are busy half of the time
// and wait for each other's results the rest. With single instead of paired multiply-adds it takes 568 us.
#include <algorithm>

#include "kda_scan.cuh"

namespace kda {
namespace {

constexpr int kWarps = kScanThreads / 32;
template <typename T>
constexpr int kBlock = 16 / sizeof(T);  // tokens that are loaded together and computed without a look at sequence ends

template <int NP>
struct Tile {  // tokens of B and C in shared memory at a time: at most 16 KB
    static constexpr int tokens = NP <= 64 ? 32 : 2048 / NP;
};

// A lane's two channels of one row.
template <typename T>
struct alignas(2 * sizeof(T)) Two {
    T a, b;
};
template <typename T>
__device__ __forceinline__ f32x2 to_pair(Two<T> v) { return pair(to_float(v.a), to_float(v.b)); }

__device__ __forceinline__ bool on_16_bytes(const float *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

__device__ __forceinline__ void copy16(void *to, const void *from) {  // global -> shared, asynchronous
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((unsigned)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copies_arrived() { asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory"); }

// What a kernel makes of its chunk:
//   kOutputs   y and the sequences' final states
//   kEnds      the end state of the chunk's last sequence (from zeros, or from its initial state if it begins in the chunk)
//   kStates    for the backward pass: that end state, and the states before every kScanWindow-th row
//   kBackEnds  for the backward pass, rows taken from the last to the first: the gradient at the state before the chunk of its
//              first sequence, from zeros, or from its final state's gradient if it ends in the chunk; B is C and u is dy here
// WIDE: every row's channels lie on 16-byte boundaries. A lane holds S states of two channels, which share the reads of B and C.
// The rows of x, dt and z come through a ring in shared memory, each warp its own channels' rows, STAGES - 1 blocks ahead:
// loads into registers were moved back to their use by the compiler, and a third of the time was spent waiting for them.
template <typename T, int S, int L, bool WIDE, int MODE>
__global__ void __launch_bounds__(kScanThreads, 2)
    scan_rows_kernel(ScanParams p, T *__restrict__ y, float *fin, ScanPlan plan, Carries carry) {
    constexpr bool OUT = MODE == kOutputs, BACK = MODE == kBackEnds;
    constexpr int BLK = kBlock<T>;
    constexpr int NP = S * L, TT = Tile<NP>::tokens, SIDES = OUT ? 2 : 1;
    constexpr int EACH = TT * SIDES * NP / kScanThreads;  // values of a tile that a thread brings
    static_assert(TT % BLK == 0 && TT * SIDES * NP % kScanThreads == 0, "tile");
    __shared__ __align__(16) float tile[2][TT][SIDES][NP];
    if ((OUT || MODE == kStates) && blockIdx.x == 0 && blockIdx.y == 0) check_seqs(p.seqs, p.err);
    const int per = p.C / p.G;
    const int blocks = (per * L + 2 * kScanThreads - 1) / (2 * kScanThreads);
    const int g = blockIdx.y / blocks;
    const int k = ((blockIdx.y % blocks) * (kScanThreads / L) + threadIdx.x / L) * 2, n0 = (threadIdx.x % L) * S;
    const bool live = k < per, live1 = k + 1 < per;
    const int c = g * per + (live ? k : 0), c1 = live1 ? c + 1 : c;
    const long long chunk_states = (long long)p.C * p.N;
    const int chunk = BACK ? blockIdx.x + 1 : blockIdx.x;  // nothing comes before the first
    const long long r0 = chunk * plan.rows;
    long long stop = min(r0 + plan.rows, p.seqs.rows);

    f32x2 h[2][S / 2], A[2][S / 2];
    auto load_states = [&](const float *from, f32x2(&to)[2][S / 2], float scale) {  // a tensor [C][N]
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float *row = from + (long long)(j ? c1 : c) * p.N + n0;
            if (p.N == NP && on_16_bytes(from)) {
#pragma unroll
                for (int i = 0; i < S / 4; ++i) {
                    const float4 v = reinterpret_cast<const float4 *>(row)[i];
                    to[j][2 * i] = pair(v.x * scale, v.y * scale);
                    to[j][2 * i + 1] = pair(v.z * scale, v.w * scale);
                }
                continue;
            }
#pragma unroll
            for (int i = 0; i < S / 2; ++i) {
                const int n = n0 + 2 * i;
                to[j][i] = pair(n < p.N ? row[2 * i] * scale : 0.f, n + 1 < p.N ? row[2 * i + 1] * scale : 0.f);
            }
        }
    };
    load_states(p.A, A, kLog2e);
    auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < S / 2; ++i) h[0][i] = h[1][i] = 0;
    };
    clear();
    auto store = [&](float *to) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (!(j ? live1 : live)) continue;
            float *row = to + (long long)(c + j) * p.N + n0;
            if (p.N == NP && on_16_bytes(to)) {
#pragma unroll
                for (int i = 0; i < S / 4; ++i) {
                    float4 v;
                    unpair(h[j][2 * i], v.x, v.y);
                    unpair(h[j][2 * i + 1], v.z, v.w);
                    reinterpret_cast<float4 *>(row)[i] = v;
                }
                continue;
            }
#pragma unroll
            for (int i = 0; i < S / 2; ++i) {
                const int n = n0 + 2 * i;
                float v0, v1;
                unpair(h[j][i], v0, v1);
                if (n < p.N) row[2 * i] = v0;
                if (n + 1 < p.N) row[2 * i + 1] = v1;
            }
        }
    };
    auto initial = [&](int n) {
        const long long slot = p.init ? state_slot(p.init_idx, p.pool, n, p.err) : -1;
        if (slot >= 0)
            load_states(p.init + slot * chunk_states, h, 1.f);
        else
            clear();
    };
    auto final_state = [&](int n) {
        if (!OUT || !fin) return;
        const long long slot = state_slot(p.fin_idx, p.pool, n, p.err);
        if (slot >= 0) store(fin + slot * chunk_states);
    };
    // After the end of sequence n: its final state, and those of the empty sequences behind it.
    auto close_sequence = [&](int n) {
        final_state(n);
        for (++n; n < p.seqs.n_seqs && p.seqs.begin(n) == p.seqs.end(n); ++n) {
            if (!OUT) continue;
            initial(n);
            final_state(n);
        }
        return n;
    };

    long long r = r0;
    int seq = 0;
    if constexpr (MODE == kEnds) {
        seq = p.seqs.at(stop - 1);
        const long long bos = p.seqs.begin(seq);
        if (bos >= r0 && bos < stop) {
            r = bos;
            initial(seq);
            store(carry.first + chunk * chunk_states);
        }
    } else if constexpr (BACK) {
        seq = p.seqs.at(r0);
        const long long eos = p.seqs.end(seq);
        if (eos <= stop && eos > r0) {
            stop = eos;
            if (fin) load_states(fin + (long long)seq * chunk_states, h, 1.f);
        }
    } else {
        if (OUT && chunk == 0)  // empty sequences before the first row
            for (; seq < p.seqs.n_seqs && p.seqs.begin(seq) == p.seqs.end(seq) && p.seqs.begin(seq) == 0; ++seq) {
                initial(seq);
                final_state(seq);
            }
        if (r0 >= stop) return;
        seq = p.seqs.at(r0);
        const long long bos = p.seqs.begin(seq);
        if (OUT && plan.carries && bos < r0) {
            if (plan.folded()) {  // from the end state of the chunk in which the sequence begins, over the chunks since
                int j = bos > 0 ? (int)(bos / plan.rows) : 0;
                load_states(carry.state + j * chunk_states, h, 1.f);
                for (++j; j < chunk; ++j) {
                    f32x2 local[2][S / 2];
                    load_states(carry.state + j * chunk_states, local, 1.f);
                    const float *time = carry.time + (long long)j * p.C;
                    const f32x2 t0 = both(time[c]), t1 = both(time[c1]);
#pragma unroll
                    for (int i = 0; i < S / 2; ++i) {
                        h[0][i] = carried2(t0, A[0][i], h[0][i], local[0][i]);
                        h[1][i] = carried2(t1, A[1][i], h[1][i], local[1][i]);
                    }
                }
            } else {
                load_states(carry.state + chunk * chunk_states, h, 1.f);
            }
        }
    }
    // The row at which the next sequence begins. The last sequence that begins here and goes on after the chunk takes
    // its initial state from the first kernel's copy, because another block may write its final state there.
    long long end = p.seqs.end(seq);
    auto begin_sequence = [&](int n) {
        end = p.seqs.end(n);
        if (OUT && plan.carries && end > stop && chunk + 1 < plan.chunks)
            load_states(carry.first + chunk * chunk_states, h, 1.f);
        else
            initial(n);
    };
    if ((OUT || MODE == kStates) && p.seqs.begin(seq) == r0) begin_sequence(seq);

    const f32x2 bias = p.dt_bias ? pair(p.dt_bias[c], p.dt_bias[c1]) : 0, skip = p.D ? pair(p.D[c], p.D[c1]) : 0;
    const T *X = static_cast<const T *>(p.x), *DT = static_cast<const T *>(p.dt), *Z = static_cast<const T *>(p.z);
    const long long B_stride = BACK ? p.C_stride : p.B_stride;
    const T *Bm = static_cast<const T *>(BACK ? p.Cm : p.Bm) + g * p.N, *Cm = static_cast<const T *>(p.Cm) + g * p.N;

    f32x2 total = 0;  // of the time steps
    T ahead[EACH];
    auto fetch = [&](long long first) {  // the next tile's values of this thread
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int v = i * kScanThreads + threadIdx.x, n = v % NP, side = (v / NP) % SIDES;
            const long long at = first + v / (NP * SIDES), row = BACK ? r0 + stop - 1 - at : at;
            ahead[i] = at < stop && n < p.N ? (side ? Cm[row * p.C_stride + n] : Bm[row * B_stride + n]) : from_float<T>(0.f);
        }
    };
    constexpr int CW = 64 / L, ROWS = OUT || BACK ? 3 : 2, STAGES = 4;  // channels of a warp, tensors
    __shared__ __align__(16) T ring[kWarps][STAGES][ROWS][BLK][CW];
    auto &mine = ring[threadIdx.x / 32];
    const int lane = threadIdx.x % 32;
    const int w0 = ((blockIdx.y % blocks) * kWarps + threadIdx.x / 32) * CW;  // the warp's first channel in the group
    auto row_at = [&](long long at) { return BACK ? r0 + stop - 1 - at : at; };
    // Brings the block of rows that starts at `first` into its stage.
    auto bring = [&](long long first, int stage) {
#pragma unroll
        for (int t = 0; t < ROWS; ++t) {
            const T *from = (t == 0 ? X : t == 1 ? DT : Z) + g * per + w0;
            const long long stride = t == 0 ? p.x_stride : t == 1 ? p.dt_stride : p.z_stride;
            if (t == 2 && !Z) break;
            if constexpr (WIDE && CW * sizeof(T) >= 16) {
                constexpr int PER = 16 / sizeof(T), WORDS = CW / PER;  // values per copy, copies per row
#pragma unroll
                for (int i = lane; i < BLK * WORDS; i += 32) {
                    const int u = i / WORDS, k0 = (i % WORDS) * PER;
                    if (first + u < stop && w0 + k0 < per) copy16(&mine[stage][t][u][k0], from + row_at(first + u) * stride + k0);
                }
            } else {
                for (int i = lane; i < BLK * CW; i += 32) {
                    const int u = i / CW, k0 = i % CW;
                    if (first + u < stop && w0 + k0 < per) mine[stage][t][u][k0] = from[row_at(first + u) * stride + k0];
                }
            }
        }
        copies_issued();
    };
    // The state before a window, and the time since the chunk's first row.
    auto keep = [&](long long window) {
        const long long at = chunk * plan.windows() + window;
        store(carry.kept + at * chunk_states);
        float t0, t1;
        unpair(total, t0, t1);
        if (live && n0 == 0) carry.kept_time[at * p.C + c] = t0;
        if (live1 && n0 == 0) carry.kept_time[at * p.C + c1] = t1;
    };
    auto row_pair = [&](int stage, int t, int u) {
        return to_pair(*reinterpret_cast<const Two<T> *>(&mine[stage][t][u][lane / L * 2]));
    };
    auto step = [&](f32x2 x, f32x2 dt, f32x2 z, const float *bc, T *out) {  // one token, with its B and C at `bc`
        dt = add2(dt, bias);
        if (p.softplus) dt = softplus2(dt);
        float dts[2], us[2];
        unpair(dt, dts[0], dts[1]);
        if constexpr (BACK) {
            if (Z) x = mul2(x, silu2(z));
            unpair(x, us[0], us[1]);
        } else {
            unpair(mul2(dt, x), us[0], us[1]);
        }
        if constexpr (!OUT) total = add2(total, dt);
        const f32x2 *B2 = reinterpret_cast<const f32x2 *>(bc), *C2 = reinterpret_cast<const f32x2 *>(bc + (SIDES - 1) * NP);
        const f32x2 t0 = both(dts[0]), t1 = both(dts[1]), u0 = both(us[0]), u1 = both(us[1]);
        f32x2 s0 = 0, s1 = 0;
#pragma unroll
        for (int i = 0; i < S / 2; ++i) {
            const f32x2 b = B2[i], a0 = decay2(t0, A[0][i]), a1 = decay2(t1, A[1][i]);
            h[0][i] = BACK ? mul2(a0, fma2(u0, b, h[0][i])) : fma2(a0, h[0][i], mul2(u0, b));
            h[1][i] = BACK ? mul2(a1, fma2(u1, b, h[1][i])) : fma2(a1, h[1][i], mul2(u1, b));
            if constexpr (OUT) {
                const f32x2 cc = C2[i];
                s0 = i == 0 ? mul2(cc, h[0][i]) : fma2(cc, h[0][i], s0);
                s1 = i == 0 ? mul2(cc, h[1][i]) : fma2(cc, h[1][i], s1);
            }
        }
        if constexpr (OUT) {
            float sums[2], other[2];
            unpair(s0, sums[0], other[0]);
            unpair(s1, sums[1], other[1]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                sums[j] += other[j];
#pragma unroll
                for (int m = L / 2; m > 0; m >>= 1) sums[j] += __shfl_xor_sync(0xffffffffu, sums[j], m);
            }
            f32x2 y2 = fma2(skip, x, pair(sums[0], sums[1]));
            if (Z) y2 = mul2(y2, silu2(z));
            unpair(y2, sums[0], sums[1]);
            if (n0 == 0) {
                if constexpr (WIDE) {
                    if (live) *reinterpret_cast<Two<T> *>(out + c) = Two<T>{from_float<T>(sums[0]), from_float<T>(sums[1])};
                } else {
                    if (live) out[c] = from_float<T>(sums[0]);
                    if (live1) out[c1] = from_float<T>(sums[1]);
                }
            }
        }
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) bring(r + i * BLK, i);
    int stage = 0;
    fetch(r);
    for (int buf = 0; r < stop; buf ^= 1) {
        float *bc = &tile[buf][0][0][0];
#pragma unroll
        for (int i = 0; i < EACH; ++i) bc[i * kScanThreads + threadIdx.x] = to_float(ahead[i]);
        __syncthreads();  // two buffers: the one written next was last read before this barrier
        fetch(r + TT);
        bc += n0;
        for (int t0 = 0; t0 < TT && r < stop; t0 += BLK, bc += BLK * SIDES * NP) {
            copies_arrived<STAGES - 2>();
            __syncwarp();  // every lane's copies of this block are there, and the block before is read
            bring(r + (STAGES - 1) * BLK, stage == 0 ? STAGES - 1 : stage - 1);
            T *out = y + r * p.C;
            if (MODE == kStates && (r - r0) % kScanWindow == 0) keep((r - r0) / kScanWindow);
            if (r + BLK <= stop && (MODE == kEnds || BACK || r + BLK <= end || end < r)) {
#pragma unroll
                for (int u = 0; u < BLK; ++u)
                    step(row_pair(stage, 0, u), row_pair(stage, 1, u), (OUT || BACK) && Z ? row_pair(stage, ROWS - 1, u) : 0,
                         bc + u * SIDES * NP, out + u * p.C);
                r += BLK;
            } else {  // a sequence ends in the block, or the chunk does
#pragma unroll 1
                for (int u = 0; u < BLK && r < stop; ++u, ++r) {
                    if ((OUT || MODE == kStates) && r == end) {
                        seq = close_sequence(seq);
                        if (seq >= p.seqs.n_seqs) {  // rows past the last sequence: a bad cu_seqlens
                            copies_arrived<0>();
                            return;
                        }
                        begin_sequence(seq);
                    }
                    step(row_pair(stage, 0, u), row_pair(stage, 1, u), (OUT || BACK) && Z ? row_pair(stage, ROWS - 1, u) : 0,
                         bc + u * SIDES * NP, out + u * p.C);
                }
            }
            stage = stage == STAGES - 1 ? 0 : stage + 1;
        }
    }
    copies_arrived<0>();
    if constexpr (OUT) {
        if (stop == end) close_sequence(seq);
    } else {
        store(carry.state + chunk * chunk_states);
        float t0, t1;
        unpair(total, t0, t1);
        if (live && n0 == 0) carry.time[(long long)chunk * p.C + c] = t0;
        if (live1 && n0 == 0) carry.time[(long long)chunk * p.C + c1] = t1;
    }
}

// From the chunks' end states to the states before them, one thread per (channel, state). A batch of chunks is
// loaded before the walk over it, which is bound by the latency of those loads; places past the ends load the last one's again (as
// predicated loads they came one after another: 13 us instead of 10 for the gradients' walk below, 19 chunks of 4096 channels x 16 states).
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
        float local[kCarryBatch], root[kCarryBatch];
#pragma unroll
        for (int b = 0; b < kCarryBatch; ++b) {
            const int j = min(j0 + b, plan.chunks - 2);  // nothing follows the last chunk
            local[b] = carry.state[j * size + i];
            root[b] = root_decay(carry.time[(long long)j * p.C + c], A);
        }
#pragma unroll
        for (int b = 0; b < kCarryBatch; ++b) {
            if (j0 + b < plan.chunks) carry.state[(j0 + b) * size + i] = before;
            if (j0 + b + 1 < plan.chunks) before = fresh[j0 + b] ? local[b] : carried(root[b], before, local[b]);
        }
    }
}

// The same from the last chunk to the first for the gradients at the states.
__global__ void __launch_bounds__(128) scan_back_carry_kernel(ScanParams p, ScanPlan plan, Carries carry) {
    extern __shared__ unsigned char goes_on[];  // chunk j's first sequence goes on after it
    for (int j = threadIdx.x; j < plan.chunks; j += 128) {
        const long long r0 = j * plan.rows;
        goes_on[j] = p.seqs.end(p.seqs.at(r0)) > min(r0 + plan.rows, p.seqs.rows);
    }
    __syncthreads();
    const long long size = (long long)p.C * p.N, i = (long long)blockIdx.x * 128 + threadIdx.x;
    if (i >= size) return;
    const float A = p.A[i] * kLog2e;
    const long long c = i / p.N;
    float after = 0.f;
    for (int j0 = plan.chunks - 1; j0 >= 0; j0 -= kCarryBatch) {
        float local[kCarryBatch], root[kCarryBatch];
#pragma unroll
        for (int b = 0; b < kCarryBatch; ++b) {
            const int j = max(j0 - b, 0);  // nothing comes before the first chunk
            local[b] = carry.state[j * size + i];
            root[b] = root_decay(carry.time[(long long)j * p.C + c], A);
        }
#pragma unroll
        for (int b = 0; b < kCarryBatch; ++b) {
            if (j0 - b < 0) break;
            carry.state[(j0 - b) * size + i] = after;
            after = goes_on[j0 - b] ? carried(root[b], after, local[b]) : local[b];
        }
    }
}

// No rows: every sequence's final state is its initial one; nothing else is read, A neither.
__global__ void __launch_bounds__(128) scan_no_rows_kernel(ScanParams p, float *fin) {
    const int n = blockIdx.x;
    const long long size = (long long)p.C * p.N, from = p.init ? state_slot(p.init_idx, p.pool, n, p.err) : -1;
    const long long to = fin ? state_slot(p.fin_idx, p.pool, n, p.err) : -1;
    if (to < 0) return;
    for (long long i = threadIdx.x; i < size; i += 128) fin[to * size + i] = from >= 0 ? p.init[from * size + i] : 0.f;
}

Carries carries_in(const kda_scan_args &a, const ScanPlan &plan, void *ws) {
    const size_t states = (size_t)plan.chunks * a.D * a.N;
    float *f = static_cast<float *>(ws);
    return Carries{f, f + states, f + 2 * states, nullptr, nullptr};
}

// Every row's channels of x, dt, z and the output on 16-byte boundaries.
template <typename T>
bool wide_rows(const ScanParams &p, const void *out) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.dt) | reinterpret_cast<uintptr_t>(p.z) |
                           reinterpret_cast<uintptr_t>(out);
    constexpr int per = 16 / sizeof(T);
    return bits % 16 == 0 && (p.C / p.G) % per == 0 && p.x_stride % per == 0 && p.dt_stride % per == 0 &&
           (!p.z || p.z_stride % per == 0);
}

struct PrefillLaunch {
    ScanParams p;
    void *y;
    float *fin;
    ScanPlan plan;
    Carries carry;
    int blocks;
    cudaStream_t s;
    template <typename T, int S, int L, bool WIDE>
    void launch() {
        if (plan.carries) {
            scan_rows_kernel<T, S, L, WIDE, kEnds><<<dim3((unsigned)plan.chunks - 1, (unsigned)blocks), kScanThreads, 0, s>>>(
                p, nullptr, nullptr, plan, carry);
            const long long size = (long long)p.C * p.N;
            if (!plan.folded()) scan_carry_kernel<<<(unsigned)((size + 127) / 128), 128, (size_t)plan.chunks, s>>>(p, plan, carry);
        }
        scan_rows_kernel<T, S, L, WIDE, kOutputs><<<dim3((unsigned)plan.chunks, (unsigned)blocks), kScanThreads, 0, s>>>(
            p, static_cast<T *>(y), fin, plan, carry);
    }
    template <typename T, int S, int L>
    void operator()() {
        wide_rows<T>(p, y) ? launch<T, S, L, true>() : launch<T, S, L, false>();
    }
};

struct StatesLaunch {
    ScanParams p;
    ScanPlan plan;
    Carries carry;
    int blocks;
    cudaStream_t s;
    template <typename T, int S, int L, bool WIDE>
    void launch() {
        scan_rows_kernel<T, S, L, WIDE, kStates><<<dim3((unsigned)plan.chunks, (unsigned)blocks), kScanThreads, 0, s>>>(
            p, nullptr, nullptr, plan, carry);
        if (!plan.carries) return;
        const long long size = (long long)p.C * p.N;
        scan_carry_kernel<<<(unsigned)((size + 127) / 128), 128, (size_t)plan.chunks, s>>>(p, plan, carry);
    }
    template <typename T, int S, int L>
    void operator()() {
        wide_rows<T>(p, nullptr) ? launch<T, S, L, true>() : launch<T, S, L, false>();
    }
};

struct BackEndsLaunch {
    ScanParams p;  // x is dy
    float *d_fin;
    ScanPlan plan;
    Carries carry;
    int blocks;
    cudaStream_t s;
    template <typename T, int S, int L, bool WIDE>
    void launch() {
        scan_rows_kernel<T, S, L, WIDE, kBackEnds><<<dim3((unsigned)plan.chunks - 1, (unsigned)blocks), kScanThreads, 0, s>>>(
            p, nullptr, d_fin, plan, carry);
        const long long size = (long long)p.C * p.N;
        scan_back_carry_kernel<<<(unsigned)((size + 127) / 128), 128, (size_t)plan.chunks, s>>>(p, plan, carry);
    }
    template <typename T, int S, int L>
    void operator()() {
        wide_rows<T>(p, nullptr) ? launch<T, S, L, true>() : launch<T, S, L, false>();
    }
};

// One token: bound by HBM, the state is read and written once. LP lanes hold a channel's states, V consecutive ones each
// (16 bytes where N and the addresses allow it), so that a warp streams whole 512-byte runs of the state; the parts of y
// are added by shuffles. This form takes any sizes and addresses, two sequences per thread.
template <typename T, int LP, int V>
__global__ void __launch_bounds__(128) scan_decode_kernel(ScanParams p, float *state, T *__restrict__ y, bool wide_bc) {
    constexpr int PAIRS = 1, SEQS = 2 * PAIRS;
    const int k = blockIdx.y * (128 / LP) + threadIdx.x / LP, l = threadIdx.x % LP;
    const bool live = k < p.C;
    const int c = live ? k : p.C - 1;
    const int g = c / (p.C / p.G);
    const int first = blockIdx.x * SEQS;
    long long from[SEQS], to[SEQS];
    float x[SEQS], dt[SEQS], z[SEQS];
    Pack<float, V> h[SEQS];
    Pack<T, V> bs[SEQS], cs[SEQS];
    const T *Z = static_cast<const T *>(p.z);
    auto load = [&](int s, int n0) {  // the states n0.. of sequence s, and B and C at them
        const int n = first + s;
        if (from[s] >= 0) {
            h[s] = load_pack<float, V>(state + (from[s] * p.C + c) * p.N + n0);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) h[s].e[v] = 0.f;
        }
        const T *B = static_cast<const T *>(p.Bm) + n * p.B_stride + g * p.N + n0;
        const T *Cm = static_cast<const T *>(p.Cm) + n * p.C_stride + g * p.N + n0;
        if (wide_bc) {
            bs[s] = load_pack<T, V>(B);
            cs[s] = load_pack<T, V>(Cm);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                bs[s].e[v] = B[v];
                cs[s].e[v] = Cm[v];
            }
        }
    };
    const int start = l * V;
#pragma unroll
    for (int s = 0; s < SEQS; ++s) {
        const int n = first + s;
        from[s] = to[s] = -1;
        x[s] = dt[s] = z[s] = 0.f;
        if (n >= p.seqs.n_seqs) continue;
        from[s] = state_slot(p.init_idx, p.pool, n, p.err);
        to[s] = p.fin_idx == p.init_idx ? from[s] : state_slot(p.fin_idx, p.pool, n, p.err);
        x[s] = to_float(static_cast<const T *>(p.x)[n * p.x_stride + c]);
        dt[s] = to_float(static_cast<const T *>(p.dt)[n * p.dt_stride + c]);
        if (Z) z[s] = to_float(Z[n * p.z_stride + c]);
        if (start < p.N) load(s, start);
    }
    const float bias = p.dt_bias ? p.dt_bias[c] : 0.f, skip = p.D ? p.D[c] : 0.f;
    Pack<float, V> a;
    if (start < p.N) a = load_pack<float, V>(p.A + (long long)c * p.N + start);
#pragma unroll
    for (int q = 0; q < PAIRS; ++q) {
        f32x2 dt2 = add2(pair(dt[2 * q], dt[2 * q + 1]), both(bias));
        if (p.softplus) dt2 = softplus2(dt2);
        unpair(dt2, dt[2 * q], dt[2 * q + 1]);
    }
    float sum[SEQS];
#pragma unroll
    for (int s = 0; s < SEQS; ++s) {
        const int n = first + s;
        sum[s] = 0.f;
        if (n >= p.seqs.n_seqs) continue;
        const float u = dt[s] * x[s];
        for (int n0 = start; n0 < p.N; n0 += LP * V) {
            if (n0 != start) {
                load(s, n0);
                a = load_pack<float, V>(p.A + (long long)c * p.N + n0);
            } else if (s > 0 && start + LP * V < p.N) {
                a = load_pack<float, V>(p.A + (long long)c * p.N + n0);
            }
#pragma unroll
            for (int v = 0; v < V; ++v)
                h[s].e[v] = fmaf(decay(dt[s], a.e[v] * kLog2e), h[s].e[v], u * to_float(bs[s].e[v]));
            float part = to_float(cs[s].e[0]) * h[s].e[0];
            if constexpr (V == 4) {  // in the other form's order, so that alignment does not change a result
                const float *hv = h[s].e;
                part = fmaf(to_float(cs[s].e[0]), hv[0], to_float(cs[s].e[2]) * hv[2]) +
                       fmaf(to_float(cs[s].e[1]), hv[1], to_float(cs[s].e[3]) * hv[3]);
            }
            sum[s] = n0 == start ? part : sum[s] + part;
            if (to[s] >= 0 && live) store_pack<float, V>(state + (to[s] * p.C + c) * p.N + n0, h[s]);
        }
#pragma unroll
        for (int m = LP / 2; m > 0; m >>= 1) sum[s] += __shfl_xor_sync(0xffffffffu, sum[s], m);
    }
#pragma unroll
    for (int q = 0; q < PAIRS; ++q) {
        f32x2 y2 = fma2(both(skip), pair(x[2 * q], x[2 * q + 1]), pair(sum[2 * q], sum[2 * q + 1]));
        if (Z) y2 = mul2(y2, silu2(pair(z[2 * q], z[2 * q + 1])));
        float out[2];
        unpair(y2, out[0], out[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int n = first + 2 * q + e;
            if (live && l == 0 && n < p.seqs.n_seqs) y[(long long)n * p.C + c] = from_float<T>(out[e]);
        }
    }
}

// The same for the usual sizes (up to 64 states, rows on 4-byte boundaries): a warp keeps the A of its channels (32 of them
// with up to 16 states) and walks over sequences, whose states and inputs come through a ring in shared memory two steps of two
// sequences ahead. The time steps and the gate are computed by one lane per channel and handed to the lanes of its
// states. 256 sequences of 4096 channels x 16 states: 18.5 us, against 50 us for the form above, whose short-lived blocks have no load
// in flight half of their time and whose lanes repeat a channel's time step.
constexpr int kStreamBlocks = 4;

template <typename T, int LP>
struct Decode {
    static constexpr int R = LP < 4 ? LP : 4, CH = 32 / LP, CW = R * CH;  // words per lane, channels per word, channels
    struct Stage {
        float4 state[R][32];
        T x[CW], dt[CW], z[CW];
        T B[4 * LP], C[4 * LP];
    };
};

template <typename T, int LP>
__global__ void __launch_bounds__(128) scan_decode_stream_kernel(ScanParams p, float *state, T *__restrict__ y, int walkers) {
    using D = Decode<T, LP>;
    constexpr int R = D::R, CH = D::CH, CW = D::CW, STAGES = 3;
    extern __shared__ __align__(16) unsigned char memory[];
    const int lane = threadIdx.x % 32, l = lane % LP;
    const int block = blockIdx.x * 4 + threadIdx.x / 32;  // the warp's channel block
    if (block * CW >= p.C) return;
    const int c0 = block * CW, g = c0 / (p.C / p.G);
    const int own = lane % CW;                            // the channel that the lane computes time step and gate of
    const bool in = 4 * l < p.N;
    auto mine = reinterpret_cast<typename D::Stage(*)[2]>(memory) + threadIdx.x / 32 * STAGES;
    const int walker = blockIdx.y;
    const int count = (p.seqs.n_seqs - walker + walkers - 1) / walkers;  // the warp's sequences: walker, walker + walkers, ...
    const T *Z = static_cast<const T *>(p.z);
    int from32 = 0, to32 = 0;  // the slots of 32 of them, one per lane
    auto slots = [&](int i0) {
        const int n = walker + (i0 + lane) * walkers;
        from32 = to32 = -1;
        if (n < p.seqs.n_seqs) {
            from32 = (int)state_slot(p.init_idx, p.pool, n, p.err);
            to32 = p.fin_idx == p.init_idx ? from32 : (int)state_slot(p.fin_idx, p.pool, n, p.err);
        }
    };
    auto words = [&](T *to, const T *from, int values) {  // at most 32 words of 4 bytes, one per lane; more for fp32 B and C
        constexpr int PER = 4 / sizeof(T);
        for (int i = lane * PER; i < values; i += 32 * PER)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((unsigned)__cvta_generic_to_shared(to + i)), "l"(from + i)
                         : "memory");
    };
    const long long at_lane = (long long)(c0 + lane / LP) * p.N + 4 * l;  // of the lane's first word in a state
    auto bring = [&](int i, int stage) {  // sequences i and i + 1 of the warp's
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int slot = __shfl_sync(0xffffffffu, from32, (i + e) % 32);
            if (i + e >= count) continue;
            const long long n = walker + (long long)(i + e) * walkers;
            typename D::Stage &st = mine[stage][e];
            if (in && slot >= 0) {
                const float *from = state + (long long)slot * p.C * p.N + at_lane;
#pragma unroll
                for (int j = 0; j < R; ++j) copy16(&st.state[j][lane], from + j * CH * p.N);
            }
            words(st.x, static_cast<const T *>(p.x) + n * p.x_stride + c0, CW);
            words(st.dt, static_cast<const T *>(p.dt) + n * p.dt_stride + c0, CW);
            if (Z) words(st.z, Z + n * p.z_stride + c0, CW);
            words(st.B, static_cast<const T *>(p.Bm) + n * p.B_stride + g * p.N, p.N);
            words(st.C, static_cast<const T *>(p.Cm) + n * p.C_stride + g * p.N, p.N);
        }
        copies_issued();
    };
    f32x2 A[R][2];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const float4 v = in ? *reinterpret_cast<const float4 *>(p.A + at_lane + j * CH * p.N) : make_float4(0.f, 0.f, 0.f, 0.f);
        A[j][0] = pair(v.x * kLog2e, v.y * kLog2e);
        A[j][1] = pair(v.z * kLog2e, v.w * kLog2e);
    }
    const f32x2 bias = both(p.dt_bias ? p.dt_bias[c0 + own] : 0.f), skip = both(p.D ? p.D[c0 + own] : 0.f);
    for (int i0 = 0; i0 < count; i0 += 32) {
        slots(i0);
        const int stop = min(count, i0 + 32);
        auto bring_up_to = [&](int i, int stage) {
            if (i < stop)
                bring(i, stage);
            else
                copies_issued();
        };
#pragma unroll
        for (int k = 0; k < STAGES - 1; ++k) bring_up_to(i0 + 2 * k, k);
        int stage = 0;
        for (int i = i0; i < stop; i += 2) {
            copies_arrived<STAGES - 2>();
            __syncwarp();  // every lane's copies of this step are there, and the step before is read
            bring_up_to(i + 2 * (STAGES - 1), stage == 0 ? STAGES - 1 : stage - 1);
            const auto &st = mine[stage];
            f32x2 dt = add2(pair(to_float(st[0].dt[own]), to_float(st[1].dt[own])), bias);
            if (p.softplus) dt = softplus2(dt);
            const f32x2 x = pair(to_float(st[0].x[own]), to_float(st[1].x[own]));
            float dts[2], us[2], sums[2];
            unpair(dt, dts[0], dts[1]);
            unpair(mul2(dt, x), us[0], us[1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int from = __shfl_sync(0xffffffffu, from32, (i + e) % 32), to = __shfl_sync(0xffffffffu, to32, (i + e) % 32);
                f32x2 b01 = 0, b23 = 0, c01 = 0, c23 = 0;
                if (in) {
                    const T *b = st[e].B + 4 * l, *cc = st[e].C + 4 * l;
                    b01 = pair(to_float(b[0]), to_float(b[1]));
                    b23 = pair(to_float(b[2]), to_float(b[3]));
                    c01 = pair(to_float(cc[0]), to_float(cc[1]));
                    c23 = pair(to_float(cc[2]), to_float(cc[3]));
                }
                float v[R];  // the lane's part of y of its channels
                float *out = state + (long long)to * p.C * p.N + at_lane;
                const bool write = i + e < stop && to >= 0 && in;
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    const float4 h = in && from >= 0 ? st[e].state[j][lane] : make_float4(0.f, 0.f, 0.f, 0.f);
                    const f32x2 t2 = both(__shfl_sync(0xffffffffu, dts[e], j * CH + lane / LP));
                    const f32x2 u2 = both(__shfl_sync(0xffffffffu, us[e], j * CH + lane / LP));
                    const f32x2 h01 = fma2(decay2(t2, A[j][0]), pair(h.x, h.y), mul2(u2, b01));
                    const f32x2 h23 = fma2(decay2(t2, A[j][1]), pair(h.z, h.w), mul2(u2, b23));
                    float lo, hi;
                    unpair(fma2(c01, h01, mul2(c23, h23)), lo, hi);
                    v[j] = lo + hi;
                    if (write) {
                        float4 o;
                        unpair(h01, o.x, o.y);
                        unpair(h23, o.z, o.w);
                        *reinterpret_cast<float4 *>(out + j * CH * p.N) = o;
                    }
                }
                // Over the lanes of a channel, each step halving the channels that a lane keeps.
#pragma unroll
                for (int m = LP / 2; m >= R; m >>= 1)
#pragma unroll
                    for (int j = 0; j < R; ++j) v[j] += __shfl_xor_sync(0xffffffffu, v[j], m);
                int left = R;
#pragma unroll
                for (int m = R / 2; m > 0; m >>= 1) {
                    left /= 2;
                    const bool upper = l & m;
#pragma unroll
                    for (int j = 0; j < R / 2; ++j) {
                        if (j >= left) break;
                        const float keep = upper ? v[left + j] : v[j], send = upper ? v[j] : v[left + j];
                        v[j] = keep + __shfl_xor_sync(0xffffffffu, send, m);
                    }
                }
                sums[e] = __shfl_sync(0xffffffffu, v[0], own % CH * LP + own / CH);  // to the lane that owns the channel
            }
            f32x2 y2 = fma2(skip, x, pair(sums[0], sums[1]));
            if (Z) y2 = mul2(y2, silu2(pair(to_float(st[0].z[own]), to_float(st[1].z[own]))));
            unpair(y2, sums[0], sums[1]);
            if (lane < CW) {
                const long long n = walker + (long long)i * walkers;
                y[n * p.C + c0 + own] = from_float<T>(sums[0]);
                if (i + 1 < stop) y[(n + walkers) * p.C + c0 + own] = from_float<T>(sums[1]);
            }
            stage = stage == STAGES - 1 ? 0 : stage + 1;
        }
        copies_arrived<0>();
        __syncwarp();
    }
}

template <typename T, int LP>
cudaError_t launch_stream(const ScanParams &p, float *state, void *y, cudaStream_t s) {
    using D = Decode<T, LP>;
    constexpr int bytes = 4 * 3 * 2 * sizeof(typename D::Stage);
    static_assert(bytes <= 100 * 1024, "two blocks per SM");
    const cudaError_t e = cudaFuncSetAttribute(scan_decode_stream_kernel<T, LP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    // Walkers per channel block: kStreamBlocks blocks per SM in all, two sequences at least for each.
    const unsigned cols = (unsigned)((p.C / D::CW + 3) / 4);
    const int most = (p.seqs.n_seqs + 1) / 2;
    int walkers = (int)(152LL * kStreamBlocks / cols);
    walkers = walkers < 1 ? 1 : walkers > most ? most : walkers;
    scan_decode_stream_kernel<T, LP><<<dim3(cols, (unsigned)walkers), 128, bytes, s>>>(p, state, static_cast<T *>(y), walkers);
    return cudaGetLastError();
}

// Whether the streaming form fits the call, and its launch.
template <typename T>
bool launch_decode_stream(const ScanParams &p, float *state, void *y, cudaStream_t s, cudaError_t &e) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.dt) | reinterpret_cast<uintptr_t>(p.z) |
                           reinterpret_cast<uintptr_t>(p.Bm) | reinterpret_cast<uintptr_t>(p.Cm);
    const long long strides = p.x_stride | p.dt_stride | p.z_stride | p.B_stride | p.C_stride;
    int LP = 1;
    while (4 * LP < p.N) LP *= 2;
    const int channels = LP <= 4 ? 32 : 128 / LP;
    if (p.N % 4 != 0 || LP > 16 || bits % 4 != 0 || strides % (4 / (long long)sizeof(T)) != 0 || (p.C / p.G) % channels != 0 ||
        !aligned16(state) || !aligned16(p.A))
        return false;
    switch (LP) {
        case 1: e = launch_stream<T, 1>(p, state, y, s); break;
        case 2: e = launch_stream<T, 2>(p, state, y, s); break;
        case 4: e = launch_stream<T, 4>(p, state, y, s); break;
        case 8: e = launch_stream<T, 8>(p, state, y, s); break;
        default: e = launch_stream<T, 16>(p, state, y, s); break;
    }
    return true;
}

template <typename T, int V>
void launch_decode(const ScanParams &p, float *state, void *y, cudaStream_t s) {
    const int words = (p.N + V - 1) / V;
    T *out = static_cast<T *>(y);
    const bool wide_bc = (reinterpret_cast<uintptr_t>(p.Bm) | reinterpret_cast<uintptr_t>(p.Cm)) % (V * sizeof(T)) == 0 &&
                         p.B_stride % V == 0 && p.C_stride % V == 0;
#define KDA_DECODE(LP)                                                                                                    \
    scan_decode_kernel<T, LP, V><<<dim3((unsigned)(p.seqs.n_seqs + 1) / 2, (unsigned)((p.C + 128 / LP - 1) / (128 / LP))), \
                                   128, 0, s>>>(p, state, out, wide_bc)
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

// Whole sequences where they give every SM a block; otherwise chunks that give it two: with three or
// four, and registers for as many, one sequence of 16384 rows and 4096 channels took 3 and 8 % longer. A row of a short chunk costs 0.35 us in both kernels together, a
// chunk 1/16 us in the walk over them, so a chunk has at least sqrt(rows / 6) rows.
ScanPlan scan_plan(const kda_scan_args &a, int sms) {
    const long long rows = (long long)a.B * a.T, blocks = scan_blocks(a);
    if (rows == 0) return ScanPlan{0, 1, false};
    if (sms <= 0) sms = 152;
    if (!a.cu_seqlens && (a.B * blocks >= sms || a.T <= 32)) return ScanPlan{a.B, a.T, false};
    long long least = 16;
    while (least * least * 6 < rows) least += 16;
    const long long chunks = std::max(1LL, std::min((rows + least - 1) / least, 2LL * sms / blocks));
    const long long per = ((rows + chunks - 1) / chunks + 15) / 16 * 16;
    const int count = (int)((rows + per - 1) / per);
    return ScanPlan{count, per, count > 1};
}

size_t scan_prefill_workspace_bytes(const kda_scan_args &a, int sms) {
    const ScanPlan plan = scan_plan(a, sms);
    return plan.carries ? (size_t)plan.chunks * a.D * (2 * a.N + 1) * sizeof(float) : 0;
}

cudaError_t launch_scan_prefill(const kda_scan_args &a, void *y, float *final_state, void *ws, int sms, unsigned *err,
                                cudaStream_t s) {
    if ((long long)a.B * a.T == 0) {
        const ScanParams p = scan_params(a, err);
        scan_no_rows_kernel<<<(unsigned)p.seqs.n_seqs, 128, 0, s>>>(p, final_state);
        return cudaGetLastError();
    }
    const ScanPlan plan = scan_plan(a, sms);
    return scan_by_type(a, PrefillLaunch{scan_params(a, err), y, final_state, plan, carries_in(a, plan, ws), scan_blocks(a), s});
}

cudaError_t launch_scan_states(const kda_scan_args &a, const ScanPlan &plan, const Carries &carry, unsigned *err, cudaStream_t s) {
    return scan_by_type(a, StatesLaunch{scan_params(a, err), plan, carry, scan_blocks(a), s});
}

cudaError_t launch_scan_back_ends(const kda_scan_args &a, const void *dy, const float *d_final, const ScanPlan &plan,
                                  const Carries &carry, unsigned *err, cudaStream_t s) {
    ScanParams p = scan_params(a, err);
    p.x = dy;
    p.x_stride = a.D;
    return scan_by_type(a, BackEndsLaunch{p, const_cast<float *>(d_final), plan, carry, scan_blocks(a), s});
}

cudaError_t launch_scan_decode(const kda_scan_args &a, float *state, void *y, unsigned *err, cudaStream_t s) {
    ScanParams p = scan_params(a, err);
    if (!p.fin_idx) p.fin_idx = p.init_idx;
    cudaError_t e = cudaSuccess;
    if (a.dtype == KDA_BF16 ? launch_decode_stream<__nv_bfloat16>(p, state, y, s, e) : launch_decode_stream<float>(p, state, y, s, e))
        return e;
    const bool wide = p.N % 4 == 0 && aligned16(state) && aligned16(p.A);  // four states per load
    if (a.dtype == KDA_BF16)
        wide ? launch_decode<__nv_bfloat16, 4>(p, state, y, s) : launch_decode<__nv_bfloat16, 1>(p, state, y, s);
    else
        wide ? launch_decode<float, 4>(p, state, y, s) : launch_decode<float, 1>(p, state, y, s);
    return cudaGetLastError();
}

}  // namespace kda
