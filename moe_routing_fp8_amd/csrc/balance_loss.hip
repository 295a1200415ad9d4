// The router's balance loss over packed sequences, its per-expert counts and
// its gradient.
//
// With p[t, :] the normalised scores of token t (softmax of the logits, or
// their sigmoids divided by the row's sum), n_s the live tokens of sequence
// s, c[s, e] the copies its live tokens send to expert e and P[s, e] the sum
// of their p[t, e]:
//   loss[s]  = E / (K n_s^2) * sum_e c[s, e] P[s, e]
//   dz[t, j] = g_s p_j (c[s, j] - sum_e c[s, e] p_e)   [* (1 - sigmoid(z_j))]
//   g_s      = grad_loss[s] * E / (K n_s^2)
// (the counts are whole numbers and carry no gradient).
//
// Forward, one to three launches.  The tokens are cut into chunks of consecutive
// tokens, one workgroup each; 16 lanes (64 above 256 experts) hold a token's
// whole row of logits in registers and keep their running sums of p there
// too.  A chunk may meet several sequences: each (chunk, sequence) piece is
// summed over the workgroup's waves in a fixed order and written to a slot of its own,
// number chunk + sequence (along the pieces in token order either index
// grows, so no two pieces share a slot, and a sequence's slots are
// consecutive).  Then each sequence's slots are added in a fixed order: by one
// workgroup per sequence in a second launch where it has few, else by
// workgroups that take a few columns each, with the loss in a third launch.  A
// batch of one chunk takes its losses in the first launch.
// No floating atomics: the results do not depend on timing.
//
// Kernel traces (sums, slots, [loss], gradient); a kernel that does nothing takes 1.3 us there:
//   32768 x 256 fp32, one sequence      11.5 + 4.8 + 2.4 + 12.4 us; the sums read 2.9 to 3.3 TB/s: as many
//                                       steps of the row reductions and exponentials as loads
//   the same with sigmoid scores        14.6 + 4.8 + 2.4 + 15.6 us
//   the same in 20 sequences, one of    17.0 + 26.5 + 11.8 us: one workgroup adds the long one's thousand slots
//   30000 tokens
//   4096 x 256 bf16, eight sequences    8.8 + 5.2 + 5.4 us, latency (sigmoid scores)
//   10007 x 61 fp32, 311 sequences      9.2 + 4.1 + 5.8 us, latency
//   64 x 16 fp32, one sequence          4.4 us in one launch, latency
// Backward, one launch: the same lanes per token read the row again, with the
// sequence's counts in registers.
//
// Sixteen lanes per row let the four row reductions of a wave run in the same
// four DPP steps; with a row over all 64 lanes the reductions, six steps for
// each row, took as many instructions as the exponentials.
#include <hip/hip_runtime.h>

#include "api_common.hpp"
#include "math_device.hpp"
#include "moe_fp8.h"

namespace moe {
namespace {

constexpr int kMaxWaves = 16;
constexpr int kNarrowExperts = 256;  // rows of up to this many experts lie over 16 lanes

// How a row lies over the lanes: L lanes hold it, P values each; a wave has
// 64 / L rows side by side.
template <int L_, int P_>
struct RowShape {
    static constexpr int L = L_, P = P_;
    static constexpr int kRows = kWave / L;
};
int rows_per_wave(int E) { return E > kNarrowExperts ? RowShape<64, 16>::kRows : RowShape<16, 16>::kRows; }

// Chunks of a batch.  One sequence (or few): about one for each of the 256
// compute units, since all their slots have to be added up for one result
// (32768 tokens, 256 experts: sums and their reduction take 10.7 + 5.1 us in
// 256 chunks, 15.3 + 6.4 us in 512).  Many sequences: smaller chunks, which
// meet fewer of them one after another.
constexpr int64_t kFewSeqsChunks = 256;
constexpr int64_t kManySeqsChunks = 1024;
constexpr int kManySeqs = 4;
// Batches of one chunk take one launch: up to this many steps of a workgroup of kMaxWaves waves (256 tokens up to
// 256 experts), which take less than a second launch, and this many sequences, whose losses are taken in turn.
constexpr int64_t kOneLaunchSteps = 4;
constexpr int kOneLaunchSeqs = 8;
// Up to this many slots per sequence, on average, one workgroup adds all of a sequence's; above, its columns are
// split over workgroups and the loss takes a launch of its own.  The offsets are on the device, so the average is
// all that the host knows: one sequence that has most of the slots of 20 takes 26 us here.
constexpr int64_t kOneLevelSlots = 64;
constexpr int kReduceCols = 16;  // columns of a workgroup of the split sum: 64-byte pieces of each slot

struct BalancePlan {
    bool one_launch;     // one chunk, whose workgroup also takes the losses
    int waves;           // of a workgroup
    int64_t chunk;       // tokens per workgroup: a multiple of waves * rows_per_wave
    int64_t num_chunks;
    int64_t num_slots;   // num_chunks + num_seqs
    size_t sums_bytes, counts_bytes, tokens_bytes;
    size_t means_offset;  // a table [S, E] for calls that do not take prob_mean
    size_t workspace_bytes;
};

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

BalancePlan plan_balance(int64_t T, int E, int S) {
    BalancePlan p;
    const int64_t most = S >= kManySeqs ? kManySeqsChunks : kFewSeqsChunks;
    const int64_t rows = rows_per_wave(E);
    p.one_launch = T > 0 && T <= kOneLaunchSteps * kMaxWaves * rows && S <= kOneLaunchSeqs;
    p.waves = p.one_launch ? kMaxWaves : 4;
    while (p.one_launch && p.waves > 4 && T <= p.waves / 2 * rows) p.waves /= 2;
    while (!p.one_launch && p.waves < kMaxWaves && T > p.waves * rows * most) p.waves *= 2;
    const int64_t step = p.waves * rows;
    const int64_t chunks = p.one_launch ? 1 : most;
    const int64_t steps = (T + step * chunks - 1) / (step * chunks);
    p.chunk = step * (steps > 1 ? steps : 1);
    p.num_chunks = (T + p.chunk - 1) / p.chunk;
    p.num_slots = p.num_chunks + S;
    p.sums_bytes = round256(static_cast<size_t>(p.num_slots) * E * sizeof(float));
    p.counts_bytes = round256(static_cast<size_t>(p.num_slots) * E * sizeof(int32_t));
    p.tokens_bytes = round256(static_cast<size_t>(p.num_slots) * sizeof(int32_t));
    p.means_offset = p.sums_bytes + p.counts_bytes + p.tokens_bytes;
    p.workspace_bytes = p.means_offset + round256(static_cast<size_t>(S) * E * sizeof(float));
    return p;
}

// The sequences: offsets == nullptr is one sequence of all tokens.  Offsets
// are clamped to [0, T], so no value of theirs leads out of range.
struct Seqs {
    const int32_t* offsets;
    int64_t num_tokens;
    int num_seqs;
    __device__ int64_t edge(int s) const {
        if (offsets == nullptr) return s <= 0 ? 0 : num_tokens;
        const int64_t o = offsets[s];
        return o < 0 ? 0 : o > num_tokens ? num_tokens : o;
    }
    // The number of sequence ends at or before token t: the sequence that
    // holds t, if t >= edge(it); num_seqs past the last one.  Every lane of
    // the wave takes part.
    __device__ int find(int64_t t, int lane) const {
        if (offsets == nullptr) return 0;
        int n = 0;
        for (int i = 1 + lane; i - lane <= num_seqs; i += 4 * kWave) {
            int32_t o[4];  // four loads in flight
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = i + k * kWave <= num_seqs ? offsets[i + k * kWave] : INT32_MAX;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool before = i + k * kWave <= num_seqs && min(static_cast<int64_t>(o[k]), num_tokens) <= t;
                n += __builtin_popcountll(__ballot(before));
            }
        }
        return n;
    }
};

// edge(i) for consecutive i, 64 of them held over the wave's lanes.
struct EdgeWindow {
    const Seqs& seqs;
    int base;
    int64_t held;  // of lane l: edge(base + l)
    __device__ void load(int i, int lane) {
        base = i;
        held = seqs.edge(min(i + lane, seqs.num_seqs));
    }
    __device__ int64_t get(int i, int lane) {  // i uniform over the wave
        if (i < base || i >= base + kWave) load(i, lane);
        return __builtin_amdgcn_readlane(static_cast<int>(held), i - base);  // at most num_tokens < 2^31
    }
};

// The expert of lane l's j-th value: vectors of V in turn over the lanes.
template <typename S, int V>
__device__ __forceinline__ int expert_of(int l, int j) { return ((j / V) * S::L + l) * V + j % V; }

// Lane l's values of a row of E (V > 1: E % V == 0 and aligned vectors); the padding gets `fill`.
template <typename TL, typename S, int V>
__device__ __forceinline__ void load_row(const void* p, int64_t at, int E, int l, float fill, float (&z)[S::P]) {
#pragma unroll
    for (int j = 0; j < S::P; j += V) {
        const int e = expert_of<S, V>(l, j);
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = fill;
        if (e < E) TL::template load<V>(p, at + e, v);
#pragma unroll
        for (int i = 0; i < V; ++i) z[j + i] = v[i];
    }
}
template <typename TL, typename S, int V>
__device__ __forceinline__ void store_row(void* p, int64_t at, int E, int l, const float (&d)[S::P]) {
#pragma unroll
    for (int j = 0; j < S::P; j += V) {
        const int e = expert_of<S, V>(l, j);
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = d[j + i];
        if (e < E) TL::template store<V>(p, at + e, v);
    }
}

// 1 / v for v in [1, 2]: the hardware's estimate and one Newton step (1 ulp).
__device__ __forceinline__ float rcp_f32(float v) {
    const float r = __builtin_amdgcn_rcpf(v);
    return __builtin_fmaf(__builtin_fmaf(-v, r, 1.0f), r, r);
}

// The unnormalised scores w of a row (0 at the padding, whose logit is -inf)
// and the factor that makes them p; comp = 1 - sigmoid(z) with SIGMOID.  A
// row of nothing but -inf gives p = 0.
//
// sigmoid(z) = r or t r with t = exp(-|z|), r = 1 / (1 + t).  Where every
// logit of a row is below -60 the sigmoids leave the range in which their
// ratio keeps 24 bits, so they are taken relative to the largest logit m:
// sigmoid(z) exp(-m) = exp(z - m) r.
template <typename S, bool SIGMOID>
__device__ __forceinline__ float row_scores(const float (&z)[S::P], float (&w)[S::P], float (&comp)[S::P]) {
    float m = z[0];
#pragma unroll
    for (int j = 1; j < S::P; ++j) m = fmaxf(m, z[j]);
    m = group_max_f32<S::L>(m);
    const bool nothing = m == -INFINITY;
    if (nothing) m = 0.0f;
    float sum = 0.0f;
    if constexpr (SIGMOID) {
        const bool low = m < -60.0f;
#pragma unroll
        for (int j = 0; j < S::P; ++j) {
            const float t = exp_nonpos_exact(-fabsf(z[j]));
            const float r = rcp_f32(1.0f + t);
            w[j] = z[j] > 0.0f ? r : t * r;
            comp[j] = z[j] > 0.0f ? t * r : r;
            if (low) w[j] = exp_nonpos(z[j] - m) * r;
        }
    } else {
#pragma unroll
        for (int j = 0; j < S::P; ++j) w[j] = exp_nonpos(z[j] - m);
    }
#pragma unroll
    for (int j = 0; j < S::P; ++j) sum += w[j];
    sum = group_sum_f32<S::L>(sum);
    return nothing ? 0.0f : 1.0f / sum;
}

// loss = E / (K n) * sum over e of count * mean, from that sum.
__device__ __forceinline__ float loss_value(float dot, int E, int K, float many) {
    return dot * (static_cast<float>(E) / static_cast<float>(K)) / many;
}

// The outputs, for a batch of one chunk (else all nullptr).
struct Outputs {
    float* loss;
    int32_t* counts;
    int32_t* seq_tokens;
    float* prob_mean;
};

template <typename TL, typename S, int V, bool SIGMOID>
__global__ __launch_bounds__(kMaxWaves* kWave) void balance_sums_kernel(
    const void* __restrict__ logits, int64_t stride, int E, const int64_t* __restrict__ topk_idx, int K,
    const uint8_t* __restrict__ mask, Seqs seqs, int64_t chunk, float* __restrict__ sums,
    int32_t* __restrict__ counts, int32_t* __restrict__ tokens, Outputs out) {
    constexpr int P = S::P;
    extern __shared__ float lds[];  // waves x E sums, then E counts, one token count and a sum of each wave
    const int waves = blockDim.x / kWave;
    int32_t* hist = reinterpret_cast<int32_t*>(lds + waves * E);
    int32_t* live = hist + E;
    float* wave_dot = reinterpret_cast<float*>(live + 1);
    const int lane = threadIdx.x & (kWave - 1), l = lane % S::L, row = lane / S::L;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t t0 = blockIdx.x * chunk;
    const int64_t t1 = min(t0 + chunk, seqs.num_tokens);
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
    if (threadIdx.x == 0) *live = 0;
    if (out.loss != nullptr) {  // sequences without tokens; the others are written once, below
        for (int i = 0; i < seqs.num_seqs; ++i) {
            if (seqs.edge(i) < seqs.edge(i + 1)) continue;
            for (int e = threadIdx.x; e < E; e += blockDim.x) {
                out.counts[i * E + e] = 0;
                if (out.prob_mean != nullptr) out.prob_mean[i * E + e] = 0.0f;
            }
            if (threadIdx.x == 0) {
                out.loss[i] = 0.0f;
                out.seq_tokens[i] = 0;
            }
        }
    }

    float acc[P];
#pragma unroll
    for (int j = 0; j < P; ++j) acc[j] = 0.0f;
    int n = 0;  // live tokens of the lane's row
    int s = 0;
    EdgeWindow edges{seqs, 0, 0};
    // Writes sequence s's slot and starts afresh (every wave of the workgroup).
    auto flush = [&]() {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int e = expert_of<S, V>(l, j);
            if constexpr (S::L < kWave) acc[j] = join_rows(acc[j], [](float a, float b) { return a + b; });
            if (row == 0 && e < E) lds[wave * E + e] = acc[j];
            acc[j] = 0.0f;
        }
        if (l == 0 && n != 0) atomicAdd(live, n);
        n = 0;
        __syncthreads();
        const int64_t slot = blockIdx.x + static_cast<int64_t>(s);
        const int all = *live;
        const float many = all > 0 ? static_cast<float>(all) : 1.0f;
        float dot = 0.0f;
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            float v = 0.0f;
#pragma unroll 4
            for (int w = 0; w < waves; ++w) v += lds[w * E + e];
            if (out.loss != nullptr) {
                v /= many;
                out.counts[s * E + e] = hist[e];
                if (out.prob_mean != nullptr) out.prob_mean[s * E + e] = v;
                dot += static_cast<float>(hist[e]) * v;
            } else {
                sums[slot * E + e] = v;
                counts[slot * E + e] = hist[e];
            }
            hist[e] = 0;
        }
        if (out.loss != nullptr) {
            dot = wave_sum_f32(dot);
            if (lane == 0) wave_dot[wave] = dot;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            *live = 0;
            if (out.loss != nullptr) {
                dot = 0.0f;
                for (int w = 0; w < waves; ++w) dot += wave_dot[w];
                out.loss[s] = loss_value(dot, E, K, many);
                out.seq_tokens[s] = all;
            } else {
                tokens[slot] = all;
            }
        }
        __syncthreads();
    };

    // A step's rows, masks and ids: none of them waits for the sequences, and
    // the next step's are on their way while this one's are worked on.
    float z[P];
    int64_t id;  // of the lane's copy, l < K
    bool on;
    auto load_step = [&](int64_t t) {
        const int64_t safe = min(t, t1 - 1);
        load_row<TL, S, V>(logits, safe * stride, E, l, -INFINITY, z);
        on = t < t1;
        if (mask != nullptr) on = on && mask[safe] != 0;
        id = -1;
        if (l < K) id = topk_idx[safe * K + l];
    };
    const int64_t step = static_cast<int64_t>(waves) * S::kRows;
    const int64_t ahead = wave * S::kRows + row;  // of the lane's token in a step
    load_step(t0 + ahead);
    s = seqs.find(t0, lane);
    edges.load(s, lane);
    __syncthreads();  // the counts are zero
    for (int64_t g = t0; g < t1; g += step) {
        const int64_t t = g + ahead;
        float w[P], comp[P];
        const float inv = row_scores<S, SIGMOID>(z, w, comp);
        const int64_t now_id = id;
        const bool now = on;
        if (g + step < t1) load_step(t + step);
        const int64_t gend = min(g + step, t1);
        while (s < seqs.num_seqs) {
            const int64_t begin = edges.get(s, lane), end = edges.get(s + 1, lane);
            if (begin >= gend) break;
            if (now && t >= begin && t < end) {
                ++n;
                if (now_id >= 0 && now_id < E) atomicAdd(&hist[now_id], 1);
#pragma unroll
                for (int j = 0; j < P; ++j) acc[j] = __builtin_fmaf(w[j], inv, acc[j]);
            }
            if (end > gend) break;  // the sequence goes on in the next step
            if (max(begin, t0) < end) flush();
            ++s;
        }
    }
    // the sequence that the chunk's end cuts
    if (s < seqs.num_seqs && edges.get(s, lane) < t1 && edges.get(s + 1, lane) > t1) flush();
}

// The slots of sequence s: first .. last (first > last: none).
__device__ __forceinline__ void seq_slots(const Seqs& seqs, int64_t chunk, int s, int64_t& first, int64_t& last) {
    const int64_t begin = seqs.edge(s), end = seqs.edge(s + 1);
    first = 0;
    last = -1;
    if (begin < end) {
        first = begin / chunk + s;
        last = (end - 1) / chunk + s;
    }
}

// The lane's share of the live tokens of slots first .. last; wave_sum_i32 adds them.
__device__ __forceinline__ int live_tokens(const int32_t* tokens, int64_t first, int64_t last, int lane) {
    int n = 0;
    for (int64_t i = first + lane; i <= last; i += kWave) n += tokens[i];
    return n;
}

// One workgroup per sequence: `cols` threads (a power of two >= E) for each
// of blockDim / cols slots at a time; each thread's slots in order, then the
// threads of a column in order, then the loss.
__global__ __launch_bounds__(1024) void balance_loss_kernel(const float* __restrict__ sums,
                                                             const int32_t* __restrict__ slot_counts,
                                                             const int32_t* __restrict__ slot_tokens, Seqs seqs,
                                                             int64_t chunk, int E, int K, int cols,
                                                             float* __restrict__ loss, int32_t* __restrict__ counts,
                                                             int32_t* __restrict__ seq_tokens,
                                                             float* __restrict__ prob_mean) {
    __shared__ float part[1024];
    __shared__ int32_t part_count[1024];
    __shared__ float part_dot[1024 / kWave];
    const int s = blockIdx.x, lane = threadIdx.x & (kWave - 1);
    const int e = threadIdx.x & (cols - 1), row = threadIdx.x / cols, rows = blockDim.x / cols;
    int64_t first, last;
    seq_slots(seqs, chunk, s, first, last);
    int n = live_tokens(slot_tokens, first, last, lane);
    float sum = 0.0f;
    int c = 0;
    if (e < E) {
#pragma unroll 4
        for (int64_t i = first + row; i <= last; i += rows) {
            sum += sums[i * E + e];
            c += slot_counts[i * E + e];
        }
    }
    part[threadIdx.x] = sum;
    part_count[threadIdx.x] = c;
    n = wave_sum_i32(n);
    const float many = n > 0 ? static_cast<float>(n) : 1.0f;
    __syncthreads();
    float dot = 0.0f;
    if (row == 0 && e < E) {
        for (int r = 1; r < rows; ++r) {
            sum += part[r * cols + e];
            c += part_count[r * cols + e];
        }
        const float mean = sum / many;
        counts[static_cast<int64_t>(s) * E + e] = c;
        if (prob_mean != nullptr) prob_mean[static_cast<int64_t>(s) * E + e] = mean;
        dot = static_cast<float>(c) * mean;
    }
    dot = wave_sum_f32(dot);
    if (lane == 0) part_dot[threadIdx.x / kWave] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < cols / kWave; ++w) dot += part_dot[w];
        loss[s] = loss_value(dot, E, K, many);
        seq_tokens[s] = n;
    }
}

// A sequence of many chunks: a workgroup adds kReduceCols columns of one sequence's slots,
// blockDim / kReduceCols of them at a time; each thread's slots in order, then
// the threads of a column in order.  Leaves the means in `means` (prob_mean,
// or a table of the workspace).
__global__ __launch_bounds__(1024) void balance_reduce_kernel(const float* __restrict__ sums,
                                                               const int32_t* __restrict__ slot_counts,
                                                               const int32_t* __restrict__ slot_tokens, Seqs seqs,
                                                               int64_t chunk, int E, int32_t* __restrict__ counts,
                                                               int32_t* __restrict__ seq_tokens,
                                                               float* __restrict__ means) {
    __shared__ float part[1024];
    __shared__ int32_t part_count[1024];
    const int s = blockIdx.y;
    const int col = threadIdx.x % kReduceCols, row = threadIdx.x / kReduceCols;
    const int rows = blockDim.x / kReduceCols;
    const int e = blockIdx.x * kReduceCols + col;
    int64_t first, last;
    seq_slots(seqs, chunk, s, first, last);
    float sum = 0.0f;
    int c = 0;
    if (e < E) {
#pragma unroll 4
        for (int64_t i = first + row; i <= last; i += rows) {
            sum += sums[i * E + e];
            c += slot_counts[i * E + e];
        }
    }
    part[threadIdx.x] = sum;
    part_count[threadIdx.x] = c;
    __syncthreads();
    if (threadIdx.x >= kWave) return;
    const int n = wave_sum_i32(live_tokens(slot_tokens, first, last, threadIdx.x));
    if (blockIdx.x == 0 && threadIdx.x == 0) seq_tokens[s] = n;
    if (row == 0 && e < E) {
        sum = 0.0f;
        c = 0;
        for (int r = 0; r < rows; ++r) {
            sum += part[r * kReduceCols + col];
            c += part_count[r * kReduceCols + col];
        }
        counts[static_cast<int64_t>(s) * E + e] = c;
        means[static_cast<int64_t>(s) * E + e] = sum / (n > 0 ? static_cast<float>(n) : 1.0f);
    }
}

// One wave per sequence: the loss from its counts and means.
__global__ __launch_bounds__(256) void balance_dot_kernel(const int32_t* __restrict__ counts,
                                                           const float* __restrict__ means,
                                                           const int32_t* __restrict__ seq_tokens, int S, int E, int K,
                                                           float* __restrict__ loss) {
    const int lane = threadIdx.x & (kWave - 1);
    const int s = blockIdx.x * (256 / kWave) + threadIdx.x / kWave;
    if (s >= S) return;
    const int64_t at = static_cast<int64_t>(s) * E;
    float dot = 0.0f;
    for (int e = lane; e < E; e += kWave) dot += static_cast<float>(counts[at + e]) * means[at + e];
    dot = wave_sum_f32(dot);
    const int n = seq_tokens[s];
    if (lane == 0) loss[s] = loss_value(dot, E, K, n > 0 ? static_cast<float>(n) : 1.0f);
}

constexpr int kGradThreads = 256;
// Waves of a large batch's gradient: 16 for each of the 256 compute units; a
// wave then has the next set's loads in flight while it works on one.
constexpr int64_t kGradWaves = 4096;

// A wave takes `sets` sets of S::kRows consecutive tokens.
template <typename TL, typename S, int V, bool SIGMOID>
__global__ __launch_bounds__(kGradThreads) void balance_grad_kernel(
    const void* __restrict__ logits, int64_t stride, int E, int K, const uint8_t* __restrict__ mask, Seqs seqs,
    int64_t sets, const int32_t* __restrict__ counts, const int32_t* __restrict__ seq_tokens,
    const float* __restrict__ grad_loss, void* __restrict__ grad) {
    constexpr int P = S::P;
    const int lane = threadIdx.x & (kWave - 1), l = lane % S::L, row = lane / S::L;
    const int64_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t t0 = (blockIdx.x * static_cast<int64_t>(kGradThreads / kWave) + wave) * sets * S::kRows;
    const int64_t t1 = min(t0 + sets * S::kRows, seqs.num_tokens);
    if (t0 >= t1) return;
    float z[P];
    bool on;
    auto load_set = [&](int64_t t) {
        const int64_t safe = min(t, t1 - 1);
        load_row<TL, S, V>(logits, safe * stride, E, l, -INFINITY, z);
        on = t < t1;
        if (mask != nullptr) on = on && mask[safe] != 0;
    };
    load_set(t0 + row);
    int s = seqs.find(t0, lane);
    EdgeWindow edges{seqs, 0, 0};
    edges.load(s, lane);
    int held = -1;  // the sequence whose scaled counts are in a[]
    float a[P] = {};
    for (int64_t g = t0; g < t1; g += S::kRows) {
        float w[P], comp[P];
        const float inv = row_scores<S, SIGMOID>(z, w, comp);
        const bool now = on;
        if (g + S::kRows < t1) load_set(g + S::kRows + row);
        // each row's own sequence: step through the ends up to the set's last row
        const int64_t t = g + row, last = min(g + S::kRows, t1) - 1;
        while (s < seqs.num_seqs && edges.get(s + 1, lane) <= g) ++s;
        int own = s;
        int64_t begin = edges.get(s, lane);
        for (int i = s; i < seqs.num_seqs; ++i) {
            const int64_t end = edges.get(i + 1, lane);
            if (end > last) break;
            if (end <= t) {
                own = i + 1;
                begin = end;
            }
        }
        const bool live = now && own < seqs.num_seqs && begin <= t;
        if (__any(live && own != held)) {
            held = min(own, seqs.num_seqs - 1);
            const float n = static_cast<float>(max(seq_tokens[held], 1));
            const float scale = grad_loss[held] * (static_cast<float>(E) / static_cast<float>(K)) / (n * n);
            load_row<I32, S, V>(counts, static_cast<int64_t>(held) * E, E, l, 0.0f, a);
#pragma unroll
            for (int j = 0; j < P; ++j) a[j] *= scale;
        }
        float mean = 0.0f, d[P];
#pragma unroll
        for (int j = 0; j < P; ++j) mean = __builtin_fmaf(a[j], w[j], mean);
        mean = group_sum_f32<S::L>(mean) * inv;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            d[j] = w[j] * inv * (a[j] - mean);
            if constexpr (SIGMOID) d[j] *= comp[j];
            d[j] = live ? d[j] : 0.0f;
        }
        if (t <= last) store_row<TL, S, V>(grad, t * E, E, l, d);
    }
}

// Calls f.template operator()<TL, S, V, SIGMOID>() for the row shape.  V: 16
// bytes of logits (8 where a lane holds four bf16 values) where every row
// starts on a 16-byte boundary (gradients and counts as well) and E fills
// whole vectors, else single values.  131072 x 64 bf16, forward and backward:
// 18.8 and 13.4 us, with single values 23.0 and 15.6; 131072 x 24 fp32: 17.6
// and 12.5 against 19.1 and 12.8.  Up to 16 experts a lane holds one value.
template <typename TL, typename S, typename F>
hipError_t with_vec(bool vec, int score, F&& f) {
    constexpr int V = S::P * TL::kBytes < 16 ? S::P : 16 / TL::kBytes;
    if (vec)
        return score == MOE_SCORE_SIGMOID ? f.template operator()<TL, S, V, true>()
                                          : f.template operator()<TL, S, V, false>();
    return score == MOE_SCORE_SIGMOID ? f.template operator()<TL, S, 1, true>()
                                      : f.template operator()<TL, S, 1, false>();
}
template <typename TL, typename F>
hipError_t with_row(const void* logits, const void* grad, const void* counts, int64_t stride, int E, int score,
                    F&& f) {
    const bool vec = E % (16 / TL::kBytes) == 0 && aligned(logits, 16) && aligned(grad, 16) &&
                     aligned(counts, 16) && stride * TL::kBytes % 16 == 0;
    if (E <= 16) return with_vec<TL, RowShape<16, 1>>(false, score, f);
    if (E <= 64) return with_vec<TL, RowShape<16, 4>>(vec, score, f);
    if (E <= 128) return with_vec<TL, RowShape<16, 8>>(vec, score, f);
    if (E <= kNarrowExperts) return with_vec<TL, RowShape<16, 16>>(vec, score, f);
    if (E <= 512) return with_vec<TL, RowShape<64, 8>>(vec, score, f);
    return with_vec<TL, RowShape<64, 16>>(vec, score, f);
}

struct SumsLauncher {
    const void* logits;
    int64_t stride;
    int E;
    const int64_t* topk_idx;
    int K;
    const uint8_t* mask;
    Seqs seqs;
    BalancePlan plan;
    float* sums;
    int32_t *counts, *tokens;
    Outputs out;
    hipStream_t stream;
    template <typename TL, typename S, int V, bool SIGMOID>
    hipError_t operator()() const {
        const size_t lds = (static_cast<size_t>(plan.waves + 1) * E + 1 + plan.waves) * sizeof(float);
        hipLaunchKernelGGL((balance_sums_kernel<TL, S, V, SIGMOID>), dim3(static_cast<unsigned>(plan.num_chunks)),
                           dim3(plan.waves * kWave), lds, stream, logits, stride, E, topk_idx, K, mask, seqs,
                           plan.chunk, sums, counts, tokens, out);
        return hipGetLastError();
    }
};

struct GradLauncher {
    const void* logits;
    int64_t stride;
    int E, K;
    const uint8_t* mask;
    Seqs seqs;
    const int32_t *counts, *seq_tokens;
    const float* grad_loss;
    void* grad;
    hipStream_t stream;
    template <typename TL, typename S, int V, bool SIGMOID>
    hipError_t operator()() const {
        const int64_t all = (seqs.num_tokens + S::kRows - 1) / S::kRows;
        const int64_t sets = (all + kGradWaves - 1) / kGradWaves;
        const int64_t per_block = sets * S::kRows * (kGradThreads / kWave);
        const int64_t blocks = (seqs.num_tokens + per_block - 1) / per_block;
        hipLaunchKernelGGL((balance_grad_kernel<TL, S, V, SIGMOID>), dim3(static_cast<unsigned>(blocks)),
                           dim3(kGradThreads), 0, stream, logits, stride, E, K, mask, seqs, sets, counts,
                           seq_tokens, grad_loss, grad);
        return hipGetLastError();
    }
};

bool balance_shape_ok(int64_t T, int32_t E, int32_t K, int32_t S) {
    return T >= 0 && T <= INT32_MAX / kMaxTopk && E >= 1 && E <= kMaxExperts && K >= 1 && K <= kMaxTopk && K <= E &&
           S >= 1 && S <= MOE_BALANCE_MAX_SEQS;
}

// What both directions check of the logits, the mask and the sequences.
bool balance_input_ok(const void* logits, int32_t dtype, int64_t stride, int64_t T, int32_t E, int32_t score,
                      const int32_t* seq_offsets, int32_t S) {
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F32) return false;
    if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return false;
    if (stride < E) return false;
    if ((seq_offsets == nullptr && S != 1) || !aligned(seq_offsets, 4)) return false;
    return T == 0 || (logits != nullptr && aligned(logits, dtype == MOE_DTYPE_BF16 ? 2 : 4));
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_balance_loss_workspace_bytes(int64_t num_tokens, int32_t num_experts, int32_t num_seqs) {
    if (!moe::balance_shape_ok(num_tokens, num_experts, 1, num_seqs)) return 0;
    return moe::plan_balance(num_tokens, num_experts, num_seqs).workspace_bytes;
}

moe_status moe_balance_loss(const void* logits, int32_t logits_dtype, int64_t row_stride, int64_t num_tokens,
                            int32_t num_experts, int32_t score, const int64_t* topk_idx, int32_t num_topk,
                            const uint8_t* token_mask, const int32_t* seq_offsets, int32_t num_seqs, float* loss,
                            int32_t* counts, int32_t* seq_tokens, float* prob_mean, void* workspace,
                            size_t workspace_bytes, hipStream_t stream) {
    using namespace moe;
    if (!balance_shape_ok(num_tokens, num_experts, num_topk, num_seqs)) return MOE_ERR_INVALID_ARGUMENT;
    if (!balance_input_ok(logits, logits_dtype, row_stride, num_tokens, num_experts, score, seq_offsets, num_seqs))
        return MOE_ERR_INVALID_ARGUMENT;
    if (loss == nullptr || counts == nullptr || seq_tokens == nullptr) return MOE_ERR_INVALID_ARGUMENT;
    if (!aligned(loss, 4) || !aligned(counts, 4) || !aligned(seq_tokens, 4) || !aligned(prob_mean, 4))
        return MOE_ERR_INVALID_ARGUMENT;
    if (num_tokens > 0 && (topk_idx == nullptr || !aligned(topk_idx, 8))) return MOE_ERR_INVALID_ARGUMENT;
    if (workspace == nullptr || !aligned(workspace, 256)) return MOE_ERR_INVALID_ARGUMENT;
    const BalancePlan plan = plan_balance(num_tokens, num_experts, num_seqs);
    if (workspace_bytes < plan.workspace_bytes) return MOE_ERR_WORKSPACE_TOO_SMALL;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    float* sums = reinterpret_cast<float*>(ws);
    int32_t* slot_counts = reinterpret_cast<int32_t*>(ws + plan.sums_bytes);
    int32_t* slot_tokens = reinterpret_cast<int32_t*>(ws + plan.sums_bytes + plan.counts_bytes);
    const Seqs seqs{seq_offsets, num_tokens, num_seqs};
    if (num_tokens > 0) {
        const Outputs out = plan.one_launch ? Outputs{loss, counts, seq_tokens, prob_mean} : Outputs{};
        const SumsLauncher go{logits, row_stride, num_experts, topk_idx, num_topk, token_mask, seqs,
                              plan,   sums,       slot_counts, slot_tokens, out, stream};
        const hipError_t err = logits_dtype == MOE_DTYPE_BF16
                                   ? with_row<Bf16>(logits, nullptr, nullptr, row_stride, num_experts, score, go)
                                   : with_row<F32>(logits, nullptr, nullptr, row_stride, num_experts, score, go);
        if (err != hipSuccess || plan.one_launch) return hip_status(err);
    }
    const int64_t slots = plan.num_slots / num_seqs;  // of a sequence, on average
    if (slots <= kOneLevelSlots) {
        int cols = kWave, rows = 1;
        while (cols < num_experts) cols *= 2;
        while (rows < slots && cols * rows < 1024) rows *= 2;
        hipLaunchKernelGGL(balance_loss_kernel, dim3(num_seqs), dim3(cols * rows), 0, stream, sums, slot_counts,
                           slot_tokens, seqs, plan.chunk, num_experts, num_topk, cols, loss, counts, seq_tokens,
                           prob_mean);
        return hip_status(hipGetLastError());
    }
    float* means = prob_mean != nullptr ? prob_mean : reinterpret_cast<float*>(ws + plan.means_offset);
    hipLaunchKernelGGL(balance_reduce_kernel, dim3((num_experts + kReduceCols - 1) / kReduceCols, num_seqs),
                       dim3(1024), 0, stream, sums, slot_counts, slot_tokens, seqs, plan.chunk, num_experts, counts,
                       seq_tokens, means);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return hip_status(err);
    hipLaunchKernelGGL(balance_dot_kernel, dim3((num_seqs + 3) / 4), dim3(256), 0, stream, counts, means, seq_tokens,
                       num_seqs, num_experts, num_topk, loss);
    return hip_status(hipGetLastError());
}

moe_status moe_balance_loss_backward(const float* grad_loss, const void* logits, int32_t logits_dtype,
                                     int64_t row_stride, int64_t num_tokens, int32_t num_experts, int32_t score,
                                     int32_t num_topk, const uint8_t* token_mask, const int32_t* seq_offsets,
                                     int32_t num_seqs, const int32_t* counts, const int32_t* seq_tokens,
                                     void* grad_logits, hipStream_t stream) {
    using namespace moe;
    if (!balance_shape_ok(num_tokens, num_experts, num_topk, num_seqs)) return MOE_ERR_INVALID_ARGUMENT;
    if (!balance_input_ok(logits, logits_dtype, row_stride, num_tokens, num_experts, score, seq_offsets, num_seqs))
        return MOE_ERR_INVALID_ARGUMENT;
    if (num_tokens == 0) return MOE_OK;
    if (grad_loss == nullptr || counts == nullptr || seq_tokens == nullptr || grad_logits == nullptr)
        return MOE_ERR_INVALID_ARGUMENT;
    if (!aligned(grad_loss, 4) || !aligned(counts, 4) || !aligned(seq_tokens, 4) ||
        !aligned(grad_logits, logits_dtype == MOE_DTYPE_BF16 ? 2 : 4))
        return MOE_ERR_INVALID_ARGUMENT;
    const Seqs seqs{seq_offsets, num_tokens, num_seqs};
    const GradLauncher go{logits, row_stride, num_experts, num_topk,    token_mask, seqs,
                          counts, seq_tokens, grad_loss,   grad_logits, stream};
    return hip_status(logits_dtype == MOE_DTYPE_BF16
                          ? with_row<Bf16>(logits, grad_logits, counts, row_stride, num_experts, score, go)
                          : with_row<F32>(logits, grad_logits, counts, row_stride, num_experts, score, go));
}

}  // extern "C"
