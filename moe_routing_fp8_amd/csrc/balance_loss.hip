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
// Forward, two launches.  The tokens are cut into chunks of consecutive
// tokens, one workgroup each; a wave holds a token's whole row of logits in
// registers and keeps its running sums of p there too.  A chunk may meet
// several sequences: each (chunk, sequence) piece is summed over the
// workgroup's waves in a fixed order and written to a slot of its own,
// number chunk + sequence (along the pieces in token order either index
// grows, so no two pieces share a slot, and a sequence's slots are
// consecutive).  The second launch sums each sequence's slots in order.  No
// floating atomics: the results do not depend on timing.
// Backward, one launch: a wave per token reads the row again, with the
// sequence's counts in registers.
#include <hip/hip_runtime.h>

#include "api_common.hpp"
#include "math_device.hpp"
#include "moe_fp8.h"

namespace moe {
namespace {

constexpr int kBalanceThreads = 256;
constexpr int kBalanceWaves = kBalanceThreads / kWave;
// Chunks of a large batch: two workgroups for each of the 256 compute units.
constexpr int64_t kBalanceMaxChunks = 512;
constexpr int64_t kBalanceMinChunkTokens = 8;

struct BalancePlan {
    int64_t chunk;       // tokens per workgroup
    int64_t num_chunks;
    int64_t num_slots;   // num_chunks + num_seqs
    size_t sums_bytes, counts_bytes, tokens_bytes;
    size_t workspace_bytes;
};

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

BalancePlan plan_balance(int64_t T, int E, int S) {
    BalancePlan p;
    p.chunk = (T + kBalanceMaxChunks - 1) / kBalanceMaxChunks;
    if (p.chunk < kBalanceMinChunkTokens) p.chunk = kBalanceMinChunkTokens;
    p.num_chunks = (T + p.chunk - 1) / p.chunk;
    p.num_slots = p.num_chunks + S;
    p.sums_bytes = round256(static_cast<size_t>(p.num_slots) * E * sizeof(float));
    p.counts_bytes = round256(static_cast<size_t>(p.num_slots) * E * sizeof(int32_t));
    p.tokens_bytes = round256(static_cast<size_t>(p.num_slots) * sizeof(int32_t));
    p.workspace_bytes = p.sums_bytes + p.counts_bytes + p.tokens_bytes;
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
        for (int i = 1; i <= num_seqs; i += kWave) {
            const bool before = i + lane <= num_seqs && edge(i + lane) <= t;
            n += __builtin_popcountll(__ballot(before));
        }
        return n;
    }
};

// A token's row over the wave: lane's experts are lane * P .. lane * P + P - 1
// (VEC: E == 64 * P and aligned rows) or lane + 64 j.
template <int P, bool VEC>
__device__ __forceinline__ int expert_of(int lane, int j) { return VEC ? lane * P + j : lane + kWave * j; }

template <typename TL, int P, bool VEC>
__device__ __forceinline__ void load_row(const void* logits, int64_t at, int E, int lane, float (&z)[P]) {
    if constexpr (VEC) {
        TL::template load<P>(logits, at + lane * P, z);
    } else {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int e = lane + kWave * j;
            float one[1] = {-INFINITY};
            if (e < E) TL::template load<1>(logits, at + e, one);
            z[j] = one[0];
        }
    }
}

// p of the row (0 at the padding, whose logit is -inf); comp[j] = 1 -
// sigmoid(z[j]) with SIGMOID.  A row of nothing but -inf gives p = 0.
//
// sigmoid(z) = r or t r with t = exp(-|z|), r = 1 / (1 + t).  Where every
// logit of a row is below -60 the sigmoids leave the range in which their
// ratio keeps 24 bits, so they are taken relative to the largest logit m:
// sigmoid(z) exp(-m) = exp(z - m) r.
template <int P, bool SIGMOID>
__device__ __forceinline__ void row_probs(const float (&z)[P], float (&p)[P], float (&comp)[P]) {
    float m = z[0];
#pragma unroll
    for (int j = 1; j < P; ++j) m = fmaxf(m, z[j]);
    m = wave_max_f32(m);
    float sum = 0.0f;
    if constexpr (SIGMOID) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const float t = exp_nonpos(-fabsf(z[j]));
            const float r = 1.0f / (1.0f + t);
            p[j] = z[j] > 0.0f ? r : t * r;
            comp[j] = z[j] > 0.0f ? t * r : r;
            if (m < -60.0f) p[j] = exp_nonpos(z[j] - m) * r;
        }
    } else {
#pragma unroll
        for (int j = 0; j < P; ++j) p[j] = exp_nonpos(z[j] - m);
    }
#pragma unroll
    for (int j = 0; j < P; ++j) sum += p[j];
    sum = wave_sum_f32(sum);
    const float inv = 1.0f / sum;
#pragma unroll
    for (int j = 0; j < P; ++j) p[j] = m == -INFINITY ? 0.0f : p[j] * inv;
}

template <typename TL, int P, bool VEC, bool SIGMOID>
__global__ __launch_bounds__(kBalanceThreads) void balance_sums_kernel(
    const void* __restrict__ logits, int64_t stride, int E, const int64_t* __restrict__ topk_idx, int K,
    const uint8_t* __restrict__ mask, Seqs seqs, int64_t chunk, float* __restrict__ sums,
    int32_t* __restrict__ counts, int32_t* __restrict__ tokens) {
    extern __shared__ float lds[];  // kBalanceWaves x E sums, then E counts, then one token count
    int32_t* hist = reinterpret_cast<int32_t*>(lds + kBalanceWaves * E);
    int32_t* live = hist + E;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = threadIdx.x / kWave;
    const int64_t t0 = blockIdx.x * chunk;
    const int64_t t1 = min(t0 + chunk, seqs.num_tokens);
    for (int e = threadIdx.x; e < E; e += kBalanceThreads) hist[e] = 0;
    if (threadIdx.x == 0) *live = 0;
    __syncthreads();
    for (int s = seqs.find(t0, lane); s < seqs.num_seqs; ++s) {
        const int64_t begin = max(t0, seqs.edge(s)), end = min(t1, seqs.edge(s + 1));
        if (begin >= t1) break;
        if (begin >= end) continue;
        float acc[P];
#pragma unroll
        for (int j = 0; j < P; ++j) acc[j] = 0.0f;
        int n = 0;
        for (int64_t t = begin + wave; t < end; t += kBalanceWaves) {
            if (mask != nullptr && mask[t] == 0) continue;
            float z[P], p[P], comp[P];
            load_row<TL, P, VEC>(logits, t * stride, E, lane, z);
            if (lane < K) {
                const int64_t id = topk_idx[t * K + lane];
                if (id >= 0 && id < E) atomicAdd(&hist[id], 1);
            }
            row_probs<P, SIGMOID>(z, p, comp);
#pragma unroll
            for (int j = 0; j < P; ++j) acc[j] += p[j];
            ++n;
        }
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int e = expert_of<P, VEC>(lane, j);
            if (e < E) lds[wave * E + e] = acc[j];
        }
        if (lane == 0) atomicAdd(live, n);
        __syncthreads();
        const int64_t slot = blockIdx.x + static_cast<int64_t>(s);
        for (int e = threadIdx.x; e < E; e += kBalanceThreads) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kBalanceWaves; ++w) v += lds[w * E + e];
            sums[slot * E + e] = v;
            counts[slot * E + e] = hist[e];
            hist[e] = 0;
        }
        if (threadIdx.x == 0) {
            tokens[slot] = *live;
            *live = 0;
        }
        __syncthreads();
    }
}

// One workgroup per sequence: its slots, in order.
__global__ __launch_bounds__(kBalanceThreads) void balance_loss_kernel(
    const float* __restrict__ sums, const int32_t* __restrict__ slot_counts,
    const int32_t* __restrict__ slot_tokens, Seqs seqs, int64_t chunk, int E, int K, float* __restrict__ loss,
    int32_t* __restrict__ counts, int32_t* __restrict__ seq_tokens, float* __restrict__ prob_mean) {
    __shared__ float part[kBalanceWaves];
    const int s = blockIdx.x;
    const int64_t begin = seqs.edge(s), end = seqs.edge(s + 1);
    int64_t first = 0, last = -1;  // slots
    if (begin < end) {
        first = begin / chunk + s;
        last = (end - 1) / chunk + s;
    }
    int n = 0;
    for (int64_t i = first; i <= last; ++i) n += slot_tokens[i];
    const float many = n > 0 ? static_cast<float>(n) : 1.0f;
    float dot = 0.0f;
    for (int e = threadIdx.x; e < E; e += kBalanceThreads) {
        float sum = 0.0f;
        int c = 0;
        for (int64_t i = first; i <= last; ++i) {
            sum += sums[i * E + e];
            c += slot_counts[i * E + e];
        }
        const float mean = sum / many;
        counts[static_cast<int64_t>(s) * E + e] = c;
        if (prob_mean != nullptr) prob_mean[static_cast<int64_t>(s) * E + e] = mean;
        dot += static_cast<float>(c) * mean;
    }
    dot = wave_sum_f32(dot);
    if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
        float v = 0.0f;
        for (int w = 0; w < kBalanceWaves; ++w) v += part[w];
        loss[s] = v * (static_cast<float>(E) / static_cast<float>(K)) / many;
        seq_tokens[s] = n;
    }
}

template <typename TL, int P, bool VEC, bool SIGMOID>
__global__ __launch_bounds__(kBalanceThreads) void balance_grad_kernel(
    const void* __restrict__ logits, int64_t stride, int E, int K, const uint8_t* __restrict__ mask, Seqs seqs,
    int64_t chunk, const int32_t* __restrict__ counts, const int32_t* __restrict__ seq_tokens,
    const float* __restrict__ grad_loss, void* __restrict__ grad) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t first = (blockIdx.x * static_cast<int64_t>(kBalanceWaves) + threadIdx.x / kWave) * chunk;
    const int64_t last = min(first + chunk, seqs.num_tokens);
    if (first >= last) return;
    int s = seqs.find(first, lane);
    int held = -1;  // the sequence whose scaled counts are in a[]
    float a[P];
    for (int64_t t = first; t < last; ++t) {
        while (s < seqs.num_seqs && seqs.edge(s + 1) <= t) ++s;
        float d[P];
        const bool live = s < seqs.num_seqs && seqs.edge(s) <= t && (mask == nullptr || mask[t] != 0);
        if (live) {
            if (held != s) {
                held = s;
                const float n = static_cast<float>(max(seq_tokens[s], 1));
                const float g = grad_loss[s] * (static_cast<float>(E) / static_cast<float>(K)) / (n * n);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const int e = expert_of<P, VEC>(lane, j);
                    a[j] = e < E ? g * static_cast<float>(counts[static_cast<int64_t>(s) * E + e]) : 0.0f;
                }
            }
            float z[P], p[P], comp[P];
            load_row<TL, P, VEC>(logits, t * stride, E, lane, z);
            row_probs<P, SIGMOID>(z, p, comp);
            float mean = 0.0f;
#pragma unroll
            for (int j = 0; j < P; ++j) mean += a[j] * p[j];
            mean = wave_sum_f32(mean);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                d[j] = p[j] * (a[j] - mean);
                if constexpr (SIGMOID) d[j] *= comp[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < P; ++j) d[j] = 0.0f;
        }
        if constexpr (VEC) {
            TL::template store<P>(grad, t * E + lane * P, d);
        } else {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int e = lane + kWave * j;
                const float one[1] = {d[j]};
                if (e < E) TL::template store<1>(grad, t * E + e, one);
            }
        }
    }
}

// Calls f.template operator()<TL, P, VEC, SIGMOID>() for the row shape: P the
// least power of two with 64 * P >= E, VEC where E == 64 * P and every
// vector of P logits (and gradients) is aligned to min(16, its bytes).
template <typename TL, int P, bool VEC, typename F>
hipError_t with_score(int score, F&& f) {
    return score == MOE_SCORE_SIGMOID ? f.template operator()<TL, P, VEC, true>()
                                      : f.template operator()<TL, P, VEC, false>();
}
template <typename TL, int P, typename F>
hipError_t with_vec(const void* logits, const void* grad, int64_t stride, int E, int score, F&& f) {
    constexpr int bytes = P * TL::kBytes < 16 ? P * TL::kBytes : 16;
    const bool vec = E == kWave * P && aligned(logits, bytes) && aligned(grad, bytes) &&
                     stride * TL::kBytes % bytes == 0;
    return vec ? with_score<TL, P, true>(score, f) : with_score<TL, P, false>(score, f);
}
template <typename TL, typename F>
hipError_t with_row(const void* logits, const void* grad, int64_t stride, int E, int score, F&& f) {
    if (E <= 64) return with_vec<TL, 1>(logits, grad, stride, E, score, f);
    if (E <= 128) return with_vec<TL, 2>(logits, grad, stride, E, score, f);
    if (E <= 256) return with_vec<TL, 4>(logits, grad, stride, E, score, f);
    if (E <= 512) return with_vec<TL, 8>(logits, grad, stride, E, score, f);
    return with_vec<TL, 16>(logits, grad, stride, E, score, f);
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
    hipStream_t stream;
    template <typename TL, int P, bool VEC, bool SIGMOID>
    hipError_t operator()() const {
        const size_t lds = (static_cast<size_t>(kBalanceWaves + 1) * E + 1) * sizeof(float);
        hipLaunchKernelGGL((balance_sums_kernel<TL, P, VEC, SIGMOID>), dim3(static_cast<unsigned>(plan.num_chunks)),
                           dim3(kBalanceThreads), lds, stream, logits, stride, E, topk_idx, K, mask, seqs, plan.chunk,
                           sums, counts, tokens);
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
    template <typename TL, int P, bool VEC, bool SIGMOID>
    hipError_t operator()() const {
        constexpr int64_t kChunk = 8;  // consecutive tokens of a wave
        const int64_t per_block = kChunk * kBalanceWaves;
        const int64_t blocks = (seqs.num_tokens + per_block - 1) / per_block;
        hipLaunchKernelGGL((balance_grad_kernel<TL, P, VEC, SIGMOID>), dim3(static_cast<unsigned>(blocks)),
                           dim3(kBalanceThreads), 0, stream, logits, stride, E, K, mask, seqs, kChunk, counts,
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
        const SumsLauncher go{logits, row_stride, num_experts, topk_idx, num_topk, token_mask, seqs,
                              plan,   sums,       slot_counts, slot_tokens, stream};
        const hipError_t err = logits_dtype == MOE_DTYPE_BF16
                                   ? with_row<Bf16>(logits, nullptr, row_stride, num_experts, score, go)
                                   : with_row<F32>(logits, nullptr, row_stride, num_experts, score, go);
        if (err != hipSuccess) return hip_status(err);
    }
    hipLaunchKernelGGL(balance_loss_kernel, dim3(num_seqs), dim3(kBalanceThreads), 0, stream, sums, slot_counts,
                       slot_tokens, seqs, plan.chunk, num_experts, num_topk, loss, counts, seq_tokens, prob_mean);
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
                          ? with_row<Bf16>(logits, grad_logits, row_stride, num_experts, score, go)
                          : with_row<F32>(logits, grad_logits, row_stride, num_experts, score, go));
}

}  // extern "C"
