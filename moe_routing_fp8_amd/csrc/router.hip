// Routing from the router's logits, and its gradient.
//
// With z the logits of a token, s = softmax(z) or sigmoid(z) and c = s + bias:
// the experts are taken in descending order of c, among those of the
// topk_groups groups with the largest group scores, and their weights are
//   w_k = scale * s_k   or, renormalised,   scale * s_k / sum_j s_j.
//
// Forward, one launch: a row lies over 16 lanes (64 above 256 experts), expert
// e in slot e / L of lane e % L.  Every lane sorts its keys once, then each of
// the K rounds takes the maximum over the lanes' heads, four rows of a wave
// side by side.
//
// The order is that of the values in 64 bits, while the keys hold 28 bits of
// an fp32 value and the slot (larger keys are lower slots, so equal values go
// to the lowest expert without another comparison).  Neighbours of the
// resulting order, and the last one taken and the best one left, are compared
// once at the end: only a row where two of them lie closer than the keys'
// error, without being equal bit by bit in what they are made of, is ordered
// again, in 64 bits, by its whole wave.
//
// Backward, one launch: the chosen experts' derivatives are laid into a row of
// zeros in LDS, from where the row is written in whole vectors; softmax
// weights without renormalisation add the term of every other expert.
#include <hip/hip_runtime.h>

#include <float.h>

#include "api_common.hpp"
#include "kernels.hpp"
#include "math_device.hpp"
#include "moe_fp8.h"
#include "topk_device.hpp"

namespace moe {
namespace {

constexpr int kWaves = 4;            // of a workgroup
constexpr int kNarrowExperts = 256;  // rows of up to this many experts lie over 16 lanes
constexpr int kMaxGroups = 64;       // MOE_ROUTER_MAX_GROUPS
constexpr uint32_t kSlotMask = 15;   // the key's bits that hold the slot
constexpr uint32_t kNone = 0;        // the key of an expert that cannot be taken: below every value's

struct RouterArgs {
    const void* logits;
    int64_t row_stride, num_tokens;
    int E, K, sigmoid;
    const float* bias;
    int groups, topk_groups, group_size, top2;
    int lanes_per_group;  // lanes that share the scan of one group
    uint32_t group_magic;  // e / group_size == umulhi(e, group_magic) (group_size > 1)
    int renormalize;
    float scale;
    const uint8_t* token_mask;
    int64_t* idx;
    float* weights;
};

// A logit as it counts: NaN takes its expert out like -inf, +inf is the
// largest finite value.
__device__ __forceinline__ float clean(float z) { return z != z ? -INFINITY : fminf(z, FLT_MAX); }

__device__ __forceinline__ bool takeable(float z, const float* bias, int e) {
    return z > -INFINITY && (bias == nullptr || bias[e] > -INFINITY);
}

// sigmoid(z) to 4 ulp: the exponential of an exact argument to 1.5 ulp, a sum,
// the hardware reciprocal and a product.
__device__ __forceinline__ float sigmoid_key(float z) {
    const float e = exp_nonpos_exact(-fabsf(z));
    const float r = __builtin_amdgcn_rcpf(1.0f + e);
    return z < 0.0f ? e * r : r;
}

template <int L>
__device__ __forceinline__ uint32_t group_max_u32(uint32_t x) {
    if constexpr (L == 16) return row16_max_u32(x);
    else
        return topk::wave_max_u32(x);
}

// Batcher's odd-even merge sort, descending (P a power of two).
template <int P>
__device__ __forceinline__ void sort_desc(uint32_t (&key)[P]) {
#pragma unroll
    for (int p = 1; p < P; p *= 2) {
#pragma unroll
        for (int k = p; k >= 1; k /= 2) {
#pragma unroll
            for (int j = k % p; j + k < P; j += 2 * k) {
#pragma unroll
                for (int i = 0; i < k; ++i) {
                    if (i + j + k < P && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t a = key[i + j], b = key[i + j + k];
                        key[i + j] = max(a, b);
                        key[i + j + k] = min(a, b);
                    }
                }
            }
        }
    }
}

__device__ __forceinline__ uint32_t order_key(float v) { return topk::score_key(v); }
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

__device__ __forceinline__ uint64_t order_key64(double v) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ void lds_handoff() {
    // lanes of one wave hand values over through LDS: its accesses complete in
    // order, so only the compiler has to be kept from moving them
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// LDS of a wave.  `value` holds the scores that the groups are judged by: fp32
// [rows][E], or 64-bit [E] while a row is ordered exactly.
template <int L, int P>
struct WaveLds {
    static constexpr int kRows = kWave / L;
    double value[L * P > kNarrowExperts ? L * P : kRows * L * P / 2];
    double group[kMaxGroups];
    int taken[kRows][kMaxGroups];
    int winner[kRows][16];
};

// The order of one row in 64 bits, by the whole wave: expert e is value e / 64
// of lane e % 64.
template <typename T, int Q>
__device__ __forceinline__ void exact_row(const RouterArgs& a, int64_t t, double* value, double* group, int* taken,
                                       int* winner, int lane) {
    float z[Q];
    double c[Q];
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < Q; ++j) {
        const int e = j * kWave + lane;
        float f[1] = {-INFINITY};
        if (e < a.E) T::template load<1>(a.logits, t * a.row_stride + e, f);
        z[j] = clean(f[0]);
        top = fmaxf(top, z[j]);
    }
    if (!a.sigmoid) {
        top = group_max_f32<kWave>(top);
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < Q; ++j) {
            c[j] = z[j] > -INFINITY ? exp(static_cast<double>(z[j]) - static_cast<double>(top)) : 0.0;
            sum += c[j];
        }
        for (int o = 1; o < kWave; o *= 2) sum += __shfl_xor(sum, o);
#pragma unroll
        for (int j = 0; j < Q; ++j) c[j] /= sum;
    } else {
#pragma unroll
        for (int j = 0; j < Q; ++j) c[j] = 1.0 / (1.0 + exp(-static_cast<double>(z[j])));
    }
    const bool by_value = a.bias != nullptr;
#pragma unroll
    for (int j = 0; j < Q; ++j) {
        const int e = j * kWave + lane;
        const bool open = e < a.E && takeable(z[j], a.bias, e);
        if (by_value && open) c[j] += static_cast<double>(fminf(a.bias[e], FLT_MAX));
        if (!open) c[j] = -INFINITY;
        if (!by_value && !a.top2) c[j] = open ? static_cast<double>(z[j]) : -INFINITY;
    }
    if (a.groups > 1) {
#pragma unroll
        for (int j = 0; j < Q; ++j) {
            const int e = j * kWave + lane;
            if (e < a.E) value[e] = c[j];
        }
        lds_handoff();
        if (lane < a.groups) {
            double b1 = -INFINITY, b2 = -INFINITY;
            for (int i = 0; i < a.group_size; ++i) {
                const double v = value[lane * a.group_size + i];
                b2 = fmax(b2, fmin(b1, v));
                b1 = fmax(b1, v);
            }
            group[lane] = a.top2 ? b1 + b2 : b1;
        }
        lds_handoff();
        if (lane < a.groups) {
            const double mine = group[lane];
            int rank = 0;
            for (int h = 0; h < a.groups; ++h) {
                const double o = group[h];
                rank += o > mine || (o == mine && h < lane);
            }
            taken[lane] = rank < a.topk_groups;
        }
        lds_handoff();
#pragma unroll
        for (int j = 0; j < Q; ++j) {
            const int e = j * kWave + lane;
            if (e >= a.E) continue;
            if (!taken[e / a.group_size])
                c[j] = -INFINITY;
            else if (!by_value && c[j] > -INFINITY)
                c[j] = static_cast<double>(z[j]);
        }
    } else if (!by_value) {
#pragma unroll
        for (int j = 0; j < Q; ++j)
            if (c[j] > -INFINITY) c[j] = static_cast<double>(z[j]);
    }
    for (int k = 0; k < a.K; ++k) {
        double best = -INFINITY;
        int slot = 0;
#pragma unroll
        for (int j = 0; j < Q; ++j) {
            if (c[j] > best) {
                best = c[j];
                slot = j;
            }
        }
        const uint64_t key = best > -INFINITY ? order_key64(best) : 0;
        const uint32_t hi = static_cast<uint32_t>(key >> 32), lo = static_cast<uint32_t>(key);
        const uint32_t top_hi = topk::wave_max_u32(hi);
        const uint32_t top_lo = topk::wave_max_u32(hi == top_hi ? lo : 0);
        const bool mine = best > -INFINITY && hi == top_hi && lo == top_lo;
        // the lowest expert of equal ones
        const uint32_t inv = topk::wave_max_u32(mine ? ~static_cast<uint32_t>(slot * kWave + lane) : 0);
        const int e = inv == 0 ? -1 : static_cast<int>(~inv);
        if (lane == 0) winner[k] = e;
#pragma unroll
        for (int j = 0; j < Q; ++j)
            if (j * kWave + lane == e) c[j] = -INFINITY;
    }
    lds_handoff();
}

template <typename T, int L, int P>
__global__ __launch_bounds__(kWaves* kWave) void router_kernel(RouterArgs a) {
    constexpr int kRows = kWave / L;
    constexpr int Q = L * P > kNarrowExperts ? L * P / kWave : kNarrowExperts / kWave;
    __shared__ WaveLds<L, P> lds[kWaves];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int sub = lane % L, row = lane / L;
    WaveLds<L, P>& m = lds[wave];
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * kWaves + wave) * kRows;
    if (first >= a.num_tokens) return;  // whole waves; no barrier follows
    const int64_t t = first + row;
    const bool inside = t < a.num_tokens;
    const bool live = inside && (a.token_mask == nullptr || a.token_mask[t] != 0);
    const int64_t base = (inside ? t : first) * a.row_stride;

    float z[P], c[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
        const int e = j * L + sub;
        float f[1] = {-INFINITY};
        if (e < a.E) T::template load<1>(a.logits, base + e, f);
        z[j] = live ? clean(f[0]) : -INFINITY;
    }
    // the softmax's maximum and sum, where the order or the weights need them
    const bool scored = a.bias != nullptr || (a.top2 && a.groups > 1);
    float top = 0.0f, inv_sum = 0.0f, sum = 0.0f;
    if (!a.sigmoid && (scored || !a.renormalize)) {
        top = z[0];
#pragma unroll
        for (int j = 1; j < P; ++j) top = fmaxf(top, z[j]);
        top = group_max_f32<L>(top);
        const float at = top > -INFINITY ? top : 0.0f;  // a row of nothing: every exponential is 0
#pragma unroll
        for (int j = 0; j < P; ++j) {
            c[j] = exp_nonpos(z[j] - at);
            sum += c[j];
        }
        sum = group_sum_f32<L>(sum);
        inv_sum = 1.0f / sum;
        top = at;
    }
    if (scored) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int e = j * L + sub;
            const float s = a.sigmoid ? sigmoid_key(z[j]) : c[j] * inv_sum;
            float b = 0.0f;
            if (a.bias != nullptr && e < a.E) b = a.bias[e];
            c[j] = (z[j] > -INFINITY && b > -INFINITY) ? s + fminf(b, FLT_MAX) : -INFINITY;
        }
    } else {
#pragma unroll
        for (int j = 0; j < P; ++j) c[j] = z[j];
    }
    // two values closer than this may be in the other order: each key is cut
    // by up to 2^-19 of its value, and errs by the rounding of c, 4 ulp of s
    // (a softmax's sum of 16 terms a lane: 2^-19 of the largest s, which is
    // 1 / sum) and the sigmoid's exponent, whose error times s is below 2^-22
    const float most = a.sigmoid ? 1.0f : inv_sum;
    const float slack = scored ? 0x1p-17f * most + (a.sigmoid ? 0x1p-22f : 0.0f) : 0.0f;
    bool near = false;

    if (a.groups > 1) {
        float* value = reinterpret_cast<float*>(m.value) + row * a.E;
#pragma unroll
        for (int j = 0; j < P; ++j)
            if (j * L + sub < a.E) value[j * L + sub] = c[j];
        lds_handoff();
        // several lanes scan a group where there are more lanes than groups
        const int lpg = a.lanes_per_group, per_pass = L / lpg, part = sub % lpg;
        float kept = INFINITY, left = -INFINITY;
        float mine[L == 16 ? 4 : 1];
#pragma unroll
        for (int pass = 0; pass < (L == 16 ? 4 : 1); ++pass) {
            const int g = pass * per_pass + sub / lpg;
            float b1 = -INFINITY, b2 = -INFINITY;
            if (pass * per_pass < a.groups) {
                if (g < a.groups) {
                    // every lane starts elsewhere in its group: other banks
                    int i = part + lpg * (lane % ((a.group_size + lpg - 1) / lpg));
                    for (int n = part; n < a.group_size; n += lpg) {
                        if (i >= a.group_size) i = part;
                        const float v = value[g * a.group_size + i];
                        b2 = fmaxf(b2, fminf(b1, v));
                        b1 = fmaxf(b1, v);
                        i += lpg;
                    }
                }
                for (int o = 1; o < lpg; o *= 2) {
                    const float o1 = __shfl_xor(b1, o), o2 = __shfl_xor(b2, o);
                    b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
                    b1 = fmaxf(b1, o1);
                }
            }
            mine[pass] = a.top2 ? b1 + b2 : b1;
        }
        // ranks over the row's groups; the scores pass through `taken`
        float* score = reinterpret_cast<float*>(m.taken[row]);
#pragma unroll
        for (int pass = 0; pass < (L == 16 ? 4 : 1); ++pass) {
            const int g = pass * per_pass + sub / lpg;
            if (g < a.groups && part == 0) score[g] = mine[pass];
        }
        lds_handoff();
        bool in[L == 16 ? 4 : 1];
#pragma unroll
        for (int pass = 0; pass < (L == 16 ? 4 : 1); ++pass) {
            const int g = pass * per_pass + sub / lpg;
            in[pass] = false;
            if (g < a.groups) {
                int rank = 0;
                for (int h = 0; h < a.groups; ++h) {
                    const float o = score[h];
                    rank += o > mine[pass] || (o == mine[pass] && h < g);
                }
                in[pass] = rank < a.topk_groups;
                if (in[pass]) kept = fminf(kept, mine[pass]);
                else
                    left = fmaxf(left, mine[pass]);
            }
        }
        lds_handoff();
#pragma unroll
        for (int pass = 0; pass < (L == 16 ? 4 : 1); ++pass) {
            const int g = pass * per_pass + sub / lpg;
            if (g < a.groups && part == 0) m.taken[row][g] = in[pass];
        }
        lds_handoff();
        kept = -group_max_f32<L>(-kept);
        left = group_max_f32<L>(left);
        // two sums of two values each, not cut to a key
        near = scored && left > -INFINITY && !(kept - left > 0x1p-21f * (fabsf(kept) + fabsf(left)) + 2 * slack);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int e = j * L + sub;
            if (e < a.E) {
                const int g = a.group_size > 1 ? __umulhi(static_cast<uint32_t>(e), a.group_magic) : e;
                if (!m.taken[row][g]) c[j] = -INFINITY;
            }
        }
    }
    // without a bias the logits order as the scores do, and exactly
    const bool by_value = a.bias != nullptr;
    uint32_t key[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
        const float v = by_value ? c[j] : z[j];
        key[j] = c[j] > -INFINITY ? (order_key(v) & ~kSlotMask) | (kSlotMask - j) : kNone;
    }
    sort_desc<P>(key);

    uint32_t my_key = kNone;
    m.winner[row][sub % 16] = -1;
    lds_handoff();
    for (int k = 0; k < a.K; ++k) {
        const uint32_t best = group_max_u32<L>(key[0]);
        const bool hit = key[0] == best && best != kNone;
        const uint64_t who = __ballot(hit);
        // the lowest lane of the row's that hold it
        const uint64_t below = who & ((L == kWave ? ~0ull : ((1ull << L) - 1) << (row * L)) & ((1ull << lane) - 1));
        if (sub == k) my_key = best;
        if (hit && below == 0) {
            m.winner[row][k] = static_cast<int>(kSlotMask - (key[0] & kSlotMask)) * L + sub;
#pragma unroll
            for (int j = 0; j + 1 < P; ++j) key[j] = key[j + 1];
            key[P - 1] = kNone;
        }
    }
    lds_handoff();

    // is the order proven?
    {
        const int e = sub < 16 ? m.winner[row][sub] : -1;
        float ze = -INFINITY, be = 0.0f;
        if (sub < a.K && e >= 0) {
            float f[1];
            T::template load<1>(a.logits, base + e, f);
            ze = clean(f[0]);
            if (by_value) be = a.bias[e];
        }
        const uint32_t cut = my_key & ~kSlotMask;
        const float v = key_value(cut);
        // the next winner, one lane up
        const uint32_t next = __shfl_down(my_key, 1) & ~kSlotMask;
        const float zn = __shfl_down(ze, 1), bn = __shfl_down(be, 1);
        const bool exact_keys = !by_value && T::kBytes == 2;  // bf16 logits lose nothing
        if (!exact_keys && sub + 1 < a.K && next != kNone) {
            const bool same = ze == zn && be == bn;
            const float vn = key_value(next);
            const bool close =
                by_value ? v - vn <= 0x1p-18f * (fabsf(v) + fabsf(vn)) + slack : cut == next;
            near = near || (close && !same);
        }
        // what is left within the last winner's reach has to be equal to it
        const int last = row * L + a.K - 1;
        const uint32_t cut_last = __shfl(cut, last);
        const float z_last = __shfl(ze, last), b_last = __shfl(be, last);
        if (!exact_keys && cut_last != kNone) {
            const float vl = key_value(cut_last);
            const uint32_t reach =
                by_value ? order_key(vl - (0x1p-16f * fabsf(vl) + 2 * slack)) & ~kSlotMask : cut_last;
            for (int j = 0; j < P; ++j) {
                if (key[0] < reach || key[0] == kNone) break;
                const int o = static_cast<int>(kSlotMask - (key[0] & kSlotMask)) * L + sub;
                float f[1];
                T::template load<1>(a.logits, base + o, f);
                near = near || clean(f[0]) != z_last || (by_value && a.bias[o] != b_last);
#pragma unroll
                for (int i = 0; i + 1 < P; ++i) key[i] = key[i + 1];
                key[P - 1] = kNone;
            }
        }
        uint64_t todo = __ballot(near);
        while (todo != 0) {
            const int r = __builtin_ctzll(todo) / L;
            exact_row<T, Q>(a, first + r, m.value, m.group, m.taken[r], m.winner[r], lane);
            todo &= L == kWave ? 0 : ~(((1ull << L) - 1) << (r * L));
        }
    }

    // the weights, lane k of a row its k-th
    const int e = sub < 16 ? m.winner[row][sub] : -1;
    const bool mine = sub < a.K && e >= 0;
    float ze = -INFINITY;
    if (mine) {
        float f[1];
        T::template load<1>(a.logits, base + e, f);
        ze = clean(f[0]);
    }
    float w = 0.0f;
    if (a.renormalize) {
        // shifted by the largest logit chosen, so that a row whose scores all
        // vanish in fp32 still has its weights; the shift cancels
        const float high = group_max_f32<L>(ze);
        const float shift = a.sigmoid ? fminf(high, 0.0f) : high;
        float r = 0.0f;
        if (mine) {
            r = exp_nonpos_exact(fminf(ze - shift, 0.0f));
            if (a.sigmoid) r = ze < 0.0f ? r / (1.0f + exp_nonpos_exact(ze)) : 1.0f / (1.0f + exp_nonpos_exact(-ze));
        }
        const float total = group_sum_f32<L>(r);
        if (mine) w = a.scale * (r / total);
    } else if (mine) {
        if (a.sigmoid) {
            const float x = exp_nonpos_exact(-fabsf(ze));
            w = a.scale * ((ze < 0.0f ? x : 1.0f) / (1.0f + x));
        } else {
            w = a.scale * (exp_nonpos(ze - top) / sum);
        }
    }
    if (inside && sub < a.K) {
        a.idx[t * a.K + sub] = e;
        a.weights[t * a.K + sub] = w;
    }
}

struct BackwardArgs {
    const float* grad_weights;
    const void* logits;
    int64_t row_stride, num_tokens;
    int E, K, sigmoid, renormalize;
    float scale;
    const int64_t* idx;
    void* grad;
};

// Four consecutive values a lane and step, at once where every row's accesses
// are aligned (VEC); else one by one in the same places, so that the sums'
// order, and with it every bit, does not depend on the alignment.
template <typename T, int L, bool VEC>
__global__ __launch_bounds__(kWaves* kWave) void router_backward_kernel(BackwardArgs a) {
    constexpr int kRows = kWave / L;
    constexpr int kWidth = L == 16 ? kNarrowExperts : kMaxExperts;
    constexpr int N = kWidth / (L * 4);
    __shared__ float4 lds[kWaves][kRows][kWidth / 4];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int sub = lane % L, row = lane / L;
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * kWaves + wave) * kRows;
    if (first >= a.num_tokens) return;  // whole waves; no barrier follows
    const int64_t t = first + row;
    const bool inside = t < a.num_tokens;
    const int64_t base = (inside ? t : first) * a.row_stride;
    const bool dense = !a.sigmoid && !a.renormalize;

    // lane k of a row: its k-th expert, if that is one
    int e = -1;
    float g = 0.0f, ze = -INFINITY;
    if (inside && sub < a.K) {
        const int64_t id = a.idx[t * a.K + sub];
        if (id >= 0 && id < a.E) {
            e = static_cast<int>(id);
            g = a.scale * a.grad_weights[t * a.K + sub];
            float f[1];
            T::template load<1>(a.logits, base + e, f);
            ze = clean(f[0]);
        }
    }
    float4* whole = lds[wave][row];
    float* out = reinterpret_cast<float*>(whole);
#pragma unroll
    for (int j = 0; j < kWidth / 4 / L; ++j)
        if ((j * L + sub) * 4 < a.E) whole[j * L + sub] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    lds_handoff();

    float z[N][4];
    float top = -INFINITY, inv_sum = 0.0f;
    if (dense) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int i = (n * L + sub) * 4;
#pragma unroll
            for (int v = 0; v < 4; ++v) z[n][v] = -INFINITY;
            if constexpr (VEC) {
                if (i < a.E) T::template load<4>(a.logits, base + i, z[n]);
            } else {
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (i + v < a.E) T::template load<1>(a.logits, base + i + v, *reinterpret_cast<float(*)[1]>(&z[n][v]));
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                z[n][v] = clean(z[n][v]);
                top = fmaxf(top, z[n][v]);
            }
        }
        top = group_max_f32<L>(top);
        if (top == -INFINITY) top = 0.0f;
        float sum = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                z[n][v] = exp_nonpos(z[n][v] - top);
                sum += z[n][v];
            }
        }
        sum = group_sum_f32<L>(sum);
        inv_sum = sum > 0.0f ? 1.0f / sum : 0.0f;
    }
    float d = g, dot = 0.0f;
    if (a.renormalize) {
        const float high = group_max_f32<L>(ze);
        const float shift = a.sigmoid ? fminf(high, 0.0f) : high;
        float r = 0.0f, rest = 1.0f;
        if (e >= 0 && ze > -INFINITY) {
            r = exp_nonpos_exact(fminf(ze - shift, 0.0f));
            if (a.sigmoid) {
                const float x = exp_nonpos_exact(-fabsf(ze));
                r = ze < 0.0f ? r / (1.0f + x) : 1.0f / (1.0f + x);
                rest = (ze < 0.0f ? 1.0f : x) / (1.0f + x);  // 1 - sigmoid
            }
        }
        const float total = group_sum_f32<L>(r);
        const float p = total > 0.0f ? r / total : 0.0f;
        d = p * (g - group_sum_f32<L>(g * p)) * rest;
    } else if (a.sigmoid) {
        const float x = exp_nonpos_exact(-fabsf(ze));  // s (1 - s) = x / (1 + x)^2
        d = e >= 0 ? g * (x / (1.0f + x)) / (1.0f + x) : 0.0f;
    } else {
        dot = group_sum_f32<L>(e >= 0 ? g * (exp_nonpos(ze - top) * inv_sum) : 0.0f);
    }
    if (e >= 0) out[e] = d;
    lds_handoff();
    if (!inside) return;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = (n * L + sub) * 4;
        if (i >= a.E) continue;
        const float4 d4 = whole[n * L + sub];  // past E: not stored
        float f[4] = {d4.x, d4.y, d4.z, d4.w};
        if (dense) {
#pragma unroll
            for (int v = 0; v < 4; ++v) f[v] = z[n][v] * inv_sum * (f[v] - dot);
        }
        if constexpr (VEC) {
            T::template store<4>(a.grad, t * a.E + i, f);
        } else {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                if (i + v < a.E) {
                    const float one[1] = {f[v]};
                    T::template store<1>(a.grad, t * a.E + i + v, one);
                }
            }
        }
    }
}

template <typename T, int L, int P>
void launch_router_shape(const RouterArgs& a, hipStream_t stream) {
    const int64_t per = kWaves * (kWave / L);
    hipLaunchKernelGGL((router_kernel<T, L, P>), dim3(static_cast<unsigned>((a.num_tokens + per - 1) / per)),
                       dim3(kWaves * kWave), 0, stream, a);
}

template <typename T>
hipError_t launch_router(const RouterArgs& a, hipStream_t stream) {
    if (a.E <= 32) launch_router_shape<T, 16, 2>(a, stream);
    else if (a.E <= 64)
        launch_router_shape<T, 16, 4>(a, stream);
    else if (a.E <= 128)
        launch_router_shape<T, 16, 8>(a, stream);
    else if (a.E <= kNarrowExperts)
        launch_router_shape<T, 16, 16>(a, stream);
    else if (a.E <= 512)
        launch_router_shape<T, 64, 8>(a, stream);
    else
        launch_router_shape<T, 64, 16>(a, stream);
    return hipGetLastError();
}

template <typename T, int L, bool VEC>
void launch_backward_shape(const BackwardArgs& a, hipStream_t stream) {
    const int64_t per = kWaves * (kWave / L);
    hipLaunchKernelGGL((router_backward_kernel<T, L, VEC>), dim3(static_cast<unsigned>((a.num_tokens + per - 1) / per)),
                       dim3(kWaves * kWave), 0, stream, a);
}

template <typename T>
hipError_t launch_backward(const BackwardArgs& a, hipStream_t stream) {
    const uintptr_t bytes = 4 * T::kBytes;
    const bool vec = a.E % 4 == 0 && a.row_stride % 4 == 0 && aligned(a.logits, bytes) && aligned(a.grad, bytes);
    if (a.E <= kNarrowExperts) {
        if (vec) launch_backward_shape<T, 16, true>(a, stream);
        else
            launch_backward_shape<T, 16, false>(a, stream);
    } else if (vec) {
        launch_backward_shape<T, 64, true>(a, stream);
    } else {
        launch_backward_shape<T, 64, false>(a, stream);
    }
    return hipGetLastError();
}

// What both directions check.
bool valid_router(int32_t dtype, int64_t row_stride, int64_t T, int32_t E, int32_t K, int32_t score, int32_t renorm,
                  float scale) {
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F32) return false;
    if (T < 0 || T > INT32_MAX / kMaxTopk || E < 1 || E > kMaxExperts || row_stride < E) return false;
    if (K < 1 || K > kMaxTopk || K > E) return false;
    if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return false;
    return (renorm == 0 || renorm == 1) && scale - scale == 0.0f;
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_router(const void* logits, int32_t logits_dtype, int64_t row_stride, int64_t num_tokens,
                                 int32_t num_experts, int32_t num_topk, int32_t score, const float* bias,
                                 int32_t num_groups, int32_t topk_groups, int32_t group_score, int32_t renormalize,
                                 float scale, const uint8_t* token_mask, int64_t* topk_idx, float* topk_weights,
                                 hipStream_t stream) {
    using namespace moe;
    if (!valid_router(logits_dtype, row_stride, num_tokens, num_experts, num_topk, score, renormalize, scale))
        return MOE_ERR_INVALID_ARGUMENT;
    if (num_groups < 1 || num_experts % num_groups != 0 || topk_groups < 1 || topk_groups > num_groups)
        return MOE_ERR_INVALID_ARGUMENT;
    const int32_t size = num_experts / num_groups;
    if (group_score != MOE_GROUP_MAX && group_score != MOE_GROUP_TOP2) return MOE_ERR_INVALID_ARGUMENT;
    if (num_groups > 1 && group_score == MOE_GROUP_TOP2 && size < 2) return MOE_ERR_INVALID_ARGUMENT;
    if (num_topk > topk_groups * size) return MOE_ERR_INVALID_ARGUMENT;
    if (num_groups > MOE_ROUTER_MAX_GROUPS) return MOE_ERR_UNSUPPORTED;
    if (num_tokens == 0) return MOE_OK;
    if (logits == nullptr || topk_idx == nullptr || topk_weights == nullptr) return MOE_ERR_INVALID_ARGUMENT;
    if (!aligned(logits, logits_dtype == MOE_DTYPE_BF16 ? 2 : 4) || !aligned(bias, 4) || !aligned(topk_idx, 8) ||
        !aligned(topk_weights, 4))
        return MOE_ERR_INVALID_ARGUMENT;
    const int L = num_experts <= kNarrowExperts ? 16 : kWave;
    int lanes = 1;
    while (lanes * 2 * num_groups <= L && lanes * 2 <= size) lanes *= 2;
    RouterArgs a{};
    a.logits = logits;
    a.row_stride = row_stride;
    a.num_tokens = num_tokens;
    a.E = num_experts;
    a.K = num_topk;
    a.sigmoid = score == MOE_SCORE_SIGMOID;
    a.bias = bias;
    a.groups = topk_groups == num_groups ? 1 : num_groups;  // all groups taken: as good as one
    a.topk_groups = topk_groups;
    a.group_size = size;
    a.top2 = a.groups > 1 && group_score == MOE_GROUP_TOP2;
    a.lanes_per_group = lanes;
    // exact for e < 2^16: the excess of the rounded-up reciprocal is below 2^-32, times e below 1 / size
    a.group_magic = size > 1 ? static_cast<uint32_t>(0xFFFFFFFFu / static_cast<uint32_t>(size) + 1) : 0;
    a.renormalize = renormalize;
    a.scale = scale;
    a.token_mask = token_mask;
    a.idx = topk_idx;
    a.weights = topk_weights;
    return hip_status(logits_dtype == MOE_DTYPE_BF16 ? launch_router<Bf16>(a, stream)
                                                     : launch_router<F32>(a, stream));
}

extern "C" moe_status moe_router_backward(const float* grad_weights, const void* logits, int32_t logits_dtype,
                                          int64_t row_stride, int64_t num_tokens, int32_t num_experts,
                                          const int64_t* topk_idx, int32_t num_topk, int32_t score,
                                          int32_t renormalize, float scale, void* grad_logits, hipStream_t stream) {
    using namespace moe;
    if (!valid_router(logits_dtype, row_stride, num_tokens, num_experts, num_topk, score, renormalize, scale))
        return MOE_ERR_INVALID_ARGUMENT;
    if (num_tokens == 0) return MOE_OK;
    if (grad_weights == nullptr || logits == nullptr || topk_idx == nullptr || grad_logits == nullptr)
        return MOE_ERR_INVALID_ARGUMENT;
    const uintptr_t size = logits_dtype == MOE_DTYPE_BF16 ? 2 : 4;
    if (!aligned(grad_weights, 4) || !aligned(logits, size) || !aligned(topk_idx, 8) || !aligned(grad_logits, size))
        return MOE_ERR_INVALID_ARGUMENT;
    const BackwardArgs a{grad_weights, logits,      row_stride, num_tokens, num_experts, num_topk,
                         score == MOE_SCORE_SIGMOID, renormalize, scale,      topk_idx,   grad_logits};
    return hip_status(logits_dtype == MOE_DTYPE_BF16 ? launch_backward<Bf16>(a, stream)
                                                     : launch_backward<F32>(a, stream));
}
