// Routing from the router's logits, and its gradient.
//
// With z the logits of a token, s = softmax(z) or sigmoid(z) and c = s + bias:
// the experts are taken in descending order of c, among those of the
// topk_groups groups with the largest group scores, and their weights are
//   w_k = scale * s_k   or, renormalised,   scale * s_k / sum_j s_j.
//
// Forward, one launch: a row lies over 16 lanes (64 above 256 experts), P
// consecutive experts a lane.  Every lane sorts its keys once, then each of the K
// rounds takes the maximum over the lanes' heads, four rows of a wave side by
// side.  Where a group is made of whole lanes, as 8 groups of 32 are, its best
// experts are the lanes' first ones.
//
// The order is that of the values in 64 bits, while a key holds 28 bits of an
// fp32 value (26 above 256 experts) and the slot, or in a round's maximum the
// lane: larger keys are lower ones, so equal values go to the lowest expert.
// Neighbours of the resulting order, and the last expert taken and the best one
// left, are compared once at the end.  Only a row where two of them lie closer
// than the keys' error, without being equal bit by bit in what they are made of,
// is ordered again, about one of a hundred: the experts taken and the one left
// that is near them by their values in 64 bits, a lane each; or, where more than
// one is near, one that equals the last taken is left or groups are near, all of
// them, by the whole wave.
//
// Backward, one launch: the chosen experts' derivatives are laid into a row of
// zeros in LDS, from where the row is written in whole vectors; softmax
// weights without renormalisation add the term of every other expert.
//
// Kernel traces, the chip idle before each call, median (least) of 20:
//   32768 x 256 fp32, sigmoid, bias, 4 of 8 groups    25.2 (19.8) us (7.2 of bytes), back to back 19.7:
//                                                     about 1000 vector instructions a wave of four
//                                                     rows, part of them for groups already refused
//   32768 x 256 bf16, softmax; its whole gradient     14.9 (14.6) + 9.1 (8.2) us (3.3 and 6.6 of bytes)
//   10007 x 61 fp32, softmax, bias; its gradient      7.0 (6.5) + 3.9 (3.6) us
//   1 x 256 fp32, sigmoid, bias, groups               4.7 (4.6) us: two trips to memory, the logits and,
//                                                     once ranked, the chosen ones again
// Where every row has to be ordered again, back to back: 32768 x 256 bf16 sigmoids around
// 8 with a bias of zeros 87 us, all logits 0 in 8 groups judged by their two best 141 us.
// Sixteen lanes a row: a round's maximum takes four DPP steps for four rows; with
// a row over all 64 lanes, as many steps and more for each.
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
constexpr int kMaxGroups = MOE_ROUTER_MAX_GROUPS;
constexpr int kDppRowShl1 = 0x101;  // lane i + 1 of the same row (lane 15 of a row reads 0)
constexpr uint32_t kNone = 0x007FFFFF;  // keys up to -inf's: no expert

struct RouterArgs {
    const void* logits;
    int64_t row_stride, num_tokens;
    int E, K, sigmoid;
    const float* bias;
    int groups, topk_groups, group_size, top2;
    int lanes_per_group;   // of whole lanes, if a group is; else lanes that share its scan
    int whole_lanes;
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

// sigmoid(z) to order by: 3 ulp, and the exponent's rounding, |z| 2^-23 of an
// exponential that counts s (1 - s): below 2^-22 in all.
__device__ __forceinline__ float sigmoid_key(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896340736f));
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

__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}
// -0 becomes +0; no NaN comes here.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
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

// LDS of a wave.  `value` holds what groups that are not whole lanes are judged
// by, fp32 [rows][E], or the 64-bit values [E] of a row that is ordered exactly.
template <int L, int P>
struct WaveLds {
    static constexpr int kRows = kWave / L;
    static constexpr int kValues = kRows == 1 ? L * P : kRows * L * P / 2;
    double value[kValues];
    union {
        float best[kRows][2 * L > kMaxGroups ? 2 * L : kMaxGroups];  // of a lane or a group; then whether it is taken
        int winner[kRows][16];                                       // once the groups are chosen
    };
};

template <typename T>
__device__ __forceinline__ float logit(const RouterArgs& a, int64_t i) {
    float f[1];
    T::template load<1>(a.logits, i, f);
    return clean(f[0]);
}

// One row in 64 bits, by the whole wave, through LDS.  Rare, so these take few
// registers; but what they take, the last wave of a launch adds to its time, most
// of it for code that no other wave has fetched.
//
// The values that experts, or with `groups` groups, are judged by: -inf for an
// expert that cannot be taken.
template <typename T, int Q>
__device__ __forceinline__ void exact_values(const RouterArgs& a, int64_t t, double* value, bool scores, int lane) {
    const int64_t base = t * a.row_stride;
    const bool by_value = a.bias != nullptr;
    float high = -INFINITY;
#pragma unroll
    for (int j = 0; j < Q; ++j) {
        const int e = j * kWave + lane;
        if (e >= a.E) continue;
        const float z = logit<T>(a, base + e);
        high = fmaxf(high, z);
        value[e] = by_value && !(a.bias[e] > -INFINITY) ? -INFINITY : static_cast<double>(z);
    }
    if (scores) {
        double top = 0.0, sum = 1.0;
        if (!a.sigmoid) {
            top = static_cast<double>(group_max_f32<kWave>(high));
            sum = 0.0;
#pragma unroll 1
            for (int e = lane; e < a.E; e += kWave) {
                // an expert that only its bias takes out has its part in the sum
                const double z = by_value ? static_cast<double>(logit<T>(a, base + e)) : value[e];
                if (z > -INFINITY) sum += exp(z - top);
            }
            for (int o = 1; o < kWave; o *= 2) sum += __shfl_xor(sum, o);
        }
#pragma unroll 1
        for (int e = lane; e < a.E; e += kWave) {
            const double z = value[e];
            if (!(z > -INFINITY)) continue;
            const double x = exp(a.sigmoid ? -z : z - top);
            double c = a.sigmoid ? 1.0 / (1.0 + x) : x / sum;
            if (by_value) c += static_cast<double>(fminf(a.bias[e], FLT_MAX));
            value[e] = c;
        }
    }
    lds_handoff();
}
// The groups taken, a bit each.
__device__ __forceinline__ uint64_t exact_groups(const RouterArgs& a, const double* value, int lane) {
    double b1 = -INFINITY, b2 = -INFINITY;  // lane g: of group g
#pragma unroll 1
    for (int i = 0; lane < a.groups && i < a.group_size; ++i) {
        const double v = value[lane * a.group_size + i];
        b2 = fmax(b2, fmin(b1, v));
        b1 = fmax(b1, v);
    }
    const double mine = a.top2 ? b1 + b2 : b1;
    int rank = 0;
#pragma unroll 1
    for (int h = 0; h < a.groups; ++h) {
        const double o = __shfl(mine, h);
        rank += o > mine || (o == mine && h < lane);
    }
    return __ballot(lane < a.groups && rank < a.topk_groups);
}
// The winners, of the groups `taken`.
template <typename T, int Q>
__device__ __forceinline__ void exact_row(const RouterArgs& a, int64_t t, double* value, uint64_t taken, int* winner,
                                          int lane) {
    exact_values<T, Q>(a, t, value, a.bias != nullptr, lane);
    for (int k = 0; k < a.K; ++k) {
        double best = -INFINITY;
        int at = 0;
#pragma unroll 1
        for (int e = lane; e < a.E; e += kWave) {
            const double v = value[e];
            if (v > best && (a.groups <= 1 || ((taken >> (e / a.group_size)) & 1) != 0)) {
                best = v;
                at = e;
            }
        }
        const uint64_t key = best > -INFINITY ? order_key64(best) : 0;
        const uint32_t hi = static_cast<uint32_t>(key >> 32), lo = static_cast<uint32_t>(key);
        const uint32_t top_hi = topk::wave_max_u32(hi);
        const uint32_t top_lo = topk::wave_max_u32(hi == top_hi ? lo : 0);
        const bool mine = best > -INFINITY && hi == top_hi && lo == top_lo;
        // the lowest expert of equal ones
        const uint32_t inv = topk::wave_max_u32(mine ? ~static_cast<uint32_t>(at) : 0);
        const int e = inv == 0 ? -1 : static_cast<int>(~inv);
        if (lane == 0) winner[k] = e;
        if (mine && at == e) value[e] = -INFINITY;
        lds_handoff();
    }
}

// P consecutive values from element i on; those past the row's E are -inf.  VEC:
// in pieces of up to 16 bytes, which E is a multiple of.
template <typename T, int P, bool VEC>
__device__ __forceinline__ void load_values(const void* p, int64_t i, int left, float (&f)[P]) {
    constexpr int N = VEC ? (P < 16 / T::kBytes ? P : 16 / T::kBytes) : 1;
#pragma unroll
    for (int j = 0; j < P; j += N) {
        float v[N];
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = -INFINITY;
        if constexpr (N == 2) {
            if (j < left) {
                T::template load<1>(p, i + j, *reinterpret_cast<float(*)[1]>(&v[0]));
                T::template load<1>(p, i + j + 1, *reinterpret_cast<float(*)[1]>(&v[1]));
            }
        } else {
            if (j < left) T::template load<N>(p, i + j, v);
        }
#pragma unroll
        for (int k = 0; k < N; ++k) f[j + k] = v[k];
    }
}

// DEPTH: a lane's keys that can come up, the K largest and the next.
template <typename T, int L, int P, int DEPTH, bool VEC>
__global__ __launch_bounds__(kWaves* kWave) void router_kernel(RouterArgs a) {
    constexpr int kRows = kWave / L, Q = (L * P + kWave - 1) / kWave;
    constexpr uint32_t kCut = L == 16 ? 15 : 63;  // the key's bits that hold a slot or a lane
    constexpr float kCutError = L == 16 ? 0x1p-19f : 0x1p-17f;  // of a value
    static_assert(P <= 16 && L * P <= kMaxExperts, "slots");
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
    const bool by_value = a.bias != nullptr;
    auto row_lanes = [](int r) { return L == kWave ? ~0ull : ((1ull << (L % kWave)) - 1) << (r * L); };

    float z[P], c[P];
    load_values<T, P, VEC>(a.logits, base + sub * P, live ? a.E - sub * P : 0, z);
    if (by_value) load_values<F32, P, VEC>(a.bias, sub * P, a.E - sub * P, c);
#pragma unroll
    for (int j = 0; j < P; ++j) z[j] = clean(z[j]);
    // the softmax's maximum and sum, where the order or the weights need them
    const bool scored = by_value || a.top2;
    float top = 0.0f, inv_sum = 1.0f, sum = 1.0f;
    if (!a.sigmoid && (scored || !a.renormalize)) {
        top = z[0];
#pragma unroll
        for (int j = 1; j < P; ++j) top = fmaxf(top, z[j]);
        top = group_max_f32<L>(top);
        if (top == -INFINITY) top = 0.0f;  // a row of nothing: every exponential is 0
        sum = 0.0f;
#pragma unroll
        for (int j = 0; j < P; ++j) sum += exp_nonpos(z[j] - top);
        sum = group_sum_f32<L>(sum);
        inv_sum = __builtin_amdgcn_rcpf(sum);
    }
    if (scored) {
        float s[P];
        if (a.sigmoid) {
#pragma unroll
            for (int j = 0; j < P; ++j) s[j] = sigmoid_key(z[j]);
        } else {
#pragma unroll
            for (int j = 0; j < P; ++j) s[j] = exp_nonpos(z[j] - top) * inv_sum;
        }
        if (by_value) {
#pragma unroll
            for (int j = 0; j < P; ++j) s[j] = c[j] > -INFINITY ? s[j] + fminf(c[j], FLT_MAX) : -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < P; ++j) c[j] = z[j] > -INFINITY ? s[j] : -INFINITY;
    } else {
#pragma unroll
        for (int j = 0; j < P; ++j) c[j] = z[j];
    }
    // Two values closer than this may be in the other order: twice the sigmoid's
    // error, or that of a softmax's score (its sum of up to 16 terms a lane and the
    // steps over the lanes: below 2^-19 of the largest, which is 1 / sum), and the
    // rounding of c, which the callers add with the cut of the keys.
    const float slack = scored ? (a.sigmoid ? 0x1p-21f : 0x1p-17f * inv_sum) : 0.0f;
    bool open = true;        // this lane's experts can be taken (of whole-lane groups)
    uint64_t taken = ~0ull;  // the row's groups, a bit each

    if (a.groups > 1) {
        // How far a group's score may be off for the roundings of its values, of their
        // sum and of what is made of it below: 4 of 2^-24 of |b1| + |b2|, which may be far
        // more than the sum (two large biases that cancel); with a margin of two.
        auto rounding = [&](float b1, float b2) {
            return 0x1p-21f * fabsf(b1) + (a.top2 ? 0x1p-21f * fabsf(b2) : 0.0f);
        };
        // the least that a group taken may be worth, the most that one left may be
        float kept = INFINITY, left = -INFINITY;
        const int n = a.lanes_per_group;
        if (a.whole_lanes) {
            float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                b2 = fmaxf(b2, fminf(b1, c[j]));
                b1 = fmaxf(b1, c[j]);
            }
            const int g = sub / n;
            if (n > 1) {
                float2* each = reinterpret_cast<float2*>(m.best[row]);
                each[sub] = make_float2(b1, b2);
                lds_handoff();
                for (int i = 0; i < n; ++i) {
                    const float2 o = each[min(g * n + i, L - 1)];  // lanes past the last group: any
                    const float lo = i == 0 ? -INFINITY : fminf(b1, o.x);
                    b2 = i == 0 ? o.y : fmaxf(fmaxf(b2, o.y), lo);
                    b1 = i == 0 ? o.x : fmaxf(b1, o.x);
                }
                lds_handoff();
            }
            const float mine = a.top2 ? b1 + b2 : b1;
            float* score = m.best[row];
            if (g < a.groups) score[g] = mine;  // the same from every lane of a group
            lds_handoff();
            int rank = 0;
            for (int h = 0; h < a.groups; ++h) {
                const float o = score[h];
                rank += o > mine || (o == mine && h < g);
            }
            open = g < a.groups && rank < a.topk_groups;
            if (open) kept = mine - rounding(b1, b2);
            else if (g < a.groups && mine > -INFINITY)
                left = mine + rounding(b1, b2);
        } else {
            float* value = reinterpret_cast<float*>(m.value) + row * a.E;
#pragma unroll
            for (int j = 0; j < P; ++j)
                if (sub * P + j < a.E) value[sub * P + j] = c[j];
            lds_handoff();
            // several lanes scan a group where there are more lanes than groups
            const int part = sub % n;
            for (int g = sub / n; g < kMaxGroups; g += L / n) {
                float b1 = -INFINITY, b2 = -INFINITY;
                if (g < a.groups) {
                    for (int i = part; i < a.group_size; i += n) {
                        const float v = value[g * a.group_size + i];
                        b2 = fmaxf(b2, fminf(b1, v));
                        b1 = fmaxf(b1, v);
                    }
                }
                for (int o = 1; o < n; o *= 2) {
                    const float o1 = __shfl_xor(b1, o), o2 = __shfl_xor(b2, o);
                    b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
                    b1 = fmaxf(b1, o1);
                }
                // place g is one of a group up to g, and those have been read
                lds_handoff();
                if (g < a.groups && part == 0) {
                    m.best[row][g] = a.top2 ? b1 + b2 : b1;
                    value[g] = rounding(b1, b2);
                }
                if (n > 1) break;  // then the lanes cover the groups at once
            }
            lds_handoff();
            taken = 0;
#pragma unroll
            for (int i = 0; i < kMaxGroups / L; ++i) {
                const int g = i * L + sub;
                bool in = false;
                if (g < a.groups) {
                    const float mine = m.best[row][g];
                    int rank = 0;
                    for (int h = 0; h < a.groups; ++h) {
                        const float o = m.best[row][h];
                        rank += o > mine || (o == mine && h < g);
                    }
                    in = rank < a.topk_groups;
                    if (in) kept = fminf(kept, mine - value[g]);
                    else if (mine > -INFINITY)
                        left = fmaxf(left, mine + value[g]);
                }
                taken |= ((__ballot(in) >> (row * L)) & (L == kWave ? ~0ull : (1ull << L) - 1)) << (i * L % kWave);
            }
        }
        if (scored) {  // logits are compared as they are
            kept = -group_max_f32<L>(-kept);
            left = group_max_f32<L>(left);
            // the errors of four scores
            uint64_t todo = __ballot(left > -INFINITY && !(kept - left > 2 * slack));
            while (todo != 0) {
                const int r = __builtin_ctzll(todo) / L;
                exact_values<T, Q>(a, first + r, m.value, true, lane);
                const uint64_t of_row = exact_groups(a, m.value, lane);
                lds_handoff();
                if (row == r) {
                    taken = of_row;
                    open = !a.whole_lanes || ((of_row >> (sub / n)) & 1) != 0;
                }
                todo &= ~row_lanes(r);
            }
        }
        if (!a.whole_lanes) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int e = sub * P + j;
                const int g = a.group_size > 1 ? __umulhi(static_cast<uint32_t>(e), a.group_magic) : e;
                if (e < a.E && ((taken >> g) & 1) == 0) c[j] = z[j] = -INFINITY;
            }
        }
    }
    if (!by_value) {  // the logits order as the scores do, and exactly
#pragma unroll
        for (int j = 0; j < P; ++j) c[j] = z[j];
    }
    uint32_t key[P];
#pragma unroll
    for (int j = 0; j < P; ++j) key[j] = (order_key(c[j]) & ~kCut) | (kCut - j);
    sort_desc<P>(key);

    uint32_t my_key = 0, best = 0;
    lds_handoff();  // the groups' scores, in the same place, have been read
    m.winner[row][sub % 16] = -1;
    lds_handoff();
    for (int k = 0; k < a.K; ++k) {
        const uint32_t head = open ? (key[0] & ~kCut) | (kCut - sub) : 0;
        best = group_max_u32<L>(head);
        if (sub == k) my_key = best;
        if (head == best && best > kNone) {
            m.winner[row][k] = sub * P + static_cast<int>(kCut - (key[0] & kCut));
#pragma unroll
            for (int j = 0; j < DEPTH && j + 1 < P; ++j) key[j] = key[j + 1];
            if (DEPTH >= P) key[P - 1] = 0;
        }
    }
    lds_handoff();

    // Is the order proven?  Not where the next winner, one lane up, or something
    // left is within the reach of this one; then they have to be equal bit by bit.
    bool near = false;
    if (by_value || T::kBytes == 4) {  // keys of bf16 logits lose nothing
        const uint32_t cut = my_key & ~kCut, next = dpp_u32<kDppRowShl1>(my_key) & ~kCut;
        const float v = key_value(cut), vn = key_value(next);
        const bool pair =
            sub + 1 < a.K && next > kNone &&
            (by_value ? !(v - vn > (kCutError + 0x1p-23f) * (fabsf(v) + fabsf(vn)) + slack) : cut == next);
        const uint32_t last = best & ~kCut;
        const float vl = key_value(last);
        const uint32_t reach =
            by_value ? order_key(vl - ((2 * kCutError + 0x1p-22f) * 2 * fabsf(vl) + 2 * slack)) & ~kCut : last;
        const bool rest = open && best > kNone && key[0] > kNone && (key[0] & ~kCut) >= reach;
        if (__ballot(pair || rest) != 0) {
            int e = sub < 16 ? m.winner[row][sub] : -1;
            float ze = -INFINITY, be = 0.0f;
            if (sub < a.K && e >= 0) {
                ze = logit<T>(a, base + e);
                if (by_value) be = a.bias[e];
            }
            const float zn = dpp_f32<kDppRowShl1>(ze), bn = dpp_f32<kDppRowShl1>(be);
            bool again = pair && !(ze == zn && be == bn);
            const int from = row * L + a.K - 1;
            const float z_last = __shfl(ze, from), b_last = __shfl(be, from);
            int found = 0, candidate = -1;  // left, within reach, and not equal to the last
            bool tied = false;              // something left is equal to the last
            for (int j = 0; rest && j < P; ++j) {
                if (key[0] <= kNone || (key[0] & ~kCut) < reach) break;
                if (j == DEPTH) {
                    found = 2;  // more than the lane has kept: as good as several
                    break;
                }
                const int o = sub * P + static_cast<int>(kCut - (key[0] & kCut));
                if (logit<T>(a, base + o) != z_last || (by_value && a.bias[o] != b_last)) {
                    ++found;
                    candidate = o;
                } else {
                    tied = true;
                }
#pragma unroll
                for (int i = 0; i + 1 < P; ++i) key[i] = key[i + 1];
                key[P - 1] = 0;
            }
            const uint64_t mine_only = row_lanes(row);
            const uint64_t with = __ballot(found > 0) & mine_only;
            bool many = (__ballot(found > 1) & mine_only) != 0 || (with & (with - 1)) != 0;
            again = (__ballot(again) & mine_only) != 0;  // of the row: two of the taken may be in the other order
            // What equals the last expert taken, at a higher index, comes after it, so with the taken in their
            // order it stays out.  Where one of them may belong behind the last, it may take that one's place.
            many = many || (again && (__ballot(tied) & mine_only) != 0);
            again = again || with != 0;
            near = near || (many && again) || (with != 0 && a.K == 16);
            if (__ballot(again && !near) != 0) {
                // the candidate is one more, in lane K
                if (found == 1 && !near) m.winner[row][a.K] = candidate;
                lds_handoff();
                const bool in = again && !near && sub <= a.K && sub < 16;
                e = in ? m.winner[row][sub] : -1;
                if (in && sub == a.K && e >= 0) {
                    ze = logit<T>(a, base + e);
                    if (by_value) be = a.bias[e];
                }
                double high = 0.0, total = 1.0;
                if (by_value && !a.sigmoid) {
                    high = static_cast<double>(top);
                    total = 0.0;
#pragma unroll 1
                    for (int o = sub; o < a.E; o += L) {
                        const float f = live ? logit<T>(a, base + o) : -INFINITY;
                        if (f > -INFINITY) total += exp(static_cast<double>(f) - high);
                    }
                    for (int o = 1; o < L; o *= 2) total += __shfl_xor(total, o);
                }
                double value = static_cast<double>(ze);
                if (by_value) {
                    const double x = exp(a.sigmoid ? -value : value - high);
                    value = (a.sigmoid ? 1.0 / (1.0 + x) : x / total) + static_cast<double>(fminf(be, FLT_MAX));
                }
                if (e < 0) value = -INFINITY;
                int rank = 0;
                for (int k = 0; k <= a.K && k < 16; ++k) {
                    const double o = __shfl(value, row * L + k);
                    const int oe = __shfl(e, row * L + k);
                    rank += oe >= 0 && (o > value || (o == value && oe < e));
                }
                if (e >= 0 && rank < 16) m.winner[row][rank] = e;
                lds_handoff();
            }
        }
    }
    uint64_t todo = __ballot(near);
    while (todo != 0) {
        const int r = __builtin_ctzll(todo) / L;
        uint64_t groups = taken;  // of row r
        if (a.groups > 1) {
            if (a.whole_lanes) {
                groups = 0;
                const uint64_t lanes = __ballot(open);
                for (int g = 0; g < a.groups; ++g) groups |= ((lanes >> (r * L + g * a.lanes_per_group)) & 1) << g;
            } else {
                groups = __shfl(static_cast<unsigned long long>(taken), r * L);
            }
        }
        exact_row<T, Q>(a, first + r, m.value, groups, m.winner[r], lane);
        todo &= ~row_lanes(r);
    }

    // the weights, lane k of a row its k-th
    const int e = sub < 16 ? m.winner[row][sub] : -1;
    const bool mine = sub < a.K && e >= 0;
    float ze = -INFINITY;
    if (mine) ze = logit<T>(a, base + e);
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

template <typename T, int L, int P, int DEPTH, bool VEC>
void launch_router_form(const RouterArgs& a, hipStream_t stream) {
    const int64_t per = kWaves * (kWave / L);
    hipLaunchKernelGGL((router_kernel<T, L, P, DEPTH, VEC>),
                       dim3(static_cast<unsigned>((a.num_tokens + per - 1) / per)), dim3(kWaves * kWave), 0, stream, a);
}

template <typename T, int L, int P>
hipError_t launch_router_shape(RouterArgs a, hipStream_t stream) {
    // a group of whole lanes; or the lanes, a power of two, that share the scan of one
    a.whole_lanes = a.group_size % P == 0;
    a.lanes_per_group = a.whole_lanes ? a.group_size / P : 1;
    while (!a.whole_lanes && a.lanes_per_group * 2 * a.groups <= L && a.lanes_per_group * 2 <= a.group_size)
        a.lanes_per_group *= 2;
    constexpr int N = P < 16 / T::kBytes ? P : 16 / T::kBytes, B = P < 4 ? P : 4;
    const bool vec = a.E % (N > B ? N : B) == 0 && a.row_stride % N == 0 && aligned(a.logits, N * T::kBytes) &&
                     aligned(a.bias, 4 * B);
    constexpr int kFew = P > 8 ? 8 : P;  // the usual K: half the moves when a lane's key has been taken
    if (a.K <= kFew) {
        if (vec) launch_router_form<T, L, P, kFew, true>(a, stream);
        else
            launch_router_form<T, L, P, kFew, false>(a, stream);
    } else if (vec) {
        launch_router_form<T, L, P, P, true>(a, stream);
    } else {
        launch_router_form<T, L, P, P, false>(a, stream);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t launch_router(const RouterArgs& a, hipStream_t stream) {
    if (a.E <= 32) return launch_router_shape<T, 16, 2>(a, stream);
    if (a.E <= 64) return launch_router_shape<T, 16, 4>(a, stream);
    if (a.E <= 128) return launch_router_shape<T, 16, 8>(a, stream);
    if (a.E <= kNarrowExperts) return launch_router_shape<T, 16, 16>(a, stream);
    if (a.E <= 512) return launch_router_shape<T, 64, 8>(a, stream);
    return launch_router_shape<T, 64, 16>(a, stream);
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

// A launch takes fewer than 2^32 threads: rows over 64 lanes reach that before the limit of T does.
bool fits_launch(int64_t T, int32_t E) { return E <= kNarrowExperts || T < (int64_t{1} << 32) / kWave; }

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
    if (num_groups > MOE_ROUTER_MAX_GROUPS || !fits_launch(num_tokens, num_experts)) return MOE_ERR_UNSUPPORTED;
    if (num_tokens == 0) return MOE_OK;
    if (logits == nullptr || topk_idx == nullptr || topk_weights == nullptr) return MOE_ERR_INVALID_ARGUMENT;
    if (!aligned(logits, logits_dtype == MOE_DTYPE_BF16 ? 2 : 4) || !aligned(bias, 4) || !aligned(topk_idx, 8) ||
        !aligned(topk_weights, 4))
        return MOE_ERR_INVALID_ARGUMENT;
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
    if (!fits_launch(num_tokens, num_experts)) return MOE_ERR_UNSUPPORTED;
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
