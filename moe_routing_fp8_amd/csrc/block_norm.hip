// The norms after and before a block of the residual stream, fused with the
// block's gate and the residual scale, and their gradients.
//
// For a row of the residual r and of the block's output y (both H wide):
//   u  = y * rsqrt(mean(y^2) + eps) * post_weight     (no post_weight: u = y)
//   r' = residual_scale * r + gate * u                (no y: r' = r)
//   n  = r' * rsqrt(mean(r'^2) + eps) * pre_weight
// n is taken from r' in fp32, before r' is rounded for storage.
//
// One pass: a row is held in registers by one wave (short rows) or one
// workgroup, so y and r are read once and r' and n written once; the two sums
// of squares are the only exchanges between lanes.  The backward pass holds
// the four arrays of a row the same way.  Its parameter gradients are sums
// over rows: a workgroup walks over rows with a stride, keeps its columns'
// running sums in registers, and writes them once; a second launch adds the
// workgroups' sums in order.
//
// Kernel traces (a kernel that does nothing: 1.3 us; a large copy runs at 5.2
// TB/s).  Bound by the bytes of the rows:
//   forward, 4096 x 7168, bf16                     48.6 us  4.8 TB/s
//   forward, no norm after the block and no gate   41.7 us  5.6 TB/s
//   backward, 4096 x 7168, fp32 r and bf16 y       105.2 + 5.4 us  4.8 TB/s
//   backward, 4096 x 7168, fp32                    146.3 + 5.4 us  4.6 TB/s, with 12 registers spilled
// and by the latency of a row's dependent sums:
//   forward, one row of 7168, bf16                 4.0 us
//   backward, 4096 x 7168, bf16                    87.5 + 5.3 us  3.8 TB/s
//   backward, 1021 x 2049, bf16 (cached)           16.4 + 4.0 us, two rows in turn; its bytes take 4.9
//   backward, 16384 x 256, bf16 (cached)           30.7 + 4.7 us, 16 rows in turn; its bytes take 9.8
//   backward, 2048 x 16384, bf16                   250.7 + 9.0 us, with 80 registers spilled
#include <hip/hip_runtime.h>

#include "api_common.hpp"
#include "math_device.hpp"
#include "moe_fp8.h"

namespace moe {
namespace {

constexpr int kMaxRowThreads = 1024;
constexpr int kMaxHidden = MOE_BLOCK_NORM_MAX_HIDDEN;
// The backward pass takes one workgroup for each compute unit, two up to
// eight waves a row and four up to four, no more than 16 waves a compute unit
// (a single one for rows of one wave gives it four); each leaves one row of
// partial sums.
constexpr int64_t kComputeUnits = 256;

// 1 / sqrt(v): the hardware's estimate and one Newton step, which brings it
// to within 1 ulp (0 and infinity keep the estimate's value).  The estimate
// takes a subnormal v, which eps = 0 lets through, for 0: v is scaled by 2^24
// there, and the root by 2^12.
__device__ __forceinline__ float rsqrt_f32(float v) {
    const bool tiny = v < 0x1p-126f;
    const float s = tiny ? v * 0x1p24f : v;
    const float r = __builtin_amdgcn_rsqf(s);
    const float e = __builtin_fmaf(-s * r, r, 1.0f);
    float n = __builtin_fmaf(0.5f * r, e, r);
    n = s > 0.0f && s < INFINITY ? n : r;
    return tiny ? n * 0x1p12f : n;
}

// Rows of more bytes than this in all are read and written past the caches
// (half of the 256 MB of Infinity Cache: what is larger finds nothing there
// when it comes round again).  4096 x 7168 bf16: 48.0 us against 54.8.  The
// backward pass streams its stores only (119.1 us against 121.8 before its
// rows took one shape of access for all alignments, which made it 110; with
// streaming loads 131).
constexpr int64_t kStreamBytes = int64_t{128} << 20;

// Sum over the workgroup, in a fixed order; every thread receives it.  `part`
// holds one float per wave and is not written again before another barrier.
__device__ __forceinline__ float block_sum(float v, float* part) {
    v = wave_sum_f32(v);
    const int waves = blockDim.x / kWave;
    if (waves == 1) return v;
    if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < waves; ++w) s += part[w];
    return s;
}

struct NormArgs {
    const void* residual;
    int64_t residual_stride;
    const void* y;
    int64_t y_stride;
    int64_t num_tokens;
    int hidden;
    const float* post_weight;
    const float* gate;
    int gate_mode;
    float residual_scale;
    const float* pre_weight;
    float eps;
    void* res_out;
    void* normed;
    float* post_rstd;
    float* pre_rstd;
};

// Parameters are read where the next row finds them again: never streaming.
template <Access AS>
using Param8 = Vec8<F32, AS == kOdd ? kOdd : kAligned>;

// Thread i's j-th vector of a row starts at element (i + j * blockDim.x) * 8.
template <typename TR, typename TA, int VPT, Access AS>
__global__ __launch_bounds__(kMaxRowThreads) void block_norm_kernel(NormArgs a) {
    __shared__ float part[2][kMaxRowThreads / kWave];
    const int64_t t = blockIdx.x;
    const int H = a.hidden;
    const float inv_h = 1.0f / static_cast<float>(H);
    float r[VPT][8], u[VPT][8];
    float sq = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int e = (threadIdx.x + j * blockDim.x) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) r[j][i] = u[j][i] = 0.0f;
        if (e < H) {
            Vec8<TR, AS>::load(a.residual, t * a.residual_stride + e, H - e, r[j]);
            if (a.y != nullptr) Vec8<TA, AS>::load(a.y, t * a.y_stride + e, H - e, u[j]);
        }
    }
    if (a.y != nullptr) {
        float rstd = 1.0f;
        if (a.post_weight != nullptr) {
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) sq += u[j][i] * u[j][i];
            rstd = rsqrt_f32(block_sum(sq, part[0]) * inv_h + a.eps);
            if (threadIdx.x == 0 && a.post_rstd != nullptr) a.post_rstd[t] = rstd;
        }
        const float token_gate = a.gate_mode == MOE_GATE_TOKEN ? a.gate[t] : 1.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int e = (threadIdx.x + j * blockDim.x) * 8;
            if (e >= H) continue;
            float w[8], g[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                w[i] = 1.0f;
                g[i] = token_gate;
            }
            if (a.post_weight != nullptr) Param8<AS>::load(a.post_weight, e, H - e, w);
            if (a.gate_mode == MOE_GATE_CHANNEL) Param8<AS>::load(a.gate, e, H - e, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) r[j][i] = a.residual_scale * r[j][i] + g[i] * (u[j][i] * rstd * w[i]);
            Vec8<TR, AS>::store(a.res_out, t * H + e, H - e, r[j]);
        }
    }
    if (a.normed == nullptr) return;
    sq = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) sq += r[j][i] * r[j][i];
    const float rstd = rsqrt_f32(block_sum(sq, part[1]) * inv_h + a.eps);
    if (threadIdx.x == 0 && a.pre_rstd != nullptr) a.pre_rstd[t] = rstd;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int e = (threadIdx.x + j * blockDim.x) * 8;
        if (e >= H) continue;
        float w[8];
        Param8<AS>::load(a.pre_weight, e, H - e, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = r[j][i] * rstd * w[i];
        Vec8<TA, AS>::store(a.normed, t * H + e, H - e, w);
    }
}

struct NormGradArgs {
    const void* grad_res_out;  // or nullptr: zero
    const void* grad_normed;   // or nullptr: no norm before the next block
    const void* res_out;
    int64_t res_out_stride;
    const void* y;
    int64_t y_stride;
    int64_t num_tokens;
    int hidden;
    const float* post_weight;
    const float* gate;
    int gate_mode;
    float residual_scale;
    const float* pre_weight;
    const float* post_rstd;
    const float* pre_rstd;
    void* grad_residual;
    void* grad_y;
    float* grad_token_gate;
    float* partials;  // [workgroup][parameter][H rounded up to 8]: post weight, channel gate, pre weight (those given)
    int num_params;
};

// A row's four arrays as loaded.
template <typename TR, typename TA, int VPT, Access AS>
struct GradRow {
    Vec8<TR, AS> grad_res_out[VPT], res_out[VPT];
    Vec8<TA, AS> grad_normed[VPT], y[VPT];
    float pre_rstd, post_rstd, token_gate;
};

// HELD: the next row's loads are in flight while a row is worked on, and the
// parameters stay in registers.  The workgroup's waves fill a compute unit at
// hidden 7168, so nothing else would cover a row's loads; reading the three
// parameters again for each row would add 86 KB from the caches to the 129 KB
// of the row.  Without (rows of more than 8 values a thread): neither fits.
// A workgroup of up to 1024 threads leaves a thread 128 registers: that holds
// one vector of a row unless both streams are fp32 (12 to 25 spilled), and two
// vectors not at all (78 to 702 spilled).
// AS: of the loads; OUT: of the stores.
template <typename TR, typename TA, int VPT, Access AS, Access OUT>
__global__ __launch_bounds__(kMaxRowThreads) void block_norm_grad_kernel(NormGradArgs a) {
    constexpr bool HELD = VPT == 1;
    // two sets in turn: a row's sums have been read before the next row but one writes there
    __shared__ float part[2][3][kMaxRowThreads / kWave];
    int turn = 0;
    const int H = a.hidden;
    const float inv_h = 1.0f / static_cast<float>(H);
    const bool pre = a.grad_normed != nullptr, block = a.y != nullptr, post = a.post_weight != nullptr;
    const bool channel = a.gate_mode == MOE_GATE_CHANNEL;
    float sum_post[VPT][8], sum_gate[VPT][8], sum_pre[VPT][8];
    float held_post[HELD ? VPT : 1][8], held_gate[HELD ? VPT : 1][8], held_pre[HELD ? VPT : 1][8];
    auto load_params = [&](int e, float(&wp)[8], float(&wg)[8], float(&wn)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            wp[i] = wg[i] = 1.0f;
            wn[i] = 0.0f;
        }
        if (post) Param8<AS>::load(a.post_weight, e, H - e, wp);
        if (channel) Param8<AS>::load(a.gate, e, H - e, wg);
        if (pre) Param8<AS>::load(a.pre_weight, e, H - e, wn);
    };
    auto load = [&](GradRow<TR, TA, VPT, AS>& row, int64_t t) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int e = (threadIdx.x + j * blockDim.x) * 8;
            if (e >= H) continue;
            if (a.grad_res_out != nullptr) row.grad_res_out[j].load(a.grad_res_out, t * H + e, H - e);
            if (pre) {
                row.res_out[j].load(a.res_out, t * a.res_out_stride + e, H - e);
                row.grad_normed[j].load(a.grad_normed, t * H + e, H - e);
            }
            if (block) row.y[j].load(a.y, t * a.y_stride + e, H - e);
        }
        row.pre_rstd = pre ? a.pre_rstd[t] : 0.0f;
        row.post_rstd = post ? a.post_rstd[t] : 1.0f;
        row.token_gate = a.gate_mode == MOE_GATE_TOKEN ? a.gate[t] : 1.0f;
    };
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sum_post[j][i] = sum_gate[j][i] = sum_pre[j][i] = 0.0f;
        const int e = (threadIdx.x + j * blockDim.x) * 8;
        if constexpr (HELD)
            if (e < H) load_params(e, held_post[j], held_gate[j], held_pre[j]);
    }
    GradRow<TR, TA, VPT, AS> row;
    if constexpr (HELD) load(row, blockIdx.x);
    for (int64_t t = blockIdx.x; t < a.num_tokens; t += gridDim.x, turn ^= 1) {
        if constexpr (!HELD) load(row, t);
        float d[VPT][8], yh[VPT][8], xh[VPT][8], g[VPT][8];
        const float pre_rstd = row.pre_rstd, post_rstd = row.post_rstd, token_gate = row.token_gate;
        float dot = 0.0f;
        // D = dr' + rstd * (g - xh * mean(g * xh)), g = dn * pre_weight
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int e = (threadIdx.x + j * blockDim.x) * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) d[j][i] = yh[j][i] = xh[j][i] = g[j][i] = 0.0f;
            if (e >= H) continue;
            if (a.grad_res_out != nullptr) row.grad_res_out[j].unpack(d[j]);
            if (block) row.y[j].unpack(yh[j]);
            if (pre) {
                row.res_out[j].unpack(xh[j]);
                row.grad_normed[j].unpack(g[j]);
                float wn[8];
                if constexpr (!HELD) Param8<AS>::load(a.pre_weight, e, H - e, wn);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    xh[j][i] *= pre_rstd;
                    sum_pre[j][i] = __builtin_fmaf(g[j][i], xh[j][i], sum_pre[j][i]);
                    g[j][i] *= HELD ? held_pre[HELD ? j : 0][i] : wn[i];
                    dot = __builtin_fmaf(g[j][i], xh[j][i], dot);
                }
            }
        }
        if constexpr (HELD)
            if (t + gridDim.x < a.num_tokens) load(row, t + gridDim.x);
        if (pre) {
            const float mean = block_sum(dot, part[turn][0]) * inv_h;
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) d[j][i] += pre_rstd * (g[j][i] - xh[j][i] * mean);
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int e = (threadIdx.x + j * blockDim.x) * 8;
            if (e >= H) continue;
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = a.residual_scale * d[j][i];
            Vec8<TR, OUT>::store(a.grad_residual, t * H + e, H - e, o);
        }
        if (block) {
            float dot_gate = 0.0f;
            dot = 0.0f;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int e = (threadIdx.x + j * blockDim.x) * 8;
                if (e >= H) continue;
                float wp[8], wg[8], wn[8];
                if constexpr (!HELD) load_params(e, wp, wg, wn);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float w = HELD ? held_post[HELD ? j : 0][i] : wp[i];
                    const float gate = channel ? (HELD ? held_gate[HELD ? j : 0][i] : wg[i]) : token_gate;
                    yh[j][i] *= post_rstd;
                    const float along = d[j][i] * (yh[j][i] * w);
                    dot_gate += along;
                    sum_gate[j][i] += along;
                    d[j][i] *= gate;  // du
                    sum_post[j][i] = __builtin_fmaf(d[j][i], yh[j][i], sum_post[j][i]);
                    d[j][i] *= w;
                    dot = __builtin_fmaf(d[j][i], yh[j][i], dot);
                }
            }
            if (a.gate_mode == MOE_GATE_TOKEN) {
                dot_gate = block_sum(dot_gate, part[turn][1]);
                if (threadIdx.x == 0) a.grad_token_gate[t] = dot_gate;
            }
            if (post) {
                const float mean = block_sum(dot, part[turn][2]) * inv_h;
#pragma unroll
                for (int j = 0; j < VPT; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i) d[j][i] = post_rstd * (d[j][i] - yh[j][i] * mean);
            }
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int e = (threadIdx.x + j * blockDim.x) * 8;
                if (e < H) Vec8<TA, OUT>::store(a.grad_y, t * H + e, H - e, d[j]);
            }
        }
    }
    const int width = (H + 7) / 8 * 8;
    float* out = a.partials + static_cast<int64_t>(blockIdx.x) * a.num_params * width;
    using Out8 = Vec8<F32, kAligned>;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int e = (threadIdx.x + j * blockDim.x) * 8;
        if (e >= H) continue;
        int64_t at = e;
        if (post) {
            Out8::store(out, at, 8, sum_post[j]);
            at += width;
        }
        if (channel) {
            Out8::store(out, at, 8, sum_gate[j]);
            at += width;
        }
        if (pre) Out8::store(out, at, 8, sum_pre[j]);
    }
}

// The parameters' gradients: column sums of the workgroups' partials, each of
// kSumWaves waves every kSumWaves-th row in order, then the waves in order.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(kSumWaves* kWave) void block_norm_param_kernel(const float* __restrict__ partials,
                                                                             int64_t blocks, int params, int H,
                                                                             float* o0, float* o1, float* o2) {
    __shared__ float lds[kSumWaves][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int c = blockIdx.x * kWave + lane, padded = (H + 7) / 8 * 8, width = params * padded;
    float v = 0.0f;
    if (c < width)
#pragma unroll 8
        for (int64_t b = wave; b < blocks; b += kSumWaves) v += partials[b * width + c];
    lds[wave][lane] = v;
    __syncthreads();
    if (wave == 0 && c < width) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kSumWaves; ++w) s += lds[w][lane];
        float* const outs[3] = {o0, o1, o2};
        int left = c;
        for (int k = 0; k < 3; ++k) {
            if (outs[k] == nullptr) continue;
            if (left < padded) {
                if (left < H) outs[k][left] = s;
                break;
            }
            left -= padded;
        }
    }
}

// Threads of a row: enough that VPT vectors of 8 each cover it, in whole waves.
int row_threads(int H, int vpt) {
    const int n = (H + 8 * vpt - 1) / (8 * vpt);
    return (n + kWave - 1) / kWave * kWave;
}

template <typename TR, typename TA, int VPT, Access AS>
hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL((block_norm_kernel<TR, TA, VPT, AS>), dim3(static_cast<unsigned>(a.num_tokens)),
                       dim3(row_threads(a.hidden, VPT)), 0, stream, a);
    return hipGetLastError();
}
// Two vectors a thread where the rows fill the chip (their shorter workgroups
// overlap: 48.0 us against 50.8 with one) or do not fit otherwise; one where
// the latency of a few rows counts.
template <typename TR, typename TA, Access AS>
hipError_t launch_norm_rows(const NormArgs& a, hipStream_t stream) {
    if (AS != kStreaming && a.hidden <= 8 * kMaxRowThreads && a.num_tokens <= 2 * kComputeUnits)
        return launch_norm<TR, TA, 1, AS>(a, stream);
    return launch_norm<TR, TA, 2, AS>(a, stream);
}

template <typename TR, typename TA, int VPT, Access AS, Access OUT>
hipError_t launch_grad(const NormGradArgs& a, int64_t blocks, hipStream_t stream) {
    hipLaunchKernelGGL((block_norm_grad_kernel<TR, TA, VPT, AS, OUT>), dim3(static_cast<unsigned>(blocks)),
                       dim3(row_threads(a.hidden, VPT)), 0, stream, a);
    return hipGetLastError();
}
template <typename TR, typename TA, Access AS, Access OUT>
hipError_t launch_grad_rows(const NormGradArgs& a, int64_t blocks, hipStream_t stream) {
    if (a.hidden > 8 * kMaxRowThreads) return launch_grad<TR, TA, 2, AS, AS>(a, blocks, stream);
    return launch_grad<TR, TA, 1, AS, OUT>(a, blocks, stream);
}

// Calls f with the two element types.
template <typename F>
hipError_t with_types(int res, int act, F&& f) {
    if (res == MOE_DTYPE_BF16) return act == MOE_DTYPE_BF16 ? f(Bf16{}, Bf16{}) : f(Bf16{}, F32{});
    return act == MOE_DTYPE_BF16 ? f(F32{}, Bf16{}) : f(F32{}, F32{});
}

bool dtype_ok(int32_t d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F32; }
int dtype_bytes(int32_t d) { return d == MOE_DTYPE_BF16 ? 2 : 4; }
// Rows of 8-element vectors: 16-byte aligned start and stride (a null pointer passes).
bool vec_rows(const void* p, int64_t stride, int32_t dtype) {
    return aligned(p, 16) && stride * dtype_bytes(dtype) % 16 == 0;
}

// Whether a gate (or its gradient) is there iff its mode asks for one; of no tokens' gate either is right.
bool gate_given(int mode, const void* gate, int64_t num_tokens) {
    if (mode == MOE_GATE_TOKEN && num_tokens == 0) return true;
    return (mode != MOE_GATE_NONE) == (gate != nullptr);
}

int64_t grad_blocks(int64_t T, int H) {
    const int waves = row_threads(H, 1) / kWave;
    const int64_t most = kComputeUnits * (waves > 8 ? 1 : waves > 4 ? 2 : 4);
    return T < most ? T : most;
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_block_norm(const void* residual, int64_t residual_stride, int32_t residual_dtype, const void* y,
                          int64_t y_stride, int32_t act_dtype, int64_t num_tokens, int32_t hidden,
                          const float* post_weight, const float* gate, int32_t gate_mode, float residual_scale,
                          const float* pre_weight, float eps, void* res_out, void* normed, float* post_rstd,
                          float* pre_rstd, hipStream_t stream) {
    using namespace moe;
    if (num_tokens < 0 || hidden < 1 || !dtype_ok(residual_dtype) || !dtype_ok(act_dtype))
        return MOE_ERR_INVALID_ARGUMENT;
    if (gate_mode != MOE_GATE_NONE && gate_mode != MOE_GATE_CHANNEL && gate_mode != MOE_GATE_TOKEN)
        return MOE_ERR_INVALID_ARGUMENT;
    if (!(eps >= 0.0f) || residual_scale != residual_scale) return MOE_ERR_INVALID_ARGUMENT;
    if (!gate_given(gate_mode, gate, num_tokens)) return MOE_ERR_INVALID_ARGUMENT;
    if (post_rstd != nullptr && post_weight == nullptr) return MOE_ERR_INVALID_ARGUMENT;
    if (residual_stride < hidden) return MOE_ERR_INVALID_ARGUMENT;
    if (hidden > kMaxHidden || num_tokens > MOE_BLOCK_NORM_MAX_TOKENS) return MOE_ERR_UNSUPPORTED;
    if (num_tokens == 0) return MOE_OK;  // tensors without elements may be null
    if ((normed != nullptr) != (pre_weight != nullptr)) return MOE_ERR_INVALID_ARGUMENT;
    if (pre_rstd != nullptr && normed == nullptr) return MOE_ERR_INVALID_ARGUMENT;
    const bool block = y != nullptr;
    if (residual == nullptr || block != (res_out != nullptr)) return MOE_ERR_INVALID_ARGUMENT;
    if (block) {
        if (y_stride < hidden) return MOE_ERR_INVALID_ARGUMENT;
    } else if (normed == nullptr || post_weight != nullptr || gate != nullptr || residual_scale != 1.0f) {
        return MOE_ERR_INVALID_ARGUMENT;  // without a block only the norm before the next one is left
    }
    const int rb = dtype_bytes(residual_dtype), ab = dtype_bytes(act_dtype);
    if (!aligned(residual, rb) || !aligned(res_out, rb) || !aligned(y, ab) || !aligned(normed, ab) ||
        !aligned(post_weight, 4) || !aligned(gate, 4) || !aligned(pre_weight, 4) || !aligned(post_rstd, 4) ||
        !aligned(pre_rstd, 4))
        return MOE_ERR_INVALID_ARGUMENT;
    const bool vec = hidden % 8 == 0 && vec_rows(residual, residual_stride, residual_dtype) &&
                     vec_rows(y, y == nullptr ? 8 : y_stride, act_dtype) && aligned(res_out, 16) &&
                     aligned(normed, 16) && aligned(post_weight, 16) && aligned(pre_weight, 16) &&
                     (gate_mode != MOE_GATE_CHANNEL || aligned(gate, 16));
    const NormArgs a{residual,  residual_stride, y,          y_stride, num_tokens, hidden, post_weight, gate,
                     gate_mode, residual_scale,  pre_weight, eps,      res_out,    normed, post_rstd,   pre_rstd};
    const int64_t row_bytes = int64_t{2} * hidden * (rb + ab);
    const bool far = num_tokens * row_bytes > kStreamBytes;
    return hip_status(with_types(residual_dtype, act_dtype, [&](auto r, auto x) {
        using R = decltype(r);
        using A = decltype(x);
        return !vec  ? launch_norm_rows<R, A, kOdd>(a, stream)
               : far ? launch_norm_rows<R, A, kStreaming>(a, stream)
                     : launch_norm_rows<R, A, kAligned>(a, stream);
    }));
}

size_t moe_block_norm_backward_workspace_bytes(int64_t num_tokens, int32_t hidden) {
    if (num_tokens < 0 || num_tokens > MOE_BLOCK_NORM_MAX_TOKENS || hidden < 1 || hidden > moe::kMaxHidden) return 0;
    const size_t n = static_cast<size_t>(moe::grad_blocks(num_tokens, hidden)) * 3 * ((hidden + 7) / 8 * 8) * 4;
    return (n + 255) / 256 * 256;
}

moe_status moe_block_norm_backward(const void* grad_res_out, const void* grad_normed, const void* res_out,
                                   int64_t res_out_stride, int32_t residual_dtype, const void* y, int64_t y_stride,
                                   int32_t act_dtype, int64_t num_tokens, int32_t hidden, const float* post_weight,
                                   const float* gate, int32_t gate_mode, float residual_scale,
                                   const float* pre_weight, const float* post_rstd, const float* pre_rstd,
                                   void* grad_residual, void* grad_y, float* grad_post_weight, float* grad_gate,
                                   float* grad_pre_weight, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream) {
    using namespace moe;
    if (num_tokens < 0 || hidden < 1 || !dtype_ok(residual_dtype) || !dtype_ok(act_dtype))
        return MOE_ERR_INVALID_ARGUMENT;
    if (gate_mode != MOE_GATE_NONE && gate_mode != MOE_GATE_CHANNEL && gate_mode != MOE_GATE_TOKEN)
        return MOE_ERR_INVALID_ARGUMENT;
    if (residual_scale != residual_scale) return MOE_ERR_INVALID_ARGUMENT;
    if (!gate_given(gate_mode, gate, num_tokens) || !gate_given(gate_mode, grad_gate, num_tokens))
        return MOE_ERR_INVALID_ARGUMENT;
    if ((post_weight != nullptr) != (grad_post_weight != nullptr) ||
        (pre_weight != nullptr) != (grad_pre_weight != nullptr))
        return MOE_ERR_INVALID_ARGUMENT;
    const bool pre = pre_weight != nullptr, block = y != nullptr;
    if (pre && res_out_stride < hidden) return MOE_ERR_INVALID_ARGUMENT;
    if (hidden > kMaxHidden || num_tokens > MOE_BLOCK_NORM_MAX_TOKENS) return MOE_ERR_UNSUPPORTED;
    const int rb = dtype_bytes(residual_dtype), ab = dtype_bytes(act_dtype);
    if (num_tokens > 0) {
        if (grad_residual == nullptr || (grad_res_out == nullptr && !pre)) return MOE_ERR_INVALID_ARGUMENT;
        if (block != (grad_y != nullptr)) return MOE_ERR_INVALID_ARGUMENT;
        if (block) {
            if (y_stride < hidden) return MOE_ERR_INVALID_ARGUMENT;
        } else if (post_weight != nullptr || gate != nullptr || residual_scale != 1.0f) {
            return MOE_ERR_INVALID_ARGUMENT;
        }
        if (pre ? (grad_normed == nullptr || res_out == nullptr || pre_rstd == nullptr) : grad_normed != nullptr)
            return MOE_ERR_INVALID_ARGUMENT;
        if (post_weight != nullptr && post_rstd == nullptr) return MOE_ERR_INVALID_ARGUMENT;
        if (!aligned(grad_res_out, rb) || !aligned(res_out, rb) || !aligned(grad_residual, rb) ||
            !aligned(grad_normed, ab) || !aligned(y, ab) || !aligned(grad_y, ab))
            return MOE_ERR_INVALID_ARGUMENT;
    }
    for (const void* p : {static_cast<const void*>(post_weight), static_cast<const void*>(gate),
                          static_cast<const void*>(pre_weight), static_cast<const void*>(post_rstd),
                          static_cast<const void*>(pre_rstd), static_cast<const void*>(grad_post_weight),
                          static_cast<const void*>(grad_gate), static_cast<const void*>(grad_pre_weight)})
        if (!aligned(p, 4)) return MOE_ERR_INVALID_ARGUMENT;
    const bool channel = gate_mode == MOE_GATE_CHANNEL;
    const int params = (post_weight != nullptr) + channel + pre;
    if (num_tokens > 0 && params > 0) {
        if (workspace == nullptr || !aligned(workspace, 256)) return MOE_ERR_INVALID_ARGUMENT;
        if (workspace_bytes < moe_block_norm_backward_workspace_bytes(num_tokens, hidden))
            return MOE_ERR_WORKSPACE_TOO_SMALL;
    }
    const int64_t blocks = grad_blocks(num_tokens, hidden);
    float* partials = static_cast<float*>(workspace);
    if (num_tokens > 0) {
        const bool vec = hidden % 8 == 0 && aligned(grad_res_out, 16) && aligned(grad_normed, 16) &&
                         (!pre || vec_rows(res_out, res_out_stride, residual_dtype)) &&
                         (!block || vec_rows(y, y_stride, act_dtype)) && aligned(grad_residual, 16) &&
                         aligned(grad_y, 16) && aligned(post_weight, 16) && aligned(pre_weight, 16) &&
                         (!channel || aligned(gate, 16));
        const NormGradArgs a{grad_res_out,
                             pre ? grad_normed : nullptr,
                             res_out,
                             res_out_stride,
                             y,
                             y_stride,
                             num_tokens,
                             hidden,
                             post_weight,
                             gate,
                             gate_mode,
                             residual_scale,
                             pre_weight,
                             post_rstd,
                             pre_rstd,
                             grad_residual,
                             grad_y,
                             gate_mode == MOE_GATE_TOKEN ? grad_gate : nullptr,
                             partials,
                             params};
        const bool far = num_tokens * (int64_t{3} * hidden * (rb + ab)) > kStreamBytes;
        const hipError_t err = with_types(residual_dtype, act_dtype, [&](auto r, auto x) {
            using R = decltype(r);
            using A = decltype(x);
            return !vec  ? launch_grad_rows<R, A, kOdd, kOdd>(a, blocks, stream)
                   : far ? launch_grad_rows<R, A, kAligned, kStreaming>(a, blocks, stream)
                         : launch_grad_rows<R, A, kAligned, kAligned>(a, blocks, stream);
        });
        if (err != hipSuccess) return hip_status(err);
    }
    if (params == 0) return MOE_OK;
    // with no tokens the parameters' gradients are zero: the same sums over no workgroups
    const int width = params * ((hidden + 7) / 8 * 8);
    hipLaunchKernelGGL(block_norm_param_kernel, dim3((width + kWave - 1) / kWave), dim3(kSumWaves * kWave), 0, stream,
                       partials, blocks, params, hidden, grad_post_weight, channel ? grad_gate : nullptr,
                       grad_pre_weight);
    return hip_status(hipGetLastError());
}

}  // extern "C"
