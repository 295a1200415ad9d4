// Rows to 8-bit integers with one scale a row: of a tensor as it is, and of
// SwiGLU's result, for the experts' products in 8-bit integers.
//
// Per row: sf = max(amax, 127 * 2^-126) / 127 and inv = 1 / sf, correctly
// rounded, then code = round to nearest even of v * inv, within [-127, 127]
// (|v| * inv <= 127 (1 + 2^-22)).  The clamp keeps sf normal.
//
// The scale needs the whole row before the first code: a wave (rows of up to
// 512 channels) or a workgroup holds the row in registers, 8 channels a lane
// and step, so it is read once; wider rows than kMaxSteps steps of a workgroup
// are read again.  Bound by bytes and, at these sizes, by start and drain: 2048 x
// 7168 bf16 take 12.1 us (3.6 TB/s), SwiGLU of 4096 x 2 x 2048 10.8 us (3.9 TB/s;
// medians of kernel traces).
#include <hip/hip_runtime.h>

#include "api_common.hpp"
#include "kernels.hpp"
#include "math_device.hpp"
#include "moe_fp8.h"
#include "swiglu_math.hpp"

namespace moe {
namespace {

constexpr int kBlock = 256;
constexpr int kMaxSteps = 4;  // steps of a row held in registers: 8192 channels

struct CastArgs {
    const void* x;        // rows; SwiGLU: bf16 [gate | up]
    int64_t row_stride;   // elements
    int64_t num_rows;
    int width;            // channels of a row of codes
    const float* row_weights;
    float clamp;
    int8_t* out;
    float* sf;
};

// Eight channels of a row, in fp32.
template <typename T, Access AS>
struct PlainRow {
    const CastArgs& a;
    int64_t base;
    __device__ PlainRow(const CastArgs& args, int64_t r) : a(args), base(r * args.row_stride) {}
    __device__ __forceinline__ void load(int i, int n, float (&f)[8]) const {
        Vec8<T, AS>::load(a.x, base + i, n, f);
    }
};
template <Access AS>
struct SwigluRow {
    const CastArgs& a;
    int64_t base;
    float w;
    __device__ SwigluRow(const CastArgs& args, int64_t r)
        : a(args), base(r * args.row_stride), w(args.row_weights != nullptr ? args.row_weights[r] : 1.0f) {}
    __device__ __forceinline__ void load(int i, int n, float (&f)[8]) const {
        float up[8];
        Vec8<Bf16, AS>::load(a.x, base + i, n, f);
        Vec8<Bf16, AS>::load(a.x, base + a.width + i, n, up);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            float v;
            if (a.clamp > 0.0f) {
                v = silu_any_arg(fminf(f[c], a.clamp)) * fmaxf(fminf(up[c], a.clamp), -a.clamp);
            } else {
                v = silu_bf16_arg(f[c]) * up[c];
            }
            f[c] = a.row_weights != nullptr ? v * w : v;
        }
    }
};

// Eight codes, the lowest channel in the lowest byte.
__device__ __forceinline__ uint32_t code(float v, float inv) {
    return static_cast<uint32_t>(static_cast<int>(__builtin_rintf(v * inv)));
}
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float inv) {
    uint2 q;
    q.x = (code(f[0], inv) & 255u) | (code(f[1], inv) & 255u) << 8 | (code(f[2], inv) & 255u) << 16 |
          code(f[3], inv) << 24;
    q.y = (code(f[4], inv) & 255u) | (code(f[5], inv) & 255u) << 8 | (code(f[6], inv) & 255u) << 16 |
          code(f[7], inv) << 24;
    return q;
}

template <Access AS>
__device__ __forceinline__ void store_codes(int8_t* p, int n, const uint2& q) {
    if constexpr (AS == kOdd) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) p[k] = static_cast<int8_t>((k < 4 ? q.x : q.y) >> (8 * (k % 4)));
    } else {
        *reinterpret_cast<uint2*>(p) = q;
    }
}

// WAVES waves a row, STEPS steps of 8 channels a lane (0: as many as it takes,
// read twice).
template <typename Row, Access AS, int WAVES, int STEPS>
__global__ __launch_bounds__(kBlock) void cast_int8_kernel(CastArgs a) {
    constexpr int kLanes = WAVES * kWave;
    __shared__ uint32_t most[kBlock / kWave];
    const int lane = threadIdx.x % kLanes;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * (kBlock / kLanes) + threadIdx.x / kLanes;
    if (r >= a.num_rows) return;  // whole waves of a row; a row of several waves is the whole workgroup's
    const Row row(a, r);
    float f[STEPS > 0 ? STEPS : 1][8];
    uint32_t amax = 0;
    if constexpr (STEPS > 0) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int i = (s * kLanes + lane) * 8;
#pragma unroll
            for (int c = 0; c < 8; ++c) f[s][c] = 0.0f;
            if (i < a.width) row.load(i, a.width - i, f[s]);
        }
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int i = (s * kLanes + lane) * 8;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (AS != kOdd || i + c < a.width) amax = max(amax, abs_bits(f[s][c]));
        }
    } else {
        for (int i = lane * 8; i < a.width; i += kLanes * 8) {
            row.load(i, a.width - i, f[0]);
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (AS != kOdd || i + c < a.width) amax = max(amax, abs_bits(f[0][c]));
        }
    }
    amax = __float_as_uint(group_max_f32<kWave>(__uint_as_float(amax)));
    if constexpr (WAVES > 1) {
        if (threadIdx.x % kWave == 0) most[threadIdx.x / kWave] = amax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WAVES; ++w) amax = max(amax, most[w]);
    }
    const float sf = fmaxf(__uint_as_float(amax), 127.0f * 0x1p-126f) / 127.0f;
    const float inv = 1.0f / sf;
    int8_t* out = a.out + r * a.width;
    if constexpr (STEPS > 0) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int i = (s * kLanes + lane) * 8;
            if (i < a.width) store_codes<AS>(out + i, a.width - i, codes8(f[s], inv));
        }
    } else {
        for (int i = lane * 8; i < a.width; i += kLanes * 8) {
            row.load(i, a.width - i, f[0]);
            store_codes<AS>(out + i, a.width - i, codes8(f[0], inv));
        }
    }
    if (lane == 0) a.sf[r] = sf;
}

template <typename Row, Access AS>
hipError_t launch_cast(const CastArgs& a, hipStream_t stream) {
    const int64_t packed = (a.num_rows + kBlock / kWave - 1) / (kBlock / kWave);
    const dim3 block(kBlock);
    if (a.width <= 8 * kWave)
        hipLaunchKernelGGL((cast_int8_kernel<Row, AS, 1, 1>), dim3(static_cast<unsigned>(packed)), block, 0, stream, a);
    else if (a.width <= 8 * kBlock)
        hipLaunchKernelGGL((cast_int8_kernel<Row, AS, 4, 1>), dim3(static_cast<unsigned>(a.num_rows)), block, 0, stream,
                           a);
    else if (a.width <= 2 * 8 * kBlock)
        hipLaunchKernelGGL((cast_int8_kernel<Row, AS, 4, 2>), dim3(static_cast<unsigned>(a.num_rows)), block, 0, stream,
                           a);
    else if (a.width <= kMaxSteps * 8 * kBlock)
        hipLaunchKernelGGL((cast_int8_kernel<Row, AS, 4, kMaxSteps>), dim3(static_cast<unsigned>(a.num_rows)), block, 0,
                           stream, a);
    else
        hipLaunchKernelGGL((cast_int8_kernel<Row, AS, 4, 0>), dim3(static_cast<unsigned>(a.num_rows)), block, 0, stream,
                           a);
    return hipGetLastError();
}

constexpr int64_t kMaxRows = 1 << 24;  // one workgroup a row: fewer than 2^32 threads

}  // namespace
}  // namespace moe

extern "C" moe_status moe_cast_int8(const void* x, int32_t x_dtype, int64_t row_stride, int64_t num_rows, int32_t width,
                                    int8_t* out, float* out_sf, hipStream_t stream) {
    using namespace moe;
    if (x_dtype != MOE_DTYPE_BF16 && x_dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARGUMENT;
    if (num_rows < 0 || width < 1 || row_stride < width) return MOE_ERR_INVALID_ARGUMENT;
    if (width > MOE_MATVEC_MAX_WIDTH || num_rows >= kMaxRows) return MOE_ERR_UNSUPPORTED;
    if (num_rows == 0) return MOE_OK;
    if (x == nullptr || out == nullptr || out_sf == nullptr) return MOE_ERR_INVALID_ARGUMENT;
    if (!aligned(x, x_dtype == MOE_DTYPE_BF16 ? 2 : 4) || !aligned(out_sf, 4)) return MOE_ERR_INVALID_ARGUMENT;
    const CastArgs a{x, row_stride, num_rows, width, nullptr, 0.0f, out, out_sf};
    const bool even = width % 8 == 0 && row_stride % 8 == 0 && aligned(x, 16) && aligned(out, 8);
    hipError_t err;
    if (x_dtype == MOE_DTYPE_BF16)
        err = even ? launch_cast<PlainRow<Bf16, kAligned>, kAligned>(a, stream)
                   : launch_cast<PlainRow<Bf16, kOdd>, kOdd>(a, stream);
    else
        err = even ? launch_cast<PlainRow<F32, kAligned>, kAligned>(a, stream)
                   : launch_cast<PlainRow<F32, kOdd>, kOdd>(a, stream);
    return hip_status(err);
}

extern "C" moe_status swiglu_cast_int8(const uint16_t* gate_up_bf16, int64_t num_rows, int32_t inter,
                                       const float* row_weights, float clamp_value, int8_t* out, float* out_sf,
                                       hipStream_t stream) {
    using namespace moe;
    if (num_rows < 0 || inter < 1 || clamp_value != clamp_value) return MOE_ERR_INVALID_ARGUMENT;
    if (inter > MOE_MATVEC_MAX_WIDTH || num_rows >= kMaxRows) return MOE_ERR_UNSUPPORTED;
    if (num_rows == 0) return MOE_OK;
    if (gate_up_bf16 == nullptr || out == nullptr || out_sf == nullptr) return MOE_ERR_INVALID_ARGUMENT;
    if (!aligned(gate_up_bf16, 2) || !aligned(row_weights, 4) || !aligned(out_sf, 4)) return MOE_ERR_INVALID_ARGUMENT;
    const CastArgs a{gate_up_bf16, 2 * static_cast<int64_t>(inter), num_rows, inter, row_weights, clamp_value, out,
                     out_sf};
    const bool even = inter % 8 == 0 && aligned(gate_up_bf16, 16) && aligned(out, 8);
    return hip_status(even ? launch_cast<SwigluRow<kAligned>, kAligned>(a, stream)
                           : launch_cast<SwigluRow<kOdd>, kOdd>(a, stream));
}
