// Wave64 fp32 reductions and the exponential shared by the block norm and
// balance loss kernels.
#pragma once

#include "device_utils.hpp"

namespace moe {

template <int CTRL>
__device__ __forceinline__ float dpp_f32(float x) {
    return __uint_as_float(dpp_u32<CTRL>(__float_as_uint(x)));
}

// The value of the lane 16 places away in the other half of each 32-lane
// half-wave (lane ^ 16), and of the lane in the other half-wave (lane ^ 32).
__device__ __forceinline__ float lane_xor16(float x) {
    return __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(x), 0x401F));
}
__device__ __forceinline__ float lane_xor32(float x) { return __shfl_xor(x, 32, kWave); }

// Sum over the wave in a fixed order; every lane receives it.
__device__ __forceinline__ float wave_sum_f32(float x) {
    x += dpp_f32<kDppQuadXor1>(x);
    x += dpp_f32<kDppQuadXor2>(x);
    x += dpp_f32<kDppRowHalfMirror>(x);
    x += dpp_f32<kDppRowMirror>(x);
    x += lane_xor16(x);
    x += lane_xor32(x);
    return x;
}

// Maximum over the wave (a NaN loses to any number); every lane receives it.
__device__ __forceinline__ float wave_max_f32(float x) {
    x = fmaxf(x, dpp_f32<kDppQuadXor1>(x));
    x = fmaxf(x, dpp_f32<kDppQuadXor2>(x));
    x = fmaxf(x, dpp_f32<kDppRowHalfMirror>(x));
    x = fmaxf(x, dpp_f32<kDppRowMirror>(x));
    x = fmaxf(x, lane_xor16(x));
    x = fmaxf(x, lane_xor32(x));
    return x;
}

// exp(x) for x <= 0 (and NaN): the hardware exp2 of the rounded product
// x * log2(e), times a first-order correction by the product's rounding error
// and the constant's low part.  Without it the error grows with |x| (the
// argument of exp2 carries an error of |x| * 2^-25); with it the result is
// within 2 ulp down to the smallest normal.  exp(-inf) = 0: the correction's
// inf - inf is kept out by the select.
__device__ __forceinline__ float exp_nonpos(float x) {
    constexpr float kLog2e = 1.44269504088896340736f;
    constexpr float kLog2eLo = 1.9259629911266175e-8f;  // log2(e) - kLog2e
    constexpr float kLn2 = 0.693147180559945309417f;
    const float p = x * kLog2e;
    float e = __builtin_fmaf(x, kLog2e, -p);
    e = __builtin_fmaf(x, kLog2eLo, e);
    const float r = __builtin_amdgcn_exp2f(p) * __builtin_fmaf(e, kLn2, 1.0f);
    return x < -104.0f ? 0.0f : r;  // exp(-104) is below half the smallest denormal
}

// bf16 bit pattern (round to nearest even) of an fp32 value, and two packed.
__device__ __forceinline__ uint16_t bf16_bits(float f) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}
__device__ __forceinline__ uint32_t bf16_pack2(float lo, float hi) {
    return static_cast<uint32_t>(bf16_bits(lo)) | (static_cast<uint32_t>(bf16_bits(hi)) << 16);
}

// Element types of the operators that take bf16 or fp32: VEC consecutive
// values to and from fp32 registers.  VEC > 1 needs the address aligned to
// min(16, VEC * sizeof(T)) bytes.
struct Bf16 {
    static constexpr int kBytes = 2;
    template <int VEC>
    static __device__ __forceinline__ void load(const void* p, int64_t i, float (&f)[VEC]) {
        const uint16_t* q = static_cast<const uint16_t*>(p) + i;
        if constexpr (VEC % 8 == 0) {
#pragma unroll
            for (int v = 0; v < VEC / 8; ++v)
                unpack8_bf16(reinterpret_cast<const uint4*>(q)[v], *reinterpret_cast<float(*)[8]>(f + 8 * v));
        } else if constexpr (VEC == 4) {
            const uint2 r = *reinterpret_cast<const uint2*>(q);
            f[0] = bf16_lo(r.x); f[1] = bf16_hi(r.x); f[2] = bf16_lo(r.y); f[3] = bf16_hi(r.y);
        } else if constexpr (VEC == 2) {
            const uint32_t r = *reinterpret_cast<const uint32_t*>(q);
            f[0] = bf16_lo(r); f[1] = bf16_hi(r);
        } else {
            static_assert(VEC == 1, "vector width");
            f[0] = __uint_as_float(static_cast<uint32_t>(*q) << 16);
        }
    }
    template <int VEC>
    static __device__ __forceinline__ void store(void* p, int64_t i, const float (&f)[VEC]) {
        uint16_t* q = static_cast<uint16_t*>(p) + i;
        if constexpr (VEC % 8 == 0) {
#pragma unroll
            for (int v = 0; v < VEC / 8; ++v) {
                const float* g = f + 8 * v;
                reinterpret_cast<uint4*>(q)[v] = make_uint4(bf16_pack2(g[0], g[1]), bf16_pack2(g[2], g[3]),
                                                            bf16_pack2(g[4], g[5]), bf16_pack2(g[6], g[7]));
            }
        } else if constexpr (VEC == 4) {
            *reinterpret_cast<uint2*>(q) = make_uint2(bf16_pack2(f[0], f[1]), bf16_pack2(f[2], f[3]));
        } else if constexpr (VEC == 2) {
            *reinterpret_cast<uint32_t*>(q) = bf16_pack2(f[0], f[1]);
        } else {
            static_assert(VEC == 1, "vector width");
            *q = bf16_bits(f[0]);
        }
    }
};

struct F32 {
    static constexpr int kBytes = 4;
    template <int VEC>
    static __device__ __forceinline__ void load(const void* p, int64_t i, float (&f)[VEC]) {
        const float* q = static_cast<const float*>(p) + i;
        if constexpr (VEC % 4 == 0) {
#pragma unroll
            for (int v = 0; v < VEC / 4; ++v) {
                const float4 r = reinterpret_cast<const float4*>(q)[v];
                f[4 * v] = r.x; f[4 * v + 1] = r.y; f[4 * v + 2] = r.z; f[4 * v + 3] = r.w;
            }
        } else if constexpr (VEC == 2) {
            const float2 r = *reinterpret_cast<const float2*>(q);
            f[0] = r.x; f[1] = r.y;
        } else {
            static_assert(VEC == 1, "vector width");
            f[0] = *q;
        }
    }
    template <int VEC>
    static __device__ __forceinline__ void store(void* p, int64_t i, const float (&f)[VEC]) {
        float* q = static_cast<float*>(p) + i;
        if constexpr (VEC % 4 == 0) {
#pragma unroll
            for (int v = 0; v < VEC / 4; ++v)
                reinterpret_cast<float4*>(q)[v] = make_float4(f[4 * v], f[4 * v + 1], f[4 * v + 2], f[4 * v + 3]);
        } else if constexpr (VEC == 2) {
            *reinterpret_cast<float2*>(q) = make_float2(f[0], f[1]);
        } else {
            static_assert(VEC == 1, "vector width");
            *q = f[0];
        }
    }
};

}  // namespace moe
