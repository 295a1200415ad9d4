// Wave64 fp32 reductions and the exponential shared by the block norm and
// balance loss kernels.
#pragma once

#include <type_traits>

#include "device_utils.hpp"

namespace moe {

template <int CTRL>
__device__ __forceinline__ float dpp_f32(float x) {
    return __uint_as_float(dpp_u32<CTRL>(__float_as_uint(x)));
}

// After the four steps within a 16-lane row, the rows meet through gfx950's
// row and half-wave swaps: swapping a register with itself leaves, in the two
// results, the two rows (halves) to be joined, in every lane.  VALU only; the
// cross-lane moves through LDS (ds_swizzle, ds_bpermute) would add their
// latency to each of the row reductions these kernels wait for.
template <typename Op>
__device__ __forceinline__ float join_rows(float x, Op op) {
    const uint32_t b = __float_as_uint(x);
    const auto rows = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    const uint32_t c = __float_as_uint(op(__uint_as_float(rows[0]), __uint_as_float(rows[1])));
    const auto halves = __builtin_amdgcn_permlane32_swap(c, c, false, false);
    return op(__uint_as_float(halves[0]), __uint_as_float(halves[1]));
}

// Sum and maximum over each group of L lanes, 16 (a DPP row) or 64.
template <int L>
__device__ __forceinline__ float group_sum_f32(float x) {
    static_assert(L == 16 || L == kWave, "a DPP row or a wave");
    x += dpp_f32<kDppQuadXor1>(x);
    x += dpp_f32<kDppQuadXor2>(x);
    x += dpp_f32<kDppRowHalfMirror>(x);
    x += dpp_f32<kDppRowMirror>(x);
    if constexpr (L == kWave) x = join_rows(x, [](float a, float b) { return a + b; });
    return x;
}
template <int L>
__device__ __forceinline__ float group_max_f32(float x) {
    static_assert(L == 16 || L == kWave, "a DPP row or a wave");
    x = fmaxf(x, dpp_f32<kDppQuadXor1>(x));
    x = fmaxf(x, dpp_f32<kDppQuadXor2>(x));
    x = fmaxf(x, dpp_f32<kDppRowHalfMirror>(x));
    x = fmaxf(x, dpp_f32<kDppRowMirror>(x));
    if constexpr (L == kWave) x = join_rows(x, [](float a, float b) { return fmaxf(a, b); });
    return x;
}

// Sum over the wave in a fixed order; every lane receives it.
__device__ __forceinline__ float wave_sum_f32(float x) { return group_sum_f32<kWave>(x); }

__device__ __forceinline__ int wave_sum_i32(int x) {
    uint32_t u = static_cast<uint32_t>(x);
    u += dpp_u32<kDppQuadXor1>(u);
    u += dpp_u32<kDppQuadXor2>(u);
    u += dpp_u32<kDppRowHalfMirror>(u);
    u += dpp_u32<kDppRowMirror>(u);
    const auto rows = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    u = rows[0] + rows[1];
    const auto halves = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return static_cast<int>(halves[0] + halves[1]);
}

// exp(x) for x <= 0 (and NaN) by the hardware exp2: the rounded product x *
// log2(e) costs a relative error of |x| * 2^-24 (about 1e-6 at x = -16, where
// the value is 1e-7), which the scores' normalisation carries over unchanged.
__device__ __forceinline__ float exp_nonpos(float x) {
    return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f);
}

// bf16 bit pattern (round to nearest even) of an fp32 value, and two packed.
__device__ __forceinline__ uint16_t bf16_bits(float f) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}
__device__ __forceinline__ uint32_t bf16_pack2(float lo, float hi) {
    return static_cast<uint32_t>(bf16_bits(lo)) | (static_cast<uint32_t>(bf16_bits(hi)) << 16);
}

template <bool STREAM>
__device__ __forceinline__ uint4 load16(const uint4* p) {
    if constexpr (STREAM) return load_stream16(p);
    return *p;
}
template <bool STREAM>
__device__ __forceinline__ void store16(uint4* p, const uint4& v) {
    if constexpr (STREAM)
        store_stream16(p, v);
    else
        *p = v;
}

// Element types of the operators that take bf16 or fp32: VEC consecutive
// values to and from fp32 registers.  VEC > 1 needs the address aligned to
// min(16, VEC * sizeof(T)) bytes.  STREAM: non-temporal 16-byte accesses.
//
// Raw<VEC>: the values as loaded, to be unpacked later.
struct Bf16 {
    static constexpr int kBytes = 2;
    template <int VEC>
    struct Raw {
        static_assert(VEC == 8 || VEC == 1, "vector width");
        typename std::conditional<VEC == 8, u32x4_t, uint16_t>::type v;
        __device__ __forceinline__ void load(const void* p, int64_t i) {
            v = *reinterpret_cast<const decltype(v)*>(static_cast<const uint16_t*>(p) + i);
        }
        __device__ __forceinline__ void unpack(float (&f)[VEC]) const {
            if constexpr (VEC == 8) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    f[2 * k] = bf16_lo(v[k]);
                    f[2 * k + 1] = bf16_hi(v[k]);
                }
            } else {
                f[0] = __uint_as_float(static_cast<uint32_t>(v) << 16);
            }
        }
    };
    template <int VEC, bool STREAM = false>
    static __device__ __forceinline__ void load(const void* p, int64_t i, float (&f)[VEC]) {
        const uint16_t* q = static_cast<const uint16_t*>(p) + i;
        if constexpr (VEC % 8 == 0) {
#pragma unroll
            for (int v = 0; v < VEC / 8; ++v)
                unpack8_bf16(load16<STREAM>(reinterpret_cast<const uint4*>(q) + v),
                             *reinterpret_cast<float(*)[8]>(f + 8 * v));
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
    template <int VEC, bool STREAM = false>
    static __device__ __forceinline__ void store(void* p, int64_t i, const float (&f)[VEC]) {
        uint16_t* q = static_cast<uint16_t*>(p) + i;
        if constexpr (VEC % 8 == 0) {
#pragma unroll
            for (int v = 0; v < VEC / 8; ++v) {
                const float* g = f + 8 * v;
                store16<STREAM>(reinterpret_cast<uint4*>(q) + v,
                                make_uint4(bf16_pack2(g[0], g[1]), bf16_pack2(g[2], g[3]), bf16_pack2(g[4], g[5]),
                                           bf16_pack2(g[6], g[7])));
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
    struct Raw {
        static_assert(VEC == 8 || VEC == 1, "vector width");
        static constexpr int N = VEC == 8 ? 2 : 1;
        typename std::conditional<VEC == 8, u32x4_t, uint32_t>::type v[N];
        __device__ __forceinline__ void load(const void* p, int64_t i) {
#pragma unroll
            for (int n = 0; n < N; ++n)
                v[n] = reinterpret_cast<const std::remove_reference_t<decltype(v[0])>*>(static_cast<const float*>(p) + i)[n];
        }
        __device__ __forceinline__ void unpack(float (&f)[VEC]) const {
            if constexpr (VEC == 8) {
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(v[k / 4][k % 4]);
            } else {
                f[0] = __uint_as_float(v[0]);
            }
        }
    };
    template <int VEC, bool STREAM = false>
    static __device__ __forceinline__ void load(const void* p, int64_t i, float (&f)[VEC]) {
        const float* q = static_cast<const float*>(p) + i;
        if constexpr (VEC % 4 == 0) {
#pragma unroll
            for (int v = 0; v < VEC / 4; ++v) {
                const uint4 r = load16<STREAM>(reinterpret_cast<const uint4*>(q) + v);
                f[4 * v] = __uint_as_float(r.x); f[4 * v + 1] = __uint_as_float(r.y);
                f[4 * v + 2] = __uint_as_float(r.z); f[4 * v + 3] = __uint_as_float(r.w);
            }
        } else if constexpr (VEC == 2) {
            const float2 r = *reinterpret_cast<const float2*>(q);
            f[0] = r.x; f[1] = r.y;
        } else {
            static_assert(VEC == 1, "vector width");
            f[0] = *q;
        }
    }
    template <int VEC, bool STREAM = false>
    static __device__ __forceinline__ void store(void* p, int64_t i, const float (&f)[VEC]) {
        float* q = static_cast<float*>(p) + i;
        if constexpr (VEC % 4 == 0) {
#pragma unroll
            for (int v = 0; v < VEC / 4; ++v)
                store16<STREAM>(reinterpret_cast<uint4*>(q) + v,
                                make_uint4(__float_as_uint(f[4 * v]), __float_as_uint(f[4 * v + 1]),
                                           __float_as_uint(f[4 * v + 2]), __float_as_uint(f[4 * v + 3])));
        } else if constexpr (VEC == 2) {
            *reinterpret_cast<float2*>(q) = make_float2(f[0], f[1]);
        } else {
            static_assert(VEC == 1, "vector width");
            *q = f[0];
        }
    }
};

// int32 values as fp32 (load only).
struct I32 {
    template <int VEC>
    static __device__ __forceinline__ void load(const void* p, int64_t i, float (&f)[VEC]) {
        float bits[VEC];
        F32::load<VEC>(p, i, bits);
#pragma unroll
        for (int v = 0; v < VEC; ++v) f[v] = static_cast<float>(__float_as_int(bits[v]));
    }
};

}  // namespace moe
