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

// exp(x) for x <= 0 (and NaN) by the hardware exp2.  The rounded product x *
// log2(e) costs a relative error of |x| * 2^-24: for an x that is a difference
// of fp32 values, as large as these are the softmax's, whose rounding costs as
// much.
__device__ __forceinline__ float exp_nonpos(float x) {
    return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f);
}

// The same for an exact x, to 1.5 ulp and |x| * 2^-28: with h the rounded
// product, exp(x) = exp2(h) * exp(x - h ln 2), where the second argument is
// below 2^-16 as long as the result is not 0.  Its clamp, which a NaN leaves
// as -1, is for x so low that the difference means nothing, -inf among them.
// (The second difference's own constant leaves the |x| * 2^-28.)
__device__ __forceinline__ float exp_nonpos_exact(float x) {
    const float h = x * 1.44269504088896340736f;
    const float e = __builtin_amdgcn_exp2f(h);
    return __builtin_fmaf(e, __builtin_amdgcn_fmed3f(__builtin_fmaf(-h, 0.693147180559945309417f, x), -1.0f, 1.0f), e);
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
                unpack8_bf16(reinterpret_cast<const uint4*>(q)[v],
                             *reinterpret_cast<float(*)[8]>(f + 8 * v));
        } else if constexpr (VEC == 4) {
            const uint2 r = *reinterpret_cast<const uint2*>(q);
            f[0] = bf16_lo(r.x); f[1] = bf16_hi(r.x); f[2] = bf16_lo(r.y); f[3] = bf16_hi(r.y);
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
                const uint4 r = reinterpret_cast<const uint4*>(q)[v];
                f[4 * v] = __uint_as_float(r.x); f[4 * v + 1] = __uint_as_float(r.y);
                f[4 * v + 2] = __uint_as_float(r.z); f[4 * v + 3] = __uint_as_float(r.w);
            }
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
        } else {
            static_assert(VEC == 1, "vector width");
            *q = f[0];
        }
    }
};

// Eight consecutive values of a row of T (Bf16 or F32), as loaded.  AS says
// how: kAligned 16-byte accesses, the same kStreaming past the caches, or
// kOdd, for rows of any alignment and length: 16-byte accesses at the
// element's alignment (the hardware splits what crosses a line) and, for the
// last n < 8 values of a row, one by one.
enum Access { kAligned, kStreaming, kOdd };

template <typename T, Access AS>
struct Vec8 {
    static constexpr int N = T::kBytes / 2;  // 16-byte pieces
    struct __attribute__((packed, aligned(T::kBytes))) Piece {
        u32x4_t v;
    };
    u32x4_t v[N];

    // n: values left in the row from i on
    __device__ __forceinline__ void load(const void* p, int64_t i, int n) {
        const uint8_t* q = static_cast<const uint8_t*>(p) + i * T::kBytes;
        if constexpr (AS == kOdd) {
            if (n >= 8) {
#pragma unroll
                for (int k = 0; k < N; ++k) v[k] = reinterpret_cast<const Piece*>(q)[k].v;
            } else {
                uint32_t w[4 * N] = {};
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (k >= n) continue;
                    if constexpr (T::kBytes == 2)
                        w[k / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(q)[k]) << (k % 2 * 16);
                    else
                        w[k] = reinterpret_cast<const uint32_t*>(q)[k];
                }
#pragma unroll
                for (int k = 0; k < 4 * N; ++k) v[k / 4][k % 4] = w[k];
            }
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const u32x4_t* a = reinterpret_cast<const u32x4_t*>(q) + k;
                v[k] = AS == kStreaming ? __builtin_nontemporal_load(a) : *a;
            }
        }
    }
    __device__ __forceinline__ void unpack(float (&f)[8]) const {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if constexpr (T::kBytes == 2)
                f[k] = k % 2 == 0 ? bf16_lo(v[0][k / 2]) : bf16_hi(v[0][k / 2]);
            else
                f[k] = __uint_as_float(v[k / 4][k % 4]);
        }
    }
    static __device__ __forceinline__ void store(void* p, int64_t i, int n, const float (&f)[8]) {
        uint8_t* q = static_cast<uint8_t*>(p) + i * T::kBytes;
        if (AS == kOdd && n < 8) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (k >= n) continue;
                if constexpr (T::kBytes == 2)
                    reinterpret_cast<uint16_t*>(q)[k] = bf16_bits(f[k]);
                else
                    reinterpret_cast<float*>(q)[k] = f[k];
            }
            return;
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            u32x4_t w;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if constexpr (T::kBytes == 2)
                    w[c] = bf16_pack2(f[2 * c], f[2 * c + 1]);
                else
                    w[c] = __float_as_uint(f[4 * k + c]);
            }
            if constexpr (AS == kOdd)
                reinterpret_cast<Piece*>(q)[k].v = w;
            else if constexpr (AS == kStreaming)
                __builtin_nontemporal_store(w, reinterpret_cast<u32x4_t*>(q) + k);
            else
                reinterpret_cast<u32x4_t*>(q)[k] = w;
        }
    }
    static __device__ __forceinline__ void load(const void* p, int64_t i, int n, float (&f)[8]) {
        Vec8 r;
        r.load(p, i, n);
        r.unpack(f);
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
