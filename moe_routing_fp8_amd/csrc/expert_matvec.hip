// The experts' products at decode: a few rows per expert times that expert's
// 4-bit weights.
//
//   out[r, n] = sum_k x[r, k] * e2m1(w[e(r), n, k]) * sf[e(r), n, k / g]
//
// Rows are grouped by expert (expert_offsets).  Up to some 64 rows per expert
// the weights' bytes bound the time, so the kernel is built around one pass
// over them: a wave reads 16 weight rows at a time, each lane 16 bytes (32
// codes) of one row, and every fragment it unpacks feeds the matrix cores
// for up to MT * 16 rows of x.
//
// Products.  An e2m1 value is exact in bf16, and so is an e4m3 value of x, so
// both go through the bf16 matrix instruction with exact products and fp32
// sums.  A UE8M0 scale is a power of two and joins the weight in the
// conversion (exact as well); a weight scale in fp32 or the 128-channel scale
// of an e4m3 row multiplies the fp32 sum of its group.  Nothing is rounded to
// fewer than 32 bits before the output's one rounding to bf16.  (The scaled
// 8-bit x 4-bit matrix instruction would skip the conversions, but it aligns
// its products to fewer bits than fp32 holds: 5e-5 relative error on random
// operands.)
//
// Fragments.  v_mfma_f32_16x16x32_bf16 takes 8 consecutive k from each lane;
// lane l holds row l % 16 of its operand and quarter l / 16 of the k range.
// The order of k within a step of 128 is free as long as both operands agree:
//   - scales of one value per 128 k, or folded ones: instruction i takes the
//     i-th dword of every lane's 16 bytes, k = 32 q + 8 i + (0..7);
//   - fp32 scales per 32 k: instruction i must cover one group, k = 32 i +
//     8 q + (0..7); four lane-row swaps transpose the dwords over the lane
//     quarters.
// The workgroup's waves split k; their sums meet in LDS in a fixed order.
#include <hip/hip_runtime.h>

#include "api_common.hpp"
#include "math_device.hpp"
#include "moe_fp8.h"

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kStep = 128;  // k per step of a wave
enum ScaleMode { kFolded = 0, kF32Group128 = 1, kF32Group32 = 2 };

struct MatvecArgs {
    const void* x;
    const float* x_sf;
    int64_t x_rows;
    const int32_t* row_token;
    int64_t num_rows;
    int K, N, E;
    const int32_t* offsets;
    const uint8_t* codes;
    const void* sf;
    int group;
    uint16_t* out;
};

union Frag {
    bf16x8_t v;
    bf16x2_t p[4];
    uint4 u;
};

// Eight e2m1 codes (low nibble first) times 2^(exponent of scale), as bf16.
__device__ __forceinline__ bf16x8_t e2m1_to_bf16(uint32_t d, float scale) {
    Frag f;
    f.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 0);
    f.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 1);
    f.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 2);
    f.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 3);
    return f.v;
}
// Eight e4m3 codes as bf16.
__device__ __forceinline__ bf16x8_t e4m3_to_bf16(uint32_t lo, uint32_t hi) {
    Frag f;
    f.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    f.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    f.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    f.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return f.v;
}

// Dword i of the lane in quarter q goes to dword q of the lane in quarter i.
__device__ __forceinline__ void transpose_quarters(uint32_t (&d)[4]) {
    const auto a = __builtin_amdgcn_permlane16_swap(d[0], d[1], false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(d[2], d[3], false, false);
    const auto even = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
    const auto odd = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
    d[0] = even[0];
    d[1] = odd[0];
    d[2] = even[1];
    d[3] = odd[1];
}

// The index-th expert that has rows; false if there are fewer.  Offsets are
// clamped to [0, num_rows].
__device__ __forceinline__ bool find_expert(const MatvecArgs& a, int index, int lane, int& e, int64_t& row0,
                                            int& rows) {
    if (a.offsets == nullptr) {
        e = 0;
        row0 = 0;
        rows = static_cast<int>(a.num_rows);
        return index == 0;
    }
    const int R = static_cast<int>(a.num_rows);
    for (int base = 0; base < a.E; base += kWave) {
        int begin = 0, end = 0;
        if (base + lane < a.E) {
            begin = min(max(a.offsets[base + lane], 0), R);
            end = min(max(a.offsets[base + lane + 1], 0), R);
        }
        const uint64_t busy = __ballot(end > begin);
        const int n = __builtin_popcountll(busy);
        if (index < n) {
            const int rank = __builtin_popcountll(busy & ((uint64_t{1} << lane) - 1));
            const int at = __builtin_ctzll(__ballot(end > begin && rank == index));
            e = base + at;
            row0 = __builtin_amdgcn_readlane(begin, at);
            rows = __builtin_amdgcn_readlane(end, at) - static_cast<int>(row0);
            return true;
        }
        index -= n;
    }
    return false;
}

template <bool E4M3, int MODE, int NT, int MT, int WAVES>
__global__ __launch_bounds__(WAVES* kWave) void expert_matvec_kernel(MatvecArgs a) {
    // the operand whose scale is per row of its own goes second: a lane's four
    // sums then share that row
    constexpr bool kXFirst = MODE != kFolded;
    __shared__ float red[WAVES > 1 ? WAVES : 1][MT * 16][NT * 16 + 1];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int lr = lane & 15, q = lane >> 4;
    int e, rows;
    int64_t row0;
    if (!find_expert(a, blockIdx.y, lane, e, row0, rows)) return;
    const int n0 = blockIdx.x * (NT * 16);
    const int K = a.K;
    const int steps = (K + kStep - 1) / kStep;
    const int first = steps * wave / WAVES, last = steps * (wave + 1) / WAVES;
    const int groups = K / a.group;

    const uint8_t* wrow[NT];
    int64_t srow[NT];  // first scale of the lane's weight row
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int64_t n = static_cast<int64_t>(e) * a.N + min(n0 + nt * 16 + lr, a.N - 1);
        wrow[nt] = a.codes + n * (K / 2) + q * 16;
        srow[nt] = n * groups;
    }

    for (int m0 = 0; m0 < rows; m0 += MT * 16) {
        int64_t xrow[MT];  // x row of the lane's row of x, or -1
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int m = m0 + mt * 16 + lr;
            int64_t r = -1;
            if (m < rows) r = a.row_token != nullptr ? a.row_token[row0 + m] : row0 + m;
            xrow[mt] = r < a.x_rows ? r : -1;
        }
        f32x4_t acc[MT][NT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

        for (int step = first; step < last; ++step) {
            const int k0 = step * kStep;
            const bool in = k0 + q * 32 < K;
            uint32_t wd[NT][4];
            float ws[NT][4];  // kFolded, kF32Group128: [0]
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint4 w = make_uint4(0, 0, 0, 0);
                if (in) w = *reinterpret_cast<const uint4*>(wrow[nt] + k0 / 2);
                wd[nt][0] = w.x; wd[nt][1] = w.y; wd[nt][2] = w.z; wd[nt][3] = w.w;
                ws[nt][0] = 1.0f;
                if constexpr (MODE == kFolded) {
                    if (in) {
                        const uint32_t b = static_cast<const uint8_t*>(a.sf)[srow[nt] + (k0 + q * 32) / a.group];
                        ws[nt][0] = __uint_as_float(b << 23);
                    }
                } else if constexpr (MODE == kF32Group128) {
                    ws[nt][0] = static_cast<const float*>(a.sf)[srow[nt] + k0 / 128];
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        ws[nt][i] = k0 + i * 32 < K ? static_cast<const float*>(a.sf)[srow[nt] + k0 / 32 + i] : 0.0f;
                    transpose_quarters(wd[nt]);
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                // the lane's k of instruction i start at ks + i * ki
                const int ks = MODE == kF32Group32 ? k0 + q * 8 : k0 + q * 32;
                constexpr int ki = MODE == kF32Group32 ? 32 : 8;
                bf16x8_t xf[4];
                float xs[4] = {1.0f, 1.0f, 1.0f, 1.0f};  // kXFirst: of the lane's four sums' rows; else [0]
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    Frag f;
                    f.u = make_uint4(0, 0, 0, 0);
                    if (xrow[mt] >= 0 && ks + i * ki < K) {
                        if constexpr (E4M3) {
                            const uint2 c = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.x) +
                                                                            xrow[mt] * K + ks + i * ki);
                            f.v = e4m3_to_bf16(c.x, c.y);
                        } else {
                            f.u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + xrow[mt] * K +
                                                                  ks + i * ki);
                        }
                    }
                    xf[i] = f.v;
                }
                if constexpr (E4M3) {
                    float own = 0.0f;
                    if (xrow[mt] >= 0) own = a.x_sf[xrow[mt] * (K / 128) + step];
                    xs[0] = own;
                    if constexpr (kXFirst) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) xs[j] = __shfl(own, q * 4 + j, kWave);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if constexpr (MODE == kFolded) {
                        f32x4_t d = E4M3 ? f32x4_t{0.0f, 0.0f, 0.0f, 0.0f} : acc[mt][nt];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e2m1_to_bf16(wd[nt][i], ws[nt][0]), xf[i], d,
                                                                        0, 0, 0);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[mt][nt][j] = E4M3 ? __builtin_fmaf(xs[0], d[j], acc[mt][nt][j]) : d[j];
                    } else if constexpr (MODE == kF32Group128) {
                        f32x4_t d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[i], e2m1_to_bf16(wd[nt][i], 1.0f), d, 0, 0,
                                                                        0);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[mt][nt][j] = __builtin_fmaf(ws[nt][0] * xs[j], d[j], acc[mt][nt][j]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            f32x4_t d = {0.0f, 0.0f, 0.0f, 0.0f};
                            d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[i], e2m1_to_bf16(wd[nt][i], 1.0f), d, 0, 0,
                                                                        0);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                acc[mt][nt][j] = __builtin_fmaf(ws[nt][i] * xs[j], d[j], acc[mt][nt][j]);
                        }
                    }
                }
            }
        }
        // the first operand's rows run along a lane's sums, the second's along the lanes
        if (m0 > 0) __syncthreads();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    red[wave][mt * 16 + (kXFirst ? q * 4 + j : lr)][nt * 16 + (kXFirst ? lr : q * 4 + j)] =
                        acc[mt][nt][j];
        __syncthreads();
        for (int i = threadIdx.x; i < MT * 16 * NT * 16; i += WAVES * kWave) {
            const int m = i / (NT * 16), n = i % (NT * 16);
            if (m0 + m >= rows || n0 + n >= a.N) continue;
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) v += red[w][m][n];
            a.out[(row0 + m0 + m) * a.N + n0 + n] = bf16_bits(v);
        }
    }
}

template <bool E4M3, int MODE>
hipError_t launch_matvec(const MatvecArgs& a, hipStream_t stream) {
    constexpr int NT = 2, MT = 1, WAVES = 4;
    const unsigned experts = static_cast<unsigned>(a.E < a.num_rows ? a.E : a.num_rows);
    const dim3 grid(static_cast<unsigned>((a.N + NT * 16 - 1) / (NT * 16)), experts);
    hipLaunchKernelGGL((expert_matvec_kernel<E4M3, MODE, NT, MT, WAVES>), grid, dim3(WAVES * kWave), 0, stream, a);
    return hipGetLastError();
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_expert_matvec(const void* x, int32_t x_dtype, const float* x_sf, int64_t x_rows,
                                        const int32_t* row_token, int64_t num_rows, int32_t inner, int32_t out_width,
                                        int32_t num_experts, const int32_t* expert_offsets, const uint8_t* w_codes,
                                        const void* w_sf, int32_t group_size, int32_t sf_ue8m0, uint16_t* out_bf16,
                                        hipStream_t stream) {
    using namespace moe;
    if (num_rows < 0 || num_rows > INT32_MAX || x_rows < 0 || x_rows > INT32_MAX) return MOE_ERR_INVALID_ARGUMENT;
    if (x_dtype != MOE_DTYPE_BF16 && x_dtype != MOE_DTYPE_E4M3) return MOE_ERR_INVALID_ARGUMENT;
    if (num_experts < 1 || num_experts > kMaxExperts || out_width < 1 || inner < 1) return MOE_ERR_INVALID_ARGUMENT;
    if (sf_ue8m0 != 0 && sf_ue8m0 != 1) return MOE_ERR_INVALID_ARGUMENT;
    if (group_size != 32 && group_size != 128) return MOE_ERR_UNSUPPORTED;
    if (inner % group_size != 0 || (x_dtype == MOE_DTYPE_E4M3 && inner % 128 != 0)) return MOE_ERR_INVALID_ARGUMENT;
    if (expert_offsets == nullptr && num_experts != 1) return MOE_ERR_INVALID_ARGUMENT;
    if (row_token == nullptr && x_rows != num_rows) return MOE_ERR_INVALID_ARGUMENT;
    if (inner > MOE_MATVEC_MAX_WIDTH || out_width > MOE_MATVEC_MAX_WIDTH) return MOE_ERR_UNSUPPORTED;
    if (num_rows == 0) return MOE_OK;
    if (w_codes == nullptr || w_sf == nullptr || out_bf16 == nullptr) return MOE_ERR_INVALID_ARGUMENT;
    if (x_rows > 0 && (x == nullptr || (x_dtype == MOE_DTYPE_E4M3) != (x_sf != nullptr)))
        return MOE_ERR_INVALID_ARGUMENT;
    if (!aligned(x, 16) || !aligned(w_codes, 16) || !aligned(x_sf, 4) || !aligned(row_token, 4) ||
        !aligned(expert_offsets, 4) || !aligned(w_sf, sf_ue8m0 ? 1 : 4) || !aligned(out_bf16, 2))
        return MOE_ERR_INVALID_ARGUMENT;
    const MatvecArgs a{x,         x_sf,           x_rows,  row_token, num_rows,   inner,   out_width,
                       num_experts, expert_offsets, w_codes, w_sf,      group_size, out_bf16};
    const bool e4m3 = x_dtype == MOE_DTYPE_E4M3;
    hipError_t err;
    if (sf_ue8m0)
        err = e4m3 ? launch_matvec<true, kFolded>(a, stream) : launch_matvec<false, kFolded>(a, stream);
    else if (group_size == 128)
        err = e4m3 ? launch_matvec<true, kF32Group128>(a, stream) : launch_matvec<false, kF32Group128>(a, stream);
    else
        err = e4m3 ? launch_matvec<true, kF32Group32>(a, stream) : launch_matvec<false, kF32Group32>(a, stream);
    return hip_status(err);
}
