// The experts' products at decode: a few rows per expert times that expert's
// 4-bit weights.
//
//   out[r, n] = sum_k x[r, k] * e2m1(w[e(r), n, k]) * sf[e(r), n, k / g]
//
// Rows are grouped by expert (expert_offsets).  Up to some 64 rows per expert
// the weights' bytes bound the time, so the kernel is built around one pass
// over them: a wave owns 32 weight rows (output columns) and walks along k in
// steps of 128; every fragment of codes that it unpacks meets up to MAXROWS
// (8, 16 or 32) rows of x in the matrix cores.
//
// Measured, from kernel traces (weights, scales, rows and results over the time):
//   one token's 8 experts, 7168 -> 4096, UE8M0 scales, bf16 x   25 us    5.0 TB/s
//   128 rows, 32 experts, 7168 -> 4096, UE8M0 scales, e4m3 x    79 to 89 us, 5.5 to 6.2 TB/s
//   128 rows, 32 experts, 7168 -> 4096, fp32 scales of 32       115 to 123 us, 4.7 to 5.0 TB/s
//   512 rows, 32 experts, 2048 -> 7168, fp32 scales, bf16 x     60 to 65 us, 4.0 to 4.3 TB/s
//   one token's 4 experts, 2880 -> 5760, UE8M0 scales, bf16 x   20 us    1.7 TB/s (k ends inside a block)
//   one row, one expert, 2048 -> 7168, UE8M0 scales, bf16 x     5.1 us   (latency: loads, one block of k, the join of
//                                                               four waves' shares; an empty kernel takes 1.3)
// A bare streaming read of such arrays reaches 6.6 to 7.0 TB/s.  With few rows
// the start and the drain of a launch of one round of waves bound it; with 16
// and more rows the registers, which allow two waves a SIMD and so bound the
// loads in flight while the matrix cores and the conversions work.  They do
// not hold everything everywhere: 2 to 10 are spilled in passes of 32 rows
// (the 512 rows above), 2 to 10 in passes of 16 with fp32 scales of 32, and
// 24 to 48 in those where k ends inside a block.
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
// Workgroups.  Where there is a tile of columns for every wave the chip holds,
// a workgroup's four waves take four tiles and share their rows of x (SHARED);
// with fewer tiles the workgroup's waves split the k of one, and their sums
// meet in LDS in a fixed order.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "api_common.hpp"
#include "expert_matvec_lds.hpp"
#include "math_device.hpp"
#include "moe_fp8.h"

namespace moe {
namespace {

using namespace matvec;

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kStep = 128;  // k per step of a wave
static_assert(kLanes == kWave, "LDS layout");
constexpr int kMaxThreads = kMaxSplit * kWave;
constexpr int64_t kWavePlaces = 8 * 256;
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
    u32x4_t u;
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

__device__ __forceinline__ u32x4_t u32x4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) { return u32x4_t{a, b, c, d}; }

// Four words and one of them at any alignment (a row of scale bytes starts anywhere).
struct __attribute__((packed, aligned(1))) Words4 {
    uint32_t w[4];
};
struct __attribute__((packed, aligned(1))) Word {
    uint32_t w;
};

// One wave's share of a tile: NT * 16 weight rows from column n0 on, k steps
// [first, last) of which [first, first + 4 * blocks) in blocks of four.
struct Share {
    int e, n0;
    int64_t row0;  // of the expert's rows
    int rows;
    int first, blocks, last;
};

// Keeps the compiler from moving LDS accesses of one lane across those of
// others that it has to stay behind; the hardware runs a wave's in order.
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The sums of rows m0 .. m0 + ROWS - 1 of the expert over the wave's share of k.
//
// Eight neighbouring lanes load one row's 128 bytes of codes (16 neighbouring
// lanes, or 8, a row's 256 or 128 bytes of x).  A load in the order of the
// matrix fragments, whose neighbouring lanes lie in different rows, occupies
// the address unit four times as long, and one that takes half a cache line
// leaves the next step's to wait in the cache for the line on its way; either
// bounded the kernel (as did one byte of scales per lane and step).  The wave's own corner of LDS then turns the data
// into fragments: lane (lr, q) reads row lr (of x_unit's).  The
// 16-byte chunks of a row are stored at (chunk XOR row), which spreads the
// eight rows that one LDS clock serves over all banks.
//
// SHARED: the workgroup's waves have tiles of their own and the same k, so
// each loads the x of one step of a block for all of them; otherwise they
// split k and each loads its own.  TAIL: k may end inside a block.
template <bool E4M3, int MODE, int MAXROWS, int ROWS, bool SHARED, bool TAIL>
__device__ __forceinline__ void multiply_rows(const MatvecArgs& a, const Share& sh, int m0, int lane, int wave,
                                              u32x4_t* lds, u32x4_t* x_lds, f32x4_t (&acc)[(ROWS + 15) / 16][kNT]) {
    constexpr bool kXFirst = MODE != kFolded;
    static_assert((ROWS & (ROWS - 1)) == 0 && ROWS <= MAXROWS, "rows of a pass");
    constexpr int MT = (ROWS + 15) / 16;
    constexpr int kChunks = E4M3 ? 8 : 16;             // 16-byte chunks of a row of x in a step
    constexpr int kRowsPerLoad = kWave / kChunks;
    constexpr int XI = (ROWS + kRowsPerLoad - 1) / kRowsPerLoad;
    constexpr int kAhead = SHARED ? 1 : kBlock;  // steps of x in the wave's registers
    constexpr int kStepX = ROWS * kChunks;             // LDS of a step's x
    constexpr int XV = E4M3 ? 2 : 4;                   // 16-byte vectors of a lane's fragments of one step
    const int lr = lane & 15, q = lane >> 4;
    const int K = a.K;
    const bool bytes32 = MODE == kFolded && a.group == 32;
    u32x4_t* lds_w = lds;
    u32x4_t* lds_s = lds + kLdsCodes;

    // codes: load i's row 8 i + lane / 8 of tile nt, scales: row `lane` of the tile pair
    const uint8_t* wp[kNT][kPair];
    const int64_t row_e = static_cast<int64_t>(sh.e) * a.N;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int i = 0; i < kPair; ++i) {
            const int64_t n = row_e + min(sh.n0 + nt * 16 + i * 8 + lane / 8, a.N - 1);
            wp[nt][i] = a.codes + n * (K / 2) + ((lane & 7) ^ (lane >> 3)) * 16;
        }
    const uint8_t* sp = static_cast<const uint8_t*>(a.sf) + (row_e + min(sh.n0 + lane % kCols, a.N - 1)) *
                                                               (K / a.group) * (MODE == kFolded ? 1 : 4);
    // x: load i's row x_load_row(i)
    auto x_row = [&](int m) -> int64_t {
        int64_t r = -1;
        if (m < sh.rows - m0 && m < ROWS) r = a.row_token != nullptr ? a.row_token[sh.row0 + m0 + m] : sh.row0 + m0 + m;
        return r < a.x_rows ? r : -1;
    };
    const uint8_t* xp[XI];
#pragma unroll
    for (int i = 0; i < XI; ++i) {
        const int64_t r = x_row(x_load_row(kChunks, i, lane));
        xp[i] = r < 0 ? nullptr
                      : static_cast<const uint8_t*>(a.x) + r * (E4M3 ? K : 2 * static_cast<int64_t>(K)) +
                            x_load_chunk(kChunks, i, lane) * 16;
    }
    const float* xsp[MT];  // scales of e4m3 row lr of each fragment
    if constexpr (E4M3)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int64_t r = x_row(mt * 16 + lr);
            xsp[mt] = r < 0 ? nullptr : a.x_sf + r * (K / 128);
        }

    auto unpack_x = [&](bf16x8_t(&xf)[4], const u32x4_t(&x)[XV]) __attribute__((always_inline)) {
        if constexpr (E4M3) {
            xf[0] = e4m3_to_bf16(x[0].x, x[0].y);
            xf[1] = e4m3_to_bf16(x[0].z, x[0].w);
            xf[2] = e4m3_to_bf16(x[1].x, x[1].y);
            xf[3] = e4m3_to_bf16(x[1].z, x[1].w);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                Frag f;
                f.u = x[i];
                xf[i] = f.v;
            }
        }
    };
    auto unpack_codes = [&](bf16x8_t(&wf)[kNT][4], const u32x4_t(&w)[kNT], const float(&ws)[kNT][4])
        __attribute__((always_inline)) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            uint32_t d[4] = {w[nt].x, w[nt].y, w[nt].z, w[nt].w};
            if constexpr (MODE == kF32Group32) transpose_quarters(d);
#pragma unroll
            for (int i = 0; i < 4; ++i) wf[nt][i] = e2m1_to_bf16(d[i], MODE == kFolded ? ws[nt][0] : 1.0f);
        }
    };
    // Sums of 16 rows from their fragments; xs_own: the scale of the lane's e4m3 row.
    auto multiply = [&](const bf16x8_t(&wf)[kNT][4], const float(&ws)[kNT][4], const u32x4_t(&x)[XV], float xs_own,
                        f32x4_t(&sum)[kNT]) __attribute__((always_inline)) {
        bf16x8_t xf[4];
        unpack_x(xf, x);
        float xs[4] = {1.0f, 1.0f, 1.0f, 1.0f};  // kXFirst: of the lane's four sums' rows; else [0]
        if constexpr (E4M3) {
            xs[0] = xs_own;
            if constexpr (kXFirst) {
#pragma unroll
                for (int j = 0; j < 4; ++j) xs[j] = __shfl(xs_own, q * 4 + j, kWave);
            }
        }
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            if constexpr (MODE == kFolded) {
                f32x4_t d = E4M3 ? f32x4_t{0.0f, 0.0f, 0.0f, 0.0f} : sum[nt];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[nt][i], xf[i], d, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[nt][j] = E4M3 ? __builtin_fmaf(xs[0], d[j], sum[nt][j]) : d[j];
            } else if constexpr (MODE == kF32Group128) {
                f32x4_t d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[i], wf[nt][i], d, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[nt][j] = __builtin_fmaf(ws[nt][0] * xs[j], d[j], sum[nt][j]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f32x4_t d = {0.0f, 0.0f, 0.0f, 0.0f};
                    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[i], wf[nt][i], d, 0, 0, 0);
#pragma unroll
                    for (int j = 0; j < 4; ++j) sum[nt][j] = __builtin_fmaf(ws[nt][i] * xs[j], d[j], sum[nt][j]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };

    // Loads complete in order, so a step's x goes out before its codes.  Lanes without a row of x load nothing:
    // their fragment rows hold anything, and only give sums that are not kept.
    auto load_x = [&](u32x4_t(&x)[XI], int step) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < XI; ++i)
            if (xp[i] != nullptr)
                x[i] = *reinterpret_cast<const u32x4_t*>(xp[i] + static_cast<int64_t>(step) * (kChunks * 16));
    };
    auto load_codes = [&](u32x4_t(&w)[kNT][kPair], int step) __attribute__((always_inline)) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int i = 0; i < kPair; ++i)
                w[nt][i] = __builtin_nontemporal_load(
                    reinterpret_cast<const u32x4_t*>(wp[nt][i] + step * (kStep / 2)));
    };
    auto load_step_scales = [&](u32x4_t& s, int step) __attribute__((always_inline)) {
        if (MODE == kF32Group32 && lane < kCols) {
            const Words4 v = *reinterpret_cast<const Words4*>(sp + 16 * step);
            s = u32x4(v.w[0], v.w[1], v.w[2], v.w[3]);
        }
    };
    // a block's scales of a weight row: 16 bytes, or one word of four steps' bytes
    auto load_scales = [&](u32x4_t& s, float4(&xs)[MT], int step) __attribute__((always_inline)) {
        if (MODE != kF32Group32 && lane < kCols) {
            if (MODE == kFolded && !bytes32) {
                s.x = reinterpret_cast<const Word*>(sp + step)->w;
            } else {
                const Words4 v = *reinterpret_cast<const Words4*>(sp + 4 * step);
                s = u32x4(v.w[0], v.w[1], v.w[2], v.w[3]);
            }
        }
        if constexpr (E4M3)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                if (xsp[mt] != nullptr) {
                    const Words4 v = *reinterpret_cast<const Words4*>(xsp[mt] + step);
                    xs[mt] = make_float4(__uint_as_float(v.w[0]), __uint_as_float(v.w[1]), __uint_as_float(v.w[2]),
                                         __uint_as_float(v.w[3]));
                }
    };
    if (sh.blocks > 0) {
        u32x4_t w[kBlock / kPair][kNT][kPair], x[kAhead][XI], s[kBlock];  // s: kF32Group32 of each step
        float4 xs[MT] = {}, xs_next[MT] = {};
        u32x4_t s_next;
        const int end = sh.first + kBlock * sh.blocks;
        load_scales(s_next, xs_next, sh.first);
#pragma unroll
        for (int j = 0; j < kBlock; ++j) {
            if (j < kAhead) load_x(x[j], sh.first + (SHARED ? wave : j));
            load_step_scales(s[j], sh.first + j);
            if (j % kPair == 0) load_codes(w[j / kPair], sh.first + j);
        }
        for (int step = sh.first; step < end; step += kBlock) {
            const bool more = step + kBlock < end;
            if (MODE != kF32Group32 && lane < kCols) lds_s[lane] = s_next;
            if constexpr (E4M3)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) xs[mt] = xs_next[mt];
            if (more) load_scales(s_next, xs_next, step + kBlock);
            if constexpr (SHARED) {
                if (step > sh.first) __syncthreads();  // the block before has been read
#pragma unroll
                for (int i = 0; i < XI; ++i) x_lds[wave * kStepX + i * kWave + lane] = x[0][i];
                if (more) load_x(x[0], step + kBlock + wave);
                __syncthreads();
            }
#pragma unroll
            for (int j = 0; j < kBlock; ++j) {
                if (j % kPair == 0)
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                        for (int i = 0; i < kPair; ++i)
                            lds_w[(nt * kPair + i) * kWave + lane] = w[j / kPair][nt][i];
                if constexpr (!SHARED)
#pragma unroll
                    for (int i = 0; i < XI; ++i) x_lds[i * kWave + lane] = x[j % kAhead][i];
                if (MODE == kF32Group32 && lane < kCols) lds_s[lane] = s[j];
                if constexpr (!SHARED)
                    if (j + kAhead < kBlock || more) load_x(x[j % kAhead], step + j + kAhead);
                if (more) {
                    load_step_scales(s[j], step + kBlock + j);
                    if (j % kPair == 0) load_codes(w[j / kPair], step + kBlock + j);
                }
                wave_lds_order();
                u32x4_t wl[kNT];
                float ws[kNT][4];
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt) {
                    wl[nt] = lds_w[nt * (kPair * kWave) + lr * 8 + ((j % kPair * 4 + q) ^ (lr & 7))];
                    const uint32_t* sw = reinterpret_cast<const uint32_t*>(lds_s + nt * 16 + lr);
                    if constexpr (MODE == kFolded) {
                        const uint32_t v = bytes32 ? sw[j] >> (8 * q) : sw[0] >> (8 * j);
                        ws[nt][0] = __uint_as_float((v & 0xFFu) << 23);
                    } else if constexpr (MODE == kF32Group128) {
                        ws[nt][0] = __uint_as_float(sw[j]);
                    } else {
                        const u32x4_t v = lds_s[nt * 16 + lr];
                        ws[nt][0] = __uint_as_float(v.x);
                        ws[nt][1] = __uint_as_float(v.y);
                        ws[nt][2] = __uint_as_float(v.z);
                        ws[nt][3] = __uint_as_float(v.w);
                    }
                }
                bf16x8_t wf[kNT][4];
                unpack_codes(wf, wl, ws);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const int m = mt * 16 + lr;
                    const u32x4_t* step_x = x_lds + (SHARED ? j * kStepX : 0);
                    u32x4_t xl[XV];
                    if constexpr (MODE == kF32Group32 && E4M3) {  // k = 32 i + 8 q of instruction i: half a chunk
                        u32x2_t c[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            c[i] = reinterpret_cast<const u32x2_t*>(
                                step_x + x_unit(MAXROWS, ROWS, kChunks, m, 2 * i + (q >> 1)))[q & 1];
                        xl[0] = u32x4(c[0].x, c[0].y, c[1].x, c[1].y);
                        xl[1] = u32x4(c[2].x, c[2].y, c[3].x, c[3].y);
                    } else {
#pragma unroll
                        for (int i = 0; i < XV; ++i)
                            xl[i] = step_x[x_unit(MAXROWS, ROWS, kChunks, m,
                                                  MODE == kF32Group32 ? 4 * i + q : XV * q + i)];
                    }
                    const float own = j == 0 ? xs[mt].x : j == 1 ? xs[mt].y : j == 2 ? xs[mt].z : xs[mt].w;
                    multiply(wf, ws, xl, own, acc[mt]);
                    // the next rows' (or step's) fragments would not fit the registers as well
                    __builtin_amdgcn_sched_barrier(0);
                }
                wave_lds_order();
            }
        }
    }
    // What is left, less than a block, straight into fragments: all of its loads first.  The last step may end inside
    // (K % 128 != 0).
    if constexpr (!TAIL) return;
    const int base = sh.first + kBlock * sh.blocks;
    int64_t frag_row[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) frag_row[mt] = x_row(mt * 16 + lr);
    u32x4_t w[kBlock][kNT], x[kBlock][MT][XV] = {};
    float ws[kBlock][kNT][4], xs[kBlock][MT] = {};
#pragma unroll
    for (int j = 0; j < kBlock; ++j) {
        const int step = base + j, k0 = step * kStep;
        if (step >= sh.last) break;
        const bool in = k0 + q * 32 < K;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            const int64_t n = row_e + min(sh.n0 + nt * 16 + lr, a.N - 1);
            w[j][nt] = u32x4(0, 0, 0, 0);
            if (in) w[j][nt] = *reinterpret_cast<const u32x4_t*>(a.codes + n * (K / 2) + k0 / 2 + q * 16);
            if constexpr (MODE == kFolded) {
                ws[j][nt][0] = 1.0f;
                if (in)
                    ws[j][nt][0] = __uint_as_float(
                        static_cast<uint32_t>(
                            static_cast<const uint8_t*>(a.sf)[n * (K / a.group) + (k0 + q * 32) / a.group])
                        << 23);
            } else if constexpr (MODE == kF32Group128) {
                ws[j][nt][0] = static_cast<const float*>(a.sf)[n * (K / 128) + step];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    ws[j][nt][i] =
                        k0 + i * 32 < K ? static_cast<const float*>(a.sf)[n * (K / 32) + 4 * step + i] : 0.0f;
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            if (frag_row[mt] < 0) continue;
            if constexpr (E4M3) {
                xs[j][mt] = a.x_sf[frag_row[mt] * (K / 128) + step];
                const uint8_t* p = static_cast<const uint8_t*>(a.x) + frag_row[mt] * K + k0;
                if constexpr (MODE == kF32Group32) {
                    u32x2_t c[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) c[i] = *reinterpret_cast<const u32x2_t*>(p + 32 * i + 8 * q);
                    x[j][mt][0] = u32x4(c[0].x, c[0].y, c[1].x, c[1].y);
                    x[j][mt][1] = u32x4(c[2].x, c[2].y, c[3].x, c[3].y);
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i) x[j][mt][i] = *reinterpret_cast<const u32x4_t*>(p + 32 * q + 16 * i);
                }
            } else {
                const uint16_t* p = static_cast<const uint16_t*>(a.x) + frag_row[mt] * K + k0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = MODE == kF32Group32 ? 32 * i + 8 * q : 32 * q + 8 * i;
                    if (k0 + k < K) x[j][mt][i] = *reinterpret_cast<const u32x4_t*>(p + k);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kBlock; ++j) {
        if (base + j >= sh.last) break;
        bf16x8_t wf[kNT][4];
        unpack_codes(wf, w[j], ws[j]);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) multiply(wf, ws[j], x[j][mt], xs[j][mt], acc[mt]);
    }
}

// A workgroup is blockDim / 64 waves.  SHARED: each has a tile of kCols output
// columns of its own; otherwise they split the k range of one tile.  MAXROWS:
// rows that one pass over the weights serves; an expert with more takes
// several, which the grid's z shares out.
template <bool E4M3, int MODE, int MAXROWS, bool SHARED, bool TAIL>
__global__ __launch_bounds__(kMaxThreads, 2) void expert_matvec_kernel(MatvecArgs a) {
    // the operand whose scale is per row of its own goes second: a lane's four
    // sums then share that row
    constexpr bool kXFirst = MODE != kFolded;
    constexpr int kLdsWave = lds_wave(SHARED, MAXROWS);
    extern __shared__ u32x4_t lds[];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int waves = blockDim.x / kWave;
    const int lr = lane & 15, q = lane >> 4;
    Share sh;
    if (!find_expert(a, blockIdx.y, lane, sh.e, sh.row0, sh.rows)) return;
    const int split = SHARED ? 1 : waves, part = SHARED ? 0 : wave;
    sh.n0 = (SHARED ? blockIdx.x * waves + wave : blockIdx.x) * kCols;  // may be past N: then nothing is written
    const int steps = (a.K + kStep - 1) / kStep;
    const int blocks = a.K / (kStep * kBlock);
    if (a.x_rows == 0) {
        sh.first = sh.blocks = sh.last = 0;
    } else {  // the last wave also takes what is left after the blocks
        sh.first = blocks * part / split * kBlock;
        sh.blocks = blocks * (part + 1) / split - blocks * part / split;
        sh.last = part == split - 1 ? steps : sh.first + kBlock * sh.blocks;
    }

    // Leaves the wave's sums in LDS, adds the shares of the tile's waves in order and writes the rows.
    u32x4_t* mine = lds + wave * kLdsWave;
    u32x4_t* x_lds = SHARED ? lds + waves * kLdsWave : mine + kLdsCodes + kLdsScales;
    const float* tile = reinterpret_cast<const float*>(lds + (wave - part) * kLdsWave);
    auto run = [&](auto rows_const, int m0) __attribute__((always_inline)) {
        constexpr int ROWS = decltype(rows_const)::value;
        constexpr int MT = (ROWS + 15) / 16;
        f32x4_t acc[MT][kNT] = {};
        multiply_rows<E4M3, MODE, MAXROWS, ROWS, SHARED, TAIL>(a, sh, m0, lane, wave, mine, x_lds, acc);
        wave_lds_order();
        float* sums = reinterpret_cast<float*>(mine);
        // the first operand's rows run along a lane's sums, the second's along the lanes
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sums[(mt * 16 + (kXFirst ? q * 4 + i : lr)) * kPitch + nt * 16 + (kXFirst ? lr : q * 4 + i)] =
                        acc[mt][nt][i];
        if constexpr (SHARED)
            wave_lds_order();
        else
            __syncthreads();
        for (int i = part * kWave + lane; i < ROWS * kCols; i += split * kWave) {
            const int m = i / kCols, n = i % kCols;
            if (m >= sh.rows - m0 || sh.n0 + n >= a.N) continue;
            float v = 0.0f;
            for (int w = 0; w < split; ++w) v += tile[w * (kLdsWave * 4) + m * kPitch + n];
            const int64_t r = sh.row0 + m0 + m;
            if (a.row_token != nullptr) {
                const int t = a.row_token[r];
                if (t < 0 || t >= a.x_rows) v = 0.0f;
            }
            a.out[r * a.N + sh.n0 + n] = bf16_bits(v);
        }
    };
    const int64_t first = int64_t{blockIdx.z} * MAXROWS, stride = int64_t{gridDim.z} * MAXROWS;
    for (int64_t m = first; m < sh.rows; m += stride) {
        if (m > first) __syncthreads();  // the sums and operands in LDS have been read
        const int m0 = static_cast<int>(m);
        const int rows = sh.rows - m0;
        if (!E4M3 && MAXROWS <= 8 && rows <= 4)
            run(std::integral_constant<int, 4>{}, m0);
        else if (MAXROWS <= 8 || rows <= 8)
            run(std::integral_constant<int, 8>{}, m0);
        else if (MAXROWS <= 16 || rows <= 16)
            run(std::integral_constant<int, MAXROWS < 16 ? MAXROWS : 16>{}, m0);
        else
            run(std::integral_constant<int, MAXROWS>{}, m0);
    }
}

template <bool E4M3, int MODE, int MAXROWS, bool TAIL>
hipError_t launch_rows(const MatvecArgs& a, int64_t experts, hipStream_t stream) {
    const int64_t tiles = (a.N + kCols - 1) / kCols;
    const int blocks = a.K / (kStep * kBlock);
    // A wave for each tile where that fills the eight places for waves of every compute unit (their registers allow
    // two a SIMD); else the waves of a workgroup split k, as far as there is a block of steps for each, until all
    // places are taken.  One token's eight experts, 1024 tiles: 25.1 us split in two, 28.5 us in four (two rounds).
    // Places still free take an expert's passes side by side (72 rows of one matrix, 1568 -> 4096: 9.3 us, 27.3 us one
    // after another); an expert with fewer passes leaves its spare workgroups at once.
    auto passes = [&](int64_t waves) {
        const int64_t most = (a.num_rows + MAXROWS - 1) / MAXROWS, free = kWavePlaces / waves;
        return static_cast<unsigned>(free < 1 ? 1 : free < most ? free : most);
    };
    constexpr bool kManyTiles = MAXROWS > 16;  // the caller's rule
    if (kManyTiles || tiles * experts >= kWavePlaces || blocks < 2) {
        const dim3 grid(static_cast<unsigned>((tiles + kSharedWaves - 1) / kSharedWaves),
                        static_cast<unsigned>(experts), passes(tiles * experts));
        hipLaunchKernelGGL((expert_matvec_kernel<E4M3, MODE, MAXROWS, true, TAIL>), grid, dim3(kSharedWaves * kWave),
                           lds_bytes(true, MAXROWS, kSharedWaves), stream, a);
    } else if constexpr (!kManyTiles) {
        int split = 2;
        while (split < kMaxSplit && tiles * experts * split < kWavePlaces && blocks >= 2 * split) split *= 2;
        hipLaunchKernelGGL((expert_matvec_kernel<E4M3, MODE, MAXROWS, false, TAIL>),
                           dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(experts),
                                passes(tiles * experts * split)),
                           dim3(split * kWave), lds_bytes(false, MAXROWS, split), stream, a);
    }
    return hipGetLastError();
}

// The rows that a pass over the weights serves.  No expert has more rows than
// there are, and of many experts few have many times the average; fewer rows
// take less LDS and fewer registers (128 rows over 32 experts: 83 us with 16,
// 95 us with 32), but an expert with more reads its weights again (512 rows
// over 32: 77 us with 16, 65 us with 32), unless there are places for its
// passes side by side (200 rows of one matrix, 7168 -> 512: 12.1 us with 16,
// 18.0 us with 32).  k that ends inside a block takes 16:
// the code for its last steps costs the registers of a wave in four (65
// against 69 us without it).  So do fp32 scales of 32 channels, whose sums of
// 32 rows would not fit.
template <bool E4M3, int MODE>
hipError_t launch_matvec(const MatvecArgs& a, hipStream_t stream) {
    const int64_t experts = a.E < a.num_rows ? a.E : a.num_rows;
    if (a.K % (kStep * kBlock) != 0) return launch_rows<E4M3, MODE, 16, true>(a, experts, stream);
    if (a.num_rows <= 8 || a.num_rows <= 2 * static_cast<int64_t>(a.E))
        return launch_rows<E4M3, MODE, 8, false>(a, experts, stream);
    if constexpr (MODE != kF32Group32)
        if (a.num_rows > 16 && a.num_rows > 8 * static_cast<int64_t>(a.E) &&
            (a.N + kCols - 1) / kCols * experts >= kWavePlaces)
            return launch_rows<E4M3, MODE, 32, false>(a, experts, stream);
    return launch_rows<E4M3, MODE, 16, false>(a, experts, stream);
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
    if (inner > MOE_MATVEC_MAX_WIDTH || out_width > MOE_MATVEC_MAX_WIDTH) return MOE_ERR_UNSUPPORTED;
    if (num_rows == 0) return MOE_OK;  // an empty row_token may be null: x_rows is then anything
    if (row_token == nullptr && x_rows != num_rows) return MOE_ERR_INVALID_ARGUMENT;
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
