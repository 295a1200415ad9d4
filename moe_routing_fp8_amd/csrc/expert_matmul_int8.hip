// The experts' products in 8-bit integers: rows grouped by expert times that
// expert's matrix, with one scale a row and one an output channel,
//   out[r, n] = (fp32(sum_k x[r', k] * w[e, n, k]) * x_sf[r']) * w_sf[e, n].
// The sums are whole numbers in 32 bits, exact in any order.
//
// One workgroup computes a tile of BM rows of one expert and BN channels.  The
// x rows and w rows of BK bytes of k go from memory to LDS without passing
// registers (16 bytes a lane, 1024 consecutive LDS bytes a wave), STAGES steps
// of k in flight; the matrix instruction takes 16 rows of each with 64 bytes
// of k from there.
#include <hip/hip_runtime.h>

#include "api_common.hpp"
#include "device_utils.hpp"
#include "kernels.hpp"
#include "math_device.hpp"
#include "moe_fp8.h"

namespace moe {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr int kXcds = 8;        // dies, each with an L2 of its own; workgroups go to them in turn
constexpr int kMinRows = 16, kMinChannels = 64;  // of the smallest tile
constexpr int kGroupTiles = 8;  // row tiles of an expert that share its w tiles side by side

struct MatmulArgs {
    const uint8_t* x;
    const float* x_sf;
    int64_t x_rows;
    const int32_t* row_token;
    int64_t num_rows;
    int K, N, E;
    const int32_t* expert_offsets;
    const uint8_t* w;
    const float* w_sf;
    void* out;
    int out_f32, vec4;  // vec4: four channels are stored at once
    int n_tiles;
};

__device__ const uint4 kZeroChunk = {0, 0, 0, 0};

// Where the 16-byte chunk c of row r lies in its row of a stage: rows that a
// matrix instruction's lanes read together have it in different banks.
template <int BK>
__device__ __forceinline__ int swizzle(int r, int c) {
    return c ^ (r & (BK / 16 - 1));
}

template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ int row_tiles(const MatmulArgs& a, int e, int bm, int64_t& begin, int64_t& count) {
    if (a.expert_offsets == nullptr) {
        begin = 0;
        count = a.num_rows;
    } else {
        int64_t b = a.expert_offsets[e], c = a.expert_offsets[e + 1];
        b = b < 0 ? 0 : b > a.num_rows ? a.num_rows : b;
        c = c < b ? b : c > a.num_rows ? a.num_rows : c;
        begin = b;
        count = c - b;
    }
    return static_cast<int>((count + bm - 1) / bm);
}

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
    for (int o = 1; o < kWave; o *= 2) {
        const int u = __shfl_up(v, o);
        if (lane >= o) v += u;
    }
    return v;
}

struct Tile {
    int expert;
    int64_t row;   // first row
    int rows;      // rows of the tile
    int channel;   // first channel
};

// The workgroup's tile.  Tiles are numbered expert by expert; within an
// expert, kGroupTiles row tiles of one channel tile after another, so that
// tiles that run together share rows of w and x.  Each die takes a run of
// consecutive tiles.  Every wave finds the same tile by itself.
template <int BM, int BN>
__device__ __forceinline__ bool find_tile(const MatmulArgs& a, Tile& t) {
    const int lane = threadIdx.x % kWave;
    const int chunk = (a.E + kWave - 1) / kWave;
    int64_t begin, count;
    int mine = 0;
    for (int i = 0; i < chunk; ++i) {
        const int e = lane * chunk + i;
        if (e < a.E) mine += row_tiles(a, e, BM, begin, count);
    }
    int incl = wave_scan(mine, lane);
    const int total = __builtin_amdgcn_readlane(incl, kWave - 1);
    const int64_t tiles = static_cast<int64_t>(total) * a.n_tiles;
    const int64_t per = (tiles + kXcds - 1) / kXcds;
    const int64_t turn = blockIdx.x / kXcds;
    const int64_t id = (blockIdx.x % kXcds) * per + turn;
    if (turn >= per || id >= tiles) return false;
    const int slot = static_cast<int>(id / a.n_tiles);
    int owner = __popcll(__ballot(incl <= slot));
    int before = __builtin_amdgcn_readlane(incl - mine, owner);
    int e = owner;
    if (chunk > 1) {
        const int first = owner * chunk;
        mine = lane < chunk && first + lane < a.E ? row_tiles(a, first + lane, BM, begin, count) : 0;
        incl = before + wave_scan(mine, lane);
        owner = __popcll(__ballot(incl <= slot));
        before = __builtin_amdgcn_readlane(incl - mine, owner);
        e = first + owner;
    }
    const int m_tiles = row_tiles(a, e, BM, begin, count);
    const int64_t local = id - static_cast<int64_t>(before) * a.n_tiles;
    const int64_t per_group = static_cast<int64_t>(kGroupTiles) * a.n_tiles;
    const int g = static_cast<int>(local / per_group);
    const int in_group = static_cast<int>(local - g * per_group);
    const int width = min(kGroupTiles, m_tiles - g * kGroupTiles);
    const int n = in_group / width, m = g * kGroupTiles + in_group % width;
    t.expert = e;
    t.row = begin + static_cast<int64_t>(m) * BM;
    t.rows = static_cast<int>(min<int64_t>(BM, count - static_cast<int64_t>(m) * BM));
    t.channel = n * BN;
    return true;
}

// Sixteen bytes at any address; past `left` bytes zeros.
struct __attribute__((packed, aligned(1))) Unaligned16 {
    u32x4_t v;
};
__device__ __forceinline__ u32x4_t load_any(const uint8_t* p, int left) {
    if (left >= 16) return reinterpret_cast<const Unaligned16*>(p)->v;
    u32x4_t v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 15; ++i)
        if (i < left) v[i / 4] |= static_cast<uint32_t>(p[i]) << (8 * (i % 4));
    return v;
}

// WM x WN waves, each BM / WM rows and BN / WN channels.  DIRECT: rows are 16-byte
// aligned and go straight to LDS; else through registers, one step ahead.
template <int BM, int BN, int BK, int STAGES, int WM, int WN, bool DIRECT>
__global__ __launch_bounds__(WM* WN* kWave) void expert_matmul_int8_kernel(MatmulArgs a) {
    constexpr int kWaves = WM * WN;
    constexpr int kChunks = BK / 16;                     // of a row
    constexpr int kRowsPerLoad = kWave / kChunks;        // rows that a wave's load covers
    constexpr int kLoads = (BM + BN) / kRowsPerLoad / kWaves;  // of a wave and step
    constexpr int kStage = (BM + BN) * BK;
    constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
    static_assert((BM + BN) % (kRowsPerLoad * kWaves) == 0 && BM % (16 * WM) == 0 && BN % (16 * WN) == 0, "tile");
    static_assert(BM % kRowsPerLoad == 0, "a load lies in x or in w");
    static_assert(DIRECT || STAGES == 2, "two stages through registers");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[STAGES][kStage];

    Tile t;
    if (!find_tile<BM, BN>(a, t)) return;
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);

    // this lane's chunk of each of its wave's loads
    const uint8_t* src[kLoads];
    int at[kLoads];  // its k within a step
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
        const int r = (wave + j * kWaves) * kRowsPerLoad + lane / kChunks;  // row of the stage
        const int c = swizzle<BK>(r, lane % kChunks);
        int64_t row;
        if (r < BM) {  // x: rows past the tile's read its last one again and are not stored
            row = t.row + min(r, t.rows - 1);
            if (a.row_token != nullptr) row = a.row_token[row];
            if (row < 0 || row >= a.x_rows) row = 0;  // stored as zeros
            src[j] = a.x + row * a.K;
        } else {
            row = static_cast<int64_t>(t.expert) * a.N + min(t.channel + r - BM, a.N - 1);
            src[j] = a.w + row * a.K;
        }
        at[j] = c * 16;
        src[j] += at[j];
    }
    const int steps = (a.K + BK - 1) / BK;
    auto issue = [&](int step, int stage) {
        const bool last = (step + 1) * BK > a.K;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const uint8_t* p = src[j] + static_cast<int64_t>(step) * BK;
            if (last && step * BK + at[j] >= a.K) p = reinterpret_cast<const uint8_t*>(&kZeroChunk);
            __builtin_amdgcn_global_load_lds(
                reinterpret_cast<const __attribute__((address_space(1))) void*>(reinterpret_cast<uintptr_t>(p)),
                (__attribute__((address_space(3))) void*)(lds[stage] + (wave + j * kWaves) * 1024), 16, 0, 0);
        }
    };
    u32x4_t held[DIRECT ? 1 : kLoads];
    auto fetch = [&](int step) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            held[j] = load_any(src[j] + static_cast<int64_t>(step) * BK, a.K - step * BK - at[j]);
    };

    const int wm = wave / WN, wn = wave % WN;
    const int x_row = wm * (BM / WM) + lane % 16, w_row = BM + wn * (BN / WN) + lane % 16;
    const bool busy = wm * (BM / WM) < t.rows;  // a wave whose rows are all past the tile's has nothing to sum
    i32x4_t acc[TM][TN];
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int n = 0; n < TN; ++n) acc[m][n] = i32x4_t{0, 0, 0, 0};
    auto multiply = [&](int stage) {
        const uint8_t* s = lds[stage];
#pragma unroll
        for (int k = 0; k < BK / 64; ++k) {
            i32x4_t xf[TM], wf[TN];
            const int c = k * 4 + lane / 16;
#pragma unroll
            for (int n = 0; n < TN; ++n)
                wf[n] = *reinterpret_cast<const i32x4_t*>(s + (w_row + n * 16) * BK + swizzle<BK>(w_row, c) * 16);
#pragma unroll
            for (int m = 0; m < TM; ++m)
                xf[m] = *reinterpret_cast<const i32x4_t*>(s + (x_row + m * 16) * BK + swizzle<BK>(x_row, c) * 16);
#pragma unroll
            for (int m = 0; m < TM; ++m)
#pragma unroll
                for (int n = 0; n < TN; ++n)
                    acc[m][n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[n], xf[m], acc[m][n], 0, 0, 0);
        }
    };

    if constexpr (DIRECT) {
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i)
            if (i < steps) issue(i, i);
        int stage = 0;
        for (int i = 0; i < steps; ++i) {
            if (i + STAGES - 2 < steps) wait_loads<(STAGES - 2) * kLoads>();
            else
                wait_loads<0>();
            // every wave's part of this step is there, and every wave is done with the step before it
            __builtin_amdgcn_s_barrier();
            if (i + STAGES - 1 < steps) issue(i + STAGES - 1, stage == 0 ? STAGES - 1 : stage - 1);
            if (busy) multiply(stage);
            stage = stage + 1 == STAGES ? 0 : stage + 1;
        }
    } else {
        fetch(0);
        for (int i = 0; i < steps; ++i) {
            uint8_t* s = lds[i & 1];
#pragma unroll
            for (int j = 0; j < kLoads; ++j)
                *reinterpret_cast<u32x4_t*>(s + (wave + j * kWaves) * 1024 + lane * 16) = held[j];
            if (i + 1 < steps) fetch(i + 1);
            __syncthreads();
            if (busy) multiply(i & 1);
        }
    }
    if (!busy) return;

    // lane l holds four channels, 4 (l / 16) on, of row l % 16 of each 16 x 16 product
#pragma unroll
    for (int m = 0; m < TM; ++m) {
        const int r = wm * (BM / WM) + m * 16 + lane % 16;
        if (r >= t.rows) continue;
        const int64_t row = t.row + r;
        int64_t from = row;
        if (a.row_token != nullptr) from = a.row_token[row];
        const bool known = from >= 0 && from < a.x_rows;
        const float xs = known ? a.x_sf[from] : 0.0f;
#pragma unroll
        for (int n = 0; n < TN; ++n) {
            const int ch = t.channel + wn * (BN / WN) + n * 16 + lane / 16 * 4;
            const float* ws = a.w_sf + static_cast<int64_t>(t.expert) * a.N + ch;
            const int64_t o = row * a.N + ch;
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = known && ch + i < a.N ? static_cast<float>(acc[m][n][i]) * xs * ws[i] : 0.0f;
            if (a.vec4) {
                if (ch >= a.N) continue;
                if (a.out_f32) F32::store<4>(a.out, o, v);
                else
                    Bf16::store<4>(a.out, o, v);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (ch + i >= a.N) continue;
                    float one[1] = {v[i]};
                    if (a.out_f32) F32::store<1>(a.out, o + i, one);
                    else
                        Bf16::store<1>(a.out, o + i, one);
                }
            }
        }
    }
}

template <int BM, int BN, int BK, int STAGES, int WM, int WN, bool DIRECT>
hipError_t launch_tiles(MatmulArgs a, hipStream_t stream) {
    a.n_tiles = (a.N + BN - 1) / BN;
    // an expert adds at most one partly filled tile; the kernel counts the tiles that there are
    const int64_t experts = a.E < a.num_rows ? a.E : a.num_rows;
    int64_t slots = a.num_rows / BM + experts;
    if (slots > a.num_rows) slots = a.num_rows;
    const int64_t blocks = (slots * a.n_tiles + kXcds - 1) / kXcds * kXcds;
    hipLaunchKernelGGL((expert_matmul_int8_kernel<BM, BN, BK, STAGES, WM, WN, DIRECT>),
                       dim3(static_cast<unsigned>(blocks)), dim3(WM * WN * kWave), 0, stream, a);
    return hipGetLastError();
}

template <bool DIRECT>
hipError_t launch_matmul(const MatmulArgs& a, hipStream_t stream) {
    const int64_t mean = a.num_rows / a.E;
    if constexpr (!DIRECT) {
        if (mean <= 16) return launch_tiles<16, 64, 256, 2, 1, 4, false>(a, stream);
        return launch_tiles<64, 64, 128, 2, 2, 2, false>(a, stream);
    } else {
        if (mean <= 16) return launch_tiles<16, 64, 256, 4, 1, 4, true>(a, stream);
        if (mean <= 64) return launch_tiles<64, 64, 128, 4, 1, 4, true>(a, stream);
        return launch_tiles<256, 256, 128, 2, 2, 4, true>(a, stream);
    }
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_expert_matmul_int8(const int8_t* x, const float* x_sf, int64_t x_rows,
                                             const int32_t* row_token, int64_t num_rows, int32_t inner,
                                             int32_t out_width, int32_t num_experts, const int32_t* expert_offsets,
                                             const int8_t* w, const float* w_sf, int32_t out_dtype, void* out,
                                             hipStream_t stream) {
    using namespace moe;
    if (num_rows < 0 || num_rows > INT32_MAX || x_rows < 0 || x_rows > INT32_MAX) return MOE_ERR_INVALID_ARGUMENT;
    if (out_dtype != MOE_DTYPE_BF16 && out_dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARGUMENT;
    if (num_experts < 1 || num_experts > kMaxExperts || out_width < 1 || inner < 1) return MOE_ERR_INVALID_ARGUMENT;
    if (expert_offsets == nullptr && num_experts != 1) return MOE_ERR_INVALID_ARGUMENT;
    // beyond it a sum of products of codes could leave 32 bits
    if (inner > MOE_MATMUL_INT8_MAX_INNER || out_width > MOE_MATVEC_MAX_WIDTH) return MOE_ERR_UNSUPPORTED;
    if ((num_rows / kMinRows + num_experts) * ((out_width + kMinChannels - 1) / kMinChannels) >= MOE_MATMUL_INT8_MAX_TILES)
        return MOE_ERR_UNSUPPORTED;
    if (num_rows == 0) return MOE_OK;  // an empty row_token may be null: x_rows is then anything
    if (row_token == nullptr && x_rows != num_rows) return MOE_ERR_INVALID_ARGUMENT;
    if (w == nullptr || w_sf == nullptr || out == nullptr) return MOE_ERR_INVALID_ARGUMENT;
    if (x_rows > 0 && (x == nullptr || x_sf == nullptr)) return MOE_ERR_INVALID_ARGUMENT;
    const uintptr_t size = out_dtype == MOE_DTYPE_BF16 ? 2 : 4;
    if (!aligned(x_sf, 4) || !aligned(w_sf, 4) || !aligned(row_token, 4) || !aligned(expert_offsets, 4) ||
        !aligned(out, size))
        return MOE_ERR_INVALID_ARGUMENT;
    MatmulArgs a{};
    // without x rows every row is one of zeros; what is read in its place is w
    a.x = reinterpret_cast<const uint8_t*>(x_rows > 0 ? x : w);
    a.x_sf = x_sf;
    a.x_rows = x_rows;
    a.row_token = row_token;
    a.num_rows = num_rows;
    a.K = inner;
    a.N = out_width;
    a.E = num_experts;
    a.expert_offsets = expert_offsets;
    a.w = reinterpret_cast<const uint8_t*>(w);
    a.w_sf = w_sf;
    a.out = out;
    a.out_f32 = out_dtype == MOE_DTYPE_F32;
    a.vec4 = out_width % 4 == 0 && aligned(out, 4 * size);
    const bool direct = inner % 16 == 0 && aligned(a.x, 16) && aligned(w, 16);
    return hip_status(direct ? launch_matmul<true>(a, stream) : launch_matmul<false>(a, stream));
}
