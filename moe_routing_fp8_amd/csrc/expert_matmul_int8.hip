// The experts' products in 8-bit integers: rows grouped by expert times that
// expert's matrix, with one scale a row and one an output channel,
//   out[r, n] = (fp32(sum_k x[r', k] * w[e, n, k]) * x_sf[r']) * w_sf[e, n].
// The sums are whole numbers in 32 bits, exact in any order.
//
// A workgroup computes tiles of up to BM rows of one expert by BN channels.  The
// x rows and w rows of BK bytes of k go from memory to LDS without passing
// registers (16 bytes a lane, 1024 consecutive LDS bytes a wave), one or two steps of
// k ahead; the matrix instruction takes 16 rows of each with 64 bytes of k from
// there.
//
// 32 experts, 7168 -> 4096, bf16 out (back to back, rotating inputs):
//   128 rows             96 to 108 us    bytes of the weights: 20 experts have rows, 5.5 to 6.2 TB/s
//   4096 rows by token   246 to 288 us   loads into LDS, waits at the tiles' ends, 2.1 to 3.0 tiles a compute unit
//   16384 rows by token  587 to 621 us   1.55 to 1.64 POPS: the same, unequal experts
// One matrix, 16384 rows, 8192 -> 8192: 943 to 985 us, 2.2 to 2.3 POPS.  Multiplying
// alone takes 74% of that, loading alone 79%; random codes in registers reach 4.1 POPS.
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
    int out_f32, vec;  // vec: channels that lie side by side are stored at once
    int n_tiles;
};

__device__ const uint4 kZeroChunk = {0, 0, 0, 0};

// The tile's place: BM rows of an expert, BN channels.
struct Tile {
    int expert;
    int rows;     // rows of the tile
    int channel;  // first channel
    int64_t row;  // first row
};

// The rows of expert e, whatever the offsets hold within [0, num_rows].
__device__ __forceinline__ void expert_rows(const MatmulArgs& a, int e, int& begin, int& count) {
    begin = 0;
    count = static_cast<int>(a.num_rows);
    if (a.expert_offsets == nullptr) return;
    const int most = static_cast<int>(a.num_rows);
    begin = min(max(a.expert_offsets[e], 0), most);
    count = min(max(a.expert_offsets[e + 1], begin), most) - begin;
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

// Numbers the tiles expert by expert: an expert's rows are shared evenly, in
// whole blocks of 16, by as few tiles of up to BM rows as hold them.  Within an
// expert, kGroupTiles row tiles of one channel tile after another, so that tiles
// that run together share rows of w and x.  Every wave holds the sums of each
// lane's experts, and finds the same tiles by itself.
template <int BM, int BN>
struct Tiles {
    const MatmulArgs& a;
    int lane, chunk;        // experts a lane
    int begin, count;       // the lane's expert, if chunk is 1
    int mine, weight;       // row tiles of the lane's experts, and what they cost
    int tiles_to, cost_to;  // the same up to and with this lane's
    int total, cost;        // of all experts

    static __device__ __forceinline__ int row_tiles(int count) { return (count + BM - 1) / BM; }
    static __device__ __forceinline__ int tile_rows(int count, int tiles) {
        return tiles == 0 ? 0 : ((count + tiles - 1) / tiles + 15) / 16 * 16;
    }
    // A tile's time, in sixteenths of what its rows add: its loads take about as long as half of them.
    static __device__ __forceinline__ int tile_cost(int rows) { return (rows + BM / 2) / 16 + 1; }

    __device__ __forceinline__ explicit Tiles(const MatmulArgs& args)
        : a(args), lane(threadIdx.x % kWave), chunk((args.E + kWave - 1) / kWave), begin(0), count(0), mine(0),
          weight(0) {
        for (int i = 0; i < chunk; ++i) {
            const int e = lane * chunk + i;
            if (e >= a.E) continue;
            expert_rows(a, e, begin, count);
            const int n = row_tiles(count);
            mine += n;
            weight += n * tile_cost(tile_rows(count, n));
        }
        // Offsets that decrease can give many experts the same rows.  Up to 2^30 of cost they
        // are computed all the same; beyond that, where the sums would leave 32 bits (a lane's
        // own, of at most 16 experts of 2^28 rows, does not), there are no tiles.
        if (__builtin_amdgcn_readlane(wave_scan(weight / kWave, lane), kWave - 1) >= (1 << 30) / kWave)
            mine = weight = 0;
        tiles_to = wave_scan(mine, lane);
        cost_to = wave_scan(weight, lane);
        total = __builtin_amdgcn_readlane(tiles_to, kWave - 1);
        cost = __builtin_amdgcn_readlane(cost_to, kWave - 1);
    }

    // An expert, and the row tiles and their cost before it.
    struct Found {
        int expert, begin, count, tiles_before, cost_before;
    };
    // The expert at which the sum picked by `value` passes `at`, 0 <= at < its total.
    template <typename V>
    __device__ __forceinline__ Found search(int at, V value) const {
        const int to = value(tiles_to, cost_to);
        int owner = __popcll(__ballot(to <= at));
        Found f;
        f.expert = owner;
        f.tiles_before = __builtin_amdgcn_readlane(tiles_to - mine, owner);
        f.cost_before = __builtin_amdgcn_readlane(cost_to - weight, owner);
        int first = begin, rows = count;
        if (chunk > 1) {
            const int e = owner * chunk + lane;
            int n = 0, c = 0;
            first = rows = 0;
            if (lane < chunk && e < a.E) {
                expert_rows(a, e, first, rows);
                n = row_tiles(rows);
                c = n * tile_cost(tile_rows(rows, n));
            }
            const int n_to = f.tiles_before + wave_scan(n, lane), c_to = f.cost_before + wave_scan(c, lane);
            const int in = __popcll(__ballot(value(n_to, c_to) <= at));
            f.expert = owner * chunk + in;
            f.tiles_before = __builtin_amdgcn_readlane(n_to - n, in);
            f.cost_before = __builtin_amdgcn_readlane(c_to - c, in);
            owner = in;
        }
        f.begin = __builtin_amdgcn_readlane(first, owner);
        f.count = __builtin_amdgcn_readlane(rows, owner);
        return f;
    }

    // The first tile of part `part` of `parts` of about the same cost.
    __device__ __forceinline__ int64_t start_of(int part, int parts) const {
        if (part >= parts || total == 0) return static_cast<int64_t>(total) * a.n_tiles;
        const int64_t target = static_cast<int64_t>(cost) * a.n_tiles * part / parts;
        const Found f = search(static_cast<int>(target / a.n_tiles), [](int, int c) { return c; });
        const int64_t into = target - static_cast<int64_t>(f.cost_before) * a.n_tiles;
        return static_cast<int64_t>(f.tiles_before) * a.n_tiles +
               into / tile_cost(tile_rows(f.count, row_tiles(f.count)));
    }

    // Tile number id, 0 <= id < total * n_tiles.
    __device__ __forceinline__ Tile find(int64_t id) const {
        const Found f = search(static_cast<int>(id / a.n_tiles), [](int n, int) { return n; });
        const int m_tiles = row_tiles(f.count), rows = tile_rows(f.count, m_tiles);
        const int64_t local = id - static_cast<int64_t>(f.tiles_before) * a.n_tiles;
        const int64_t per_group = static_cast<int64_t>(kGroupTiles) * a.n_tiles;
        const int g = static_cast<int>(local / per_group);
        const int in_group = static_cast<int>(local - g * per_group);
        const int width = min(kGroupTiles, m_tiles - g * kGroupTiles);
        const int n = in_group / width, m = g * kGroupTiles + in_group % width;
        Tile t;
        t.expert = f.expert;
        t.rows = min(rows, f.count - m * rows);
        t.channel = n * BN;
        t.row = static_cast<int64_t>(f.begin) + static_cast<int64_t>(m) * rows;
        return t;
    }
};

// How a tile's products lie over the waves and lanes, and its rows in LDS.
//
// A wave multiplies TM x TN blocks of 16 rows by 16 channels.  Its row blocks
// are WM apart, so that a tile that is not full leaves all waves an equal share.
// Lane l holds, of each block, row l % 16 and four channels, those of block
// 2 j + 1 next to those of block 2 j: eight channels in a row, 64 bytes of four
// lanes, are stored together.
//
// LDS holds the BM rows of x and the BN rows of w, BK bytes each.  The 16-byte
// chunk c of a row lies at c ^ swizzle(row): eight or sixteen consecutive lanes,
// which read together, have it in different banks.
template <int BM, int BN, int BK, int WM, int WN>
struct Layout {
    static constexpr int kWaves = WM * WN;
    static constexpr int kChunks = BK / 16;
    static constexpr int kRowsPerLoad = kWave / kChunks;  // rows that a wave's 1024-byte load covers
    static constexpr int kXLoads = BM / kRowsPerLoad, kWLoads = BN / kRowsPerLoad;  // of a step, all waves together
    static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
    static constexpr bool kPairs = TN % 2 == 0;
    static_assert(BM % kRowsPerLoad == 0 && BN % (kRowsPerLoad * kWaves) == 0 && BM % (16 * WM) == 0 &&
                      BN % (16 * WN) == 0, "tile");
    typedef i32x4_t Sums[TM][TN];

    static __device__ __forceinline__ int x_swizzle(int r) { return r & (kChunks - 1); }
    static __device__ __forceinline__ int w_swizzle(int r) {
        return (kPairs ? (r & 3) | ((r >> 3) & 3) << 2 : r) & (kChunks - 1);
    }
    // channel of a wave's block n that line i (0 to 15) of the instruction has
    static __device__ __forceinline__ int channel(int n, int i) {
        return kPairs ? n / 2 * 32 + i / 4 * 8 + n % 2 * 4 + i % 4 : n * 16 + i;
    }

    // Adds the products of one step for the wave's first `used` row blocks.  Each
    // block's rows of x are read two blocks before they are multiplied, the next
    // 64 bytes of w along with them; the scheduler, left alone, reads them just
    // before (32 experts, 16384 rows: 612 against 596 us).
    static __device__ __forceinline__ void multiply(const uint8_t* x, const uint8_t* w, int used, int wm, int wn,
                                                    int lane, Sums& acc) {
        constexpr int U = BK / 64, kAhead = 2, kHeld = kAhead + 1;
        const int line = lane % 16;
        const int x_row = wm * 16 + line, w_row = wn * (BN / WN) + channel(0, line);
        auto read_x = [&](int i) {
            const int c = (i / TM * 4 + lane / 16) ^ x_swizzle(x_row);  // all the wave's rows of a line have one swizzle
            return *reinterpret_cast<const i32x4_t*>(x + (x_row + i % TM * WM * 16) * BK + c * 16);
        };
        auto read_w = [&](int k, int n) {
            const int row = w_row + channel(n, 0), c = (k * 4 + lane / 16) ^ w_swizzle(row);
            return *reinterpret_cast<const i32x4_t*>(w + row * BK + c * 16);
        };
        i32x4_t xf[kHeld], wf[2][TN];
#pragma unroll
        for (int n = 0; n < TN; ++n) wf[0][n] = read_w(0, n);
#pragma unroll
        for (int i = 0; i < kAhead && i < U * TM; ++i) xf[i] = read_x(i);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < U * TM; ++i) {
            const int k = i / TM, m = i % TM;
            if (i + kAhead < U * TM) xf[(i + kAhead) % kHeld] = read_x(i + kAhead);
#pragma unroll
            for (int n = 0; n < TN; ++n)
                if (k + 1 < U && n * TM / TN == m) wf[(k + 1) % 2][n] = read_w(k + 1, n);
            if (m < used) {
#pragma unroll
                for (int n = 0; n < TN; ++n)
                    acc[m][n] =
                        __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[k % 2][n], xf[i % kHeld], acc[m][n], 0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // The row blocks of wave row wm that a tile of `rows` rows reaches.
    static __device__ __forceinline__ int used_blocks(int rows, int wm) {
        return max((rows + 15) / 16 - wm + WM - 1, 0) / WM;
    }

    // Writes the wave's results.  xs(r) gives a row's scale and whether it has
    // one, ws(c) a channel's.
    template <typename XS, typename WS>
    static __device__ __forceinline__ void store(const MatmulArgs& a, const Tile& t, int wm, int wn, int lane,
                                                 const Sums& acc, XS xs, WS ws) {
        constexpr int V = kPairs ? 8 : 4;  // channels that lie side by side
        const int c0 = wn * (BN / WN) + lane / 16 * V;
#pragma unroll
        for (int n = 0; n < TN; n += V / 4) {
            const int c = c0 + channel(n, 0);
            float scale[V];
#pragma unroll
            for (int i = 0; i < V; ++i) scale[i] = ws(c + i);
#pragma unroll
            for (int m = 0; m < TM; ++m) {
                const int r = (m * WM + wm) * 16 + lane % 16;
                if (r >= t.rows || t.channel + c >= a.N) continue;
                bool known;
                const float x_scale = xs(r, known);
                float v[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    v[i] = static_cast<float>(acc[m][n + i / 4][i % 4]) * x_scale * scale[i];
                    if (!known) v[i] = 0.0f;
                }
                const int64_t o = (t.row + r) * a.N + t.channel + c;
                if (a.vec) {
                    if (a.out_f32) F32::store<V>(a.out, o, v);
                    else
                        Bf16::store<V>(a.out, o, v);
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        if (t.channel + c + i >= a.N) continue;
                        const float one[1] = {v[i]};
                        if (a.out_f32) F32::store<1>(a.out, o + i, one);
                        else
                            Bf16::store<1>(a.out, o + i, one);
                    }
                }
            }
        }
    }
};

template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// 16 (4) bytes a lane from memory to consecutive LDS addresses, past the registers.
// The builtin for this makes the compiler wait for all of them before the next
// read of LDS (a large matrix: 1230 against 1010 us); here wait_loads and the
// barrier behind it order them.  No register is written, so there is no output
// that the compiler could take as ready; m0's write needs one wait state.
// The LDS address, one for the wave, is that of a __shared__ array plus an offset.
#define MOE_LDS_ADDRESS(array) \
    static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) void*)(array)))

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // that m0 is named as overwritten
__device__ __forceinline__ void load16_to_lds(const void* p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(
                     __builtin_amdgcn_readfirstlane(lds)), "v"(p)
                 : "memory", "m0");
}
__device__ __forceinline__ void load4_to_lds(const void* p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(
                     __builtin_amdgcn_readfirstlane(lds)), "v"(p)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// Rows of whole, aligned 16-byte chunks.  The workgroup stays and takes one tile
// after another; its loads run ahead of the products, SX - 1 steps those of x and
// SW - 1 those of w, across the tiles' ends.  A tile's scales are loaded with its
// first steps.  SX is SW, or 2 where LDS has no room for more: x comes from the L2
// mostly, w from memory.
//
// A tile's border is not free: the compiler does not know of the loads into LDS and
// waits for everything under way where it uses the tile's row tokens, and before it
// writes their registers again; the tile's stores count in the first wait_loads
// behind them.  Up to three such waits a tile, of 16 steps with 2048 of k.
template <int BM, int BN, int BK, int SX, int SW, int WM, int WN>
__global__ __launch_bounds__(WM* WN* kWave) void expert_matmul_int8_kernel(MatmulArgs a) {
    using Y = Layout<BM, BN, BK, WM, WN>;
    constexpr int kWaves = Y::kWaves, kThreads = kWaves * kWave;
    constexpr int kX = (Y::kXLoads + kWaves - 1) / kWaves, kW = Y::kWLoads / kWaves;  // loads of a wave and step
    constexpr bool kEven = Y::kXLoads % kWaves == 0;  // else the first waves have one more of x
    static_assert(SX == SW ? SW == 2 || kEven : SX == 2 && SW == 3, "what the waits count");
    // the loads that may be under way still when a step's have to be there: those
    // of later steps, if they come after the step's own
    constexpr int kLater = SX == SW ? (SW - 2) * (kX + kW) : kW;
    static_assert(BM <= kThreads && BN % kWave == 0, "a thread for each row's scale, whole waves for the channels'");
    constexpr int kScales = (BM + kWave - 1) / kWave * kWave;  // whole waves load them
    __shared__ __attribute__((aligned(1024))) uint8_t x_stages[SX][BM * BK], w_stages[SW][BN * BK];
    // of each tile that the loads may be ahead
    __shared__ float x_scale[SW][kScales], w_scale[SW][BN];
    __shared__ uint8_t known[SW][BM];
    __shared__ Tile tiles_ahead[SW];
    const uint32_t x_lds = MOE_LDS_ADDRESS(x_stages), w_lds = MOE_LDS_ADDRESS(w_stages);
    const uint32_t x_scale_lds = MOE_LDS_ADDRESS(x_scale), w_scale_lds = MOE_LDS_ADDRESS(w_scale);

    const Tiles<BM, BN> tiles(a);
    // workgroups go to the dies in turn; a die's take one run of tiles by turns
    const int die = blockIdx.x % kXcds, stride = gridDim.x / kXcds;
    int64_t id = tiles.start_of(die, kXcds) + blockIdx.x / kXcds;
    const int64_t end = tiles.start_of(die + 1, kXcds);
    if (id >= end) return;
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int steps = (a.K + BK - 1) / BK;
    int64_t left = (end - id + stride - 1) / stride * steps;  // steps to multiply
    const int line_row = lane / Y::kChunks, line_chunk = lane % Y::kChunks;  // the lane's place in a load

    // The loads' side.  `next` is the tile that w comes to next, `after` the one
    // that x does; a tile's row tokens are read one step before x needs them.
    Tile next = tiles.find(id), after = next;
    int token[kX], my_token = 0;
    const uint8_t *x_src[kX], *w_src[kW];
    int x_step = 0, w_step = 0, x_slot = 0, w_slot = 0, x_stage = 0, w_stage = 0;
    int x_tiles = 0, w_tiles = 0;  // begun
    bool more = true;
    auto read_tokens = [&](const Tile& t) {
        after = t;
#pragma unroll
        for (int j = 0; j < kX; ++j) {
            // rows past the tile's read its last one again and are not stored
            const int64_t row = t.row + min((wave + j * kWaves) * Y::kRowsPerLoad + line_row, t.rows - 1);
            token[j] = a.row_token != nullptr ? a.row_token[row] : static_cast<int>(row);
        }
        const int64_t row = t.row + min(static_cast<int>(threadIdx.x), t.rows - 1);
        my_token = a.row_token != nullptr ? a.row_token[row] : static_cast<int>(row);
    };
    auto load_x = [&]() {
        if (x_step == 0) {
            if (x_tiles == w_tiles + (SX == SW && more)) return;  // no tile left
            ++x_tiles;
#pragma unroll
            for (int j = 0; j < kX; ++j) {
                const int r = (wave + j * kWaves) * Y::kRowsPerLoad + line_row;
                // a row without a token is stored as zeros, whatever it reads
                const int x = token[j] >= 0 && token[j] < a.x_rows ? token[j] : 0;
                x_src[j] = a.x + static_cast<int64_t>(x) * a.K + (line_chunk ^ Y::x_swizzle(r)) * 16;
            }
            const bool has = my_token >= 0 && my_token < a.x_rows;
            if (threadIdx.x < BM) known[x_slot][threadIdx.x] = has;
            if (threadIdx.x == 0) tiles_ahead[x_slot] = after;
            if (wave * kWave < BM)
                load4_to_lds(has ? static_cast<const void*>(a.x_sf + my_token) : &kZeroChunk,
                             x_scale_lds + (x_slot * kScales + wave * kWave) * 4);
        }
#pragma unroll
        for (int j = 0; j < kX; ++j) {
            if (!kEven && wave + j * kWaves >= Y::kXLoads) continue;
            const uint8_t* p = x_src[j];
            if ((x_step + 1) * BK > a.K) {  // past the end of k: zeros
                const int r = (wave + j * kWaves) * Y::kRowsPerLoad + line_row;
                if (x_step * BK + (line_chunk ^ Y::x_swizzle(r)) * 16 >= a.K)
                    p = reinterpret_cast<const uint8_t*>(&kZeroChunk);
            }
            load16_to_lds(p, x_lds + x_stage * (BM * BK) + (wave + j * kWaves) * 1024);
            x_src[j] += BK;
        }
        x_stage = x_stage + 1 == SX ? 0 : x_stage + 1;
        if (++x_step == steps) {
            x_step = 0;
            x_slot = x_slot + 1 == SW ? 0 : x_slot + 1;
        }
    };
    auto load_w = [&]() {
        if (w_step == 0) {
            ++w_tiles;
            const int64_t first = static_cast<int64_t>(next.expert) * a.N;
#pragma unroll
            for (int j = 0; j < kW; ++j) {
                const int r = (wave + j * kWaves) * Y::kRowsPerLoad + line_row;
                w_src[j] = a.w + (first + min(next.channel + r, a.N - 1)) * a.K + (line_chunk ^ Y::w_swizzle(r)) * 16;
            }
#pragma unroll
            for (int i = 0; i < (BN + kThreads - 1) / kThreads; ++i) {
                const int c = i * kThreads + wave * kWave;
                if (c < BN)
                    load4_to_lds(a.w_sf + first + min(next.channel + c + lane, a.N - 1),
                                 w_scale_lds + (w_slot * BN + c) * 4);
            }
        }
#pragma unroll
        for (int j = 0; j < kW; ++j) {
            const uint8_t* p = w_src[j];
            if ((w_step + 1) * BK > a.K) {
                const int r = (wave + j * kWaves) * Y::kRowsPerLoad + line_row;
                if (w_step * BK + (line_chunk ^ Y::w_swizzle(r)) * 16 >= a.K)
                    p = reinterpret_cast<const uint8_t*>(&kZeroChunk);
            }
            load16_to_lds(p, w_lds + w_stage * (BN * BK) + (wave + j * kWaves) * 1024);
            w_src[j] += BK;
        }
        if (SX != SW && w_step == 0) read_tokens(next);  // x comes to this tile one step later
        w_stage = w_stage + 1 == SW ? 0 : w_stage + 1;
        if (++w_step == steps) {
            w_step = 0;
            w_slot = w_slot + 1 == SW ? 0 : w_slot + 1;
            id += stride;
            more = id < end;
            if (more) {
                next = tiles.find(id);
                if (SX == SW) read_tokens(next);
            }
        }
    };

    if (SX == SW) read_tokens(next);
    int ahead = 0;  // steps of w loaded or loading
    for (int i = 0; i < SW - 1; ++i) {
        if (i >= SW - SX) load_x();
        if (more) {
            load_w();
            ++ahead;
        }
    }

    const int wm = wave / WN, wn = wave % WN;
    typename Y::Sums acc;
    int xs = 0, ws = 0, slot = 0, step = 0, used = 0;
    for (; left > 0; --left) {
        if (ahead == SW - 1) wait_loads<kLater>();
        else
            wait_loads<0>();
        // every wave's part of this step is there, and every wave is done with the step before it
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");  // the compiler's reads of LDS stay behind it
        if (step == 0) {
            used = Y::used_blocks(__builtin_amdgcn_readfirstlane(tiles_ahead[slot].rows), wm);
#pragma unroll
            for (int m = 0; m < Y::TM; ++m)
#pragma unroll
                for (int n = 0; n < Y::TN; ++n) acc[m][n] = i32x4_t{0, 0, 0, 0};
        }
        --ahead;
        load_x();
        if (more) {
            load_w();
            ++ahead;
        }
        Y::multiply(x_stages[xs], w_stages[ws], used, wm, wn, lane, acc);
        xs = xs + 1 == SX ? 0 : xs + 1;
        ws = ws + 1 == SW ? 0 : ws + 1;
        if (++step < steps) continue;
        step = 0;
        const Tile t = tiles_ahead[slot];
        Y::store(
            a, t, wm, wn, lane, acc,
            [&](int r, bool& has) {
                has = known[slot][r];
                return x_scale[slot][r];
            },
            [&](int c) { return w_scale[slot][c]; });
        slot = slot + 1 == SW ? 0 : slot + 1;
    }
}

// A row's sixteen bytes from p on, at any address, of which `left` (or fewer, or
// none) are the row's: those before its end instead where it ends sooner, so that
// no byte outside it is read and no lane takes another path.
struct __attribute__((packed, aligned(1))) Unaligned16 {
    u32x4_t v;
};
__device__ __forceinline__ u32x4_t load_odd(const uint8_t* p, int left) {
    return reinterpret_cast<const Unaligned16*>(p + min(left - 16, 0))->v;
}
// Those bytes in their places, with zeros behind the row's end.
__device__ __forceinline__ u32x4_t shift_odd(u32x4_t v, int left) {
    const int n = 16 - min(max(left, 0), 16);  // bytes that came before p
    u32x4_t r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t lo = 0, hi = 0;  // words i + n / 4 and the next
#pragma unroll
        for (int k = i; k < 4; ++k) {
            lo = k == i + n / 4 ? v[k] : lo;
            hi = k == i + n / 4 + 1 ? v[k] : hi;
        }
        r[i] = __builtin_amdgcn_alignbyte(hi, lo, n % 4);
    }
    return r;
}
// The same of a row of fewer than sixteen bytes, byte by byte.
__device__ __forceinline__ u32x4_t load_short(const uint8_t* p, int left) {
    u32x4_t v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 15; ++i)
        if (i < left) v[i / 4] |= static_cast<uint32_t>(p[i]) << (8 * (i % 4));
    return v;
}

// Rows of any length at any address: the next step's chunks are in registers
// while this one's are multiplied.
template <int BM, int BN, int BK, int WM, int WN>
__global__ __launch_bounds__(WM* WN* kWave) void expert_matmul_int8_odd_kernel(MatmulArgs a) {
    using Y = Layout<BM, BN, BK, WM, WN>;
    constexpr int kLoads = (Y::kXLoads + Y::kWLoads) / Y::kWaves;
    static_assert(Y::kXLoads % Y::kWaves == 0, "a load lies in x or in w");
    __shared__ __attribute__((aligned(1024))) uint8_t stages[2][(BM + BN) * BK];
    const Tiles<BM, BN> tiles(a);
    const int die = blockIdx.x % kXcds, stride = gridDim.x / kXcds;
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / WN, wn = wave % WN;
    const int steps = (a.K + BK - 1) / BK;
    const int64_t end = tiles.start_of(die + 1, kXcds);
    for (int64_t id = tiles.start_of(die, kXcds) + blockIdx.x / kXcds; id < end; id += stride) {
        const Tile t = tiles.find(id);
        const uint8_t* src[kLoads];
        int left[kLoads];  // bytes of the row from this lane's chunk on
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int r = (wave + j * Y::kWaves) * Y::kRowsPerLoad + lane / Y::kChunks;
            const int place = lane % Y::kChunks, c = place ^ (r < BM ? Y::x_swizzle(r) : Y::w_swizzle(r - BM));
            if (r < BM) {
                int64_t row = t.row + min(r, t.rows - 1);
                if (a.row_token != nullptr) row = a.row_token[row];
                src[j] = a.x + (row >= 0 && row < a.x_rows ? row : 0) * a.K + c * 16;
            } else {
                src[j] = a.w + (static_cast<int64_t>(t.expert) * a.N + min(t.channel + r - BM, a.N - 1)) * a.K + c * 16;
            }
            left[j] = a.K - c * 16;
        }
        u32x4_t held[kLoads];
        auto fetch = [&]() {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                held[j] = a.K < 16 ? load_short(src[j], left[j]) : load_odd(src[j], left[j]);
                src[j] += BK;
                left[j] -= BK;
            }
        };
        const int used = Y::used_blocks(t.rows, wm);
        typename Y::Sums acc;
#pragma unroll
        for (int m = 0; m < Y::TM; ++m)
#pragma unroll
            for (int n = 0; n < Y::TN; ++n) acc[m][n] = i32x4_t{0, 0, 0, 0};
        __syncthreads();  // every wave is done with the tile before
        fetch();
        for (int i = 0; i < steps; ++i) {
            uint8_t* s = stages[i & 1];
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                u32x4_t v = held[j];
                if (i + 1 == steps && a.K >= 16) v = shift_odd(v, left[j] + BK);
                *reinterpret_cast<u32x4_t*>(s + (wave + j * Y::kWaves) * 1024 + lane * 16) = v;
            }
            if (i + 1 < steps) fetch();
            __syncthreads();
            Y::multiply(s, s + BM * BK, used, wm, wn, lane, acc);
        }
        Y::store(
            a, t, wm, wn, lane, acc,
            [&](int r, bool& has) {
                int64_t row = t.row + r;
                if (a.row_token != nullptr) row = a.row_token[row];
                has = row >= 0 && row < a.x_rows;
                return has ? a.x_sf[row] : 0.0f;
            },
            [&](int c) { return t.channel + c < a.N ? a.w_sf[static_cast<int64_t>(t.expert) * a.N + t.channel + c] : 0.0f; });
    }
}

// The most tiles that there can be: an expert adds at most one that is not full.
int64_t most_tiles(const MatmulArgs& a, int bm) {
    const int64_t experts = a.E < a.num_rows ? a.E : a.num_rows;
    const int64_t slots = a.num_rows / bm + experts;
    return (slots < a.num_rows ? slots : a.num_rows) * a.n_tiles;
}
unsigned whole_dies(int64_t blocks) { return static_cast<unsigned>((blocks + kXcds - 1) / kXcds * kXcds); }

// PER_CU workgroups fit a compute unit's LDS.
template <int BM, int BN, int BK, int SX, int SW, int WM, int WN, int PER_CU>
hipError_t launch_tiles(MatmulArgs a, hipStream_t stream) {
    a.n_tiles = (a.N + BN - 1) / BN;
    const int64_t places = static_cast<int64_t>(device_cu_count()) * PER_CU, tiles = most_tiles(a, BM);
    hipLaunchKernelGGL((expert_matmul_int8_kernel<BM, BN, BK, SX, SW, WM, WN>),
                       dim3(whole_dies(tiles < places ? tiles : places)), dim3(WM * WN * kWave), 0, stream, a);
    return hipGetLastError();
}

template <int BM, int BN, int BK, int WM, int WN>
hipError_t launch_odd(MatmulArgs a, hipStream_t stream) {
    a.n_tiles = (a.N + BN - 1) / BN;
    constexpr int64_t kPerCu = 8;  // more than fit at once
    const int64_t places = device_cu_count() * kPerCu, tiles = most_tiles(a, BM);
    hipLaunchKernelGGL((expert_matmul_int8_odd_kernel<BM, BN, BK, WM, WN>),
                       dim3(whole_dies(tiles < places ? tiles : places)), dim3(WM * WN * kWave), 0, stream, a);
    return hipGetLastError();
}

// The form for a batch.  Large tiles read x and w less often and keep the matrix
// units busier; small ones fill the chip where there are few, and read no more
// rows than there are.  The host knows the experts' mean row count, not each one's.
hipError_t launch_matmul(const MatmulArgs& a, bool direct, hipStream_t stream) {
    const int64_t busy = a.E < a.num_rows ? a.E : a.num_rows, mean = (a.num_rows + busy - 1) / busy;
    auto tiles = [&](int64_t bm, int64_t bn) { return busy * ((mean + bm - 1) / bm) * ((a.N + bn - 1) / bn); };
    const int64_t cus = device_cu_count();
    if (!direct) {
        // 700 rows of one matrix, 1000 -> 500: 8.8 against 10.4 us in tiles of 64 x 64; 5 experts of 156 rows, 1999 ->
        // 1021, 800 of these: 26.8 against 17.4 us
        if (mean <= 8 || tiles(16, 64) <= 2 * cus) return launch_odd<16, 64, 256, 1, 4>(a, stream);
        // 16 experts of 125 rows, 3001 -> 1000: 34.5 against 43.3 us; those 5 experts, 80 of these: 25.6 us
        if (tiles(128, 128) >= cus / 2) return launch_odd<128, 128, 128, 2, 4>(a, stream);
        return launch_odd<64, 64, 128, 2, 2>(a, stream);
    }
    // one tile holds most experts' rows (32 experts, 7168 -> 4096, 128 rows: 98 us; 108 us in tiles of 32 x 128), or
    // the places of two workgroups a compute unit are not all taken (256 rows of one matrix, 4096 -> 2048: 15.4
    // against 21.2 us; 1024 rows, 1024 -> 1024, two for each place: 11.5 against 8.9 us)
    if (mean <= 8 || tiles(16, 64) <= 2 * cus) return launch_tiles<16, 64, 256, 3, 3, 1, 4, 2>(a, stream);
    // 32 experts, 7168 -> 4096, 1024 rows an expert: 1060 against 1120 us in the next; 512: 635 against 596 us
    if (mean > 768 && tiles(256, 256) >= 2 * cus) return launch_tiles<256, 256, 128, 2, 2, 2, 4, 1>(a, stream);
    // the same, 512 rows: 598 against 668 us in the next; 8192 rows over 32 experts, 2048 -> 7168: 212 against 224 us;
    // 128 rows, 7168 -> 4096: 306 against 288 us
    if (mean > 192 && tiles(192, 256) >= cus) return launch_tiles<192, 256, 128, 2, 3, 2, 4, 1>(a, stream);
    // the same, 64 rows: 191 against 218 us in the next; 2048 rows of one matrix, 2048 -> 2048, 128 tiles of this
    // size: 23.1 against 20.6 us
    if (tiles(128, 256) >= cus) return launch_tiles<128, 256, 128, 3, 3, 2, 4, 1>(a, stream);
    // 4096 rows of one matrix, 7168 -> 512: 38 against 40 us in the last; 1024 rows, 1024 -> 1024, 128 tiles of this
    // size: 9.9 against 8.9 us
    if (tiles(64, 128) >= cus) return launch_tiles<64, 128, 128, 3, 3, 2, 4, 2>(a, stream);
    return launch_tiles<32, 128, 128, 3, 3, 1, 4, 2>(a, stream);
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
    // the sums over the experts' row tiles and their costs, 32 bits, and the rows' rounding up to whole tiles hold for
    // fewer than 2^28 rows, which the second condition leaves; tiles are numbered in 64 bits
    if (num_rows >= MOE_MATMUL_INT8_ANY_WIDTH_ROWS &&
        (num_rows / kMinRows + num_experts) * ((out_width + kMinChannels - 1) / kMinChannels) >=
            MOE_MATMUL_INT8_MAX_TILES)
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
    a.vec = out_width % 8 == 0 && aligned(out, 16);
    const bool direct = inner % 16 == 0 && aligned(a.x, 16) && aligned(w, 16);
    return hip_status(launch_matmul(a, direct, stream));
}
