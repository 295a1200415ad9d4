// How the expert products' kernel lays its operands out in LDS, in units of 16
// bytes: host and device code, without HIP.
//
// Of each wave: codes of two steps, scales of a block (fp32 scales of 32
// channels: of a step), and its x of a step (private) or the workgroup's x of
// a block (shared).  After the loop the sums of up to `rows` rows lie there.
#pragma once

#include <cstddef>

namespace moe {
namespace matvec {

constexpr int kLanes = 64;
constexpr int kNT = 2;             // 16-column tiles of a wave
constexpr int kCols = kNT * 16;
constexpr int kBlock = 4;          // steps of a block: one 16-byte load of scales, and the depth of the loads in flight
constexpr int kPair = 2;           // steps whose codes are loaded together: a row's 128 bytes, one cache line
constexpr int kPitch = kCols + 1;  // floats of a row of sums in LDS
constexpr int kSharedWaves = kBlock;  // waves of a workgroup that shares its x: one for each step of a block
constexpr int kMaxSplit = 4;       // waves that share a tile's k range

constexpr int kUnit = 16;
constexpr int kXUnits = 16;  // of a row of x in a step: 128 bf16 values (e4m3 rows take half of it)

constexpr int kLdsCodes = kNT * kPair * kLanes;
constexpr int kLdsScales = kCols;
constexpr int lds_x(bool shared, int rows) { return rows * kXUnits * (shared ? kBlock : 1); }
constexpr int lds_wave(bool shared, int rows) { return kLdsCodes + kLdsScales + (shared ? 0 : lds_x(false, rows)); }
constexpr std::size_t lds_bytes(bool shared, int rows, int waves) {
    return kUnit * (static_cast<std::size_t>(waves) * lds_wave(shared, rows) + (shared ? lds_x(true, rows) : 0));
}
static_assert(32 * kPitch * 4 <= lds_wave(true, 32) * kUnit, "a wave's sums fit where its operands were");

// x.  The wave's i-th load of a step covers rows i * kLanes / chunks onwards,
// `chunks` neighbouring lanes a row; it is stored lane by lane, so the chunk
// that a lane loads says where that chunk lies: chunk c of row m at c XOR m,
// which spreads the eight rows that one LDS clock serves over all banks.
constexpr int x_load_row(int chunks, int i, int lane) { return i * (kLanes / chunks) + lane / chunks; }
constexpr int x_load_chunk(int chunks, int i, int lane) { return (lane ^ x_load_row(chunks, i, lane)) & (chunks - 1); }
// Where chunk c of row m of the matrix fragments lies in the x of a step, for a
// pass of `rows` rows (a power of two) in a kernel whose x holds `most`.  A
// fragment has 16 rows also where a pass has 4 or 8; what its rows past them
// read only gives sums that are not kept, but it has to lie in the x: where
// that holds fewer than 16 rows, they read the pass's rows again.  (Elsewhere
// that would take registers that the kernels of 16 and 32 rows do not have.)
constexpr int x_unit(int most, int rows, int chunks, int m, int c) {
    const int r = most < 16 ? m & (rows - 1) : m;
    return r * chunks + (c ^ (r & (chunks - 1)));
}

}  // namespace matvec
}  // namespace moe
