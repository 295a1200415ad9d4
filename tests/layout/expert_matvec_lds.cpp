// Host check of the expert products' LDS layout (csrc/expert_matvec_lds.hpp): every store and read of x that a lane
// makes, for every form of the kernel, lies in the wave's or the workgroup's x, and the pass's rows are found there.
// Prints the first fault of each form and "ok" if there is none.
#include <cstdio>
#include <vector>

#include "expert_matvec_lds.hpp"

using namespace moe::matvec;

namespace {

int faults = 0;

// One block of steps of a form: `chunks` 16-byte chunks of a row of x in a step (16: bf16, 8: e4m3), passes of `rows`
// rows in a kernel made for `most`, `waves` waves.
void check(int chunks, int most, int rows, bool shared, int waves) {
    const int step_units = rows * chunks;
    const int loads = (rows + kLanes / chunks - 1) / (kLanes / chunks);
    const int fragments = (rows + 15) / 16;
    // the workgroup's LDS; what a unit holds: owner (wave, or step of a shared block) * 1000 + row * 16 + chunk
    std::vector<int> lds(lds_bytes(shared, most, waves) / kUnit, -1);
    auto x_at = [&](int wave) {
        return shared ? waves * lds_wave(true, most) : wave * lds_wave(false, most) + kLdsCodes + kLdsScales;
    };
    auto region_end = [&](int wave) {
        return shared ? static_cast<int>(lds.size()) : (wave + 1) * lds_wave(false, most);
    };
    const char* what = "";
    int at = 0;
    auto fail = [&](const char* w, int unit) {
        if (*what == 0) {
            what = w;
            at = unit;
        }
    };
    for (int wave = 0; wave < waves; ++wave)  // shared: wave w stores step w of the block
        for (int i = 0; i < loads; ++i)
            for (int lane = 0; lane < kLanes; ++lane) {
                const int unit = x_at(wave) + (shared ? wave * step_units : 0) + i * kLanes + lane;
                if (unit >= region_end(wave)) {
                    fail("store past the x", unit);
                    continue;
                }
                lds[unit] = wave * 1000 + x_load_row(chunks, i, lane) * 16 + x_load_chunk(chunks, i, lane);
            }
    for (int wave = 0; wave < waves; ++wave)
        for (int step = 0; step < (shared ? kBlock : 1); ++step)
            for (int mt = 0; mt < fragments; ++mt)
                for (int lr = 0; lr < 16; ++lr)
                    for (int c = 0; c < chunks; ++c) {
                        const int m = mt * 16 + lr;
                        const int unit =
                            x_at(wave) + (shared ? step * step_units : 0) + x_unit(most, rows, chunks, m, c);
                        if (unit < x_at(wave) || unit >= region_end(wave))
                            fail("read past the x", unit);
                        else if (m < rows && lds[unit] != (shared ? step : wave) * 1000 + m * 16 + c)
                            fail("read of another wave's, step's or row's x", unit);
                    }
    // the sums that take the operands' place, before the next wave's
    if (fragments * 16 * kPitch * 4 > lds_wave(shared, most) * kUnit) fail("sums past the wave's operands", 0);
    if (*what != 0) {
        ++faults;
        std::printf("%s, unit %d of %zu: %s x, passes of %d rows, made for %d, %s, %d waves\n", what, at, lds.size(),
                    chunks == 16 ? "bf16" : "e4m3", rows, most, shared ? "shared" : "private", waves);
    }
}

}  // namespace

int main() {
    const int forms[][2] = {{8, 4}, {8, 8}, {16, 8}, {16, 16}, {32, 8}, {32, 16}, {32, 32}};  // made for, rows
    for (const auto& f : forms)
        for (int chunks : {16, 8}) {
            if (chunks == 8 && f[1] == 4) continue;  // e4m3 rows take passes of 8 and more
            check(chunks, f[0], f[1], true, kSharedWaves);
            if (f[0] > 16) continue;  // shared only
            for (int waves = 2; waves <= kMaxSplit; waves *= 2) check(chunks, f[0], f[1], false, waves);
        }
    if (faults == 0) std::printf("ok\n");
    return faults != 0;
}
