// Drives the host side of the block operators' entry points (norms, balance loss, expert products) -- argument
// validation, size queries up to the largest shapes and empty batches, none of which launches a kernel -- for a host
// build with AddressSanitizer and UndefinedBehaviorSanitizer.  Prints "ok" on success.
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "moe_fp8.h"

#define EXPECT(cond)                                                 \
    do {                                                             \
        if (!(cond)) {                                               \
            std::printf("failed at line %d: %s\n", __LINE__, #cond); \
            return 1;                                                \
        }                                                            \
    } while (0)

int main() {
    // a non-null, 256-byte aligned address that is never dereferenced on the host
    void* p = reinterpret_cast<void*>(uintptr_t{0x10000});
    void* odd = reinterpret_cast<void*>(uintptr_t{0x10001});
    auto* f = static_cast<float*>(p);
    auto* i32 = static_cast<int32_t*>(p);
    auto* i64 = static_cast<int64_t*>(p);
    auto* u8 = static_cast<uint8_t*>(p);
    auto* u16 = static_cast<uint16_t*>(p);
    const moe_status bad = MOE_ERR_INVALID_ARGUMENT, no = MOE_ERR_UNSUPPORTED, small = MOE_ERR_WORKSPACE_TOO_SMALL;
    const int64_t far = INT64_MAX;

    auto norm = [&](const void* r, int64_t stride, int64_t T, int32_t H, int32_t mode, const float* gate, float eps) {
        return moe_block_norm(r, stride, MOE_DTYPE_F32, p, stride, MOE_DTYPE_BF16, T, H, f, gate, mode, 1.0f, f, eps,
                              p, p, f, f, nullptr);
    };
    EXPECT(norm(p, 64, -1, 64, MOE_GATE_NONE, nullptr, 0.0f) == bad);
    EXPECT(norm(p, 64, far, 64, MOE_GATE_NONE, nullptr, 0.0f) == no);
    EXPECT(norm(p, 64, 4, 64, MOE_GATE_CHANNEL, nullptr, 0.0f) == bad);
    EXPECT(norm(p, 64, 4, 64, MOE_GATE_NONE, nullptr, std::nanf("")) == bad);
    EXPECT(norm(odd, 64, 4, 64, MOE_GATE_NONE, nullptr, 0.0f) == bad);
    EXPECT(norm(nullptr, far, 0, 64, MOE_GATE_TOKEN, nullptr, 0.0f) == MOE_OK);
    EXPECT(moe_block_norm_backward_workspace_bytes(MOE_BLOCK_NORM_MAX_TOKENS, MOE_BLOCK_NORM_MAX_HIDDEN) > 0);
    EXPECT(moe_block_norm_backward_workspace_bytes(far, 64) == 0);
    EXPECT(moe_block_norm_backward_workspace_bytes(4, INT32_MAX) == 0);
    auto norm_back = [&](int64_t T, float* gate, const float* w, size_t ws) {
        return moe_block_norm_backward(p, p, p, 64, MOE_DTYPE_BF16, p, 64, MOE_DTYPE_BF16, T, 64, w, gate,
                                       MOE_GATE_TOKEN, 1.0f, w, f, f, p, p, f, gate, f, p, ws, nullptr);
    };
    EXPECT(norm_back(4, nullptr, f, 1 << 30) == bad);
    EXPECT(norm_back(4, f, f, 16) == small);
    EXPECT(norm_back(4, f, nullptr, 1 << 30) == bad);
    EXPECT(norm_back(-4, f, f, 1 << 30) == bad);
    EXPECT(norm_back(far, f, f, 1 << 30) == no);

    EXPECT(moe_balance_loss_workspace_bytes(INT32_MAX / 16, 1024, MOE_BALANCE_MAX_SEQS) > 0);
    EXPECT(moe_balance_loss_workspace_bytes(0, 1, 1) > 0);
    EXPECT(moe_balance_loss_workspace_bytes(far, 16, 1) == 0);
    EXPECT(moe_balance_loss_workspace_bytes(100, INT32_MAX, 1) == 0);
    auto balance = [&](const void* z, int64_t stride, int64_t T, int32_t S, const int32_t* off, size_t ws) {
        return moe_balance_loss(z, MOE_DTYPE_BF16, stride, T, 64, MOE_SCORE_SIGMOID, i64, 4, nullptr, off, S, f, i32,
                                i32, nullptr, p, ws, nullptr);
    };
    EXPECT(balance(p, 63, 100, 1, nullptr, 1 << 30) == bad);
    EXPECT(balance(odd, 64, 100, 1, nullptr, 1 << 30) == bad);
    EXPECT(balance(p, 64, 100, 2, nullptr, 1 << 30) == bad);
    EXPECT(balance(p, 64, INT32_MAX / 16, MOE_BALANCE_MAX_SEQS, i32, 1) == small);
    EXPECT(moe_balance_loss_backward(f, p, MOE_DTYPE_F32, 63, 100, 64, MOE_SCORE_SOFTMAX, 4, nullptr, nullptr, 1, i32,
                                     i32, p, nullptr) == bad);
    EXPECT(moe_balance_loss_backward(nullptr, nullptr, MOE_DTYPE_F32, far, 0, 64, MOE_SCORE_SOFTMAX, 4, nullptr,
                                     nullptr, 1, nullptr, nullptr, nullptr, nullptr) == MOE_OK);

    auto products = [&](int64_t X, const int32_t* token, int64_t R, int32_t K, int32_t N, int32_t E, int32_t g) {
        return moe_expert_matvec(p, MOE_DTYPE_BF16, nullptr, X, token, R, K, N, E, i32, u8, p, g, 1, u16, nullptr);
    };
    EXPECT(products(far, i32, 4, 256, 8, 2, 32) == bad);
    EXPECT(products(5, i32, far, 256, 8, 2, 32) == bad);
    EXPECT(products(5, nullptr, 4, 256, 8, 2, 32) == bad);
    EXPECT(products(5, i32, 4, INT32_MAX - 31, 8, 2, 32) == no);
    EXPECT(products(5, i32, 4, 256, INT32_MAX, 2, 32) == no);
    EXPECT(products(5, i32, 4, 256, 8, 2, 0) == no);
    EXPECT(products(5, nullptr, 0, 256, 8, 2, 32) == MOE_OK);
    std::puts("ok");
    return 0;
}
