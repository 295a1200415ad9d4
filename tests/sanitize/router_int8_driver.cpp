// Drives the host side of the routing's and the 8-bit integer entry points -- argument validation up to the largest
// shapes and empty batches, none of which launches a kernel -- for a host build with AddressSanitizer and
// UndefinedBehaviorSanitizer.  Prints "ok" on success.
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
    auto* i8 = static_cast<int8_t*>(p);
    auto* u16 = static_cast<uint16_t*>(p);
    const moe_status bad = MOE_ERR_INVALID_ARGUMENT, no = MOE_ERR_UNSUPPORTED;
    const int64_t far = INT64_MAX;

    auto route = [&](const void* z, int64_t stride, int64_t T, int32_t E, int32_t K, int32_t G, int32_t kept, float s) {
        return moe_router(z, MOE_DTYPE_F32, stride, T, E, K, MOE_SCORE_SIGMOID, f, G, kept, MOE_GROUP_TOP2, 1, s,
                          nullptr, i64, f, nullptr);
    };
    EXPECT(route(p, 64, -1, 64, 4, 8, 4, 1.0f) == bad);
    EXPECT(route(p, 64, far, 64, 4, 8, 4, 1.0f) == bad);
    EXPECT(route(p, 63, 4, 64, 4, 8, 4, 1.0f) == bad);
    EXPECT(route(p, far, 0, 64, 4, 8, 4, 1.0f) == MOE_OK);
    EXPECT(route(odd, 64, 4, 64, 4, 8, 4, 1.0f) == bad);
    EXPECT(route(p, 64, 4, 64, 4, INT32_MAX, 4, 1.0f) == bad);
    EXPECT(route(p, 64, 4, 64, 4, 0, 4, 1.0f) == bad);
    EXPECT(route(p, 64, 4, 64, 4, 8, INT32_MAX, 1.0f) == bad);
    EXPECT(route(p, 1024, 4, 1024, 16, 512, 300, 1.0f) == no);
    EXPECT(route(p, 64, 4, 64, 4, 8, 4, std::nanf("")) == bad);
    EXPECT(route(p, 64, 4, 64, 4, 8, 4, INFINITY) == bad);
    auto back = [&](const float* g, int64_t T, int32_t E, int32_t K, void* out) {
        return moe_router_backward(g, p, MOE_DTYPE_BF16, E, T, E, i64, K, MOE_SCORE_SOFTMAX, 0, 1.0f, out, nullptr);
    };
    EXPECT(back(f, far, 64, 4, p) == bad);
    EXPECT(back(f, 4, INT32_MAX, 4, p) == bad);
    EXPECT(back(nullptr, 4, 64, 4, p) == bad);
    EXPECT(back(f, 4, 64, 4, odd) == bad);
    EXPECT(back(nullptr, 0, 64, 4, nullptr) == MOE_OK);

    EXPECT(moe_cast_int8(p, MOE_DTYPE_F32, far, far, 64, i8, f, nullptr) == no);
    EXPECT(moe_cast_int8(p, MOE_DTYPE_F32, far, 4, INT32_MAX, i8, f, nullptr) == no);
    EXPECT(moe_cast_int8(odd, MOE_DTYPE_BF16, 64, 4, 64, i8, f, nullptr) == bad);
    EXPECT(moe_cast_int8(nullptr, MOE_DTYPE_BF16, 64, 0, 64, nullptr, nullptr, nullptr) == MOE_OK);
    EXPECT(swiglu_cast_int8(u16, far, 64, f, 0.0f, i8, f, nullptr) == no);
    EXPECT(swiglu_cast_int8(u16, 4, INT32_MAX, f, 0.0f, i8, f, nullptr) == no);
    EXPECT(swiglu_cast_int8(u16, 4, 64, f, std::nanf(""), i8, f, nullptr) == bad);
    EXPECT(swiglu_cast_int8(nullptr, 0, 64, nullptr, 0.0f, nullptr, nullptr, nullptr) == MOE_OK);

    auto products = [&](int64_t X, const int32_t* token, int64_t R, int32_t K, int32_t N, int32_t E) {
        return moe_expert_matmul_int8(i8, f, X, token, R, K, N, E, i32, i8, f, MOE_DTYPE_BF16, p, nullptr);
    };
    EXPECT(products(far, i32, 4, 256, 8, 2) == bad);
    EXPECT(products(5, i32, far, 256, 8, 2) == bad);
    EXPECT(products(5, nullptr, 4, 256, 8, 2) == bad);
    EXPECT(products(5, i32, 4, INT32_MAX, 8, 2) == no);
    EXPECT(products(5, i32, 4, 256, INT32_MAX, 2) == no);
    EXPECT(products(5, i32, INT32_MAX, 256, MOE_MATVEC_MAX_WIDTH, 1024) == no);
    EXPECT(products(5, i32, 4, 256, 8, INT32_MAX) == bad);
    EXPECT(products(5, nullptr, 0, 256, 8, 2) == MOE_OK);
    std::puts("ok");
    return 0;
}
