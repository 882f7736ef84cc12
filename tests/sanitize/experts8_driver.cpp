// Sanitizer driver for the host side of the operators of 8-bit experts (test infrastructure):
// argument checks and the size functions over many sizes, none of which touches a GPU.  Exit
// status 0 = clean.
#include <limits.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/seedmm.h"

#define CHECK(c) do { if (!(c)) { fprintf(stderr, "check failed: %s (line %d)\n", #c, __LINE__); return 1; } } while (0)

static uint64_t rng = 0xFEEDu;
static uint32_t next32() {
    rng ^= rng >> 12; rng ^= rng << 25; rng ^= rng >> 27;
    return (uint32_t)((rng * 2685821657736338717ull) >> 32);
}
static int any(int most) { return (int)(next32() % (uint32_t)most) >> next32() % 31; }

int main() {
    char* F = (char*)(uintptr_t)0x100000;    // aligned, never dereferenced (validation fails first)
    const int8_t* W = (const int8_t*)F;
    int32_t* I32 = (int32_t*)F;
    float* X = (float*)F;
    for (int i = 0; i < 300000; ++i) {
        const int T = any(INT_MAX), k = any(80), E = any(5000), H = any(INT_MAX), I = any(INT_MAX);
        const size_t s = seedmm_moe_sort_workspace_bytes(T, k, E), n = seedmm_moe_i8_workspace_bytes(T, k, E, H, I);
        const int64_t P = (int64_t)T * k;
        if (k < 1 || k > 64 || E < 1 || E > 4096 || P > INT_MAX) {
            CHECK(s == 0 && n == 0);
        } else {
            if (P <= 1024) CHECK(s == 0);
            else CHECK(s % 16 == 0 && s >= (size_t)(P + 1023) / 1024 * (size_t)E * 4);
            if (H < 1 || I < 1 || H > 131071 || I > 131071 || P > 1 << 30) CHECK(n == 0);
            else CHECK(n % 16 == 0 && n >= s + (size_t)P * ((size_t)H + (size_t)I * 5));
        }
    }
    CHECK(seedmm_moe_i8_workspace_bytes(1 << 24, 64, 4096, 131071, 131071) > (size_t)1 << 46);
    CHECK(seedmm_moe_sort_workspace_bytes(INT_MAX, 1, 4096) > (size_t)1 << 34);
    CHECK(seedmm_moe_sort_workspace_bytes(-1, 1, 4) == 0 && seedmm_moe_i8_workspace_bytes(-1, 1, 4, 8, 8) == 0);
    // argument errors and empty calls: each returns before any HIP call
    const int S = SEEDMM_F32, B = SEEDMM_BF16, C = SEEDMM_I8;
    CHECK(seedmm_i8_gemv(W, X, S, 1, nullptr, W, 64, X, X, S, 64, INT_MAX, 64, 1, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_i8_gemv(W, X, S, 1, nullptr, W, INT64_MAX, X, X, S, INT64_MAX, 64, 131072, 1, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_i8_gemv(W, X, S, 2, nullptr, W, 64, X, X, S, 64, 64, 64, 1, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_i8_gemv(W, X, S, 4097, I32, W, 64, X, X, S, 64, 64, 64, 1, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_i8_gemv(W, F + 2, S, 1, nullptr, W, 64, X, X, S, 64, 64, 64, 1, nullptr) == SEEDMM_EALIGN);
    CHECK(seedmm_i8_gemv(W, F + 1, B, 1, nullptr, W, 64, X, X, S, 64, 64, 64, 1, nullptr) == SEEDMM_EALIGN);
    CHECK(seedmm_i8_gemv(nullptr, nullptr, S, 1, nullptr, nullptr, 64, nullptr, nullptr, S, 64, 64, 64, 0, nullptr) == SEEDMM_OK);
    CHECK(seedmm_moe_sort(I32, INT_MAX, 2, 4, F, B, 8, nullptr, F, 8, nullptr, 8, I32, I32, F, 1 << 20, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_moe_sort(I32, INT_MAX, 1, 4, F, B, 8, nullptr, F, 8, nullptr, 8, I32, I32, F, 1 << 10, nullptr) == SEEDMM_EWORKSPACE);
    CHECK(seedmm_moe_sort(I32, 5000, 1, 4, F, B, 8, nullptr, F, 8, nullptr, 8, I32, I32, F + 4, 1 << 20, nullptr) == SEEDMM_EALIGN);
    CHECK(seedmm_moe_sort(I32, 5, 1, 4, F, B, 8, X, F, 8, nullptr, 8, I32, I32, nullptr, 0, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_moe_sort(I32, 5, 1, 4, F + 1, B, 8, nullptr, F, 8, nullptr, 8, I32, I32, nullptr, 0, nullptr) == SEEDMM_EALIGN);
    CHECK(seedmm_moe_unsort(F, B, INT64_MAX, INT_MAX, I32, X, F, S, INT64_MAX, 4, 65, 8, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_moe_unsort(F, C, 8, 8, I32, X, F, S, 8, 4, 2, 8, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_moe_unsort(nullptr, B, 8, 8, nullptr, nullptr, nullptr, S, 8, 0, 2, 8, nullptr) == SEEDMM_OK);
    CHECK(seedmm_moe_unsort_grad(F, S, 8, F, B, 8, 8, I32, X, F, 16, X, 4, 2, 8, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_moe_unsort_grad(F, S, 8, F, B, 8, 8, I32, X, nullptr, 0, nullptr, 4, 2, 8, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_moe_unsort_grad(F, S, 8, F, B, 8, 8, I32, nullptr, F, 8, X, 4, 2, 8, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_swiglu(F, B, INT64_MAX, F, B, INT64_MAX, nullptr, nullptr, 4, INT_MAX, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_swiglu(F, B, 16, F, C, 8, nullptr, nullptr, 4, 8, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_swiglu(F, B, 16, F, B, 8, X, nullptr, 4, 8, nullptr) == SEEDMM_EINVAL);
    const seedmm_i8mat m = {W, X, S}, none = {nullptr, X, S}, bad = {W, X, C};
    CHECK(seedmm_moe_i8(I32, X, 4, 2, W, X, X, 8, 64, 32, m, m, F, 16, nullptr) == SEEDMM_EWORKSPACE);
    CHECK(seedmm_moe_i8(I32, X, 4, 2, W, X, X, 8, 64, 32, none, m, F, 1 << 20, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_moe_i8(I32, X, 4, 2, W, X, X, 8, 64, 32, m, bad, F, 1 << 20, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_moe_i8(I32, X, INT_MAX, 2, W, X, X, 8, 64, 32, m, m, F, (size_t)-1, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_moe_i8(I32, X, 4, 2, W, X, X, 8, 64, 32, m, m, F + 8, 1 << 20, nullptr) == SEEDMM_EALIGN);
    printf("clean\n");
    return 0;
}
