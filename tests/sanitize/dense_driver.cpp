// Sanitizer driver for the host side of the dense operators (test infrastructure): argument
// validation, the size functions and the plans behind them over many sizes, none of which
// touches a GPU.  Exit status 0 = clean.
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/seedmm.h"

#define CHECK(c) do { if (!(c)) { fprintf(stderr, "check failed: %s (line %d)\n", #c, __LINE__); return 1; } } while (0)

static uint64_t rng = 0xBEEFu;
static uint32_t next32() {
    rng ^= rng >> 12; rng ^= rng << 25; rng ^= rng >> 27;
    return (uint32_t)((rng * 2685821657736338717ull) >> 32);
}

int main() {
    void* F = (void*)(uintptr_t)0x100000;   // aligned, never dereferenced (validation fails first)
    const uint32_t* W = (const uint32_t*)F;
    float* X = (float*)F;
    // sizes: none for few rows; fp32 and many rows are laid out
    for (int i = 0; i < 200000; ++i) {
        const int group = 32 << next32() % 3, dt = next32() % 3;
        const int K = group * (int)(next32() % 600), M = (int)(next32() % 200000), N = (int)(next32() % 5000);
        const size_t n = seedmm_q4_workspace_bytes(dt, group, M, K, N);
        const int pl = dt == SEEDMM_F32 ? 3 : 1;
        if (N * pl <= 16 || M == 0 || K == 0) CHECK(n == 0);
        else CHECK(n % 256 == 0);
        if (N * pl > 16 && M && K && (pl == 3 || (N >= 4096 && M >= 1024))) CHECK(n >= (size_t)pl * N * K * 2);
    }
    CHECK(seedmm_q4_workspace_bytes(SEEDMM_BF16, 64, 1 << 30, 1 << 30, 1 << 30) > ((size_t)1 << 40));
    CHECK(seedmm_q4_workspace_bytes(SEEDMM_BF16, 48, 64, 96, 64) == 0);
    // argument errors: each returns before any HIP call
    CHECK(seedmm_q4_gemv(W, F, F, SEEDMM_BF16, 64, F, SEEDMM_BF16, 64, nullptr, F, SEEDMM_F32, 16, 16, 96, 1, nullptr, 0, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_q4_gemv(W, F, F, SEEDMM_BF16, 64, F, SEEDMM_BF16, 2048, nullptr, F, SEEDMM_F32, 16, 16, 2048, 99, nullptr, 0, nullptr) == SEEDMM_EWORKSPACE);
    CHECK(seedmm_q4_gemv(W, F, F, SEEDMM_BF16, 64, (char*)F + 8, SEEDMM_BF16, 64, nullptr, F, SEEDMM_F32, 16, 16, 64, 1, nullptr, 0, nullptr) == SEEDMM_EALIGN);
    // more than 2^31 tiles
    CHECK(seedmm_q4_gemv(W, F, F, SEEDMM_BF16, 64, F, SEEDMM_BF16, 64, nullptr, F, SEEDMM_F32, 1 << 30, 1 << 30, 64, 1 << 30, F, (size_t)-1, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_q4_workspace_bytes(SEEDMM_BF16, 64, 64, 64, 0x7FFFFFFF) == 0);
    CHECK(seedmm_add_norm(F, SEEDMM_F32, 8, nullptr, 0, 0, nullptr, 0, NAN, nullptr, 0, F, SEEDMM_F32, 8, nullptr, 1, 8, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_add_norm(F, SEEDMM_F32, 8, nullptr, 0, 0, nullptr, 0, 1e-6f, nullptr, 0, F, SEEDMM_I8, 8, nullptr, 1, 8, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_add_norm(F, SEEDMM_BF16, 8, (char*)F + 1, SEEDMM_BF16, 8, nullptr, 0, 1e-6f, nullptr, 0, F, SEEDMM_F32, 8, nullptr, 1, 8, nullptr) == SEEDMM_EALIGN);
    CHECK(seedmm_route(F, SEEDMM_F32, 8, nullptr, 2, 1, 8, 2, (int32_t*)F, X, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_route(F, SEEDMM_F32, 8, X, SEEDMM_SOFTMAX, 1, 8, 2, (int32_t*)F, X, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_route(F, SEEDMM_F32, 8, nullptr, SEEDMM_SOFTMAX, 1, 8, 2, nullptr, X, nullptr) == SEEDMM_EINVAL);
    seedmm_mat m = {(const uint16_t*)F, (const uint16_t*)F, (const uint8_t*)F, (const int32_t*)F};
    seedmm_block b = {F, W, F, F, nullptr, nullptr, m, m, m, 1e-6f, SEEDMM_BF16, SEEDMM_BF16, 64, SEEDMM_SOFTMAX, 2, 8, 64, 32, 4};
    for (int T = 0; T < 3000; T += 7) {
        const size_t n = seedmm_moe_block_workspace_bytes(&b, T);
        CHECK(n >= seedmm_moe_workspace_bytes(T, 2, 8, 64, 32) + seedmm_q4_workspace_bytes(SEEDMM_BF16, 64, 8, 64, T));
    }
    CHECK(seedmm_moe_block(nullptr, F, 0, nullptr, 0, X, nullptr, nullptr, 1, F, 1 << 20, nullptr, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_moe_block(&b, F, 0, nullptr, 0, X, nullptr, nullptr, 4, F, 16, nullptr, nullptr) == SEEDMM_EWORKSPACE);
    CHECK(seedmm_moe_block(&b, F, 0, nullptr, 0, X, nullptr, nullptr, 0, nullptr, 0, nullptr, nullptr) == SEEDMM_OK);
    b.top_k = 9;
    CHECK(seedmm_moe_block(&b, F, 0, nullptr, 0, X, nullptr, nullptr, 4, F, 1 << 20, nullptr, nullptr) == SEEDMM_EINVAL);
    CHECK(seedmm_moe_block_workspace_bytes(&b, -1) == 0);
    printf("clean\n");
    return 0;
}
