// What the sources of the dense operators and of the 8-bit experts share: vector types and
// conversions, reductions over a wave, pieces of rows, and the launches' host helpers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/seedmm.h"

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t f32_to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// ----------------------------------------------------------------------------------
// Reductions over a wave in vector registers: exchanges within 16 lanes (quads by 1 and 2,
// then mirrored halves), then between the four 16-lane rows.
// ----------------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

template <typename F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, F f) {
    v = f(v, dpp<0xB1>(v));    // lane ^ 1
    v = f(v, dpp<0x4E>(v));    // lane ^ 2
    v = f(v, dpp<0x141>(v));   // 7 - lane of 8
    v = f(v, dpp<0x140>(v));   // 15 - lane of 16
    auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = f(a[0], a[1]);
    auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return f(b[0], b[1]);
}

__device__ __forceinline__ float wave_sum(float v) {
    return __uint_as_float(wave_reduce(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}
__device__ __forceinline__ float wave_max(float v) {
    return __uint_as_float(wave_reduce(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
    return wave_reduce(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ uint32_t wave_umin(uint32_t v) {
    return wave_reduce(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}

// 8 elements from index i, of which the first n (1 .. 8) exist (the others read as 0).  The
// vector accesses need the alignment of one element only.
template <int DT>
struct Eight {
    uint32_t u[DT == SEEDMM_F32 ? 8 : 4];
    __device__ __forceinline__ void load(const void* p, int64_t i, int n) {
        const char* at = (const char*)p + i * (DT == SEEDMM_F32 ? 4 : 2);
        if (n >= 8) {
            __builtin_memcpy(u, at, sizeof(u));
        } else {
#pragma unroll
            for (int j = 0; j < (int)(sizeof(u) / 4); ++j) u[j] = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) {
                    if constexpr (DT == SEEDMM_F32) u[j] = ((const uint32_t*)at)[j];
                    else u[j / 2] |= (uint32_t)((const uint16_t*)at)[j] << (16 * (j & 1));
                }
        }
    }
    __device__ __forceinline__ float get(int j) const {
        if constexpr (DT == SEEDMM_F32) return __uint_as_float(u[j]);
        else return __uint_as_float((j & 1) ? u[j / 2] & 0xFFFF0000u : u[j / 2] << 16);
    }
};

template <int DT>
__device__ __forceinline__ void store8(void* p, int64_t i, int n, const float (&v)[8]) {
    constexpr int B = DT == SEEDMM_F32 ? 4 : DT == SEEDMM_BF16 ? 2 : 1;
    uint32_t u[2 * B];
    if constexpr (DT == SEEDMM_F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(v[j]);
    } else if constexpr (DT == SEEDMM_BF16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = (uint32_t)f32_to_bf16(v[2 * j]) | (uint32_t)f32_to_bf16(v[2 * j + 1]) << 16;
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            u[j] = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) u[j] |= ((uint32_t)(int)v[4 * j + k] & 255u) << (8 * k);
        }
    }
    char* at = (char*)p + i * B;
    if (n >= 8) {
        __builtin_memcpy(at, u, sizeof(u));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) {
                if constexpr (DT == SEEDMM_F32) ((uint32_t*)at)[j] = u[j];
                else if constexpr (DT == SEEDMM_BF16) ((uint16_t*)at)[j] = (uint16_t)(u[j / 2] >> (16 * (j & 1)));
                else ((uint8_t*)at)[j] = (uint8_t)(u[j / 4] >> (8 * (j & 3)));
            }
    }
}

__device__ __forceinline__ float code_of(float v, float inv) {
    return inv == 0.f ? 0.f : fminf(fmaxf(rintf(v * inv), -127.f), 127.f);
}

// ---- host ------------------------------------------------------------------------
size_t align_up(size_t v) { return (v + 255) & ~(size_t)255; }
bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
int launch_status() { return hipGetLastError() == hipSuccess ? SEEDMM_OK : SEEDMM_EHIP; }

// HIP takes fewer than 2^32 threads of a grid in one dimension: larger calls are launched in
// parts of this many, over rows or tokens.
constexpr int64_t kLaunchThreads = 1 << 30;
int64_t type_bytes(int dt) { return dt == SEEDMM_F32 ? 4 : dt == SEEDMM_BF16 ? 2 : 1; }

bool float_type(int dt) { return dt == SEEDMM_F32 || dt == SEEDMM_BF16; }

}  // namespace
