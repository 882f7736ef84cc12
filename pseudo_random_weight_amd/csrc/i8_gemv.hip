// i8_gemv.hip -- gfx950 kernels of the product of 8-bit integers with a scale a row and a
// channel (seedmm_i8_gemv), for one matrix or one an expert, and their C ABI.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/seedmm.h"
#include "device_rows.hpp"

namespace {

constexpr int kMaxDim = 1 << 30;
constexpr int kMaxSum = 131071;      // K: 128 * 128 * K stays below 2^31
constexpr int kMaxExperts = 4096;

struct I8Args {
    const int8_t* w;          // [E][M][K]
    const void* s;            // [E][M]
    const int32_t* offsets;   // [E + 1] or null
    const int8_t* x;          // [N][ldx]
    const float* xs;          // [N]
    void* y;                  // [N][ldy]
    int64_t ldx, ldy, first;  // tiles from `first` on
    int E, M, K, N, tm;       // tm: tiles of channels
    int s_f32, y_bf16;
};

// The rows of a tile: those of one expert.
struct Rows {
    int e, row0, n;
};

__device__ __forceinline__ int clamp_row(int32_t v, int N) { return v < 0 ? 0 : v < N ? v : N; }

// Tile j of `tile` rows, counting each expert's tiles in turn; n = 0 past the last one.  Every
// wave finds it for itself: 64 experts at a time, their tile counts summed over the lanes.
__device__ __forceinline__ Rows find_rows(const I8Args& a, int64_t j, int tile) {
    if (!a.offsets) {
        const int64_t r = j * tile;
        return {0, (int)r, r >= a.N ? 0 : (int)(a.N - r < tile ? a.N - r : tile)};
    }
    const int lane = threadIdx.x & 63;
    int64_t front = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e < a.E) {
            lo = clamp_row(a.offsets[e], a.N);
            hi = clamp_row(a.offsets[e + 1], a.N);
        }
        const int tiles = hi > lo ? (hi - lo - 1) / tile + 1 : 0;
        int upto = tiles;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(upto, d);
            if (lane >= d) upto += o;
        }
        const unsigned long long past = __ballot(front + upto > j);
        if (past) {
            const int l = __builtin_ctzll(past);
            const int64_t in = j - front - (__shfl(upto, l) - __shfl(tiles, l));
            const int r0 = __shfl(lo, l) + (int)in * tile, end = __shfl(hi, l);
            return {__builtin_amdgcn_readfirstlane(e0 + l), __builtin_amdgcn_readfirstlane(r0),
                    __builtin_amdgcn_readfirstlane(end - r0 < tile ? end - r0 : tile)};
        }
        front += __shfl(upto, 63);
    }
    return {0, 0, 0};
}

// 16 bytes from column k of a row, zeros past K.  Any alignment.
__device__ __forceinline__ u32x4 load16(const int8_t* row, int k, int K) {
    u32x4 v = {0, 0, 0, 0};
    if (k + 16 <= K) {
        __builtin_memcpy(&v, row + k, 16);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (k + i < K) v[i / 4] |= (uint32_t)(uint8_t)row[k + i] << (8 * (i & 3));
    }
    return v;
}

// A tile of 64 channels by 64 rows; each of four waves a quarter of it in 16 x 16 x 64
// instructions, both operands through LDS.
__global__ __launch_bounds__(256) void k_i8_tile(const I8Args a) {
    __shared__ u32x4 ws[64][5], xs[64][5];
    const int64_t b = a.first + blockIdx.x;
    const Rows r = find_rows(a, b / a.tm, 64);
    if (r.n == 0) return;
    const int64_t m0 = b % a.tm * 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int c = lane & 15, q = lane >> 4, wm = wave & 1, wn = wave >> 1;
    const int lr = tid >> 2, lc = tid & 3;
    const int8_t* wrow = a.w + ((int64_t)r.e * a.M + (m0 + lr < a.M ? m0 + lr : a.M - 1)) * a.K;
    const int8_t* xrow = a.x + (r.row0 + (int64_t)(lr < r.n ? lr : r.n - 1)) * a.ldx;
    i32x4 acc[2][2] = {};
    for (int k0 = 0; k0 < a.K; k0 += 64) {
        const u32x4 wv = load16(wrow, k0 + 16 * lc, a.K), xv = load16(xrow, k0 + 16 * lc, a.K);
        __syncthreads();
        ws[lr][lc] = wv;
        xs[lr][lc] = xv;
        __syncthreads();
        i32x4 wf[2], xf[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            wf[i] = __builtin_bit_cast(i32x4, ws[wm * 32 + i * 16 + c][q]);
            xf[i] = __builtin_bit_cast(i32x4, xs[wn * 32 + i * 16 + c][q]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[i], xf[j], acc[i][j], 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int n = wn * 32 + j * 16 + c;
        if (n >= r.n) continue;
        const float sx = a.xs[r.row0 + (int64_t)n];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int64_t m = m0 + wm * 32 + i * 16 + q * 4 + v;
                if (m >= a.M) continue;
                const int64_t at = (int64_t)r.e * a.M + m;
                const float s = a.s_f32 ? ((const float*)a.s)[at] : bf16_to_f32(((const uint16_t*)a.s)[at]);
                const float f = (float)acc[i][j][v] * sx * s;
                const int64_t o = (r.row0 + (int64_t)n) * a.ldy + m;
                if (a.y_bf16) ((uint16_t*)a.y)[o] = f32_to_bf16(f);
                else ((float*)a.y)[o] = f;
            }
    }
}

}  // namespace

extern "C" {

int seedmm_i8_gemv(const int8_t* weight, const void* scales, int s_dtype, int E,
                   const int32_t* offsets, const int8_t* x, int64_t ldx, const float* x_scale,
                   void* y, int y_dtype, int64_t ldy, int M, int K, int N, void* hip_stream) {
    if (M < 0 || K < 0 || N < 0 || M > kMaxDim || N > kMaxDim || K > kMaxSum || E < 1 || E > kMaxExperts)
        return SEEDMM_EINVAL;
    if ((!offsets && E != 1) || ldx < K || ldy < M || !float_type(s_dtype) || !float_type(y_dtype)) return SEEDMM_EINVAL;
    if (M == 0 || N == 0) return SEEDMM_OK;
    if (!scales || !x_scale || !y || (K > 0 && (!weight || !x))) return SEEDMM_EINVAL;
    if (((uintptr_t)scales & (s_dtype == SEEDMM_F32 ? 3 : 1)) || ((uintptr_t)x_scale & 3) || ((uintptr_t)offsets & 3) ||
        ((uintptr_t)y & (y_dtype == SEEDMM_F32 ? 3 : 1)))
        return SEEDMM_EALIGN;
    I8Args a = {weight, scales, offsets, x, x_scale, y, ldx, ldy, 0, E, M, K, N, (M - 1) / 64 + 1,
                s_dtype == SEEDMM_F32, y_dtype == SEEDMM_BF16};
    hipStream_t st = (hipStream_t)hip_stream;
    // an expert's last tile may be partly filled: one more tile each, at most one a row
    int64_t tn = ((int64_t)N + 63) / 64;
    if (offsets) tn = N / 64 + (E < N ? E : N);
    const int64_t tiles = tn * a.tm, most = kLaunchThreads / 256;
    for (a.first = 0; a.first < tiles; a.first += most)
        hipLaunchKernelGGL(k_i8_tile, dim3((unsigned)(tiles - a.first < most ? tiles - a.first : most)), dim3(256), 0, st, a);
    return launch_status();
}

}  // extern "C"
