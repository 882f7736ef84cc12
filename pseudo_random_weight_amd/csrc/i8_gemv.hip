// i8_gemv.hip -- gfx950 kernels of the product of 8-bit integers with a scale a row and a
// channel (seedmm_i8_gemv), for one matrix or one an expert, and their C ABI.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

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

// ----------------------------------------------------------------------------------
// Many rows.  A workgroup of four waves takes 256 channels by TN = 64 NB rows, each wave 128
// channels by 32 NB rows in 32 x 32 x 32 instructions (two by two waves), K in steps of 128
// bytes.  Both operands pass through LDS in two buffers: a step's are loaded to registers two
// steps ahead and written one step ahead, so that one barrier a step is enough, and it stands in
// front of the step's last quarter, whose operands are in registers: the matrix unit has work
// while the next step's first operands are read.
//
// LDS holds rows of 128 bytes in 16-byte pieces; piece c of row r lies at c ^ (r / 2 % 8), so
// that 16 lanes reading a piece of 16 rows (and writing two rows) meet 64 different banks.
//
// Columns past K: a piece that would pass the row's end is loaded from the row's last 16 bytes,
// in both operands alike, and the bytes of x in it that belong to earlier pieces are zeroed.
// ----------------------------------------------------------------------------------
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

constexpr int kStep = 128;             // bytes of K
constexpr int kTileM = 256, kTileN = 256;
constexpr int kPiece = 32 * 128;       // a wave's 32 rows of 64 channels in bf16, or of 32 in fp32

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}

// LDS accesses of one wave keep their order across this point (they run in order; the
// compiler must not exchange them).
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

typedef __attribute__((address_space(3))) void* lds_ptr;

#define INLINE __attribute__((always_inline))

// f(0), f(1), ... f(N - 1) with constants, so that what they index stays in registers
template <typename F, int... I>
__device__ __forceinline__ void each_of(F f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F f) {
    each_of(f, std::make_integer_sequence<int, N>{});
}

// A buffer of `bytes` bytes from a uniform address: loads take a lane's 32-bit offset and a
// uniform one, and give zeros past the end.
#ifdef __HIP_DEVICE_COMPILE__
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, bytes, 0x00020000);
}
#endif

// A tile: where its operands lie, and the offsets of this thread's pieces in them.
struct WideTile {
    Rows r;
    int64_t m0;
    int mrows;
};

#ifdef __HIP_DEVICE_COMPILE__
struct WideBuffers {
    __amdgpu_buffer_rsrc_t w, x;
};
__device__ __forceinline__ WideBuffers wide_buffers(const I8Args& a, const WideTile& t) {
    return {buffer(a.w + ((int64_t)t.r.e * a.M + t.m0) * a.K, (uint32_t)t.mrows * (uint32_t)a.K),
            buffer(a.x + (int64_t)t.r.row0 * a.ldx, (uint32_t)(t.r.n - 1) * (uint32_t)a.ldx + (uint32_t)a.K)};
}
#endif

__device__ __forceinline__ WideTile wide_tile(const I8Args& a, int64_t tile, int64_t tiles) {
    WideTile t = {{0, 0, 0}, 0, 0};
    if (tile >= tiles) return t;
    t.r = find_rows(a, tile / a.tm, kTileN);
    t.m0 = tile % a.tm * kTileM;
    t.mrows = a.M - t.m0 < kTileM ? (int)(a.M - t.m0) : kTileM;
    return t;
}

template <bool BF, bool SF32>     // y in bf16, else fp32; scales in fp32, else bf16
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void k_i8_wide(const I8Args a, int64_t tiles) {
#ifdef __HIP_DEVICE_COMPILE__      // buffer resources and LDS loads have no host form
    constexpr int NB = 4, LW = kTileM / 32, L = LW + kTileN / 32, P = 4 * NB, O = 4 + NB;   // loads, products, operands
    __shared__ __align__(16) char w0[kTileM * kStep], w1[kTileM * kStep], x0[kTileN * kStep], x1[kTileN * kStep];
    __shared__ __align__(16) char pieces[2][4 * kPiece];
    int64_t tile = blockIdx.x;
    WideTile cur = wide_tile(a, tile, tiles);
    if (cur.r.n == 0) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    // This thread's pieces: of the rows lr + 32 i, the one that lies at lane % 8.  Rows that a tile
    // does not have lie behind its buffer.
    const int lr = tid >> 3, lc = (tid & 7) ^ (lr >> 1 & 7);
    int at[L];
#pragma unroll
    for (int i = 0; i < L; ++i) at[i] = (i < LW ? (lr + 32 * i) * a.K : (lr + 32 * (i - LW)) * (int)a.ldx) + 16 * lc;
    // the lane's operands: piece 2 s + lane / 32 of row lane % 32 of each block of 32
    const int h = lane >> 5, fr = lane & 31;
    const int wget = (wm * 128 + fr) * kStep, xget = (wn * 128 + fr) * kStep;
    const int real = (a.K + kStep - 1) / kStep, steps = (real + 1) & ~1;

    i32x16 acc[4][NB];
    i32x4 wf[2][4], xf[2][NB];
    // Of a tile's step t, piece n (0 .. L - 1) of this thread's.  Columns past K are zero in x: their
    // offset lies behind the buffer (the step's own stays inside of it).
    auto load = [&](const WideBuffers& d, int t, char* w, char* x, auto n) INLINE {
        constexpr int i = n;
        const int k = min(t, real - 1) * kStep;
        if constexpr (i < LW) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(d.w, (lds_ptr)(w + i * 32 * kStep + wave * 1024), 16, at[i], k, 0, 0);
        } else {
            const int past = t * kStep + 16 * lc < a.K ? 0 : (int)0x80000000;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(d.x, (lds_ptr)(x + (i - LW) * 32 * kStep + wave * 1024), 16, at[i] | past, k, 0, 0);
        }
    };
    auto fetch = [&](const char* w, const char* x, int s, int to, auto n) INLINE {   // n: 0 .. 3 + NB
        constexpr int i = n;
        const int p = ((2 * s + h) ^ (fr >> 1 & 7)) * 16;
        if constexpr (i < 4) wf[to][i] = *(const i32x4*)(w + wget + p + i * 32 * kStep);
        else xf[to][i - 4] = *(const i32x4*)(x + xget + p + (i - 4) * 32 * kStep);
    };
    // Every wave's loads of the next step have landed, and its reads of this step are done.
    auto arrive = [&]() INLINE { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
    constexpr std::integral_constant<int, 0> c0;
    constexpr std::integral_constant<int, 1> c1;
    constexpr std::integral_constant<int, -1> none;
    WideBuffers now = wide_buffers(a, cur);
    each<L>([&](auto i) INLINE { load(now, 0, w0, x0, i); });
    each<L / 2>([&](auto i) INLINE { load(now, 1, w1, x1, i); });
    arrive();
    each<O>([&](auto i) INLINE { fetch(w0, x0, 0, 0, i); });
    // A quarter of a step: its products, and in their shadow the next quarter's operands (read
    // from w and x) over the first half of them and, for HALF 0 or 1, that half of the loads of
    // d's step t to tw and tx over the second, in this order.
    auto quarter = [&](const char* w, const char* x, int s, auto from, auto half, const WideBuffers& d, int t, char* tw, char* tx) INLINE {
        each<P>([&](auto n) INLINE {
            constexpr int p = n, F = from, HALF = half;
            acc[p / NB][p % NB] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[F][p / NB], xf[F][p % NB], acc[p / NB][p % NB], 0, 0, 0);
            each<O>([&](auto i) INLINE {
                if constexpr (i * P / (2 * O) == p) fetch(w, x, s, F ^ 1, i);
            });
            if constexpr (HALF >= 0)
                each<L / 2>([&](auto i) INLINE {
                    if constexpr (P / 2 + i * P / L == p) load(d, t, tw, tx, std::integral_constant<int, HALF * (L / 2) + i>{});
                });
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // a step from (w, x); meanwhile the second half of d1's step t1 and the first of d2's t2
    auto step = [&](char* w, char* x, char* nw, char* nx, const WideBuffers& d1, int t1, const WideBuffers& d2, int t2) INLINE {
        quarter(w, x, 1, c0, c1, d1, t1, nw, nx);
        quarter(w, x, 2, c1, none, d1, 0, nw, nx);
        quarter(w, x, 3, c0, none, d1, 0, nw, nx);
        arrive();
        quarter(nw, nx, 0, c1, c0, d2, t2, w, x);
    };
    for (;;) {
        const WideTile next = wide_tile(a, tile + gridDim.x, tiles);
        const WideBuffers then = next.r.n ? wide_buffers(a, next) : now;
        // the scales of the lane's channels and rows (0 where the tile has none)
        f32x4 s[4][4];
        float sx[NB];
        const auto sbuf = buffer((const char*)a.s + ((int64_t)cur.r.e * a.M + cur.m0) * (SF32 ? 4 : 2), cur.mrows * (SF32 ? 4 : 2));
        const auto sxbuf = buffer(a.xs + cur.r.row0, cur.r.n * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int m = wm * 128 + 4 * h + i * 32 + 8 * g;
                if constexpr (SF32) {
                    s[i][g] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(sbuf, m * 4, 0, 0));
                } else {
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        s[i][g][v] = bf16_to_f32((uint16_t)__builtin_amdgcn_raw_buffer_load_b16(sbuf, (m + v) * 2, 0, 0));
                }
            }
#pragma unroll
        for (int j = 0; j < NB; ++j)
            sx[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(sxbuf, (wn * 128 + j * 32 + fr) * 4, 0, 0));
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[i][j] = i32x16{};
        for (int t = 0; t < steps; t += 2) {      // a step past the last one multiplies zeros
            const bool last = t + 2 >= steps;     // then the next tile's steps 0 and 1 are loaded
            const WideBuffers d = last ? then : now;
            const int t2 = last ? 0 : t + 2;
            step(w0, x0, w1, x1, now, t + 1, d, t2);
            step(w1, x1, w0, x0, d, t2, d, t2 + 1);
        }
        // Each wave's sums through its own pieces of LDS, so that whole lines of y are written: rows of
        // 128 bytes, 16-byte pieces permuted by the row, so that 16 lanes meet all banks.  One piece
        // is filled while the other is written out.
        const int mleft = cur.mrows - wm * 128;                // of this wave's 128 channels
        const int64_t corner = ((int64_t)cur.r.row0 + wn * 128) * a.ldy + cur.m0 + wm * 128;
        const int nleft = cur.r.n - wn * 128;
        int l = lane;
        asm volatile("" : "+v"(l));        // addresses of this part are not kept through the loop
        const int fr = l & 31, h = l >> 5, c = l & 7, rr = l >> 3;
        constexpr int B = BF ? 2 : 4, CH = 128 / B, PH = NB * 128 / CH;     // phases of CH channels by 32 rows
        auto fill = [&](auto n) INLINE {
            constexpr int j = n / (128 / CH), k = n % (128 / CH);
            char* piece = pieces[n & 1] + wave * kPiece + fr * 128;
            each<CH / 8>([&](auto qq) INLINE {
                constexpr int q = qq, i = k * CH / 32 + q / 4, g = q % 4;
                f32x4 f;
#pragma unroll
                for (int v = 0; v < 4; ++v) f[v] = (float)acc[i][j][4 * g + v] * sx[j] * s[i][g][v];
                // rows 16 .. 31 have the halves of a bf16 piece exchanged
                if constexpr (BF)
                    *(u32x2*)(piece + (q ^ (fr >> 1 & 7)) * 16 + (h ^ (fr >> 4)) * 8) = u32x2{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
                else
                    *(f32x4*)(piece + ((2 * q + h) ^ (fr >> 1 & 7)) * 16) = f;
            });
        };
        const bool whole = mleft >= 128;
        const uint32_t bytes = nleft > 0 && mleft > 0 ? (uint32_t)(((nleft - 1) * (int)a.ldy + min(mleft, 128)) * B) : 0;
        const auto ybuf = buffer((char*)a.y + corner * B, bytes);     // rows that the tile does not have lie behind it
        const int yat = rr * (int)a.ldy * B + c * 16;
        auto write = [&](auto n) INLINE {
            constexpr int j = n / (128 / CH), k = n % (128 / CH);
            const char* piece = pieces[n & 1] + wave * kPiece;
            if (whole) {
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                    const int r = it * 8 + rr;
                    u32x4 o = *(const u32x4*)(piece + r * 128 + (c ^ (r >> 1 & 7)) * 16);
                    if (BF && it >= 2) o = u32x4{o[2], o[3], o[0], o[1]};
                    __builtin_amdgcn_raw_buffer_store_b128(o, ybuf, yat + (j * 32 + it * 8) * (int)a.ldy * B + k * 128, 0, 0);
                }
            } else {                                  // the last channels: one at a time
#pragma nounroll
                for (int e = l; e < 32 * CH; e += 64) {
                    const int r = e / CH, m = e % CH, q = m * B / 16, in = m * B % 16;
                    const char* from = piece + r * 128 + (q ^ (r >> 1 & 7)) * 16 + (BF ? in ^ (r >> 4) * 8 : in);
                    const int to = k * CH + m < mleft ? (j * 32 + r) * (int)a.ldy * B + k * 128 + m * B : (int)0x80000000;
                    if constexpr (BF) __builtin_amdgcn_raw_buffer_store_b16(*(const uint16_t*)from, ybuf, to, 0, 0);
                    else __builtin_amdgcn_raw_buffer_store_b32(*(const uint32_t*)from, ybuf, to, 0, 0);
                }
            }
        };
        if (nleft > 0 && mleft > 0) {
            fill(c0);
            each<PH>([&](auto n) INLINE {
                wave_order();
                if constexpr (n + 1 < PH) fill(std::integral_constant<int, n + 1>{});
                write(n);
            });
        }
        if (!next.r.n) break;
        cur = next;
        now = then;
        tile += gridDim.x;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");     // loads to LDS end before the workgroup does
#endif
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
    const bool aligned = aligned16(weight) && aligned16(x) && K % 16 == 0 && ldx % 16 == 0;
    if (N >= 128 && aligned && K >= 16 && ldx <= 1 << 22 && ldy <= 1 << 20) {
        a.tm = (M - 1) / kTileM + 1;
        tn = ((int64_t)N + kTileN - 1) / kTileN;
        if (offsets) tn = N / kTileN + (E < N ? E : N);
        const int64_t tiles = tn * a.tm;
        const dim3 grid((unsigned)(tiles < 256 ? tiles : 256));
        if (a.y_bf16) {
            if (a.s_f32) hipLaunchKernelGGL((k_i8_wide<true, true>), grid, dim3(256), 0, st, a, tiles);
            else hipLaunchKernelGGL((k_i8_wide<true, false>), grid, dim3(256), 0, st, a, tiles);
        } else {
            if (a.s_f32) hipLaunchKernelGGL((k_i8_wide<false, true>), grid, dim3(256), 0, st, a, tiles);
            else hipLaunchKernelGGL((k_i8_wide<false, false>), grid, dim3(256), 0, st, a, tiles);
        }
        return launch_status();
    }
    for (a.first = 0; a.first < tiles; a.first += most)
        hipLaunchKernelGGL(k_i8_tile, dim3((unsigned)(tiles - a.first < most ? tiles - a.first : most)), dim3(256), 0, st, a);
    return launch_status();
}

}  // extern "C"
