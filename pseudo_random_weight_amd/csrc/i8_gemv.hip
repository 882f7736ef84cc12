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

// The sum over the lanes up to and with this one: within 16 lanes by shifts of 1, 2, 4 and 8, then
// each row's last lane added to the next row, and lane 31 to the upper half.
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
    return v;
}

// Where the search for a tile's expert goes on: `front` tiles belong to the experts below e0.
struct Seek {
    int e0 = 0;
    int64_t front = 0;
};

// Tile j of `tile` rows, counting each expert's tiles in turn; n = 0 past the last one.  Every
// wave finds it for itself: the tile counts of 64 experts are summed over the lanes, and the
// offsets of 256 are loaded at once.  `seek`: from an earlier tile on, for those that take several.
__device__ __forceinline__ Rows find_rows(const I8Args& a, int64_t j, int tile, Seek& seek) {
    if (!a.offsets) {
        const int64_t r = j * tile;
        return {0, (int)r, r >= a.N ? 0 : (int)(a.N - r < tile ? a.N - r : tile)};
    }
    const int lane = threadIdx.x & 63;
    for (; seek.e0 < a.E; seek.e0 += 256) {
        int lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = seek.e0 + 64 * i + lane;
            lo[i] = hi[i] = 0;
            if (e < a.E) {
                lo[i] = clamp_row(a.offsets[e], a.N);
                hi[i] = clamp_row(a.offsets[e + 1], a.N);
            }
        }
        int64_t front = seek.front;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (seek.e0 + 64 * i >= a.E) break;
            const int tiles = hi[i] > lo[i] ? (hi[i] - lo[i] - 1) / tile + 1 : 0;
            const int upto = wave_scan(tiles);
            const unsigned long long past = __ballot(front + upto > j);
            if (past) {
                const int l = __builtin_ctzll(past);
                const int64_t in = j - front - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(tiles, l));
                const int r0 = __builtin_amdgcn_readlane(lo[i], l) + (int)in * tile, end = __builtin_amdgcn_readlane(hi[i], l);
                return {seek.e0 + 64 * i + l, r0, end - r0 < tile ? end - r0 : tile};
            }
            front += __builtin_amdgcn_readlane(upto, 63);
        }
        seek.front = front;
    }
    return {0, 0, 0};
}
__device__ __forceinline__ Rows find_rows(const I8Args& a, int64_t j, int tile) {
    Seek seek;
    return find_rows(a, j, tile, seek);
}

// The tiles of all experts.
__device__ __forceinline__ int64_t count_tiles(const I8Args& a, int tile) {
    int64_t all = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        const int e = e0 + (threadIdx.x & 63);
        int n = 0;
        if (e < a.E) n = clamp_row(a.offsets[e + 1], a.N) - clamp_row(a.offsets[e], a.N);
        all += __builtin_amdgcn_readlane(wave_scan(n > 0 ? (n - 1) / tile + 1 : 0), 63);
    }
    return all;
}

#define INLINE __attribute__((always_inline))

// A table of 16-byte pieces in LDS with C of them a row, read by 16 lanes at a time from 16
// rows: the place of row `row`'s piece c, permuted so that the 16 lie in different banks
// (64 banks = 16 pieces, so 16 / C rows share a stretch of banks).
template <int C>
__device__ __forceinline__ int piece(int row, int c) {
    return row * C + (c ^ (row / (16 / C) & (C - 1)));
}

// LDS accesses of one wave keep their order across this point (they run in order; the
// compiler must not exchange them).
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Rows of fewer than 16 columns, which no 16-byte load fits: a tile of 64 channels by 64 rows, each of
// four waves a quarter of it in 16 x 16 x 64 instructions.  A thread loads a row, a byte at a time and
// zeros past K; the row is the first of the four pieces that an instruction takes, zeros the others.
// Bound by the outputs' writes, in single elements: 4096 rows of 8192 channels, 8 columns, 70 us; one row
// of 2^20 channels 31.
__global__ __launch_bounds__(256) void k_i8_tile(const I8Args a) {
    __shared__ u32x4 ws[64], xs[64];
    const int64_t b = a.first + blockIdx.x;
    const Rows r = find_rows(a, b / a.tm, 64);
    if (r.n == 0) return;
    const int64_t m0 = b % a.tm * 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int c = lane & 15, q = lane >> 4, wm = wave & 1, wn = wave >> 1;
    if (tid < 128) {
        const int lr = tid & 63;
        const int8_t* row = tid < 64 ? a.w + ((int64_t)r.e * a.M + (m0 + lr < a.M ? m0 + lr : a.M - 1)) * a.K
                                     : a.x + (r.row0 + (int64_t)(lr < r.n ? lr : r.n - 1)) * a.ldx;
        u32x4 v = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 15; ++i)
            if (i < a.K) v[i / 4] |= (uint32_t)(uint8_t)row[i] << (8 * (i & 3));
        (tid < 64 ? ws : xs)[lr] = v;
    }
    __syncthreads();
    i32x4 wf[2] = {}, xf[2] = {}, acc[2][2] = {};
    if (q == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            wf[i] = __builtin_bit_cast(i32x4, ws[wm * 32 + i * 16 + c]);
            xf[i] = __builtin_bit_cast(i32x4, xs[wn * 32 + i * 16 + c]);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[i], xf[j], acc[i][j], 0, 0, 0);
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
// Few rows: the weights are read once, at the memory's rate.  A wave takes 16 RM channels by
// 16 JN rows in 16 x 16 x 64 instructions, SB bytes of K a step; KW waves of a workgroup share a
// channel tile and take its steps in turn, the next step's loads in flight while one is
// multiplied.  Whole lines of the weights are loaded (SB / 16 lanes a row) and handed to the
// lanes that multiply them through the wave's own piece of LDS, and so are the activations of more
// than 16 rows; those of up to 16, which the caches hold, go straight to the lanes.  The sums are
// whole numbers: the waves' parts are added in LDS in any order.
//
// 131072 x 2048, 1 row: 45 us, 5.9 TB/s; 8 experts of 2048 x 2048: 8.2 us, 4.1 TB/s.  With more rows the load
// path binds: 61 x 5125 x 4150 (rows, M, K) 12.9 us; pieces of 64 bytes straight to the lanes took 18.9
// there and 28 for 64 x 8192 x 8192, which takes 21 now.
//
// Columns past K: as in the tiles of many rows, a piece that would pass the row's end is loaded
// from its last 16 bytes in both operands, and the bytes of x in it that belong to earlier
// pieces are zeroed.
// ----------------------------------------------------------------------------------
constexpr int kRowsWaves = 8;

// 16 bytes at any address.  Loads that do not start on 4 bytes take the memory path several times
// as long (61 x 5125 x 4150: 28.9 us where rows of 4160 took 11.5), so where rows may start anywhere
// (ODD) the aligned words that hold the 16 bytes are loaded and shifted; no other words are.  Up to 3
// bytes in front of and behind a tensor share a word with its own, are loaded and shifted out: a word lies
// in one page and one cache line, so these loads touch nothing that the tensor's do not.
template <bool ODD>
struct Bytes16 {
    u32x4 v;
    uint32_t over, by;
    // all: with the word behind the 16 bytes, if any of them lie in it
    __device__ __forceinline__ void load(const int8_t* p, bool all = true) {
        if constexpr (ODD) {
            by = (uint32_t)(uintptr_t)p & 3;
            const int8_t* at = p - by;
            v = *(const u32x4*)__builtin_assume_aligned(at, 4);
            if (all) over = *(const uint32_t*)(at + (by ? 16 : 12));
        } else {
            __builtin_memcpy(&v, __builtin_assume_aligned(p, 4), 16);
        }
    }
    // all: as loaded; else the word is the next lane's first (every lane calls)
    __device__ __forceinline__ u32x4 get(bool all = true) const {
        if constexpr (!ODD) return v;
        const uint32_t next = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v[0], 0x101, 0xF, 0xF, true);
        const uint32_t over = all ? this->over : next;
        u32x4 o;
        o[0] = __builtin_amdgcn_alignbyte(v[1], v[0], by);
        o[1] = __builtin_amdgcn_alignbyte(v[2], v[1], by);
        o[2] = __builtin_amdgcn_alignbyte(v[3], v[2], by);
        o[3] = __builtin_amdgcn_alignbyte(over, v[3], by);
        return o;
    }
};

template <int RM, int JN, int SB, int KW, bool ODD>
__global__ __launch_bounds__(kRowsWaves * 64, JN > 1 ? 2 : 4) void k_i8_rows(const I8Args a) {
    constexpr int RW = kRowsWaves / KW, C = SB / 16, LR = 64 / C, LW = RM * 16 / LR, S = SB / 64;
    constexpr int CH = RW * RM * 16, TK = JN * 16;          // channels and rows of the workgroup
    constexpr bool STAGED = JN > 1;                         // x through LDS, too
    constexpr int LX = STAGED ? TK / LR : JN * S;
    __shared__ u32x4 bounce[kRowsWaves][(RM * 16 + (STAGED ? TK : 0)) * C];
    __shared__ int32_t sums[TK][CH + 1];
    const int64_t tile = a.first + blockIdx.x;
    const Rows r = find_rows(a, tile / a.tm, TK);
    if (r.n == 0) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kw = wave % KW, rw = wave / KW;
    const int64_t mt = tile % a.tm * CH, m0 = mt + rw * RM * 16;
    for (int i = tid; i < TK * (CH + 1); i += kRowsWaves * 64) (&sums[0][0])[i] = 0;
    // loads: piece lc of channels (and rows) lr + LR i; operands: piece 4 s + q of channel or row c
    const int lr = lane / C, lc = lane % C, c = lane & 15, q = lane >> 4;
    const int8_t* w[LW];
#pragma unroll
    for (int i = 0; i < LW; ++i) {
        const int64_t m = m0 + lr + LR * i;
        w[i] = a.w + ((int64_t)r.e * a.M + (m < a.M ? m : a.M - 1)) * a.K;
    }
    const int8_t* x[STAGED ? LX : JN];
#pragma unroll
    for (int j = 0; j < (STAGED ? LX : JN); ++j)
        x[j] = a.x + (r.row0 + (int64_t)min(STAGED ? lr + LR * j : j * 16 + c, r.n - 1)) * a.ldx;
    Bytes16<ODD> wr[LW], xr[LX];
    // rows on any byte: the word behind a piece is the next lane's first, but for a row's last pieces of the
    // step or of K (131072 x 2049, 1 row: 59 us, 64 with every word loaded)
    auto own = [&](int k0) INLINE { return lc == C - 1 || k0 + 16 * lc + 32 > a.K; };
    auto load = [&](int k0) INLINE {
        const bool more = own(k0);
#pragma unroll
        for (int i = 0; i < LW; ++i) wr[i].load(w[i] + min(k0 + 16 * lc, a.K - 16), more);
        if constexpr (STAGED) {
#pragma unroll
            for (int j = 0; j < LX; ++j) xr[j].load(x[j] + min(k0 + 16 * lc, a.K - 16), more);
        } else {
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int j = 0; j < JN; ++j) xr[j * S + s].load(x[j] + min(k0 + 64 * s + 16 * q, a.K - 16));
        }
    };
    // x's columns in front of column k that an earlier piece has, where a piece from K - 16 on stands for it
    auto kept = [&](int k) INLINE {
        u32x4 keep = {~0u, ~0u, ~0u, ~0u};
        const int over = min(max(k - (a.K - 16), 0), 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) keep[i] = (uint32_t)(0xFFFFFFFFull << (8 * min(max(over - 4 * i, 0), 4)));
        return keep;
    };
    i32x4 acc[RM][JN] = {};
    u32x4 *mine = bounce[wave], *rows = mine + RM * 16 * C;
    load(kw * SB);
    __syncthreads();
    for (int k0 = kw * SB; k0 < a.K; k0 += KW * SB) {
        const bool last = k0 + SB > a.K, more = own(k0);
        wave_order();
#pragma unroll
        for (int i = 0; i < LW; ++i) mine[piece<C>(lr + LR * i, lc)] = wr[i].get(more);
        if constexpr (STAGED) {
            u32x4 keep = {~0u, ~0u, ~0u, ~0u};
            if (last) keep = kept(k0 + 16 * lc);
#pragma unroll
            for (int j = 0; j < LX; ++j) rows[piece<C>(lr + LR * j, lc)] = xr[j].get(more) & keep;
        }
        wave_order();
        i32x4 xf[JN][S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            u32x4 keep = {~0u, ~0u, ~0u, ~0u};
            if (!STAGED && last) keep = kept(k0 + 64 * s + 16 * q);
#pragma unroll
            for (int j = 0; j < JN; ++j) {
                if constexpr (STAGED) xf[j][s] = __builtin_bit_cast(i32x4, rows[piece<C>(j * 16 + c, 4 * s + q)]);
                else xf[j][s] = __builtin_bit_cast(i32x4, xr[j * S + s].get() & keep);
            }
        }
        load(k0 + KW * SB);
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < RM; ++i) {
                const i32x4 wf = __builtin_bit_cast(i32x4, mine[piece<C>(i * 16 + c, 4 * s + q)]);
#pragma unroll
                for (int j = 0; j < JN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf, xf[j][s], acc[i][j], 0, 0, 0);
            }
    }
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < JN; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) atomicAdd(&sums[j * 16 + c][(rw * RM + i) * 16 + 4 * q + v], acc[i][j][v]);
    __syncthreads();
    for (int i = tid; i < r.n * CH; i += kRowsWaves * 64) {
        const int n = i / CH, ch = i % CH;
        const int64_t m = mt + ch;
        if (m >= a.M) continue;
        const int64_t at = (int64_t)r.e * a.M + m;
        const float s = a.s_f32 ? ((const float*)a.s)[at] : bf16_to_f32(((const uint16_t*)a.s)[at]);
        const float f = (float)sums[n][ch] * a.xs[r.row0 + (int64_t)n] * s;
        const int64_t o = (r.row0 + (int64_t)n) * a.ldy + m;
        if (a.y_bf16) ((uint16_t*)a.y)[o] = f32_to_bf16(f);
        else ((float*)a.y)[o] = f;
    }
}

typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

constexpr int kPiece = 32 * 128;       // a wave's 32 rows of 64 channels in bf16, or of 32 in fp32

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}


typedef __attribute__((address_space(3))) void* lds_ptr;

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

#ifdef __HIP_DEVICE_COMPILE__
// A tile's sums to y, each wave's through its own pieces of LDS (PIECES of them), so that whole lines are written:
// 32 rows of 128 bytes at a time, 16-byte pieces permuted by the row, so that 16 lanes meet all
// banks.  With two pieces one is filled while the other is written out.  `scales` gives the scale of the
// lane's channels 32 i + 8 g + 4 h .. + 3, `row_scale` that of its row in block j.
template <int MB, int NB, bool BF, int PIECES = 2, typename S, typename X>
__device__ __forceinline__ void write_sums(const I8Args& a, const Rows& r, int64_t m0, int mrows, const i32x16 (&acc)[MB][NB],
                                           int wm, int wn, char* piece0, char* piece1, S scales, X row_scale) {
    const int mleft = mrows - wm * 32 * MB;                // of this wave's channels
    const int nleft = r.n - wn * 32 * NB;
    if (nleft <= 0 || mleft <= 0) return;
    int l = threadIdx.x & 63;
    asm volatile("" : "+v"(l));        // addresses of this part are not kept through the loop
    const int fr = l & 31, h = l >> 5, c = l & 7, rr = l >> 3;
    constexpr int B = BF ? 2 : 4, CH = 128 / B, PM = 32 * MB / CH, PH = NB * PM;     // phases of CH channels by 32 rows
    auto fill = [&](auto n) INLINE {
        constexpr int j = n / PM, k = n % PM;
        char* piece = (n & 1 ? piece1 : piece0) + fr * 128;
        each<CH / 8>([&](auto qq) INLINE {
            constexpr int q = qq, i = k * CH / 32 + q / 4, g = q % 4;
            const f32x4 s = scales(i, g);
            const float sx = row_scale(j);
            f32x4 f;
#pragma unroll
            for (int v = 0; v < 4; ++v) f[v] = (float)acc[i][j][4 * g + v] * sx * s[v];
            // rows 16 .. 31 have the halves of a bf16 piece exchanged
            if constexpr (BF)
                *(u32x2*)(piece + (q ^ (fr >> 1 & 7)) * 16 + (h ^ (fr >> 4)) * 8) = u32x2{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
            else
                *(f32x4*)(piece + ((2 * q + h) ^ (fr >> 1 & 7)) * 16) = f;
        });
    };
    // rows that the tile does not have lie behind the buffer
    const int64_t corner = ((int64_t)r.row0 + wn * 32 * NB) * a.ldy + m0 + wm * 32 * MB;
    const bool whole = mleft >= 32 * MB;
    const auto ybuf = buffer((char*)a.y + corner * B, (uint32_t)(((nleft - 1) * (int)a.ldy + min(mleft, 32 * MB)) * B));
    const int yat = rr * (int)a.ldy * B + c * 16;
    auto write = [&](auto n) INLINE {
        constexpr int j = n / PM, k = n % PM;
        const char* piece = n & 1 ? piece1 : piece0;
        if (whole) {
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const int n1 = it * 8 + rr;
                u32x4 o = *(const u32x4*)(piece + n1 * 128 + (c ^ (n1 >> 1 & 7)) * 16);
                if (BF && it >= 2) o = u32x4{o[2], o[3], o[0], o[1]};
                __builtin_amdgcn_raw_buffer_store_b128(o, ybuf, yat + (j * 32 + it * 8) * (int)a.ldy * B + k * 128, 0, 0);
            }
        } else {                                  // the last channels: a row's last piece one at a time
            const int left = mleft - k * CH - c * (16 / B);      // of this lane's
#pragma nounroll
            for (int n1 = rr; n1 < 32; n1 += 8) {
                u32x4 o = *(const u32x4*)(piece + n1 * 128 + (c ^ (n1 >> 1 & 7)) * 16);
                if (BF && n1 >= 16) o = u32x4{o[2], o[3], o[0], o[1]};
                const int to = (j * 32 + n1) * (int)a.ldy * B + k * 128 + c * 16;
                if (left >= 16 / B) {
                    __builtin_amdgcn_raw_buffer_store_b128(o, ybuf, to, 0, 0);
                } else {
#pragma unroll
                    for (int v = 0; v < 16 / B; ++v)
                        if (v < left) {
                            if constexpr (BF) __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(o[v / 2] >> (16 * (v & 1))), ybuf, to + v * B, 0, 0);
                            else __builtin_amdgcn_raw_buffer_store_b32(o[v], ybuf, to + v * B, 0, 0);
                        }
                }
            }
        }
    };
    if constexpr (PIECES == 2) fill(std::integral_constant<int, 0>{});
    each<PH>([&](auto n) INLINE {
        wave_order();
        if constexpr (PIECES == 1) {
            fill(n);
            wave_order();
        } else if constexpr (n + 1 < PH) {
            fill(std::integral_constant<int, n + 1>{});
        }
        write(n);
    });
}

// The last K % 16 columns of a lane's rows times those of x: pieces that LDS loads leave out.  Both
// operands are the rows' last 16 bytes, with x's earlier columns zeroed, in the lower half of the
// lanes.
template <int MB, int NB>
__device__ __forceinline__ void multiply_rest(const I8Args& a, const Rows& r, int64_t m0, int mrows, i32x16 (&acc)[MB][NB], int wm, int wn) {
    const int h = threadIdx.x >> 5 & 1, fr = threadIdx.x & 31, gone = h ? 16 : 16 - (a.K & 15);
    u32x4 keep;
#pragma unroll
    for (int v = 0; v < 4; ++v) keep[v] = (uint32_t)(0xFFFFFFFFull << (8 * min(max(gone - 4 * v, 0), 4)));
    i32x4 wf[MB], xf[NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
        __builtin_memcpy(&wf[i], a.w + ((int64_t)r.e * a.M + m0 + min((wm * MB + i) * 32 + fr, mrows - 1) + 1) * a.K - 16, 16);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        u32x4 v;
        __builtin_memcpy(&v, a.x + (r.row0 + (int64_t)min((wn * NB + j) * 32 + fr, r.n - 1)) * a.ldx + a.K - 16, 16);
        xf[j] = __builtin_bit_cast(i32x4, v & keep);
    }
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[i], xf[j], acc[i][j], 0, 0, 0);
}

// The scales of the tile's channels from m (four) and of its row n, 0 where it has none.
template <bool SF32>
struct TileScales {
    __amdgpu_buffer_rsrc_t s, x;
    __device__ __forceinline__ TileScales(const I8Args& a, const Rows& r, int64_t m0, int mrows)
        : s(buffer((const char*)a.s + ((int64_t)r.e * a.M + m0) * (SF32 ? 4 : 2), mrows * (SF32 ? 4 : 2))),
          x(buffer(a.xs + r.row0, r.n * 4)) {}
    __device__ __forceinline__ f32x4 channels(int m) const {
        if constexpr (SF32) return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(s, m * 4, 0, 0));
        f32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = bf16_to_f32((uint16_t)__builtin_amdgcn_raw_buffer_load_b16(s, (m + i) * 2, 0, 0));
        return v;
    }
    __device__ __forceinline__ float row(int n) const { return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(x, n * 4, 0, 0)); }
};
#endif

// ----------------------------------------------------------------------------------
// In between: tiles of 64 MB channels by 64 NB rows, four waves two by two, each 32 MB by 32 NB in
// 32 x 32 x 32 instructions.  K in steps of 64 bytes through a ring of four buffers in LDS: a step's
// loads are issued three steps ahead, straight to LDS, and two or three workgroups share a CU.
//
// LDS holds rows of 64 bytes in 16-byte pieces, permuted (`piece`) so that 16 lanes reading a piece
// of 16 rows meet 64 different banks.  Rows and columns that a tile does not have lie behind its
// buffers and are zeros.
//
// 256 x 8192 x 2048 (rows, M, K): 10 us, 850 TOP/s; 100 experts of 2048 x 2048 with 41 rows each: 97 us,
// 4.5 TB/s: bound by the weights there.  Tiles of 64 by 64 through registers took
// 28 us for the first.
// ----------------------------------------------------------------------------------
constexpr int kStep = 64;              // bytes of K

template <int MB, int NB, bool BF, bool SF32>
__global__ __launch_bounds__(256, 2) void k_i8_mid(const I8Args a) {
#ifdef __HIP_DEVICE_COMPILE__      // buffer resources and LDS loads have no host form
    constexpr int TM = 64 * MB, TN = 64 * NB, L = MB + NB, P = MB * NB, O = MB + NB;   // loads, products, operands
    __shared__ __align__(16) char w0[TM * kStep], w1[TM * kStep], w2[TM * kStep], w3[TM * kStep];
    __shared__ __align__(16) char x0[TN * kStep], x1[TN * kStep], x2[TN * kStep], x3[TN * kStep];
    const int64_t tile = a.first + blockIdx.x;
    const Rows r = find_rows(a, tile / a.tm, TN);
    if (r.n == 0) return;
    const int64_t m0 = tile % a.tm * TM;
    const int mrows = a.M - m0 < TM ? (int)(a.M - m0) : TM;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    // this thread's pieces: of the rows lr + 64 i, the one that lies at lane % 4
    const int lr = tid >> 2, lc = (tid & 3) ^ (lr >> 2 & 3);
    int at[L];
#pragma unroll
    for (int i = 0; i < L; ++i) at[i] = (i < MB ? (lr + 64 * i) * a.K : (lr + 64 * (i - MB)) * (int)a.ldx) + 16 * lc;
    const auto wbuf = buffer(a.w + ((int64_t)r.e * a.M + m0) * a.K, (uint32_t)mrows * (uint32_t)a.K);
    const auto xbuf = buffer(a.x + (int64_t)r.row0 * a.ldx, (uint32_t)(r.n - 1) * (uint32_t)a.ldx + (uint32_t)a.K);
    // the lane's operands: piece 2 s + lane / 32 of row lane % 32 of each block of 32
    const int h = lane >> 5, fr = lane & 31;
    const int wget = (wm * 32 * MB + fr) * kStep, xget = (wn * 32 * NB + fr) * kStep;
    i32x16 acc[MB][NB] = {};
    i32x4 wf[2][MB], xf[2][NB];
    const int steps = ((a.K & ~15) + kStep - 1) / kStep;
    auto load = [&](int t, char* w, char* x, auto n) INLINE {
        constexpr int i = n;
        const int k = min(t, steps - 1) * kStep;
        if constexpr (i < MB) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(wbuf, (lds_ptr)(w + i * 64 * kStep + wave * 1024), 16, at[i], k, 0, 0);
        } else {
            const int past = t * kStep + 16 * lc + 16 <= a.K ? 0 : (int)0x80000000;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(xbuf, (lds_ptr)(x + (i - MB) * 64 * kStep + wave * 1024), 16, at[i] | past, k, 0, 0);
        }
    };
    auto fetch = [&](const char* w, const char* x, int s, int to, auto n) INLINE {
        constexpr int i = n;
        const int p = ((2 * s + h) ^ (fr >> 2 & 3)) * 16;
        if constexpr (i < MB) wf[to][i] = *(const i32x4*)(w + wget + p + i * 32 * kStep);
        else xf[to][i - MB] = *(const i32x4*)(x + xget + p + (i - MB) * 32 * kStep);
    };
    // Every wave's loads of the next step have landed (those of the two after may fly on), and its
    // reads of this step are done.  No fence: its wait would be for all loads.
    auto arrive = [&]() INLINE { asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(2 * L) : "memory"); };
    each<L>([&](auto i) INLINE { load(0, w0, x0, i); });
    each<L>([&](auto i) INLINE { load(1, w1, x1, i); });
    each<L>([&](auto i) INLINE { load(2, w2, x2, i); });
    arrive();
    each<O>([&](auto i) INLINE { fetch(w0, x0, 0, 0, i); });
    // Half a step: its products, and in their shadow the next half's operands (from w and x) and, if
    // LOAD, the loads of step t to tw and tx.
    auto half = [&](const char* w, const char* x, int s, auto from, auto load_too, int t, char* tw, char* tx) INLINE {
        each<P>([&](auto n) INLINE {
            constexpr int p = n, F = from;
            acc[p / NB][p % NB] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[F][p / NB], xf[F][p % NB], acc[p / NB][p % NB], 0, 0, 0);
            each<O>([&](auto i) INLINE {
                if constexpr (i * P / O == p) fetch(w, x, s, F ^ 1, i);
            });
            if constexpr (load_too)
                each<L>([&](auto i) INLINE {
                    if constexpr (i * P / L == p) load(t, tw, tx, i);
                });
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    constexpr std::integral_constant<int, 0> c0;
    constexpr std::integral_constant<int, 1> c1;
    // step t from (w, x); the next step's are (nw, nx), and (tw, tx) are free: step t - 1's
    auto step = [&](int t, char* w, char* x, char* nw, char* nx, char* tw, char* tx) INLINE {
        half(w, x, 1, c0, c1, t + 3, tw, tx);
        arrive();
        half(nw, nx, 0, c1, c0, 0, nullptr, nullptr);
    };
    for (int t = 0; t < steps; t += 4) {      // steps past the last one multiply zeros
        step(t, w0, x0, w1, x1, w3, x3);
        step(t + 1, w1, x1, w2, x2, w0, x0);
        step(t + 2, w2, x2, w3, x3, w1, x1);
        step(t + 3, w3, x3, w0, x0, w2, x2);
    }
    // The loads behind the last step end before LDS is used again.
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (a.K & 15) multiply_rest(a, r, m0, mrows, acc, wm, wn);
    f32x4 s[MB][4];
    float sx[NB];
    const TileScales<SF32> sc(a, r, m0, mrows);
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) s[i][g] = sc.channels(wm * 32 * MB + 4 * h + i * 32 + 8 * g);
#pragma unroll
    for (int j = 0; j < NB; ++j) sx[j] = sc.row(wn * 32 * NB + j * 32 + fr);
    char* pieces = (wave & 2 ? (wave & 1 ? w3 : w2) : (wave & 1 ? w1 : w0));
    write_sums<MB, NB, BF>(a, r, m0, mrows, acc, wm, wn, pieces, pieces + kPiece, [&](int i, int g) INLINE { return s[i][g]; },
                           [&](int j) INLINE { return sx[j]; });
#endif
}

// The same tiles for rows that do not start on 4 bytes: operands pass through registers, where the
// words that hold a piece are shifted (Bytes16), to two buffers in LDS.  256 x 8192 x 2049 (rows, M,
// K): 25 us, 4096 rows 170; columns of 2052 take 10.5 and 81 by the kernels for 4 bytes.
template <int MB, int NB, bool BF, bool SF32>
__global__ __launch_bounds__(256, 2) void k_i8_odd(const I8Args a) {
#ifdef __HIP_DEVICE_COMPILE__
    constexpr int TM = 64 * MB, TN = 64 * NB;
    __shared__ __align__(16) u32x4 ws[2][TM * 4], xs[2][TN * 4];
    const int64_t tile = a.first + blockIdx.x;
    const Rows r = find_rows(a, tile / a.tm, TN);
    if (r.n == 0) return;
    const int64_t m0 = tile % a.tm * TM;
    const int mrows = a.M - m0 < TM ? (int)(a.M - m0) : TM;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    const int lr = tid >> 2, lc = tid & 3;            // this thread's pieces: lc of the rows lr + 64 i
    const int8_t *w[MB], *x[NB];
#pragma unroll
    for (int i = 0; i < MB; ++i) w[i] = a.w + ((int64_t)r.e * a.M + m0 + min(lr + 64 * i, mrows - 1)) * a.K;
#pragma unroll
    for (int j = 0; j < NB; ++j) x[j] = a.x + (r.row0 + (int64_t)min(lr + 64 * j, r.n - 1)) * a.ldx;
    Bytes16<true> wr[MB], xr[NB];
    auto load = [&](int t) INLINE {
        const int k = min(t * kStep + 16 * lc, a.K - 16);
#pragma unroll
        for (int i = 0; i < MB; ++i) wr[i].load(w[i] + k);
#pragma unroll
        for (int j = 0; j < NB; ++j) xr[j].load(x[j] + k);
    };
    auto store = [&](int t, int buf) INLINE {
        const int over = min(max(t * kStep + 16 * lc - (a.K - 16), 0), 16);   // bytes of earlier pieces
        u32x4 keep;
#pragma unroll
        for (int v = 0; v < 4; ++v) keep[v] = (uint32_t)(0xFFFFFFFFull << (8 * min(max(over - 4 * v, 0), 4)));
#pragma unroll
        for (int i = 0; i < MB; ++i) ws[buf][piece<4>(lr + 64 * i, lc)] = wr[i].get();
#pragma unroll
        for (int j = 0; j < NB; ++j) xs[buf][piece<4>(lr + 64 * j, lc)] = xr[j].get() & keep;
    };
    const int h = lane >> 5, fr = lane & 31;
    i32x16 acc[MB][NB] = {};
    const int steps = (a.K + kStep - 1) / kStep;
    load(0);
    store(0, 0);
    load(1);
    __syncthreads();
    for (int t = 0; t < steps; ++t) {
        const int buf = t & 1;
        store(t + 1, buf ^ 1);
        load(t + 2);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            i32x4 wf[MB], xf[NB];
#pragma unroll
            for (int i = 0; i < MB; ++i) wf[i] = __builtin_bit_cast(i32x4, ws[buf][piece<4>((wm * MB + i) * 32 + fr, 2 * s + h)]);
#pragma unroll
            for (int j = 0; j < NB; ++j) xf[j] = __builtin_bit_cast(i32x4, xs[buf][piece<4>((wn * NB + j) * 32 + fr, 2 * s + h)]);
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[i], xf[j], acc[i][j], 0, 0, 0);
        }
        __syncthreads();
    }
    f32x4 s[MB][4];
    float sx[NB];
    const TileScales<SF32> sc(a, r, m0, mrows);
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) s[i][g] = sc.channels(wm * 32 * MB + 4 * h + i * 32 + 8 * g);
#pragma unroll
    for (int j = 0; j < NB; ++j) sx[j] = sc.row(wn * 32 * NB + j * 32 + fr);
    // four pieces of LDS are there, one a wave
    char* mine = (char*)&ws[0][0] + wave * kPiece;
    static_assert(sizeof(ws) >= 4 * kPiece, "a piece a wave");
    write_sums<MB, NB, BF, 1>(a, r, m0, mrows, acc, wm, wn, mine, mine, [&](int i, int g) INLINE { return s[i][g]; },
                              [&](int j) INLINE { return sx[j]; });
#endif
}

// ----------------------------------------------------------------------------------
// Many rows.  A workgroup of four waves, alone on its CU, takes 256 channels by 256 rows, each wave
// 128 by 128 in 32 x 32 x 32 instructions: per product that reads the least from LDS.  K in steps
// of 128 bytes through two buffers in LDS, loaded straight from memory; the order of a step is fixed
// by hand.  One barrier a step is enough, and it stands in front of the step's last quarter, whose
// operands are in registers: the matrix unit has work while the next step's first operands are read.
//
// Workgroups stay, one a CU; a tile's last steps already load the next.  Without experts a workgroup
// takes every 256th tile.  With experts each XCD (every 8th workgroup) takes a stretch of the tiles,
// an expert's in a row, so that its weights and rows come from memory to one L2 and every XCD has as
// many tiles whatever the routing; and a tile of up to 128 rows, the rest of most experts, has half
// of the products.  4096 tokens to 8 of 100 experts of 2048 x 2048: 214 us, 227 without both.
//
// 4096 x 8192 x 2048 (rows, M, K): 70 us, 8192 x 8192 x 8192: 437 us or 2516 TOP/s at 1.6 GHz, the clock
// that the card's power leaves (1.9 GHz without the loads, 2.3 with a quarter of the products; another
// card reached 412, 2670 TOP/s); 73% of the cycles feed the matrix unit.  A tile's results take 7.8 us of
// 36 at K = 2048: all CUs write at 4.3 TB/s then.  Not waiting for the stores in the next tile's first
// step gained nothing.
// ----------------------------------------------------------------------------------
constexpr int kWideStep = 128, kWideM = 256, kWideN = 256;

// A tile: where its operands lie.
struct WideTile {
    Rows r;
    int64_t m0;
    int mrows;
};

__device__ __forceinline__ WideTile wide_tile(const I8Args& a, int64_t tile, int64_t tiles, Seek& seek) {
    WideTile t = {{0, 0, 0}, 0, 0};
    if (tile >= tiles) return t;
    t.r = find_rows(a, tile / a.tm, kWideN, seek);
    t.m0 = tile % a.tm * kWideM;
    t.mrows = a.M - t.m0 < kWideM ? (int)(a.M - t.m0) : kWideM;
    return t;
}

#ifdef __HIP_DEVICE_COMPILE__
struct WideBuffers {
    __amdgpu_buffer_rsrc_t w, x;
};
__device__ __forceinline__ WideBuffers wide_buffers(const I8Args& a, const WideTile& t) {
    return {buffer(a.w + ((int64_t)t.r.e * a.M + t.m0) * a.K, (uint32_t)t.mrows * (uint32_t)a.K),
            buffer(a.x + (int64_t)t.r.row0 * a.ldx, (uint32_t)(t.r.n - 1) * (uint32_t)a.ldx + (uint32_t)a.K)};
}
#endif

// REST: K is not a multiple of 16 (the code for it costs the others registers: 4 us of 76).
template <bool BF, bool SF32, bool REST>     // y in bf16, else fp32; scales in fp32, else bf16
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void k_i8_wide(const I8Args a, int64_t tiles) {
#ifdef __HIP_DEVICE_COMPILE__      // buffer resources and LDS loads have no host form
    constexpr int S = kWideStep, LW = kWideM / 32, L = LW + kWideN / 32;   // loads
    __shared__ __align__(16) char w0[kWideM * S], w1[kWideM * S], x0[kWideN * S], x1[kWideN * S];
    __shared__ __align__(16) char pieces[2][4 * kPiece];
    int64_t tile = blockIdx.x, hop = gridDim.x;
    if (a.offsets) {
        int64_t all = count_tiles(a, kWideN) * a.tm;
        all = all < tiles ? all : tiles;              // more only with wrong offsets
        const int xcd = blockIdx.x & 7;
        hop = gridDim.x >> 3;
        tile = all * xcd / 8 + (blockIdx.x >> 3);
        tiles = all * (xcd + 1) / 8;
    }
    Seek seek;
    WideTile cur = wide_tile(a, tile, tiles, seek);
    if (cur.r.n == 0) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    // This thread's pieces: of the rows lr + 32 i, the one that lies at lane % 8.  Rows that a tile
    // does not have lie behind its buffer.
    const int lr = tid >> 3, lc = (tid & 7) ^ (lr >> 1 & 7);
    int atw = lr * a.K + 16 * lc, atx = lr * (int)a.ldx + 16 * lc;
    const int hopw = 32 * a.K, hopx = 32 * (int)a.ldx;
    // the lane's operands: piece 2 s + lane / 32 of row lane % 32 of each block of 32
    const int h = lane >> 5, fr = lane & 31;
    const int wget = (wm * 128 + fr) * S;
    const int real = ((a.K & ~15) + S - 1) / S, steps = (real + 1) & ~1;

    // Of a tile's step t, piece n (0 .. L - 1) of this thread's.  Columns past K are zero in x: their
    // offset lies behind the buffer (the step's own stays inside of it).
    auto load = [&](const WideBuffers& d, int t, char* w, char* x, auto n) INLINE {
        constexpr int i = n;
        const int k = min(t, real - 1) * S;
        if constexpr (i < LW) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(d.w, (lds_ptr)(w + i * 32 * S + wave * 1024), 16, atw + i * hopw, k, 0, 0);
        } else {
            const int past = t * S + 16 * lc + 16 <= a.K ? 0 : (int)0x80000000;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(d.x, (lds_ptr)(x + (i - LW) * 32 * S + wave * 1024), 16, (atx + (i - LW) * hopx) | past, k, 0, 0);
        }
    };
    // Every wave's loads of the next step have landed, and its reads of this step are done.
    auto arrive = [&]() INLINE { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
    constexpr std::integral_constant<int, 0> c0;
    constexpr std::integral_constant<int, 1> c1;
    constexpr std::integral_constant<int, -1> none;
    WideBuffers now = wide_buffers(a, cur);
    each<L>([&](auto i) INLINE { load(now, 0, w0, x0, i); });
    each<L / 2>([&](auto i) INLINE { load(now, 1, w1, x1, i); });
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(L / 2) : "memory");
    // A tile of up to 64 NB rows, 32 NB of them a wave; `then`: the next tile's operands.
    auto multiply = [&](auto nb, const WideBuffers& then) INLINE {
        constexpr int NB = nb, P = 4 * NB, O = 4 + NB;     // products and operands of a quarter of a step
        const int xget = (wn * 32 * NB + fr) * S;
        i32x16 acc[4][NB];
        i32x4 wf[2][4], xf[2][NB];
        auto fetch = [&](const char* w, const char* x, int s, int to, auto n) INLINE {   // n: 0 .. 3 + NB
            constexpr int i = n;
            const int p = ((2 * s + h) ^ (fr >> 1 & 7)) * 16;
            if constexpr (i < 4) wf[to][i] = *(const i32x4*)(w + wget + p + i * 32 * S);
            else xf[to][i - 4] = *(const i32x4*)(x + xget + p + (i - 4) * 32 * S);
        };
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
            asm volatile("" : "+v"(atw), "+v"(atx));     // their multiples are not kept
            quarter(w, x, 1, c0, c1, d1, t1, nw, nx);
            quarter(w, x, 2, c1, none, d1, 0, nw, nx);
            quarter(w, x, 3, c0, none, d1, 0, nw, nx);
            arrive();
            quarter(nw, nx, 0, c1, c0, d2, t2, w, x);
        };
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[i][j] = i32x16{};
        each<O>([&](auto i) INLINE { fetch(w0, x0, 0, 0, i); });
        for (int t = 0; t < steps; t += 2) {      // a step past the last one multiplies zeros
            const bool last = t + 2 >= steps;     // then the next tile's steps 0 and 1 are loaded
            const WideBuffers d = last ? then : now;
            const int t2 = last ? 0 : t + 2;
            step(w0, x0, w1, x1, now, t + 1, d, t2);
            step(w1, x1, w0, x0, d, t2, d, t2 + 1);
        }
        // the sums stay where they are until each is read; the last product's end is waited for here
        asm volatile("s_nop 15\n\ts_nop 7" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) asm volatile("" : "+a"(acc[i][j]));
        // the scales of the lane's channels and rows (0 where the tile has none)
        f32x4 s[4][4];
        float sx[NB];
        const TileScales<SF32> sc(a, cur.r, cur.m0, cur.mrows);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) s[i][g] = sc.channels(wm * 128 + 4 * h + i * 32 + 8 * g);
#pragma unroll
        for (int j = 0; j < NB; ++j) sx[j] = sc.row(wn * 32 * NB + j * 32 + fr);
        if constexpr (REST) multiply_rest(a, cur.r, cur.m0, cur.mrows, acc, wm, wn);
        write_sums<4, NB, BF>(a, cur.r, cur.m0, cur.mrows, acc, wm, wn, pieces[0] + wave * kPiece, pieces[1] + wave * kPiece,
                              [&](int i, int g) INLINE { return s[i][g]; }, [&](int j) INLINE { return sx[j]; });
    };
    for (;;) {
        const WideTile next = wide_tile(a, tile += hop, tiles, seek);
        const WideBuffers then = next.r.n ? wide_buffers(a, next) : now;
        if (cur.r.n > 128) multiply(std::integral_constant<int, 4>{}, then);
        else multiply(std::integral_constant<int, 2>{}, then);
        if (!next.r.n) break;
        cur = next;
        now = then;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");     // loads to LDS end before the workgroup does
#endif
}

// ---- host ------------------------------------------------------------------------

// The tiles of `rows` rows that a call can have: an expert's last one may be partly filled, at most one a row.
int64_t row_tiles(const I8Args& a, int rows) {
    return a.offsets ? a.N / rows + (a.E < a.N ? a.E : a.N) : ((int64_t)a.N + rows - 1) / rows;
}

template <int RM, int JN, int SB, int KW, bool ODD>
void launch_rows(I8Args a, hipStream_t st) {
    constexpr int CH = kRowsWaves / KW * RM * 16;
    a.tm = (a.M - 1) / CH + 1;
    const int64_t tiles = row_tiles(a, JN * 16) * a.tm, most = kLaunchThreads / (kRowsWaves * 64);
    for (a.first = 0; a.first < tiles; a.first += most)
        hipLaunchKernelGGL((k_i8_rows<RM, JN, SB, KW, ODD>), dim3((unsigned)(tiles - a.first < most ? tiles - a.first : most)),
                           dim3(kRowsWaves * 64), 0, st, a);
}

// f(y in bf16, scales in fp32) as constants
template <typename F>
void by_types(const I8Args& a, F f) {
    constexpr std::true_type yes;
    constexpr std::false_type no;
    if (a.y_bf16) a.s_f32 ? f(yes, yes) : f(yes, no);
    else a.s_f32 ? f(no, yes) : f(no, no);
}

template <int MB, int NB, typename K>
void launch_tiles(I8Args a, K kernel, hipStream_t st) {
    a.tm = (a.M - 1) / (64 * MB) + 1;
    const int64_t tiles = row_tiles(a, 64 * NB) * a.tm, most = kLaunchThreads / 256;
    for (a.first = 0; a.first < tiles; a.first += most)
        hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles - a.first < most ? tiles - a.first : most)), dim3(256), 0, st, a);
}
template <int MB, int NB>
void launch_mid(const I8Args& a, hipStream_t st) {
    by_types(a, [&](auto bf, auto sf) { launch_tiles<MB, NB>(a, k_i8_mid<MB, NB, bf, sf>, st); });
}
template <int MB, int NB>
void launch_odd(const I8Args& a, hipStream_t st) {
    by_types(a, [&](auto bf, auto sf) { launch_tiles<MB, NB>(a, k_i8_odd<MB, NB, bf, sf>, st); });
}

void launch_wide(I8Args a, hipStream_t st) {
    a.tm = (a.M - 1) / kWideM + 1;
    const int64_t tiles = row_tiles(a, kWideN) * a.tm;
    const dim3 grid((unsigned)(tiles < 256 && !a.offsets ? tiles : 256));
    by_types(a, [&](auto bf, auto sf) {
        if (a.K & 15) hipLaunchKernelGGL((k_i8_wide<bf, sf, true>), grid, dim3(256), 0, st, a, tiles);
        else hipLaunchKernelGGL((k_i8_wide<bf, sf, false>), grid, dim3(256), 0, st, a, tiles);
    });
}

template <int RM, int JN, int SB, bool ODD>
void launch_rows_kw(const I8Args& a, hipStream_t st) {
    const int64_t tiles = row_tiles(a, JN * 16) * ((a.M - 1) / (RM * 16) + 1);     // of a wave
    const int kw = tiles >= 2048 ? 2 : tiles >= 512 && a.K < 8192 ? 4 : 8;
    if (kw == 2) launch_rows<RM, JN, SB, 2, ODD>(a, st);
    else if (kw == 4) launch_rows<RM, JN, SB, 4, ODD>(a, st);
    else launch_rows<RM, JN, SB, 8, ODD>(a, st);
}
template <bool ODD>
void launch_rows_jn(const I8Args& a, int jn, hipStream_t st) {
    if (jn == 1) launch_rows_kw<1, 1, 256, ODD>(a, st);
    else if (jn == 2) launch_rows_kw<2, 2, 128, ODD>(a, st);
    else launch_rows_kw<2, 4, 128, ODD>(a, st);
}

// Which kernel (us, each on the other's side too; M x K and rows, or rows x M x K):
//   fewer than 16 columns: k_i8_tile.
//   Few rows (an expert has on average), or a grid of few tiles: k_i8_rows reads the weights once
//   and splits K over a workgroup's waves.  8192 x 2048: 49 rows 8.3 (tiles of 64: 9.2), 64 rows 8.2
//   (9.3), 96 rows 11.0 (9.2); 4096 x 4096, 128 rows 10.7 (14.5); 16384 x 2048, 64 rows 11.7 (10.1);
//   100 experts of 2048 x 2048 with 9 rows each 92.8 (86.2).  Rows on odd bytes: 8192 x 2049, 128
//   rows 14.6 (23.9), 256 rows 26.2 (24.0); 1000 x 4097, 1024 rows 22 (46); 100 experts of 2048 x 2049
//   with 16 rows each 126 (166), with 40 rows 174 (179), with 128 rows 330 (248).
//   Tiles of 128 channels by 64 or 128 rows: by 128 where that makes most of a workgroup a CU.
//   256 x 8192 x 2048: 10.1 by 64, 11.7 by 128; 512 x 8192 x 2048: 17.1 and 14.1.
//   Tiles of 256 by 256, one a CU: where there is one for nearly each CU, and no second round for a
//   few.  By number of tiles, 256 by 256 (128 by 128), K = 512: 192 16.5 (14.6), 224 17.0 (17.1), 256
//   17.9 (17.9), 288 27.6 (20.9), 352 27.7 (24.5), 400 28.1 (27.6), 448 29.2 (29.5), 512 31.6 (33.0);
//   K = 1024: 192 22.0 (21.2), 224 22.8 (24.7), 288 36.5 (30.3), 352 37.2 (36.8), 400 38.7 (40.4), 512 43.8
//   (51.8); K = 2048: 192 32.1 (36.4), 256 36.3 (47.0), 264 53.4 (55.8), 288 56.3 (56.0), 512 70.4 (92.4); K =
//   4096: 192 51.6 (64.3), 264 89.0 (98.8), 288 96.6 (103.5).  (K = 256: 14.5 for 15.3 at 256, 24.0 for 25.4
//   at 512; a third round for a few is not looked for: K = 512, 576 tiles 42.1 (36.9), K = 1024 59.0 (59.2).)
//   With experts by their rows, counted from N, for which dropped slots count too: 100 experts of
//   2048 x 2048 with 164 rows each 152 (150), with 240 rows 176 (193), 328 rows 222 (244); 8 of
//   8192 x 4096 with 128 rows 86 (80), with 192 rows 93 (104).
bool wide_pays(const I8Args& a, int avg) {
    if (a.offsets) return avg >= 176;
    const int64_t tiles = row_tiles(a, kWideN) * ((a.M - 1) / kWideM + 1);
    return tiles >= (a.K >= 1536 ? 192 : 224) && (tiles <= 256 || a.K >= 2048 || (tiles - 256) * a.K >= 90000);
}

void launch(I8Args a, hipStream_t st) {
    if (a.K < 16) {
        a.tm = (a.M - 1) / 64 + 1;
        const int64_t tiles = row_tiles(a, 64) * a.tm, most = kLaunchThreads / 256;
        for (a.first = 0; a.first < tiles; a.first += most)
            hipLaunchKernelGGL(k_i8_tile, dim3((unsigned)(tiles - a.first < most ? tiles - a.first : most)), dim3(256), 0, st, a);
        return;
    }
    const bool odd = ((uintptr_t)a.w | (uintptr_t)a.x | (uintptr_t)a.K | (uintptr_t)(a.N > 1 ? a.ldx : 0)) & 3;
    const int avg = a.offsets ? (a.N - 1) / a.E + 1 : a.N;
    const int64_t tm = (a.M - 1) / 128 + 1, tiles64 = row_tiles(a, 64) * tm;
    // offsets inside a tile have to fit 31 bits
    const bool tiled = a.ldx <= 1 << 22 && a.ldy <= 1 << 20 && avg >= (a.offsets ? odd ? 33 : 9 : 49) &&
                       tiles64 >= (odd ? 256 : 128);
    if (!tiled) {
        // As many rows a wave as an expert has, but 32 while their workgroups (8 waves share a tile) fit
        // one a CU, and 16 where 32 give work to a quarter of the CUs.  us by 64, 32, 16 rows (rows x M x K):
        // 33 x 4090 x 4096 (256 workgroups of 32 rows) 9.1 7.2 11.0, 33 x 4130 x 4096 (260) 9.2 10.8 14.7;
        // 96 x 2720 x 4096 (255) 10.0 8.8 15.3, 96 x 2800 x 4096 (264) 9.1 9.1; 61 x 4500 x 4150 (282) 12.4
        // 15.2 28.6; 4 experts of 800 x 4096 with 50 rows each 9.8 8.9, 2 of 1900 x 4096 with 60 10.1 10.6;
        // 32 x 2048 x 4096 (64) 8.4 6.5 6.4, 40 x 700 x 8192 (44) 11.9 9.1 8.5.
        const int64_t tm32 = (a.M - 1) / 32 + 1;
        int jn = avg <= (a.offsets ? 8 : 16) ? 1 : avg <= 32 ? 2 : 4;
        if (jn == 4 && row_tiles(a, 32) * tm32 <= 256) jn = 2;
        if (jn == 2 && row_tiles(a, 32) * tm32 < 64) jn = 1;
        odd ? launch_rows_jn<true>(a, jn, st) : launch_rows_jn<false>(a, jn, st);
    } else if (!odd && wide_pays(a, avg)) {
        launch_wide(a, st);
    } else if (row_tiles(a, 128) * tm < 192) {
        odd ? launch_odd<2, 1>(a, st) : launch_mid<2, 1>(a, st);
    } else {
        odd ? launch_odd<2, 2>(a, st) : launch_mid<2, 2>(a, st);
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
    I8Args a = {weight, scales, offsets, x, x_scale, y, ldx, ldy, 0, E, M, K, N, 0, s_dtype == SEEDMM_F32, y_dtype == SEEDMM_BF16};
    launch(a, (hipStream_t)hip_stream);
    return launch_status();
}

}  // extern "C"
