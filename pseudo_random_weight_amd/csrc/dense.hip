// dense.hip -- gfx950 kernels of the dense operators around a seed-coded routed layer, and
// their C ABI: the product with affine 4-bit weights (seedmm_q4_gemv), the residual's
// addition with the root-mean-square norm (seedmm_add_norm), the router's choice
// (seedmm_route), and the layer that calls them with the routed experts (seedmm_moe_block).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/seedmm.h"
#include "device_rows.hpp"
#include "moe_layer.hpp"

namespace {

// ----------------------------------------------------------------------------------
// seedmm_q4_gemv.  y[n][m] = sx[n] sum_g ( s[m][g] D[m][g][n] + b[m][g] X[g][n] ) with
// D = sum of q x over the group's columns and X = sum of x.
//
// Products q x are exact: a code q is an integer of 4 bits, so it enters the matrix
// instruction without rounding, and the scale multiplies the group's fp32 sum afterwards
// (a weight s q + b is never rounded to the activation's type).
//   bf16 x: a code is an integer below 16, exact in bf16.
//   fp32 x: split into three bf16 of 8 bits each (truncated, so the split is exact), three
//     rows of the same instruction (few tokens), or three instructions (many).
//   int8 x: the integer instruction (few tokens), or exact bf16 (many); D is exact.
// ----------------------------------------------------------------------------------
constexpr int kQ4Waves = 8;      // of a workgroup for a few tokens

struct Q4Args {
    const uint32_t* w;   // [M][K/8], code k of a row in word k/8, bits 4 (k%8)
    const void* s;       // [M][K/group]
    const void* b;
    const void* x;       // [N][ldx]
    const float* xs;     // int8 x: [N]
    void* y;             // [N][ldy]
    int M, K, N, ldx, ldy;
    int y_bf16;
};

template <bool SF32>
__device__ __forceinline__ float load_scale(const void* p, int64_t i) {
    if constexpr (SF32) return ((const float*)p)[i];
    else return bf16_to_f32(((const uint16_t*)p)[i]);
}

// One wave's 16 bytes a lane (32 codes of row l % 16, columns 32 (l / 16) ..) become, after
// a 4 x 4 transposition over the four lane quarters, word j = codes 32 j + 8 q .. + 7 of the
// 128 columns: each word is then a lane's operand of one 32-column instruction.
__device__ __forceinline__ void transpose_quarters(uint32_t (&w)[4]) {
    auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    w[0] = c[0]; w[1] = c[1]; w[2] = d[0]; w[3] = d[1];
}

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

// 8 codes -> bf16 in the order 0 2 4 6 1 3 5 7.  A byte 0 .. 15 read as an 8-bit float
// (e4m3) is code * 2^-9 exactly, subnormal or not, so the pair conversion with scale 2^9
// gives the integers: 7 instructions for 8 codes.
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t w) {
    const uint32_t a = w & 0x0F0F0F0Fu, b = (w >> 4) & 0x0F0F0F0Fu;
    u32x4 v;
    v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 512.0f, false));
    v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 512.0f, true));
    v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.0f, false));
    v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 512.0f, true));
    return __builtin_bit_cast(bf16x8, v);
}

// 8 codes -> bytes in the same order
__device__ __forceinline__ u32x2 codes_i8(uint32_t w) {
    return u32x2{w & 0x0F0F0F0Fu, (w >> 4) & 0x0F0F0F0Fu};
}

// NG consecutive scales from index i of which the first nv exist (the others read as 0).
// Whole runs are one load of 2-byte (bf16) or 4-byte (fp32) alignment.
template <bool SF32, int NG>
struct Scales {
    uint32_t u[SF32 ? NG : (NG + 1) / 2];
    __device__ __forceinline__ void load(const void* p, int64_t i, int nv) {
        const char* at = (const char*)p + i * (SF32 ? 4 : 2);
        if (nv >= NG) {
            if constexpr (!SF32 && NG == 1) u[0] = *(const uint16_t*)at;
            else __builtin_memcpy(u, at, sizeof(u));
        } else {
#pragma unroll
            for (int g = 0; g < (int)(sizeof(u) / 4); ++g) u[g] = 0;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                if (g < nv) {
                    if constexpr (SF32) u[g] = ((const uint32_t*)at)[g];
                    else u[g / 2] |= (uint32_t)((const uint16_t*)at)[g] << (16 * (g & 1));
                }
            }
        }
    }
    __device__ __forceinline__ float get(int g) const {
        if constexpr (SF32) return __uint_as_float(u[g]);
        else return __uint_as_float((g & 1) ? u[g / 2] & 0xFFFF0000u : u[g / 2] << 16);
    }
};

// 8 columns of an activation row: load8 takes them from memory (or zeros), place8 writes
// them to LDS in the operands' order, XT rows `rowb` apart (fp32: three), and returns
// their sum.
template <int XT>
struct Raw8 {
    uint32_t u[XT == SEEDMM_F32 ? 8 : XT == SEEDMM_BF16 ? 4 : 2];
};

template <int XT>
__device__ __forceinline__ Raw8<XT> load8(const void* x, int64_t at, bool ok) {
    Raw8<XT> v = {};
    if (ok) {
        if constexpr (XT == SEEDMM_I8) *(u32x2*)v.u = *(const u32x2*)((const int8_t*)x + at);
        else if constexpr (XT == SEEDMM_BF16) *(u32x4*)v.u = *(const u32x4*)((const uint16_t*)x + at);
        else {
            *(u32x4*)v.u = *(const u32x4*)((const float*)x + at);
            *(u32x4*)(v.u + 4) = *(const u32x4*)((const float*)x + at + 4);
        }
    }
    return v;
}

template <int XT>
__device__ __forceinline__ float place8(const Raw8<XT>& x, char* dst, int64_t rowb) {
    const uint32_t* v = x.u;
    float sum = 0.f;
    if constexpr (XT == SEEDMM_I8) {
        int isum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) isum += (int)(int8_t)(v[0] >> 8 * i) + (int)(int8_t)(v[1] >> 8 * i);
        sum = (float)isum;
        u32x2 p;
        p[0] = __builtin_amdgcn_perm(v[1], v[0], 0x06040200u);
        p[1] = __builtin_amdgcn_perm(v[1], v[0], 0x07050301u);
        *(u32x2*)dst = p;
    } else if constexpr (XT == SEEDMM_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += __uint_as_float(v[i] << 16) + __uint_as_float(v[i] & 0xFFFF0000u);
        u32x4 p;
        p[0] = __builtin_amdgcn_perm(v[1], v[0], 0x05040100u);   // x0 x2
        p[1] = __builtin_amdgcn_perm(v[3], v[2], 0x05040100u);   // x4 x6
        p[2] = __builtin_amdgcn_perm(v[1], v[0], 0x07060302u);   // x1 x3
        p[3] = __builtin_amdgcn_perm(v[3], v[2], 0x07060302u);   // x5 x7
        *(u32x4*)dst = p;
    } else {
        uint32_t pl[3][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float f = __uint_as_float(v[i]);
            sum += f;
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                pl[p][i] = __float_as_uint(f) & 0xFFFF0000u;
                f -= __uint_as_float(pl[p][i]);
            }
        }
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = i < 2 ? 4 * i : 4 * i - 7;   // 0 4 1 5: first of the pair (e, e + 2)
                o[i] = (pl[p][e] >> 16) | pl[p][e + 2];
            }
            *(u32x4*)(dst + p * rowb) = o;
        }
    }
    return sum;
}

// the same for 8-bit rows as bf16 (exact)
__device__ __forceinline__ float place8_as_bf16(const Raw8<SEEDMM_I8>& x, char* dst) {
    float f[8], sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        f[i] = (float)(int8_t)(x.u[i >> 2] >> 8 * (i & 3));
        sum += f[i];
    }
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = i < 2 ? 4 * i : 4 * i - 7;
        o[i] = (__float_as_uint(f[e]) >> 16) | (__float_as_uint(f[e + 2]) & 0xFFFF0000u);
    }
    *(u32x4*)dst = o;
    return sum;
}

// A few tokens.  A wave takes 16 weight rows; KW waves of a workgroup share a row tile and
// take its slabs of 256 columns in turn, each loaded while the one before is multiplied,
// the first before the activations are staged.  8 lanes load the 128 bytes of a row, whole
// cache lines, and the wave's own piece of LDS hands them to the lanes that multiply them
// (each lane loading its own 16 bytes, 64 bytes a row, took 54 us for 131072 x 2048 at one
// token against 30 us: the texture path passes one line at a time).  That size streams
// its 152 MB at 5.2 TB/s with 3 sets of inputs in turn, 4.5 with 8; small matrices are bound by the
// latency of one launch and two dependent loads (100 x 2048: 3.4 us, 2048 x 2048: 3.5 us).
// The D tile of 16x16x32 instructions has a row a token: up to 4 activation rows sit in D
// rows 0, 4, 8, 12 (JN = 1), so each lane scales one value a group instead of four.
template <int XT, bool SF32, int GROUP, int JN, int KW>
__global__ __launch_bounds__(kQ4Waves * 64) void k_q4(const Q4Args a, int slab) {
    constexpr int PL = XT == SEEDMM_F32 ? 3 : 1;       // operand rows a token
    constexpr int EB = XT == SEEDMM_I8 ? 1 : 2;
    constexpr int NG = 128 / GROUP;                    // groups of 128 columns
    constexpr int WAVES = kQ4Waves, RW = WAVES / KW, SS = 2;
    constexpr int SXW = JN == 1 ? 4 : 16;
    constexpr int SC = SS * 128;                       // columns of a wave's slab
    __shared__ float red[KW][RW][JN * 4][17];
    constexpr int CR = 4 * SS;                         // 16-byte pieces of a row in it
    __shared__ u32x4 bounce[WAVES][16 * CR];
    extern __shared__ __align__(16) char lds[];
    const int rowb = slab * EB + 16;
    float* sx = (float*)lds;                                     // [slab / GROUP][SXW]
    char* xs = lds + (size_t)(slab / GROUP) * SXW * 4;           // [rows][rowb]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kw = wave % KW, rw = wave / KW;
    const int r = lane & 15, q = lane >> 4;
    const int rows = a.N * PL;                                   // <= 4 (JN = 1) or 16
    const int64_t m0 = ((int64_t)blockIdx.x * RW + rw) * 16;
    const int64_t row = m0 + r < a.M ? m0 + r : a.M - 1;
    const int G = a.K / GROUP;
    // this lane's piece of load i: row lrow[i], columns 32 lcol ..
    const int lcol = lane % CR, lsub = lane / CR;
    const uint32_t* lrow[SS];
#pragma unroll
    for (int i = 0; i < SS; ++i) {
        const int64_t m = m0 + 16 / SS * i + lsub;
        lrow[i] = a.w + (m < a.M ? m : a.M - 1) * (a.K / 8);
    }
    const int xrow = JN == 1 ? min(r >> 2, rows - 1) : min(r, rows - 1);
    const char* xl = xs + xrow * rowb + (XT == SEEDMM_I8 ? 8 : 16) * q;

    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < a.K; k0 += slab) {
        const int kn = min(slab, a.K - k0);
        u32x4 w[SS];
        Scales<SF32, NG * SS> ss, bs;
        // past K the last columns' codes are loaded again: they meet activations of zero
        auto load = [&](int c0) {
            const int k = k0 + c0 + 32 * lcol;
#pragma unroll
            for (int i = 0; i < SS; ++i) w[i] = *(const u32x4*)(lrow[i] + (k < a.K ? k : a.K - 32) / 8);
            const int g = (k0 + c0) / GROUP;
            ss.load(a.s, row * G + g, G - g);
            bs.load(a.b, row * G + g, G - g);
        };
        if (kw * SC < kn) load(kw * SC);
        if (k0) __syncthreads();
        const int per_row = slab / 8, units = a.N * per_row;
        constexpr int UB = 4;      // pieces in flight a thread
        for (int u0 = tid; u0 < units; u0 += WAVES * 64 * UB) {
            Raw8<XT> raw[UB];
#pragma unroll
            for (int i = 0; i < UB; ++i) {
                const int u = u0 + i * WAVES * 64, t = u / per_row, kk = (u - t * per_row) * 8;
                raw[i] = load8<XT>(a.x, (int64_t)t * a.ldx + k0 + kk, u < units && kk < kn);
            }
#pragma unroll
            for (int i = 0; i < UB; ++i) {
                const int u = u0 + i * WAVES * 64, t = u / per_row, kk = (u - t * per_row) * 8;
                if (u < units) {
                    float sum = place8<XT>(raw[i], xs + t * PL * rowb + kk * EB, rowb);
#pragma unroll
                    for (int d = 1; d < GROUP / 8; d *= 2) sum += __shfl_xor(sum, d);
                    if (kk % GROUP == 0) {
#pragma unroll
                        for (int p = 0; p < PL; ++p) sx[kk / GROUP * SXW + t * PL + p] = p ? 0.f : sum;
                    }
                }
            }
        }
        __syncthreads();
        // 128 columns from column 128 st of the staged ones: the wave's codes, and its scales
        // from group 128 j / GROUP of the slab's
        auto step = [&](const u32x4& wv, const Scales<SF32, NG * SS>& sv, const Scales<SF32, NG * SS>& bv, int st, int j0) {
            uint32_t c[4] = {wv[0], wv[1], wv[2], wv[3]};
            transpose_quarters(c);
            const char* xp = xl + st * 128 * EB;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const int gl = st * NG + g;
                f32x4 d = {0.f, 0.f, 0.f, 0.f};
                if constexpr (XT == SEEDMM_I8) {
                    i32x4 di = {0, 0, 0, 0};
                    if constexpr (GROUP == 32) {
                        const long xa = *(const long*)(xp + 32 * g);
                        di = __builtin_amdgcn_mfma_i32_16x16x32_i8(xa, __builtin_bit_cast(long, codes_i8(c[g])), di, 0, 0, 0);
                    } else {
#pragma unroll
                        for (int j = g * (GROUP / 32); j < (g + 1) * (GROUP / 32); j += 2) {
                            const u32x2 x0 = *(const u32x2*)(xp + 32 * j), x1 = *(const u32x2*)(xp + 32 * j + 32);
                            const u32x2 c0 = codes_i8(c[j]), c1 = codes_i8(c[j + 1]);
                            di = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                                i32x4{(int)x0[0], (int)x0[1], (int)x1[0], (int)x1[1]},
                                i32x4{(int)c0[0], (int)c0[1], (int)c1[0], (int)c1[1]}, di, 0, 0, 0);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < JN; ++j) d[j] = (float)di[j];
                } else {
#pragma unroll
                    for (int j = g * (GROUP / 32); j < (g + 1) * (GROUP / 32); ++j)
                        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(*(const bf16x8*)(xp + 64 * j), codes_bf16(c[j]), d, 0, 0, 0);
                }
                const float s = sv.get(j0 * NG + g), b = bv.get(j0 * NG + g);
                if constexpr (JN == 1) {
                    acc[0] = __builtin_fmaf(s, d[0], __builtin_fmaf(b, sx[gl * 4 + q], acc[0]));
                } else {
                    const f32x4 X = *(const f32x4*)&sx[gl * 16 + 4 * q];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[j] = __builtin_fmaf(s, d[j], __builtin_fmaf(b, X[j], acc[j]));
                }
            }
        };
        for (int c0 = kw * SC; c0 < kn; c0 += KW * SC) {
            const Scales<SF32, NG * SS> sc = ss, bc = bs;
            u32x4 v[SS];
            u32x4* const bw = bounce[wave];
#pragma unroll
            for (int i = 0; i < SS; ++i) {
                const int lr = 16 / SS * i + lsub;
                bw[piece<CR>(lr, lcol)] = w[i];
            }
            wave_order();
#pragma unroll
            for (int j = 0; j < SS; ++j) v[j] = bw[piece<CR>(r, 4 * j + q)];
            wave_order();
            if (c0 + KW * SC < kn) load(c0 + KW * SC);
#pragma unroll
            for (int j = 0; j < SS; ++j)
                if (c0 + 128 * j < kn) step(v[j], sc, bc, c0 / 128 + j, j);
        }
    }
    // the KW partial tiles meet in LDS in their order; D column = weight row
#pragma unroll
    for (int j = 0; j < JN; ++j) red[kw][rw][JN * q + j][r] = acc[j];
    __syncthreads();
    for (int u = tid; u < RW * 16 * a.N; u += WAVES * 64) {
        const int c = u & 15, h = (u >> 4) % RW, t = (u >> 4) / RW;
        const int64_t m = ((int64_t)blockIdx.x * RW + h) * 16 + c;
        if (m >= a.M) continue;
        float v = 0.f;
#pragma unroll
        for (int p = PL - 1; p >= 0; --p) {
            float e = red[0][h][t * PL + p][c];
#pragma unroll
            for (int k = 1; k < KW; ++k) e += red[k][h][t * PL + p][c];
            v += e;
        }
        if constexpr (XT == SEEDMM_I8) v *= a.xs[t];
        const int64_t o = (int64_t)t * a.ldy + m;
        if (a.y_bf16) ((uint16_t*)a.y)[o] = f32_to_bf16(v);
        else ((float*)a.y)[o] = v;
    }
}

// Many tokens.  k_q4_rows writes the activations once as bf16 rows in the operands' order
// (fp32: three planes) and the groups' sums as three bf16 planes; k_q4_wide multiplies tiles
// of them with the codes on 32x32x16 instructions.  In products with little to lay out it
// takes the rows as they are (RAW), with no launch before it.
//
// With laid-out rows the bias term is a product of its own over the groups, sum_g b[m][g]
// X[n][g]: it starts the accumulators with matrix instructions (3 for 16 groups; 6 with fp32
// biases, which are split as well: of the nine products of parts those of 2^-22 and less of
// the term are left out), so the vector units only add s D, one fma an element a 64 columns.
//
// A workgroup takes 128 weight rows by 32 TT tokens, a wave 32 of the rows.  Lane r + 32 h loads the
// 16 bytes of row r that hold columns 32 h .. 32 h + 31 of a 64-column step: word j is its
// operand of instruction j with no exchange (groups of 32: after one swap of the halves).
constexpr int kQ4Band = 512;
struct Q4Wide {
    Q4Args a;
    const uint16_t* xp;   // [PL][N][Kp] rows in the operands' order, zero past K
    const uint16_t* xg;   // [3][N][Gp] group sums, zero past K / group
    float* part;          // [S][N][M] partial sums (S = 1: null)
    int Kp, Gp, ksplit;   // columns a split
    int tn, tm;           // tiles of tokens and of weight rows
};

__device__ __forceinline__ void split3(float f, uint32_t (&p)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        p[i] = __float_as_uint(f) & 0xFFFF0000u;
        f -= __uint_as_float(p[i]);
    }
}

// One thread a run of 8 columns; the lanes of a group add their sums.
template <int XT, int GROUP>
__global__ __launch_bounds__(256) void k_q4_rows(const Q4Args a, uint16_t* xp, uint16_t* xg, int Kp, int Gp) {
    const int per = Kp / 8;
    const int64_t all = (int64_t)a.N * per, plane = (int64_t)a.N * Kp, gplane = (int64_t)a.N * Gp;
    // a wave's 64 runs start at a multiple of the group's, and so do the rows
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < (all + 63) / 64 * 64; u += (int64_t)gridDim.x * 256) {
        const int64_t n = u / per;
        const int kk = (int)(u - n * per) * 8;
        const bool in = u < all, ok = in && kk < a.K;
        float sum = 0.f;
        if (in) {
            if constexpr (XT == SEEDMM_I8) {
                sum = place8_as_bf16(load8<XT>(a.x, n * a.ldx + kk, ok), (char*)(xp + n * Kp + kk));
            } else {
                sum = place8<XT>(load8<XT>(a.x, n * a.ldx + kk, ok), (char*)(xp + n * Kp + kk), plane * 2);
            }
        }
#pragma unroll
        for (int d = 1; d < GROUP / 8; d *= 2) sum += __shfl_xor(sum, d);
        if (ok && kk % GROUP == 0) {
            uint32_t p[3];
            split3(sum, p);
#pragma unroll
            for (int i = 0; i < 3; ++i) xg[i * gplane + n * Gp + kk / GROUP] = (uint16_t)(p[i] >> 16);
        }
        // the padding groups of a row
        const int G = a.K / GROUP;
        if (in)
            for (int g = G + kk / 8; g < Gp; g += per)
#pragma unroll
                for (int i = 0; i < 3; ++i) xg[i * gplane + n * Gp + g] = 0;
    }
}

typedef float f32x16 __attribute__((ext_vector_type(16)));

// RAW: the type of activation rows taken as they are (-1: laid out by k_q4_rows).  They are
// put in the operands' order on their way to LDS, where the groups' sums go as well; the
// bias term is then one more fma an element and group.
template <int RAW, int PL, bool SF32, int GROUP, int TT, int SP, int OCC>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(OCC))) void k_q4_wide(const Q4Wide c) {
    constexpr int BT = 32 * TT, BM = 128, NTH = 256;
    constexpr int NST = PL * BT * 8 / NTH;      // 16-byte pieces of a step a thread stages
    constexpr int CW = 2 * SP;                  // 16-byte pieces of a weight row in a slab
    constexpr int NWT = BM * CW / NTH;
    static_assert(PL * BT * 8 % NTH == 0 && BM * CW % NTH == 0, "whole pieces");
    __shared__ u32x4 xs[SP][PL * BT * 8];
    __shared__ u32x4 ws[BM * CW];
    constexpr bool LAID = RAW < 0;
    static_assert(LAID || (PL == 1 && TT == 1), "raw rows: one tile a wave");
    constexpr int XB = RAW == SEEDMM_I8 ? 1 : 2;          // bytes of a staged element
    constexpr int NGB = 64 * SP / GROUP;                  // groups a slab
    __shared__ __align__(16) float gx[LAID ? 1 : NGB][LAID ? 4 : BT];
    const Q4Args& a = c.a;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 31, h = lane >> 5;
    // workgroups of one XCD (every eighth) take neighbouring tiles: columns of kQ4Band tokens
    // by all weight rows, so that its L2 holds the activations of a column
    const int total = c.tn * c.tm;
    int id = blockIdx.x;
    if (total % 8 == 0) id = (id & 7) * (total >> 3) + (id >> 3);
    constexpr int GT = kQ4Band / BT;
    const int col = id / (GT * c.tm), in = id - col * GT * c.tm;
    const int width = min(GT, c.tn - col * GT);
    const int n0 = (col * GT + in % width) * BT;
    const int64_t mb = (int64_t)(in / width) * BM, m0 = mb + 32 * wave;
    const int kb = blockIdx.y * c.ksplit, ke = min(a.K, kb + c.ksplit);
    const int G = a.K / GROUP;

    // Slabs of SP steps (64 columns each).  Piece u of a step = 16 bytes `u & 7` of tile row
    // u >> 3; the codes likewise, CW pieces a row.
    int64_t src[NST], wsrc[NWT];
    int dst[NST], wdst[NWT];
#pragma unroll
    for (int i = 0; i < NST; ++i) {
        const int u = i * NTH + tid, row = u >> 3, p = row / BT, t = row % BT;
        if constexpr (LAID) src[i] = ((int64_t)p * a.N + min(n0 + t, a.N - 1)) * c.Kp + 8 * (u & 7);
        else src[i] = (int64_t)min(n0 + t, a.N - 1) * a.ldx + 8 * (u & 7);
        dst[i] = piece<8>(row, u & 7);
    }
#pragma unroll
    for (int i = 0; i < NWT; ++i) {
        const int u = i * NTH + tid, row = u / CW;
        wsrc[i] = (mb + row < a.M ? mb + row : a.M - 1) * (a.K / 8);
        wdst[i] = piece<CW>(row, u % CW);
    }
    const int64_t row = m0 + r < a.M ? m0 + r : a.M - 1;
    constexpr int NG = GROUP == 32 ? 2 : 1;               // groups a step
    constexpr int NGS = 64 * SP >= GROUP ? 64 * SP / GROUP : 1;
    u32x4 stage[SP][NST], wstage[NWT];
    Scales<SF32, NGS> snext, bnext;      // (biases with raw rows only)
    // Activations are zero past K.  There the codes of the row's last columns are loaded
    // again, and scales are 0.
    auto fetch = [&](int k) {
#pragma unroll
        for (int b = 0; b < SP; ++b)
#pragma unroll
            for (int i = 0; i < NST; ++i) {
                if constexpr (LAID) {
                    stage[b][i] = *(const u32x4*)(c.xp + src[i] + k + 64 * b);
                } else {
                    const Raw8<RAW> v = load8<RAW>(a.x, src[i] + k + 64 * b, k + 64 * b + 8 * (tid & 7) < a.K);
#pragma unroll
                    for (int j = 0; j < 2 * XB; ++j) stage[b][i][j] = v.u[j];
                }
            }
#pragma unroll
        for (int i = 0; i < NWT; ++i) {
            const int kw = k + 32 * ((i * NTH + tid) % CW);
            wstage[i] = *(const u32x4*)(a.w + wsrc[i] + (kw < a.K ? kw : a.K - 32) / 8);
        }
        snext.load(a.s, row * G + k / GROUP, G - k / GROUP);
        if constexpr (!LAID) bnext.load(a.b, row * G + k / GROUP, G - k / GROUP);
    };
    auto put = [&]() {
#pragma unroll
        for (int i = 0; i < NST; ++i) {
            float sum[SP];
#pragma unroll
            for (int b = 0; b < SP; ++b) {
                if constexpr (LAID) {
                    xs[b][dst[i]] = stage[b][i];
                } else {
                    Raw8<RAW> v;
#pragma unroll
                    for (int j = 0; j < 2 * XB; ++j) v.u[j] = stage[b][i][j];
                    if constexpr (RAW == SEEDMM_I8) sum[b] = place8_as_bf16(v, (char*)&xs[b][dst[i]]);
                    else sum[b] = place8<RAW>(v, (char*)&xs[b][dst[i]], 0);
                }
            }
            if constexpr (!LAID) {
                const int t = (i * NTH + tid) >> 3;
#pragma unroll
                for (int b = 0; b < SP; ++b) {
                    if (GROUP == 128 && (b & 1)) continue;
                    float v = sum[b];
                    if constexpr (GROUP == 128) v += sum[b + 1];
#pragma unroll
                    for (int d = 1; d < (GROUP < 64 ? GROUP / 8 : 8); d *= 2) v += __shfl_xor(v, d);
                    if (GROUP == 32 ? (tid & 3) == 0 : (tid & 7) == 0)
                        gx[64 * b / GROUP + (GROUP == 32 ? (tid & 7) >> 2 : 0)][t] = v;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NWT; ++i) ws[wdst[i]] = wstage[i];
    };

    f32x16 acc[TT];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[tt][i] = 0.f;
    fetch(kb);
    if constexpr (LAID) {   // bias term: the splits take 16 groups in turn
        for (int g0 = 16 * blockIdx.y; g0 < G; g0 += 16 * gridDim.y) {
            const int gl = g0 + 8 * h;
            bf16x8 bb[SF32 ? 3 : 1];
            Scales<SF32, 8> b;
            b.load(a.b, row * G + min(gl, G), G - min(gl, G));
            if constexpr (SF32) {
                uint32_t p[8][3];
#pragma unroll
                for (int i = 0; i < 8; ++i) split3(b.get(i), p[i]);
#pragma unroll
                for (int q = 0; q < 3; ++q) {
                    u32x4 o;
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = (p[2 * i][q] >> 16) | p[2 * i + 1][q];
                    bb[q] = __builtin_bit_cast(bf16x8, o);
                }
            } else {
                bb[0] = __builtin_bit_cast(bf16x8, u32x4{b.u[0], b.u[1], b.u[2], b.u[3]});
            }
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) {
                const int n = min(n0 + 32 * tt + r, a.N - 1);
                bf16x8 xa[3];
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    xa[p] = *(const bf16x8*)(c.xg + ((int64_t)p * a.N + n) * c.Gp + gl);
#pragma unroll
                for (int q = 0; q < (SF32 ? 3 : 1); ++q)
#pragma unroll
                    for (int p = 0; p + q < 3; ++p)
                        acc[tt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xa[p], bb[q], acc[tt], 0, 0, 0);
            }
        }
    }
    put();
    __syncthreads();

    // Tile i's chain of instructions runs while the vector units add tile i - 1 (the last
    // tile's addition is carried into the next step) and unpack the next codes.
    constexpr int JC = 4 / NG, LAST = TT == 1 ? 1 : (TT - 1) & 1;   // instructions a group; the carried d
    static_assert(TT == 1 || TT % 2 == 0, "the carried tile's sums are not the first's");
    f32x16 d[2][NG];
    float sp[NG];                              // the carried tile's scales
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        sp[g] = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) d[LAST][g][i] = 0.f;
    }
    // A slab's activations, codes and scales are loaded while the one before is multiplied
    // and take its place in LDS after it.
    Scales<SF32, NGS> sc = snext, bc;
    if constexpr (!LAID) bc = bnext;
    auto step = [&](int b) {
        const int wr = 32 * wave + r;
        const u32x4 wv = ws[piece<CW>(wr, 2 * b + h)];
        uint32_t w[4] = {wv[0], wv[1], wv[2], wv[3]};
        if constexpr (GROUP == 32) {
            auto x = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
            auto y = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
            w[0] = x[0]; w[2] = x[1]; w[1] = y[0]; w[3] = y[1];
        }
        float s[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) s[g] = sc.get(64 * b / GROUP + g);
        bf16x8 bq[4], xa[PL][4];
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
            const int t = 32 * tt + r;
#pragma unroll
            for (int p = 0; p < PL; ++p)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int ch = GROUP == 32 ? 4 * (j >> 1) + 2 * h + (j & 1) : 4 * h + j;
                    xa[p][j] = __builtin_bit_cast(bf16x8, xs[b][piece<8>(p * BT + t, ch)]);
                }
            if (tt == 0) {
#pragma unroll
                for (int j = 0; j < 4; ++j) bq[j] = codes_bf16(w[j]);
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                f32x16 e = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int p = 0; p < PL; ++p)
#pragma unroll
                    for (int j = g * JC; j < (g + 1) * JC; ++j)
                        e = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xa[p][j], bq[j], e, 0, 0, 0);
                d[tt & 1][g] = e;
            }
            const int q = (tt + TT - 1) % TT;      // the tile before
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const float sq = tt == 0 ? sp[g] : s[g];
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    acc[q][v] = __builtin_fmaf(sq, d[tt == 0 ? LAST : q & 1][g][v], acc[q][v]);
            }
            if constexpr (TT == 1) {
#pragma unroll
                for (int g = 0; g < NG; ++g) d[1][g] = d[0][g];
            }
        }
        if constexpr (!LAID) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                if (GROUP == 128 && (b & 1)) continue;
                const float bv = bc.get(64 * b / GROUP + g);
                const float* const x = gx[64 * b / GROUP + g];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x4 X = *(const f32x4*)(x + 8 * q + 4 * h);
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        acc[0][4 * q + v] = __builtin_fmaf(bv, X[v], acc[0][4 * q + v]);
                }
            }
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) sp[g] = s[g];
        // spread the vector work between the instructions of a step (4096 x 8192 x 2048:
        // 200 -> 190 us; one tile a wave gains nothing by it)
        if constexpr (TT == 2 && PL == 1) {
#pragma unroll
            for (int i = 0; i < 4 * TT; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 8, 0);
            }
        }
    };
    for (int k = kb; k < ke; k += 64 * SP) {
        const bool more = k + 64 * SP < ke;
        if (more) fetch(k + 64 * SP);
#pragma unroll
        for (int b = 0; b < SP; ++b)
            if (k + 64 * b < ke) step(b);
        if (more) {
            __syncthreads();
            put();
            sc = snext;
            if constexpr (!LAID) bc = bnext;
            __syncthreads();
        }
    }
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int v = 0; v < 16; ++v)
            acc[TT - 1][v] = __builtin_fmaf(sp[g], d[LAST][g][v], acc[TT - 1][v]);

#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int n = n0 + 32 * tt + 8 * (i >> 2) + 4 * h + (i & 3);
            const int64_t m = m0 + r;
            if (n >= a.N || m >= a.M) continue;
            if (c.part) {
                c.part[((int64_t)blockIdx.y * a.N + n) * a.M + m] = acc[tt][i];
            } else {
                const float v = a.xs ? acc[tt][i] * a.xs[n] : acc[tt][i];
                const int64_t o = (int64_t)n * a.ldy + m;
                if (a.y_bf16) ((uint16_t*)a.y)[o] = f32_to_bf16(v);
                else ((float*)a.y)[o] = v;
            }
        }
}

// y = the S partial sums in their order
__global__ __launch_bounds__(256) void k_q4_join(const Q4Args a, const float* part, int S) {
    const int64_t n = (int64_t)a.N * a.M;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        float v = part[i];
        for (int s = 1; s < S; ++s) v += part[s * n + i];
        const int64_t t = i / a.M, m = i - t * a.M;
        if (a.xs) v *= a.xs[t];
        const int64_t o = t * a.ldy + m;
        if (a.y_bf16) ((uint16_t*)a.y)[o] = f32_to_bf16(v);
        else ((float*)a.y)[o] = v;
    }
}

// K = 0: y = 0
__global__ __launch_bounds__(256) void k_q4_zero(void* y, int y_bf16, int ldy, int M, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t o = i / M * ldy + i % M;
        if (y_bf16) ((uint16_t*)y)[o] = 0;
        else ((float*)y)[o] = 0.f;
    }
}

// ----------------------------------------------------------------------------------
// seedmm_add_norm.  r = x + delta in fp32; out = r rsqrt(mean r^2 + eps) w.  The 8-bit
// scale is max |r w| times the row's factor over 127: one pass finds both statistics, and
// a row stays in registers between its load and its store (rows up to 32,768 elements;
// longer ones are read twice).  A row whose mean square fp32 does not hold is multiplied by
// a power of two, exactly, and summed again (asking for it costs 0.08 us of 2.6 at one token
// and nothing that shows at 4096 x 2048).
// ----------------------------------------------------------------------------------
struct NormArgs {
    const void* x;
    const void* d;       // null: none
    const void* w;       // null: ones
    void* res;           // null: not written
    void* out;
    float* scale;
    int x_dt, d_dt, w_dt, out_dt;
    int64_t ldx, ldd, ldr, ldo;
    int N, H;
    float eps;
};

__device__ __forceinline__ float load_el(const void* p, int dt, int64_t i) {
    return dt == SEEDMM_F32 ? ((const float*)p)[i] : bf16_to_f32(((const uint16_t*)p)[i]);
}

// The mean square plus eps, where fp32 holds it: below 2^-100 the squares' underflow (2^-126 at
// most a square) could show in it, above the squares overflow.
__device__ __forceinline__ bool mean_holds(float t) { return t >= 0x1p-100f && t < INFINITY; }
// The factor of a row outside of that from the sum of its squares, the row taken times 2^up.
__device__ __forceinline__ float scaled_factor(const NormArgs& a, float ss, int up) {
    return (float)(1.0 / sqrt((double)ss / (double)a.H + ldexp((double)a.eps, 2 * up)));
}

// For 8 bits a row's scale and the scale's reciprocal (0: codes 0).
struct RowScale {
    float sc, inv;
};
__device__ __forceinline__ RowScale row_scale(const NormArgs& a, float f, float top) {
    RowScale o = {0.f, 0.f};
    if (a.out_dt == SEEDMM_I8) {
        o.sc = fmaxf(top * f / 127.0f, 1.17549435e-38f);
        // a row with an infinity or NaN: codes 0 and scale NaN
        if (!(top * f < INFINITY)) o.sc = NAN;
        o.inv = o.sc == o.sc ? 1.0f / o.sc : 0.f;
    }
    return o;
}
// TPR threads a row (a wave, or a workgroup), NP pieces of 8 elements a thread.
template <int TPR, int NP, int XT, int DT>   // DT: -1 = no delta
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_add_norm(const NormArgs a) {
    constexpr int NW = TPR / 64;
    __shared__ float red[2][NW];
    const int tid = TPR < 256 ? threadIdx.x % TPR : threadIdx.x;
    const int64_t n = TPR < 256 ? (int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR : blockIdx.x;
    if (n >= a.N) return;      // (a whole wave; workgroups of one row all have it)
    Eight<XT> x[NP];
    Eight<DT < 0 ? SEEDMM_BF16 : DT> d[NP];
    int cnt[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int h = (p * TPR + tid) * 8;
        cnt[p] = min(8, a.H - h);
        if (cnt[p] > 0) {
            x[p].load(a.x, n * a.ldx + h, cnt[p]);
            if constexpr (DT >= 0) d[p].load(a.d, n * a.ldd + h, cnt[p]);
        }
    }
    float w[NP][8];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int h = (p * TPR + tid) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) w[p][j] = 1.f;
        if (a.w && cnt[p] > 0) {
            if (a.w_dt == SEEDMM_F32) {
                Eight<SEEDMM_F32> e;
                e.load(a.w, h, cnt[p]);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[p][j] = e.get(j);
            } else {
                Eight<SEEDMM_BF16> e;
                e.load(a.w, h, cnt[p]);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[p][j] = e.get(j);
            }
        }
    }
    float r[NP][8], ss = 0.f, top = 0.f;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float v = 0.f;
            if (cnt[p] > 0) {
                v = x[p].get(j);
                if constexpr (DT >= 0) v += d[p].get(j);
            }
            r[p][j] = v;
            ss = __builtin_fmaf(v, v, ss);
        }
        if (a.res && cnt[p] > 0) store8<XT>(a.res, n * a.ldr + (p * TPR + tid) * 8, cnt[p], r[p]);
    }
    // Both are inlined at both of their places: else the row's arrays go to scratch memory
    // (1021 x 7167: 45 us, 27 inlined).
    // max |r w| of this thread; infinite where one is not finite
    auto weighted = [&]() __attribute__((always_inline)) {
        float m = 0.f;
        bool bad = false;
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = fabsf(r[p][j] * w[p][j]);
                m = fmaxf(m, v);
                bad |= !(v < INFINITY);
            }
        return bad ? INFINITY : m;
    };
    // both statistics over the row's threads
    auto row_stats = [&]() __attribute__((always_inline)) {
        ss = wave_sum(ss);
        if (a.out_dt == SEEDMM_I8) top = wave_max(top);
        if constexpr (NW > 1) {
            const int wave = threadIdx.x >> 6;
            if ((threadIdx.x & 63) == 0) { red[0][wave] = ss; red[1][wave] = top; }
            __syncthreads();
            ss = red[0][0]; top = red[1][0];
#pragma unroll
            for (int i = 1; i < NW; ++i) { ss += red[0][i]; top = fmaxf(top, red[1][i]); }
        }
    };
    if (a.out_dt == SEEDMM_I8) top = weighted();
    row_stats();
    const float t = ss / (float)a.H + a.eps;
    float f = 1.0f / sqrtf(t);
    const bool out_of_range = !mean_holds(t) || (a.out_dt == SEEDMM_I8 && !(top < INFINITY));
    if (__builtin_expect(__builtin_amdgcn_readfirstlane(out_of_range), 0)) {   // (all of the row's threads)
        float big = 0.f;
        bool bad = false;
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                big = fmaxf(big, fabsf(r[p][j]));
                bad |= !(fabsf(r[p][j]) < INFINITY);
            }
        big = wave_max(bad ? INFINITY : big);
        if constexpr (NW > 1) {
            __syncthreads();    // the statistics have been read
            if ((threadIdx.x & 63) == 0) red[0][threadIdx.x >> 6] = big;
            __syncthreads();
            big = red[0][0];
#pragma unroll
            for (int i = 1; i < NW; ++i) big = fmaxf(big, red[0][i]);
            __syncthreads();
        }
        if (big > 0.f && big < INFINITY) {
            const int up = -ilogbf(big);
            ss = 0.f;
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    r[p][j] = ldexpf(r[p][j], up);
                    ss = __builtin_fmaf(r[p][j], r[p][j], ss);
                }
            top = a.out_dt == SEEDMM_I8 ? weighted() : 0.f;
            row_stats();
            f = scaled_factor(a, ss, up);
        }
    }
    const RowScale o = row_scale(a, f, top);
    if (a.out_dt == SEEDMM_I8 && tid == 0) a.scale[n] = o.sc;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        if (cnt[p] <= 0) continue;
        const int64_t at = n * a.ldo + (p * TPR + tid) * 8;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = r[p][j] * w[p][j] * f;
        if (a.out_dt == SEEDMM_I8) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = code_of(v[j], o.inv);
            store8<SEEDMM_I8>(a.out, at, cnt[p], v);
        } else if (a.out_dt == SEEDMM_F32) {
            store8<SEEDMM_F32>(a.out, at, cnt[p], v);
        } else {
            store8<SEEDMM_BF16>(a.out, at, cnt[p], v);
        }
    }
}

// Rows of any length, read twice (four times outside of fp32's range).  The step past the end
// of a row of nearly 2^31 elements needs more than 31 bits.
__global__ __launch_bounds__(1024) void k_add_norm_long(const NormArgs a) {
    __shared__ float red[2][16];
    const int64_t n = blockIdx.x;
    // max |r w| and the sum of squares of the row times 2^up, or max |r| (up: NULL); infinite
    // where one is not finite
    float ss, top;
    auto pass = [&](const int* up) {
        ss = top = 0.f;
        bool bad = false;
        for (int64_t h = threadIdx.x; h < a.H; h += 1024) {
            float r = load_el(a.x, a.x_dt, n * a.ldx + h);
            if (a.d) r += load_el(a.d, a.d_dt, n * a.ldd + h);
            if (up) r = ldexpf(r, *up);
            const float v = up && a.w ? r * load_el(a.w, a.w_dt, h) : r;
            ss = __builtin_fmaf(r, r, ss);
            top = fmaxf(top, fabsf(v));
            bad |= !(fabsf(v) < INFINITY);
        }
        ss = wave_sum(ss);
        top = wave_max(bad ? INFINITY : top);
        __syncthreads();    // the pass before has been read
        if ((threadIdx.x & 63) == 0) { red[0][threadIdx.x >> 6] = ss; red[1][threadIdx.x >> 6] = top; }
        __syncthreads();
        ss = red[0][0]; top = red[1][0];
        for (int i = 1; i < 16; ++i) { ss += red[0][i]; top = fmaxf(top, red[1][i]); }
    };
    int up = 0;
    pass(&up);
    const float t = ss / (float)a.H + a.eps;
    float f = 1.0f / sqrtf(t);
    if (!mean_holds(t) || (a.out_dt == SEEDMM_I8 && !(top < INFINITY))) {   // (the whole workgroup)
        const float top0 = top;
        pass(nullptr);
        if (top > 0.f && top < INFINITY) {
            up = -ilogbf(top);
            pass(&up);
            f = scaled_factor(a, ss, up);
        } else {
            top = top0;
        }
    }
    const RowScale o = row_scale(a, f, top);
    if (a.out_dt == SEEDMM_I8 && threadIdx.x == 0) a.scale[n] = o.sc;
    for (int64_t h = threadIdx.x; h < a.H; h += 1024) {
        float r = load_el(a.x, a.x_dt, n * a.ldx + h);
        if (a.d) r += load_el(a.d, a.d_dt, n * a.ldd + h);
        const float rs = ldexpf(r, up), v = (a.w ? rs * load_el(a.w, a.w_dt, h) : rs) * f;
        if (a.res) {
            if (a.x_dt == SEEDMM_F32) ((float*)a.res)[n * a.ldr + h] = r;
            else ((uint16_t*)a.res)[n * a.ldr + h] = f32_to_bf16(r);
        }
        if (a.out_dt == SEEDMM_I8) ((int8_t*)a.out)[n * a.ldo + h] = (int8_t)(int)code_of(v, o.inv);
        else if (a.out_dt == SEEDMM_F32) ((float*)a.out)[n * a.ldo + h] = v;
        else ((uint16_t*)a.out)[n * a.ldo + h] = f32_to_bf16(v);
    }
}

// ----------------------------------------------------------------------------------
// seedmm_route.  One wave a token, expert i * 64 + lane in register i.  A key orders the
// eligible scores above 1 and the ineligible experts (logit NaN or -inf) at 1.
//
// The top_k-th largest of the 64 lane maxima is a lower bound of the top_k-th largest key,
// and few keys reach it (about top_k + 2 of 512 for top_k = 10).  Those go to a lane each,
// through LDS, and every one's rank is the number of larger ones (equal: of lower experts):
// rank s < top_k is slot s.  Sigmoid scores are compared in 64 bits, but bounded in fp32:
// the bound is lowered by the fp32 scores' error, and only the candidates are scored again.
// Where more than 64 reach the bound, or fewer than top_k lanes have an eligible expert,
// the largest key is taken top_k times instead.
// ----------------------------------------------------------------------------------
struct RouteArgs {
    const void* lg;
    const float* bias;
    int32_t* ids;
    float* w;
    int64_t ldl;
    int T, E, k, l_dt;
};

// order-preserving unsigned keys (-0 equals +0; every number above -inf is above 1)
__device__ __forceinline__ uint32_t key32(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unkey32(uint32_t k) {
    return __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ uint64_t key64(double f) {
    const uint64_t u = (uint64_t)__double_as_longlong(f + 0.0);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double sigmoid64(float l) { return 1.0 / (1.0 + exp(-(double)l)); }

// The largest key of the wave and the lowest expert i * 64 + lane that has it.
template <int NPL>
__device__ __forceinline__ uint32_t largest(const uint32_t (&key)[NPL], int lane, int& e) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < NPL; ++i) best = max(best, key[i]);
    best = wave_umax(best);
    e = -1;
    if constexpr (NPL <= 8) {
#pragma unroll
        for (int i = NPL - 1; i >= 0; --i) {
            const uint64_t m = __ballot(key[i] == best);
            if (m) e = i * 64 + __builtin_ctzll(m);
        }
    } else {
        uint32_t at = 0xFFFFFFFFu;
#pragma unroll
        for (int i = NPL - 1; i >= 0; --i)
            if (key[i] == best) at = i * 64 + lane;
        e = (int)wave_umin(at);
    }
    return best;
}
template <int NPL>
__device__ __forceinline__ uint64_t largest(const uint64_t (&key)[NPL], int lane, int& e) {
    uint64_t mine = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < NPL; ++i)
        if (key[i] > mine) { mine = key[i]; at = i; }
    const uint32_t hi = wave_umax((uint32_t)(mine >> 32));
    const uint32_t lo = wave_umax((uint32_t)(mine >> 32) == hi ? (uint32_t)mine : 0u);
    const uint64_t best = (uint64_t)hi << 32 | lo;
    e = (int)wave_umin(mine == best ? (uint32_t)(at * 64 + lane) : 0xFFFFFFFFu);
    return best;
}
template <int NPL, typename K>
__device__ __forceinline__ void clear_key(K (&key)[NPL], int lane, int e) {
#pragma unroll
    for (int i = 0; i < NPL; ++i)
        if (i * 64 + lane == e) key[i] = 0;
}

// sigmoid in fp32, off by less than 2^-22
__device__ __forceinline__ float sigmoid32(float l) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l * -1.44269504088896f));
}

template <int NPL, bool SIG, int LT>
__global__ __launch_bounds__(256) void k_route(const RouteArgs a) {
    __shared__ int cand[4][64];
    __shared__ float candl[4][64], candb[SIG ? 4 : 1][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    if (t >= a.T) return;
    float l[NPL], bias[SIG ? NPL : 1];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = i * 64 + lane;
        l[i] = e < a.E ? load_el(a.lg, LT, t * a.ldl + e) : 0.f;
        if constexpr (SIG) bias[i] = e < a.E && a.bias ? a.bias[e] : 0.f;
    }
    uint32_t key[NPL], top = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        float v = l[i];
        if constexpr (SIG) v = sigmoid32(l[i]) + bias[i];
        key[i] = i * 64 + lane >= a.E ? 0u : l[i] > -INFINITY && v > -INFINITY ? key32(v) : 1u;
        top = max(top, key[i]);
    }
    // the bound's bits from the top: the largest number that top_k lane maxima reach, or the
    // first that exactly top_k reach (the scalar unit counts; the vector units compare once)
    uint32_t bound = 0;
    for (uint32_t bit = 0x80000000u; bit; bit >>= 1) {
        const int c = __popcll(__ballot(top >= (bound | bit)));
        if (c >= a.k) bound |= bit;
        if (c == a.k) break;
    }
    const bool all = __popcll(__ballot(top > 1)) < a.k;      // too few lanes with an eligible expert
    // where lanes hold many experts more than 64 can reach it: raise it between bounds
    if constexpr (NPL >= 8) {
        auto reach = [&](uint32_t b) {
            int c = 0;
#pragma unroll
            for (int i = 0; i < NPL; ++i) c += __popcll(__ballot(key[i] >= b));
            return c;
        };
        if (!all && reach(bound) > 64) {
            uint32_t lo = bound, hi = 0xFFFFFFFFu;     // more than 64 reach lo
            while (lo < hi) {
                const uint32_t mid = lo + (hi - lo) / 2 + 1;
                const int c = reach(mid);
                if (c > 64) lo = mid;
                else if (c < a.k) hi = mid - 1;
                else { bound = mid; break; }
            }
        }
    }
    // fp32 scores are off by less than 2^-22 + 2^-24 |score|, two of them by twice that
    if constexpr (SIG) {
        const float b = unkey32(bound), low = b - 9.5367431640625e-7f * (1.0f + fabsf(b));
        if (low > -INFINITY) bound = key32(low);
    }
    int count = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const bool near = key[i] > 1 && key[i] >= bound;
        const uint64_t m = __ballot(near);
        const int at = count + __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
        if (near && at < 64) {
            cand[wave][at] = i * 64 + lane;
            candl[wave][at] = l[i];
            if constexpr (SIG) candb[wave][at] = bias[i];
        }
        count += __popcll(m);
    }

    int mine = 0, slot = -1;          // this lane's expert and its slot
    float ml = -INFINITY;             // its logit, -inf if it is masked
    double p = 0.0;                   // its sigmoid
    if (!all && count <= 64) {
        wave_order();
        if (lane < count) {
            mine = cand[wave][lane];
            ml = candl[wave][lane];
        }
        uint64_t k64 = 0;
        if (lane < count) {
            if constexpr (SIG) {
                p = sigmoid64(ml);
                k64 = key64(p + (double)candb[wave][lane]);
            } else {
                k64 = key32(ml);
            }
        }
        int rank = 0;
        for (int c = 0; c < count; ++c) {   // candidates are in the experts' order
            uint64_t o = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)k64, c);
            if constexpr (SIG) o |= (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(k64 >> 32), c) << 32;
            rank += o > k64 || (o == k64 && c < lane);
        }
        if (lane < count && rank < a.k) slot = rank;
    } else if constexpr (SIG) {
        uint64_t k64[NPL];
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            k64[i] = key[i] > 1 ? key64(sigmoid64(l[i]) + (double)bias[i]) : key[i];
        for (int s = 0; s < a.k; ++s) {
            int e;
            const uint64_t best = largest<NPL>(k64, lane, e);
            clear_key<NPL>(k64, lane, e);
            if (lane == s) { mine = e; slot = s; ml = best > 1 ? 0.f : -INFINITY; }
        }
        if (slot >= 0 && ml == 0.f) {
            ml = load_el(a.lg, LT, t * a.ldl + mine);
            p = sigmoid64(ml);
        }
    } else {
        for (int s = 0; s < a.k; ++s) {
            int e;
            const uint32_t best = largest<NPL>(key, lane, e);
            clear_key<NPL>(key, lane, e);
            if (lane == s) { mine = e; slot = s; ml = best > 1 ? unkey32(best) : -INFINITY; }
        }
    }

    const bool weighs = slot >= 0 && ml > -INFINITY;
    float w;
    if constexpr (SIG) {
        w = (float)p;
        // From logits of -60 up a sigmoid is an ordinary fp32 number (2^-87 at least); far below it
        // has fewer bits there, then none (e^-104): shares of the largest then, divided in 64 bits.
        if (__any(weighs && ml < -60.f)) {
            const uint64_t u = weighs ? (uint64_t)__double_as_longlong(p) : 0;   // p >= 0: in order
            const uint32_t hi = wave_umax((uint32_t)(u >> 32));
            const uint32_t lo = wave_umax((uint32_t)(u >> 32) == hi ? (uint32_t)u : 0u);
            const double most = __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
            w = most > 0.0 ? (float)(p / most) : 0.f;
        }
    } else {
        const float m = wave_max(weighs ? ml : -INFINITY);
        w = ml == m ? 1.0f : expf(ml - m);
    }
    if (!weighs) w = 0.f;
    const float sum = wave_sum(w);
    if (slot >= 0) {
        a.ids[t * a.k + slot] = mine;
        a.w[t * a.k + slot] = sum > 0.f ? w / sum : 0.f;
    }
}

constexpr int kMaxDim = 1 << 30;   // row and column indices of a tile stay in 32 bits
constexpr int kMaxTokens = kMaxDim - 64;   // and a row of token tiles in one launch

template <int XT, bool SF32, int GROUP, int JN, int KW>
void launch_q4_kw(const Q4Args& a, hipStream_t st) {
    constexpr int EB = XT == SEEDMM_I8 ? 1 : 2, PL = XT == SEEDMM_F32 ? 3 : 1, RW = kQ4Waves / KW;
    // the activation rows of a slab of columns in LDS, all columns if they fit
    const int rows = a.N * PL, unit = 256;
    const int per = unit * EB * rows + unit / GROUP * (JN == 1 ? 4 : 16) * 4;   // bytes of a unit of columns
    constexpr int room = 62 * 1024 - KW * RW * JN * 4 * 17 * 4 - kQ4Waves * 2048;
    int slab = (room - rows * 16) / per * unit;
    const int kround = (a.K + unit - 1) / unit * unit;
    if (slab > kround) slab = kround;
    const size_t lds = (size_t)slab / unit * per + rows * 16;
    const int64_t tiles = ((int64_t)a.M + 15) / 16;
    hipLaunchKernelGGL((k_q4<XT, SF32, GROUP, JN, KW>), dim3((unsigned)((tiles + RW - 1) / RW)),
                       dim3(kQ4Waves * 64), lds, st, a, slab);
}

// the product's weight rows m0 .. m0 + rows - 1
template <bool SF32, int GROUP>
Q4Args weight_rows(Q4Args a, int64_t m0, int64_t rows) {
    const int64_t g = m0 * (a.K / GROUP) * (SF32 ? 4 : 2);
    a.w += m0 * (a.K / 8);
    a.s = (const char*)a.s + g;
    a.b = (const char*)a.b + g;
    a.y = (char*)a.y + m0 * (a.y_bf16 ? 2 : 4);
    a.M = (int)(rows < a.M - m0 ? rows : a.M - m0);
    return a;
}

// The fewer row tiles, the more waves share one (us with 2, 4, 8 waves, one bf16 token:
// 131072 x 2048 30 33 39, 16384 x 8192 20 19 21, 8192 x 2048 6.0 5.1 5.1, 2048 x 2048
// 5.7 4.2 3.5; 16 tokens: 51 69 105, 35 35 51, 8.7 7.7 8.3, 7.8 6.4 5.7).
template <int XT, bool SF32, int GROUP, int JN>
void launch_q4_jn(const Q4Args& a, hipStream_t st) {
    const int64_t tiles = ((int64_t)a.M + 15) / 16;
    if (tiles >= 4096) launch_q4_kw<XT, SF32, GROUP, JN, 2>(a, st);
    else if (tiles >= 512) launch_q4_kw<XT, SF32, GROUP, JN, 4>(a, st);
    else launch_q4_kw<XT, SF32, GROUP, JN, 8>(a, st);
}

// The plan of a product with many tokens: what its workspace holds.
struct Q4Plan {
    bool wide;
    bool two;                      // tiles of 64 tokens, else of 32
    bool laid;                     // activations laid out by a launch of their own
    int Kp, Gp, S, ksplit, tn, tm;
    size_t xg, part, total;
};

Q4Plan q4_plan(int x_dtype, int group, int M, int K, int N) {
    Q4Plan p = {};
    const int PL = x_dtype == SEEDMM_F32 ? 3 : 1;
    p.wide = (int64_t)N * PL > 16 && M > 0 && K > 0;
    if (!p.wide) return p;
    p.Kp = (K + 255) / 256 * 256;
    p.Gp = (K / group + 15) / 16 * 16;
    // Tiles of 64 tokens by 128 weight rows where they make 512 workgroups (two a CU);
    // else of 32 by 128 with K split until they do (us by this rule, with tiles of 64 and K
    // split, with one split of K: 256 x 8192 x 2048 24.0 33.5 24.2, 61 x 5125 x 4160 19.9 23.0
    // 37.9, 64 x 8192 x 8192 31.1 31.6 49.5).  fp32 rows are three planes of work: always 64.
    const int64_t tm = ((int64_t)M + 127) / 128;
    p.two = PL == 3 || (((int64_t)N + 63) / 64) * tm >= 512;
    const int BT = p.two ? 64 : 32, slab = PL == 3 ? 128 : 256;
    p.tn = (int)(((int64_t)N + BT - 1) / BT);
    p.tm = (int)tm;
    const int slabs = (K + slab - 1) / slab;
    int64_t S = (511 + p.tn * tm) / (p.tn * tm);
    if (S > slabs) S = slabs;
    if (S > 16) S = 16;
    const int per = (int)((slabs + S - 1) / S);
    p.ksplit = per * slab;
    p.S = (slabs + per - 1) / per;
    // A launch that lays the rows out costs about 3 us; in the product it is done once a row
    // tile (61 x 5125 x 4160, 10 million elements so: 20.4 us laid out, 20.0 not; 64 x 8192 x
    // 8192, 34 million: 31.0 and 33.4; 4096 x 100 x 2048, 8 million: 23.4 and 16.1).
    p.laid = p.two || (int64_t)N * K > (1 << 24) / tm;
    if (p.laid) {
        p.xg = align_up((size_t)PL * (size_t)N * (size_t)p.Kp * 2);
        p.part = p.xg + align_up((size_t)3 * (size_t)N * (size_t)p.Gp * 2);
    }
    p.total = p.part + (p.S > 1 ? align_up((size_t)p.S * (size_t)N * (size_t)M * 4) : 0);
    return p;
}

template <int XT, bool SF32, int GROUP>
void launch_q4_group(const Q4Args& a, const Q4Plan& p, void* ws, hipStream_t st) {
    constexpr int PL = XT == SEEDMM_F32 ? 3 : 1;
    if (!p.wide) {
        constexpr int64_t rows = kLaunchThreads / (kQ4Waves * 64) * 16;   // a row tile a workgroup, or more
        for (int64_t m0 = 0; m0 < a.M; m0 += rows) {
            const Q4Args b = weight_rows<SF32, GROUP>(a, m0, rows);
            if (a.N * PL <= 4) launch_q4_jn<XT, SF32, GROUP, 1>(b, st);
            else launch_q4_jn<XT, SF32, GROUP, 4>(b, st);
        }
        return;
    }
    uint16_t* xp = (uint16_t*)ws;
    uint16_t* xg = (uint16_t*)((char*)ws + p.xg);
    if (p.laid) {
        const int64_t runs = (int64_t)a.N * (p.Kp / 8), blocks = (runs + 255) / 256;
        hipLaunchKernelGGL((k_q4_rows<XT, GROUP>), dim3((unsigned)(blocks < 65536 ? blocks : 65536)),
                           dim3(256), 0, st, a, xp, xg, p.Kp, p.Gp);
    }
    const int64_t most = kLaunchThreads / 256 / p.tn;     // row tiles a launch (in parts: S = 1)
    const int tms = (int)(p.tm <= most ? p.tm : most > 1 ? most : 1);
    for (int64_t m0 = 0; m0 < a.M; m0 += (int64_t)tms * 128) {
        const Q4Args b = weight_rows<SF32, GROUP>(a, m0, (int64_t)tms * 128);
        const int tm = (b.M + 127) / 128;
        Q4Wide c = {b, xp, xg, p.S > 1 ? (float*)((char*)ws + p.part) : nullptr, p.Kp, p.Gp, p.ksplit, p.tn, tm};
        const dim3 grid((unsigned)((int64_t)p.tn * tm), (unsigned)p.S);
        if constexpr (PL == 3) hipLaunchKernelGGL((k_q4_wide<-1, PL, SF32, GROUP, 2, 2, 2>), grid, dim3(256), 0, st, c);
        else if (p.two) hipLaunchKernelGGL((k_q4_wide<-1, PL, SF32, GROUP, 2, 4, 2>), grid, dim3(256), 0, st, c);
        else if (p.laid) hipLaunchKernelGGL((k_q4_wide<-1, PL, SF32, GROUP, 1, 4, 3>), grid, dim3(256), 0, st, c);
        else hipLaunchKernelGGL((k_q4_wide<XT, PL, SF32, GROUP, 1, 4, GROUP == 32 ? 2 : 3>), grid, dim3(256), 0, st, c);
    }
    if (p.S > 1) {
        const int64_t n = (int64_t)a.N * a.M, jb = (n + 255) / 256;
        hipLaunchKernelGGL(k_q4_join, dim3((unsigned)(jb < 65536 ? jb : 65536)), dim3(256), 0, st, a,
                           (const float*)((char*)ws + p.part), p.S);
    }
}

template <int XT, bool SF32>
void launch_q4(const Q4Args& a, int group, const Q4Plan& p, void* ws, hipStream_t st) {
    if (group == 32) launch_q4_group<XT, SF32, 32>(a, p, ws, st);
    else if (group == 64) launch_q4_group<XT, SF32, 64>(a, p, ws, st);
    else launch_q4_group<XT, SF32, 128>(a, p, ws, st);
}

template <bool SIG, int LT>
void launch_route_part(const RouteArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)((a.T - 1) / 4 + 1)), block(256);
    if (a.E <= 64) hipLaunchKernelGGL((k_route<1, SIG, LT>), grid, block, 0, st, a);
    else if (a.E <= 128) hipLaunchKernelGGL((k_route<2, SIG, LT>), grid, block, 0, st, a);
    else if (a.E <= 256) hipLaunchKernelGGL((k_route<4, SIG, LT>), grid, block, 0, st, a);
    else if (a.E <= 512) hipLaunchKernelGGL((k_route<8, SIG, LT>), grid, block, 0, st, a);
    else if (a.E <= 1024) hipLaunchKernelGGL((k_route<16, SIG, LT>), grid, block, 0, st, a);
    else if (a.E <= 2048) hipLaunchKernelGGL((k_route<32, SIG, LT>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_route<64, SIG, LT>), grid, block, 0, st, a);
}

template <bool SIG, int LT>
void launch_route(const RouteArgs& a, hipStream_t st) {
    constexpr int64_t tokens = kLaunchThreads / 64;
    for (int64_t t0 = 0; t0 < a.T; t0 += tokens) {
        RouteArgs p = a;
        p.lg = (const char*)a.lg + t0 * a.ldl * type_bytes(LT);
        p.ids += t0 * a.k;
        p.w += t0 * a.k;
        p.T = (int)(a.T - t0 < tokens ? a.T - t0 : tokens);
        launch_route_part<SIG, LT>(p, st);
    }
}

// the rows from n0 that one launch takes with `threads` a row
NormArgs norm_rows(NormArgs a, int64_t n0, int threads) {
    const int64_t rows = kLaunchThreads / threads;
    a.x = (const char*)a.x + n0 * a.ldx * type_bytes(a.x_dt);
    if (a.d) a.d = (const char*)a.d + n0 * a.ldd * type_bytes(a.d_dt);
    if (a.res) a.res = (char*)a.res + n0 * a.ldr * type_bytes(a.x_dt);
    a.out = (char*)a.out + n0 * a.ldo * type_bytes(a.out_dt);
    if (a.scale) a.scale += n0;
    a.N = (int)(a.N - n0 < rows ? a.N - n0 : rows);
    return a;
}

template <int TPR, int NP, int XT, int DT>
void launch_norm_as(const NormArgs& a, hipStream_t st) {
    const int rows = TPR < 256 ? 256 / TPR : 1;
    for (int64_t n0 = 0; n0 < a.N; n0 += kLaunchThreads / TPR) {
        const NormArgs p = norm_rows(a, n0, TPR);
        hipLaunchKernelGGL((k_add_norm<TPR, NP, XT, DT>), dim3((unsigned)((p.N - 1) / rows + 1)),
                           dim3(TPR < 256 ? 256 : TPR), 0, st, p);
    }
}

template <int XT, int DT>
void launch_norm(const NormArgs& a, hipStream_t st) {
    if (a.H <= 512) launch_norm_as<64, 1, XT, DT>(a, st);
    else if (a.H <= 2048) launch_norm_as<256, 1, XT, DT>(a, st);
    else if (a.H <= 4096) launch_norm_as<256, 2, XT, DT>(a, st);
    else if (a.H <= 8192) launch_norm_as<256, 4, XT, DT>(a, st);
    else if (a.H <= 16384) launch_norm_as<1024, 2, XT, DT>(a, st);
    else if (a.H <= 32768) launch_norm_as<1024, 4, XT, DT>(a, st);
    else {
        for (int64_t n0 = 0; n0 < a.N; n0 += kLaunchThreads / 1024) {
            const NormArgs p = norm_rows(a, n0, 1024);
            hipLaunchKernelGGL(k_add_norm_long, dim3((unsigned)p.N), dim3(1024), 0, st, p);
        }
    }
}

}  // namespace

extern "C" {

int seedmm_q4_gemv(const uint32_t* weight, const void* scales, const void* biases, int s_dtype,
                   int group, const void* x, int x_dtype, int ldx, const float* x_scale, void* y,
                   int y_dtype, int ldy, int M, int K, int N, void* workspace,
                   size_t workspace_bytes, void* hip_stream) {
    if (group != 32 && group != 64 && group != 128) return SEEDMM_EINVAL;
    if (M < 0 || K < 0 || N < 0 || M > kMaxDim || K > kMaxDim || N > kMaxTokens || K % group != 0 || ldx < K || ldy < M)
        return SEEDMM_EINVAL;
    if (!float_type(s_dtype) || !float_type(y_dtype)) return SEEDMM_EINVAL;
    if (!float_type(x_dtype) && x_dtype != SEEDMM_I8) return SEEDMM_EINVAL;
    if (M == 0 || N == 0) return SEEDMM_OK;
    if (!y) return SEEDMM_EINVAL;
    const int ymask = y_dtype == SEEDMM_F32 ? 3 : 1;
    if ((uintptr_t)y & ymask) return SEEDMM_EALIGN;
    hipStream_t st = (hipStream_t)hip_stream;
    if (K == 0) {   // empty product: y = 0 (a kernel, not a memset node, under capture)
        const int64_t n = (int64_t)N * M, blocks = (n + 255) / 256;
        hipLaunchKernelGGL(k_q4_zero, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256),
                           0, st, y, y_dtype == SEEDMM_BF16, ldy, M, n);
        return launch_status();
    }
    if (!weight || !scales || !biases || !x) return SEEDMM_EINVAL;
    if (x_dtype == SEEDMM_I8 ? !x_scale : x_scale != nullptr) return SEEDMM_EINVAL;
    const int smask = s_dtype == SEEDMM_F32 ? 3 : 1;
    if (!aligned16(weight) || !aligned16(x) || ((uintptr_t)scales & smask) ||
        ((uintptr_t)biases & smask) || ((uintptr_t)x_scale & 3))
        return SEEDMM_EALIGN;
    const int per16 = x_dtype == SEEDMM_F32 ? 4 : x_dtype == SEEDMM_BF16 ? 8 : 16;
    if (N > 1 && ldx % per16 != 0) return SEEDMM_EALIGN;
    const Q4Plan p = q4_plan(x_dtype, group, M, K, N);
    if (p.total && (!workspace || workspace_bytes < p.total)) return SEEDMM_EWORKSPACE;
    if (p.total && !aligned16(workspace)) return SEEDMM_EALIGN;
    Q4Args a = {weight, scales, biases, x, x_scale, y, M, K, N, ldx, ldy, y_dtype == SEEDMM_BF16};
    const bool sf = s_dtype == SEEDMM_F32;
    if (x_dtype == SEEDMM_F32) sf ? launch_q4<SEEDMM_F32, true>(a, group, p, workspace, st) : launch_q4<SEEDMM_F32, false>(a, group, p, workspace, st);
    else if (x_dtype == SEEDMM_BF16) sf ? launch_q4<SEEDMM_BF16, true>(a, group, p, workspace, st) : launch_q4<SEEDMM_BF16, false>(a, group, p, workspace, st);
    else sf ? launch_q4<SEEDMM_I8, true>(a, group, p, workspace, st) : launch_q4<SEEDMM_I8, false>(a, group, p, workspace, st);
    return launch_status();
}

size_t seedmm_q4_workspace_bytes(int x_dtype, int group, int M, int K, int N) {
    if (group != 32 && group != 64 && group != 128) return 0;
    if (M < 0 || K < 0 || N < 0 || M > kMaxDim || K > kMaxDim || N > kMaxDim || K % group != 0) return 0;
    return q4_plan(x_dtype, group, M, K, N).total;
}

int seedmm_add_norm(const void* x, int x_dtype, int64_t ldx, const void* delta, int delta_dtype,
                    int64_t ldd, const void* weight, int w_dtype, float eps, void* residual,
                    int64_t ldr, void* out, int out_dtype, int64_t ldo, float* scale, int N, int H,
                    void* hip_stream) {
    if (N < 0 || H < 0 || !(eps >= 0.f) || !(eps < INFINITY)) return SEEDMM_EINVAL;
    if (!float_type(x_dtype) || (delta && !float_type(delta_dtype)) || (weight && !float_type(w_dtype)))
        return SEEDMM_EINVAL;
    if (!float_type(out_dtype) && out_dtype != SEEDMM_I8) return SEEDMM_EINVAL;
    if (ldx < H || (delta && ldd < H) || (residual && ldr < H) || ldo < H) return SEEDMM_EINVAL;
    if (residual && residual == x && ldr != ldx && N > 1) return SEEDMM_EINVAL;   // rows over others' rows
    if ((out_dtype == SEEDMM_I8) != (scale != nullptr) && N > 0 && H > 0) return SEEDMM_EINVAL;
    if (N == 0 || H == 0) return SEEDMM_OK;
    if (!x || !out) return SEEDMM_EINVAL;
    auto off = [](const void* p, int dt) { return ((uintptr_t)p & (dt == SEEDMM_F32 ? 3 : dt == SEEDMM_BF16 ? 1 : 0)) != 0; };
    if (off(x, x_dtype) || (delta && off(delta, delta_dtype)) || (weight && off(weight, w_dtype)) ||
        (residual && off(residual, x_dtype)) || off(out, out_dtype) || ((uintptr_t)scale & 3))
        return SEEDMM_EALIGN;
    NormArgs a = {x, delta, weight, residual, out, scale, x_dtype, delta_dtype, w_dtype, out_dtype,
                  ldx, ldd, ldr, ldo, N, H, eps};
    hipStream_t st = (hipStream_t)hip_stream;
    const bool xf = x_dtype == SEEDMM_F32, df = delta_dtype == SEEDMM_F32;
    if (!delta) xf ? launch_norm<SEEDMM_F32, -1>(a, st) : launch_norm<SEEDMM_BF16, -1>(a, st);
    else if (df) xf ? launch_norm<SEEDMM_F32, SEEDMM_F32>(a, st) : launch_norm<SEEDMM_BF16, SEEDMM_F32>(a, st);
    else xf ? launch_norm<SEEDMM_F32, SEEDMM_BF16>(a, st) : launch_norm<SEEDMM_BF16, SEEDMM_BF16>(a, st);
    return launch_status();
}

int seedmm_route(const void* logits, int l_dtype, int64_t ldl, const float* bias, int score, int T,
                 int E, int top_k, int32_t* ids, float* w, void* hip_stream) {
    if (T < 0 || E < 1 || E > 4096 || top_k < 1 || top_k > E || top_k > 64) return SEEDMM_EINVAL;
    if ((int64_t)T * top_k > 0x7FFFFFFF || ldl < E || !float_type(l_dtype)) return SEEDMM_EINVAL;
    if (score != SEEDMM_SOFTMAX && score != SEEDMM_SIGMOID) return SEEDMM_EINVAL;
    if (bias && score == SEEDMM_SOFTMAX) return SEEDMM_EINVAL;
    if (T == 0) return SEEDMM_OK;
    if (!logits || !ids || !w) return SEEDMM_EINVAL;
    if (((uintptr_t)logits & (l_dtype == SEEDMM_F32 ? 3 : 1)) || ((uintptr_t)bias & 3) ||
        ((uintptr_t)ids & 3) || ((uintptr_t)w & 3))
        return SEEDMM_EALIGN;
    RouteArgs a = {logits, bias, ids, w, ldl, T, E, top_k, l_dtype};
    hipStream_t st = (hipStream_t)hip_stream;
    const bool lf = l_dtype == SEEDMM_F32;
    if (score == SEEDMM_SIGMOID) lf ? launch_route<true, SEEDMM_F32>(a, st) : launch_route<true, SEEDMM_BF16>(a, st);
    else lf ? launch_route<false, SEEDMM_F32>(a, st) : launch_route<false, SEEDMM_BF16>(a, st);
    return launch_status();
}

// Scratch of one block call: the normed rows, the logits, the routing (if the caller keeps
// none) and the routed layer's own workspace.
static bool block_layout(const seedmm_block* b, int T, size_t at[6]) {
    if (!b || T < 0 || b->E < 1 || b->H < 0) return false;
    const size_t layer = seedmm_moe_workspace_bytes(T, b->top_k, b->E, b->H, b->I);
    if (layer == 0) return false;
    at[0] = align_up((size_t)T * (size_t)b->H * 2);
    at[1] = at[0] + align_up((size_t)T * (size_t)b->E * 4);
    at[2] = at[1] + align_up((size_t)T * (size_t)b->top_k * 4);
    at[3] = at[2] + align_up((size_t)T * (size_t)b->top_k * 4);
    at[4] = at[3] + align_up(seedmm_q4_workspace_bytes(SEEDMM_BF16, b->group, b->E, b->H, T));
    at[5] = at[4] + layer;
    return true;
}

size_t seedmm_moe_block_workspace_bytes(const seedmm_block* block, int T) {
    size_t at[6];
    return block_layout(block, T, at) ? at[5] : 0;
}

int seedmm_moe_block(const seedmm_block* block, void* r, int r_dtype, const void* delta,
                     int delta_dtype, float* y, int32_t* ids, float* w, int T, void* workspace,
                     size_t workspace_bytes, void* hip_stream, const seedmm_side* side) {
    size_t at[6];
    if (!block || T < 0 || T > kMaxTokens) return SEEDMM_EINVAL;
    const seedmm_block& b = *block;
    if (!block_layout(block, T, at)) return SEEDMM_EINVAL;
    // every check of the four calls before the first launch: the routed layer's and the
    // choice's with an empty batch, whose checks stop before any launch
    if (int e = seedmm_moe_ex(nullptr, nullptr, 0, b.top_k, nullptr, nullptr, b.E, b.H, b.I, b.P,
                              b.p4mask, b.gate, b.up, b.down, nullptr, 0, hip_stream, nullptr))
        return e;
    if (int e = seedmm_route(nullptr, SEEDMM_F32, b.E, b.router_bias, b.score, 0, b.E, b.top_k,
                             nullptr, nullptr, hip_stream))
        return e;
    if (int e = seedmm_q4_gemv(nullptr, nullptr, nullptr, b.router_dtype, b.group, nullptr,
                               SEEDMM_BF16, b.H, nullptr, nullptr, SEEDMM_F32, b.E, b.E, b.H, 0,
                               nullptr, 0, hip_stream))
        return e;
    if (int e = seedmm_add_norm(nullptr, r_dtype, b.H, delta, delta_dtype, b.H, b.norm_weight,
                                b.norm_dtype, b.eps, nullptr, b.H, nullptr, SEEDMM_BF16, b.H,
                                nullptr, 0, b.H, hip_stream))
        return e;
    if (T == 0) return SEEDMM_OK;
    const seedmm_mat* mats[3] = {&b.gate, &b.up, &b.down};
    for (const seedmm_mat* m : mats)
        if (!m->seeds || !m->coefs || !m->codes || !m->exp_bias) return SEEDMM_EINVAL;
    if (!r || !y || !b.router_weight || !b.router_scales || !b.router_biases) return SEEDMM_EINVAL;
    if (side && side->stream && (!side->fork || !side->join || side->stream == hip_stream))
        return SEEDMM_EINVAL;
    if (!aligned16(r) || !aligned16(delta) || !aligned16(y) || !aligned16(b.norm_weight) ||
        !aligned16(b.router_weight) || !aligned16(b.router_scales) || !aligned16(b.router_biases) ||
        ((uintptr_t)b.router_bias & 3) || ((uintptr_t)ids & 3) || ((uintptr_t)w & 3))
        return SEEDMM_EALIGN;
    if (!workspace || workspace_bytes < at[5]) return SEEDMM_EWORKSPACE;
    if (!aligned16(workspace)) return SEEDMM_EALIGN;
    char* ws = (char*)workspace;
    float* logits = (float*)(ws + at[0]);
    if (!ids) ids = (int32_t*)(ws + at[1]);
    if (!w) w = (float*)(ws + at[2]);
    int e = seedmm_add_norm(r, r_dtype, b.H, delta, delta_dtype, b.H, b.norm_weight, b.norm_dtype,
                            b.eps, delta ? r : nullptr, b.H, ws, SEEDMM_BF16, b.H, nullptr, T, b.H,
                            hip_stream);
    if (!e)
        e = seedmm_q4_gemv(b.router_weight, b.router_scales, b.router_biases, b.router_dtype, b.group,
                           ws, SEEDMM_BF16, b.H, nullptr, logits, SEEDMM_F32, b.E, b.E, b.H, T,
                           ws + at[3], at[4] - at[3], hip_stream);
    if (!e)
        e = seedmm_route(logits, SEEDMM_F32, b.E, b.router_bias, b.score, T, b.E, b.top_k, ids, w,
                         hip_stream);
    if (!e)
        e = seedmm_moe_ex(ids, w, T, b.top_k, ws, y, b.E, b.H, b.I, b.P, b.p4mask, b.gate, b.up,
                          b.down, ws + at[4], at[5] - at[4], hip_stream, side);
    return e;
}

}  // extern "C"
