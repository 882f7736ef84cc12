// moe_rows.hip -- gfx950 kernels that move rows between the tokens of a routed batch and its
// experts, and their C ABI: rows sorted by expert (seedmm_moe_sort), back with their weights
// (seedmm_moe_unsort) and the gradients of that (seedmm_moe_unsort_grad), the SwiGLU step
// between two products (seedmm_swiglu), and the routed layer of 8-bit experts that is made of
// them (seedmm_moe_i8).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/seedmm.h"
#include "device_rows.hpp"

namespace {

constexpr int kMaxDim = 1 << 30;
constexpr int kMaxExperts = 4096, kMaxTopK = 64;

__device__ __forceinline__ uint32_t wave_usum(uint32_t v) {
    return wave_reduce(v, [](uint32_t a, uint32_t b) { return a + b; });
}

// ----------------------------------------------------------------------------------
// seedmm_moe_sort.  The place of pair p with expert e is
//     #{pairs of experts below e} + #{pairs q < p of expert e},
// a count over ids, so no pair waits for another and the order is always the same.
//   ONCE: batches of up to kSortOnce pairs count over all ids in the workgroup that moves the token:
//     one launch.
//   DIRECT: larger ones are cut into chunks, whose experts k_sort_count counts; each workgroup
//     sums the chunks' counts itself and counts ids inside its own chunk only.
//   SCANNED: where those sums are long, k_sort_scan and k_sort_base make them once for all.
// Long rows are bound by their copies: 4096 tokens of 8 slots over 100 experts, 2048 columns, bf16: 36 us,
// 3.9 TB/s, 8 bits: 20 us, 3.5 TB/s; 5 of each are k_sort_count and the launch between.  Short ones by the
// places: every token's workgroup reads its chunk's ids, so 16384 tokens of 16 slots over 512 experts take
// 47 us with 64 bf16 columns, whose bytes need 6.  One token: 2.8 us, a launch.
// ----------------------------------------------------------------------------------
constexpr int kSortOnce = 1024;      // pairs
constexpr int kSortChunk = 1024;     // pairs of a chunk, rounded down to whole tokens
constexpr int kSortDirect = 8192;    // counts that a workgroup sums itself
enum { ONCE, DIRECT, SCANNED };

struct SortArgs {
    const int32_t* ids;     // [T][k]
    const char* x;          // rows of row_bytes, ldx bytes apart
    const float* xs;        // null: no scales
    char* rows;
    float* rs;
    int32_t* offsets;       // [E + 1]
    int32_t* inverse;       // [T][k]
    int32_t* count;         // [chunks][E] pairs of the expert in the chunk; scanned: in those in front
    int32_t* total;         // [E] (scanned)
    int64_t ldx, ldr, row_bytes;
    int T, k, E, tokens, chunks;   // tokens of a chunk
};

// counts of the experts of a chunk
__global__ __launch_bounds__(256) void k_sort_count(const SortArgs a) {
    extern __shared__ int32_t hist[];
    const int64_t c = blockIdx.x;
    for (int e = threadIdx.x; e < a.E; e += 256) hist[e] = 0;
    __syncthreads();
    const int64_t p0 = c * a.tokens * a.k, all = (int64_t)a.T * a.k;
    const int n = (int)(all - p0 < a.tokens * a.k ? all - p0 : a.tokens * a.k);
    uint32_t e[kSortChunk / 256];
#pragma unroll
    for (int j = 0; j < kSortChunk / 256; ++j) {
        const int i = threadIdx.x + 256 * j;
        e[j] = i < n ? (uint32_t)a.ids[p0 + i] : ~0u;
    }
#pragma unroll
    for (int j = 0; j < kSortChunk / 256; ++j)
        if (e[j] < (uint32_t)a.E) atomicAdd(&hist[e[j]], 1);   // whole numbers: any order, one sum
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += 256) a.count[c * a.E + e] = hist[e];
}

// counts -> sums of the chunks in front, for 16 experts a workgroup; 16 threads an expert take
// a run of chunks each
__global__ __launch_bounds__(256) void k_sort_scan(const SortArgs a) {
    __shared__ int32_t part[16][17];
    const int col = threadIdx.x & 15, run = threadIdx.x >> 4;
    const int e = blockIdx.x * 16 + col;
    const int64_t per = (a.chunks + 15) / 16, c0 = run * per;
    const int64_t c1 = c0 + per < a.chunks ? c0 + per : a.chunks;
    int32_t sum = 0;
    if (e < a.E)
        for (int64_t c = c0; c < c1; ++c) sum += a.count[c * a.E + e];
    part[run][col] = sum;
    __syncthreads();
    int32_t front = 0;
    for (int r = 0; r < run; ++r) front += part[r][col];
    if (e >= a.E) return;
    for (int64_t c = c0; c < c1; ++c) {
        const int32_t v = a.count[c * a.E + e];
        a.count[c * a.E + e] = front;
        front += v;
    }
    if (run == 15) a.total[e] = front;
}

// hist[0 .. E - 1] -> offsets[0 .. E], by one workgroup of 256 threads
__device__ void write_offsets(const SortArgs& a, const int32_t* hist) {
    __shared__ int32_t wave_sums[4];
    const int tid = threadIdx.x;
    const int per = (a.E + 255) / 256, e0 = tid * per;
    int32_t sum = 0;
    for (int i = 0; i < per; ++i) sum += e0 + i < a.E ? hist[e0 + i] : 0;
    int32_t upto = sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int32_t o = __shfl_up(upto, d);
        if ((tid & 63) >= d) upto += o;
    }
    if ((tid & 63) == 63) wave_sums[tid >> 6] = upto;
    __syncthreads();
    int32_t front = upto - sum;
    for (int w = 0; w < tid >> 6; ++w) front += wave_sums[w];
    for (int i = 0; i < per && e0 + i < a.E; ++i) {
        a.offsets[e0 + i] = front;
        front += hist[e0 + i];
        if (e0 + i == a.E - 1) a.offsets[a.E] = front;
    }
}

__global__ __launch_bounds__(256) void k_sort_base(const SortArgs a) { write_offsets(a, a.total); }

// Workgroup 0 of the first part writes the offsets (k_sort_base has if SCANNED); each other one
// places a token's pairs and moves its row, read at the start.  ONCE: wave w counts for the slots w,
// w + 4, ... two at a time (a ballot counts 64 ids).  Else a table in LDS gives each expert the
// token's slot that names it, and each id in front of the token in its chunk adds one to its
// expert's (with ballots 4096 tokens of 8 slots took 37.6 us for 36.1, 16384 of 16 slots 71 for 47).
// A wave a token, four to a workgroup, took 45.5 us for 38.9: the writes then come from fewer
// tokens at once.
template <int MODE>
__global__ __launch_bounds__(256) void k_sort(const SortArgs a, int64_t first) {
    extern __shared__ int32_t lds[];      // ONCE: all ids; else a slot of each expert, behind (DIRECT) the experts' sums
    __shared__ int32_t place[kMaxTopK], named[kMaxTopK];
    __shared__ uint32_t earlier[kMaxTopK];
    const int64_t b = first + blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t t = b - 1;
    const int64_t chunk = MODE != ONCE && b > 0 ? t / a.tokens : 0;
    int32_t* total = lds;                 // DIRECT: pairs of an expert in all, and in the chunks in front
    int32_t* front = lds + a.E;
    if constexpr (MODE == DIRECT) {
        for (int e = tid; e < a.E; e += 256) {
            int32_t all = 0, before = 0;
#pragma unroll 8
            for (int c = 0; c < a.chunks; ++c) {
                const int32_t v = a.count[c * a.E + e];
                all += v;
                before += c < chunk ? v : 0;
            }
            total[e] = all;
            front[e] = before;
        }
    }
    if (b == 0) {
        if constexpr (MODE == ONCE) {
            for (int e = tid; e < a.E; e += 256) lds[e] = 0;
            __syncthreads();
            for (int i = tid; i < a.T * a.k; i += 256) {
                const uint32_t e = (uint32_t)a.ids[i];
                if (e < (uint32_t)a.E) atomicAdd(&lds[e], 1);
            }
        }
        __syncthreads();
        if constexpr (MODE != SCANNED) write_offsets(a, MODE == ONCE ? lds : total);
        return;
    }
    const char* src = a.x + t * a.ldx;
    const int64_t nv = a.row_bytes / 16;
    // short rows: several slots at a time, `per` threads each
    const int per = nv > 128 ? 256 : nv > 64 ? 128 : 64;
    const int g = tid / per, groups = 256 / per, v0 = tid % per;
    u32x4 w = {};
    if (v0 < nv) __builtin_memcpy(&w, src + v0 * 16, 16);
    const int64_t q0 = chunk * a.tokens * a.k;
    const int p0 = (int)(t * a.k - q0);                          // the token's pairs in the chunk
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if constexpr (MODE == ONCE) {
        const int n = a.T * a.k, full = (n + 255) & ~255;        // behind n: no expert
        for (int i = tid; i < full; i += 256) lds[i] = i < n ? a.ids[i] : -1;
        __syncthreads();
        for (int s = wave; s < a.k; s += 8) {
            uint32_t e[2], count[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 2; ++j) e[j] = (uint32_t)__builtin_amdgcn_readfirstlane(lds[p0 + (s + 4 * j < a.k ? s + 4 * j : s)]);
            for (int i0 = 0; i0 < n; i0 += 256) {
#pragma unroll
                for (int i = i0 + lane; i < i0 + 256; i += 64) {
                    const uint32_t q = (uint32_t)lds[i];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        count[j] += (uint32_t)__popcll(__ballot((q == e[j] && i < p0 + s + 4 * j) || q < e[j]));
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (lane == 0 && s + 4 * j < a.k) place[s + 4 * j] = e[j] < (uint32_t)a.E ? (int32_t)count[j] : -1;
        }
    } else {
        uint16_t* slot = (uint16_t*)(MODE == DIRECT ? lds + 2 * a.E : lds);
        uint32_t id[kSortChunk / 256];
#pragma unroll
        for (int j = 0; j < kSortChunk / 256; ++j) id[j] = tid + 256 * j < p0 ? (uint32_t)a.ids[q0 + tid + 256 * j] : ~0u;
        if (tid < a.k) {
            const uint32_t e = (uint32_t)a.ids[t * a.k + tid];
            named[tid] = (int32_t)e;
            earlier[tid] = 0;
            if (e < (uint32_t)a.E) slot[e] = (uint16_t)tid;      // one of its slots, if it has several
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kSortChunk / 256; ++j)
            if (id[j] < (uint32_t)a.E) {
                const uint32_t s = slot[id[j]];                  // any value where the token has no slot of the expert
                if (s < (uint32_t)a.k && (uint32_t)named[s] == id[j]) atomicAdd(&earlier[s], 1);   // whole numbers
            }
        __syncthreads();
        for (int s = wave; s < a.k; s += 4) {
            const uint32_t e = (uint32_t)__builtin_amdgcn_readfirstlane(named[s]);
            uint32_t at = ~0u;
            if (e < (uint32_t)a.E) {
                at = earlier[slot[e]] + (uint32_t)__popcll(__ballot(lane < s && (uint32_t)named[lane] == e));
                if constexpr (MODE == DIRECT) {
                    uint32_t below = 0;
                    for (int i = lane; i < (int)e; i += 64) below += (uint32_t)total[i];
                    at += wave_usum(below) + (uint32_t)front[e];
                } else {
                    at += (uint32_t)a.offsets[e] + (uint32_t)a.count[chunk * a.E + e];
                }
            }
            if (lane == 0) place[s] = (int32_t)at;
        }
    }
    __syncthreads();
    if (tid < a.k) {
        const int32_t at = place[tid];
        a.inverse[t * a.k + tid] = at;
        if (a.xs && at >= 0) a.rs[at] = a.xs[t];
    }
    for (int64_t v = v0; v < nv; v += per) {
        if (v > v0) __builtin_memcpy(&w, src + v * 16, 16);
        for (int s = g; s < a.k; s += groups) {
            const int32_t at = place[s];
            if (at >= 0) __builtin_memcpy(a.rows + at * a.ldr + v * 16, &w, 16);
        }
    }
    const int rest = (int)(a.row_bytes & 15);
    if (tid < rest) {
        const char c = src[nv * 16 + tid];
        for (int s = 0; s < a.k; ++s) {
            const int32_t at = place[s];
            if (at >= 0) a.rows[at * a.ldr + nv * 16 + tid] = c;
        }
    }
}

// ----------------------------------------------------------------------------------
// seedmm_moe_unsort and its gradients: TPR threads a token, 8 columns a thread and pass.  A lane a
// slot loads the token's places and weights, and they are handed out by lane reads (loaded by every
// lane for each slot and pass they cost 4096 tokens of 8 slots 39 us for 32.5); the rows of 8
// slots are in flight at once.  Bound by memory: 4096 tokens of 8 slots, 2048 columns, bf16 to fp32
// in 32 us (4.8 TB/s), their gradients in 58 to 61 (4.7), 1021 tokens of 6 slots and 7167 columns in fp32
// in 86 (4.3; rows start on 4 bytes); 64 tokens of 8 slots 2.9 and 4.4 us.
// ----------------------------------------------------------------------------------
struct UnsortArgs {
    const void* rows;         // [n_rows][ldr]
    const int32_t* inverse;   // [T][k]
    const float* w;           // [T][k] or null
    void* y;                  // [T][ldy]
    const void* dy;           // [T][ldy] (gradients)
    void* drows;              // [n_rows][ldg] or null
    float* dw;                // [T][k] or null
    int64_t ldr, ldy, ldg, tokens;
    uint32_t n_rows;
    int k, H, y_bf16;
};

constexpr int kSlots = 8;     // slots in flight

// A token's places and weights, a slot a lane.
struct Slots {
    int32_t at = -1;
    float w = 1.f;
    __device__ __forceinline__ void load(const UnsortArgs& a, int64_t t) {
        const int s = threadIdx.x & 63;
        if (s < a.k) {
            at = a.inverse[t * a.k + s];
            if (a.w) w = a.w[t * a.k + s];
        }
    }
    __device__ __forceinline__ uint32_t place(int s) const { return (uint32_t)__builtin_amdgcn_readlane(at, s); }
    __device__ __forceinline__ float weight(int s) const { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), s)); }
};

template <int TPR, int RT>
__global__ __launch_bounds__(256) void k_unsort(const UnsortArgs a) {
    const int tid = threadIdx.x;
    const int64_t hop = (int64_t)gridDim.x * (256 / TPR);
    int64_t t = (int64_t)blockIdx.x * (256 / TPR) + __builtin_amdgcn_readfirstlane(tid / TPR);
    for (; t < a.tokens; t += hop) {
        Slots now;
        now.load(a, t);
        for (int c0 = 0; c0 < a.H; c0 += TPR * 8) {         // all lanes: they hold the places
            const int c = c0 + tid % TPR * 8, n = a.H - c;
            float sum[8] = {};
            for (int s0 = 0; s0 < a.k; s0 += kSlots) {      // slots past k have no row
                Eight<RT> r[kSlots];
#pragma unroll
                for (int s = 0; s < kSlots; ++s) {
                    const uint32_t at = now.place(s0 + s);
                    if (at < a.n_rows) r[s].load(a.rows, at * a.ldr + c, n);
                }
#pragma unroll
                for (int s = 0; s < kSlots; ++s) {
                    if (now.place(s0 + s) >= a.n_rows) continue;
                    const float f = now.weight(s0 + s);
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[j] = __builtin_fmaf(f, r[s].get(j), sum[j]);
                }
            }
            if (a.y_bf16) store8<SEEDMM_BF16>(a.y, t * a.ldy + c, n, sum);
            else store8<SEEDMM_F32>(a.y, t * a.ldy + c, n, sum);
        }
    }
}

template <int TPR, int YT, int RT>
__global__ __launch_bounds__(256) void k_unsort_grad(const UnsortArgs a) {
    __shared__ float red[4][kSlots];
    const int tid = threadIdx.x;
    const int64_t hop = (int64_t)gridDim.x * (256 / TPR);
    int64_t t = (int64_t)blockIdx.x * (256 / TPR) + __builtin_amdgcn_readfirstlane(tid / TPR);
    for (; t < a.tokens; t += hop) {
        Slots now;
        now.load(a, t);
        for (int s0 = 0; s0 < a.k; s0 += kSlots) {
            float dot[kSlots] = {};
            for (int c0 = 0; c0 < a.H; c0 += TPR * 8) {     // all lanes: they hold the places
                const int c = c0 + tid % TPR * 8, n = a.H - c;
                Eight<YT> d;
                Eight<RT> r[kSlots];
                d.load(a.dy, t * a.ldy + c, n);
                if (a.dw) {
#pragma unroll
                    for (int s = 0; s < kSlots; ++s) {
                        const uint32_t at = now.place(s0 + s);
                        if (at < a.n_rows) r[s].load(a.rows, at * a.ldr + c, n);
                    }
                }
#pragma unroll
                for (int s = 0; s < kSlots; ++s) {
                    const uint32_t at = now.place(s0 + s);
                    if (at >= a.n_rows) continue;
                    if (a.dw) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) dot[s] = __builtin_fmaf(d.get(j), r[s].get(j), dot[s]);
                    }
                    if (a.drows) {
                        const float f = now.weight(s0 + s);
                        float v[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = f * d.get(j);
                        store8<RT>(a.drows, at * a.ldg + c, n, v);
                    }
                }
            }
            if (!a.dw) continue;
#pragma unroll
            for (int s = 0; s < kSlots; ++s) dot[s] = wave_sum(dot[s]);
            if constexpr (TPR > 64) {
                __syncthreads();                       // the last sums have been read
                if ((tid & 63) == 0) {
#pragma unroll
                    for (int s = 0; s < kSlots; ++s) red[tid >> 6][s] = dot[s];
                }
                __syncthreads();
                if (tid < kSlots && s0 + tid < a.k)
                    a.dw[t * a.k + s0 + tid] = (red[0][tid] + red[1][tid]) + (red[2][tid] + red[3][tid]);
            } else if ((tid & 63) == 0) {
#pragma unroll
                for (int s = 0; s < kSlots; ++s)
                    if (s0 + s < a.k) a.dw[t * a.k + s0 + s] = dot[s];
            }
        }
    }
}

// ----------------------------------------------------------------------------------
// seedmm_swiglu.  TPR threads a row, NP pieces of 8 columns a thread held in registers; for 8
// bits the row's largest |h| is found before the codes are written.  To floats bound by memory: 29491
// of 32768 rows of 1024, bf16 to bf16, in 37 us (4.9 TB/s; 41 with a division).  To 8 bits by the arithmetic:
// 43 to 46 us (3.3 to 3.5 TB/s; 55 with divisions), the vector units busy for 79% of the cycles.  512 rows to
// 8 bits 3.4 us, a launch.
// ----------------------------------------------------------------------------------
struct SwigluArgs {
    const void* gu;           // [N][ldg]
    void* out;                // [N][ldo]
    float* scale;             // [N] with 8-bit codes
    const int32_t* count;     // null: all rows
    int64_t ldg, ldo, n0, N;  // rows from n0 on
    int I, out_dt;
};

// exp of -|g| cannot overflow: silu(g) = n / d with d = 1 + e of 1 .. 2 and n = g or, for g < 0, g e.
// The hardware's reciprocal r is a step off: 1 - d r is exact, and n r + n r (1 - d r) rounds once, 2^-22
// of a step off a division, in 6 instructions for its 10.  (Where n is an infinity, d is 1 and the
// second term NaN; the median of it and the largest numbers is one of these, and the sum n.)
// 8-bit codes, which are bound by the arithmetic, take a corrected reciprocal times n, in 4: half a step of
// fp32 more, 2^-17 of a code's step.
template <bool CODES>
__device__ __forceinline__ float swiglu(float g, float u) {
    const float e = expf(-fabsf(g)), d = 1.f + e, n = g < 0.f ? g * e : g;
    const float r = __builtin_amdgcn_rcpf(d), off = __builtin_fmaf(-d, r, 1.f);
    if constexpr (CODES) return n * __builtin_fmaf(off, r, r) * u;
    const float more = __builtin_amdgcn_fmed3f(n * (off * r), -__FLT_MAX__, __FLT_MAX__);
    return __builtin_fmaf(n, r, more) * u;
}

// |v| as a whole number: in the order of the values, a NaN above everything
__device__ __forceinline__ uint32_t size_of(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// For 8 bits a row's scale and the scale's reciprocal (0: codes 0).
struct CodeScale {
    float sc, inv;
};
__device__ __forceinline__ CodeScale code_scale(float top) {
    CodeScale o;
    o.sc = fmaxf(top / 127.0f, 1.17549435e-38f);
    if (!(top < INFINITY)) o.sc = NAN;
    o.inv = o.sc == o.sc ? 1.0f / o.sc : 0.f;
    return o;
}

// the largest of a row's sizes; NW waves share a row
template <int NW>
__device__ __forceinline__ float row_top(uint32_t top, uint32_t* red) {
    top = wave_umax(top);
    if constexpr (NW > 1) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NW; ++i) top = top > red[i] ? top : red[i];
    }
    return __uint_as_float(top);
}

template <int TPR, int NP, int GT, bool CODES>
__global__ __launch_bounds__(256) void k_swiglu(const SwigluArgs a) {
    __shared__ uint32_t red[4];
    const int tid = threadIdx.x;
    const int64_t n = a.n0 + (int64_t)blockIdx.x * (256 / TPR) + __builtin_amdgcn_readfirstlane(tid / TPR);
    if (n >= a.N || (a.count && n >= *a.count)) return;     // a whole workgroup where waves share a row
    float h[NP][8];
    uint32_t top = 0;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int c = (p * TPR + tid % TPR) * 8, cnt = a.I - c;
        if (cnt <= 0) continue;
        Eight<GT> g, u;
        g.load(a.gu, n * a.ldg + c, cnt);
        u.load(a.gu, n * a.ldg + a.I + c, cnt);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            h[p][j] = swiglu<CODES>(g.get(j), u.get(j));
            const uint32_t v = j < cnt ? size_of(h[p][j]) : 0;
            top = top > v ? top : v;
        }
    }
    float inv = 0.f;
    if constexpr (CODES) {
        const CodeScale o = code_scale(row_top<TPR / 64>(top, red));
        if (tid % TPR == 0) a.scale[n] = o.sc;
        inv = o.inv;
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int c = (p * TPR + tid % TPR) * 8, cnt = a.I - c;
        if (cnt <= 0) continue;
        if constexpr (CODES) {
#pragma unroll
            for (int j = 0; j < 8; ++j) h[p][j] = code_of(h[p][j], inv);
            store8<SEEDMM_I8>(a.out, n * a.ldo + c, cnt, h[p]);
        } else if (a.out_dt == SEEDMM_F32) {
            store8<SEEDMM_F32>(a.out, n * a.ldo + c, cnt, h[p]);
        } else {
            store8<SEEDMM_BF16>(a.out, n * a.ldo + c, cnt, h[p]);
        }
    }
}

// rows of any length, for 8 bits read twice
template <int GT, bool CODES>
__global__ __launch_bounds__(1024) void k_swiglu_long(const SwigluArgs a) {
    __shared__ uint32_t red[16];
    const int64_t n = a.n0 + blockIdx.x;
    if (a.count && n >= *a.count) return;
    auto piece = [&](int64_t c, float (&h)[8]) {
        Eight<GT> g, u;
        const int cnt = (int)(a.I - c < 8 ? a.I - c : 8);
        g.load(a.gu, n * a.ldg + c, cnt);
        u.load(a.gu, n * a.ldg + a.I + c, cnt);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = swiglu<CODES>(g.get(j), u.get(j));
        return cnt;
    };
    float inv = 0.f;
    if constexpr (CODES) {
        uint32_t top = 0;
        for (int64_t c = threadIdx.x * 8; c < a.I; c += 8192) {
            float h[8];
            piece(c, h);
#pragma unroll
            for (int j = 0; j < 8; ++j) top = top > size_of(h[j]) ? top : size_of(h[j]);
        }
        const CodeScale o = code_scale(row_top<16>(top, red));
        if (threadIdx.x == 0) a.scale[n] = o.sc;
        inv = o.inv;
    }
    for (int64_t c = threadIdx.x * 8; c < a.I; c += 8192) {
        float h[8];
        const int cnt = piece(c, h);
        if constexpr (CODES) {
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] = code_of(h[j], inv);
            store8<SEEDMM_I8>(a.out, n * a.ldo + c, cnt, h);
        } else if (a.out_dt == SEEDMM_F32) {
            store8<SEEDMM_F32>(a.out, n * a.ldo + c, cnt, h);
        } else {
            store8<SEEDMM_BF16>(a.out, n * a.ldo + c, cnt, h);
        }
    }
}

// ---- host ------------------------------------------------------------------------
bool off_type(const void* p, int dt) {
    return ((uintptr_t)p & (dt == SEEDMM_F32 ? 3 : dt == SEEDMM_BF16 ? 1 : 0)) != 0;
}
bool off4(const void* p) { return ((uintptr_t)p & 3) != 0; }

int sort_tokens(int top_k) { return kSortChunk / top_k; }      // of a chunk
int64_t sort_chunks(int T, int top_k) { return ((int64_t)T + sort_tokens(top_k) - 1) / sort_tokens(top_k); }

bool routing_ok(int T, int top_k) {
    return T >= 0 && top_k >= 1 && top_k <= kMaxTopK && (int64_t)T * top_k <= 0x7FFFFFFF;
}

// Launches of `kernel` with `threads` a token or row, in parts that HIP takes: `first` is the
// part's first one.
template <typename A, typename K>
void launch_parts(K kernel, A a, int64_t A::* first, int64_t n, int threads, int block, hipStream_t st) {
    for (int64_t i = 0; i < n; i += kLaunchThreads / threads) {
        const int64_t m = n - i < kLaunchThreads / threads ? n - i : kLaunchThreads / threads;
        a.*first = i;
        hipLaunchKernelGGL(kernel, dim3((unsigned)((m * threads - 1) / block + 1)), dim3(block), 0, st, a);
    }
}

// a grid that HIP takes (its workgroups go on to further tokens)
unsigned bounded(int64_t groups) { return (unsigned)(groups < kLaunchThreads / 256 ? groups : kLaunchThreads / 256); }

template <int TPR, int RT>
void launch_unsort(const UnsortArgs& a, hipStream_t st) {
    hipLaunchKernelGGL((k_unsort<TPR, RT>), dim3(bounded((a.tokens - 1) / (256 / TPR) + 1)), dim3(256), 0, st, a);
}

template <int TPR, int YT, int RT>
void launch_grad(const UnsortArgs& a, hipStream_t st) {
    hipLaunchKernelGGL((k_unsort_grad<TPR, YT, RT>), dim3(bounded((a.tokens - 1) / (256 / TPR) + 1)), dim3(256), 0, st, a);
}

template <int YT, int RT>
void launch_grad(const UnsortArgs& a, hipStream_t st) {
    if (a.H <= 512) launch_grad<64, YT, RT>(a, st);
    else launch_grad<256, YT, RT>(a, st);
}

template <int TPR, int NP, int GT, bool CODES>
void launch_swiglu(const SwigluArgs& a, hipStream_t st) {
    launch_parts(k_swiglu<TPR, NP, GT, CODES>, a, &SwigluArgs::n0, a.N, TPR, 256, st);
}

template <int GT, bool CODES>
void launch_swiglu(const SwigluArgs& a, hipStream_t st) {
    if (a.I <= 512) launch_swiglu<64, 1, GT, CODES>(a, st);
    else if (a.I <= 2048) launch_swiglu<256, 1, GT, CODES>(a, st);
    else if (a.I <= 4096) launch_swiglu<256, 2, GT, CODES>(a, st);
    else if (a.I <= 8192) launch_swiglu<256, 4, GT, CODES>(a, st);
    else launch_parts(k_swiglu_long<GT, CODES>, a, &SwigluArgs::n0, a.N, 1024, 1024, st);
}

template <bool CODES>
void launch_swiglu(const SwigluArgs& a, bool f32, hipStream_t st) {
    f32 ? launch_swiglu<SEEDMM_F32, CODES>(a, st) : launch_swiglu<SEEDMM_BF16, CODES>(a, st);
}

}  // namespace

extern "C" {

size_t seedmm_moe_sort_workspace_bytes(int T, int top_k, int E) {
    if (!routing_ok(T, top_k) || E < 1 || E > kMaxExperts) return 0;
    if ((int64_t)T * top_k <= kSortOnce) return 0;
    return align_up((size_t)(sort_chunks(T, top_k) + 1) * (size_t)E * 4);
}

int seedmm_moe_sort(const int32_t* topk_ids, int T, int top_k, int E, const void* x, int x_dtype,
                    int64_t ldx, const float* x_scale, void* rows, int64_t ldr, float* row_scale,
                    int H, int32_t* offsets, int32_t* inverse, void* workspace,
                    size_t workspace_bytes, void* hip_stream) {
    if (!routing_ok(T, top_k) || E < 1 || E > kMaxExperts || H < 0 || H > kMaxDim) return SEEDMM_EINVAL;
    if (!float_type(x_dtype) && x_dtype != SEEDMM_I8) return SEEDMM_EINVAL;
    if (ldx < H || ldr < H || (x_scale != nullptr) != (row_scale != nullptr)) return SEEDMM_EINVAL;
    if (!offsets || (T > 0 && (!topk_ids || !inverse || (H > 0 && (!x || !rows))))) return SEEDMM_EINVAL;
    if (off4(topk_ids) || off4(offsets) || off4(inverse) || off4(x_scale) || off4(row_scale) ||
        off_type(x, x_dtype) || off_type(rows, x_dtype))
        return SEEDMM_EALIGN;
    const size_t need = seedmm_moe_sort_workspace_bytes(T, top_k, E);
    if (need && (!workspace || workspace_bytes < need)) return SEEDMM_EWORKSPACE;
    if (need && !aligned16(workspace)) return SEEDMM_EALIGN;
    const int64_t b = type_bytes(x_dtype);
    SortArgs a = {topk_ids, (const char*)x, x_scale, (char*)rows, row_scale, offsets, inverse, nullptr, nullptr,
                  ldx * b, ldr * b, H * b, T, top_k, E, sort_tokens(top_k), (int)sort_chunks(T, top_k)};
    hipStream_t st = (hipStream_t)hip_stream;
    const int mode = need == 0 ? ONCE : (int64_t)a.chunks * E <= kSortDirect ? DIRECT : SCANNED;
    if (mode != ONCE) {
        a.total = (int32_t*)workspace;
        a.count = a.total + E;
        hipLaunchKernelGGL(k_sort_count, dim3((unsigned)a.chunks), dim3(256), (size_t)E * 4, st, a);
    }
    if (mode == SCANNED) {
        hipLaunchKernelGGL(k_sort_scan, dim3((unsigned)((E + 15) / 16)), dim3(256), 0, st, a);
        hipLaunchKernelGGL(k_sort_base, dim3(1), dim3(256), 0, st, a);
    }
    const size_t lds = mode == ONCE ? 4 * (size_t)(E > kSortOnce ? E : kSortOnce) : (size_t)(E + 1) / 2 * 4 + (mode == DIRECT ? 8 * (size_t)E : 0);
    constexpr int64_t most = kLaunchThreads / 256;
    for (int64_t b0 = 0; b0 < (int64_t)T + 1; b0 += most) {     // the offsets, then a token a workgroup
        const dim3 grid((unsigned)((int64_t)T + 1 - b0 < most ? (int64_t)T + 1 - b0 : most));
        if (mode == ONCE) hipLaunchKernelGGL((k_sort<ONCE>), grid, dim3(256), lds, st, a, b0);
        else if (mode == DIRECT) hipLaunchKernelGGL((k_sort<DIRECT>), grid, dim3(256), lds, st, a, b0);
        else hipLaunchKernelGGL((k_sort<SCANNED>), grid, dim3(256), lds, st, a, b0);
    }
    return launch_status();
}

int seedmm_moe_unsort(const void* rows, int r_dtype, int64_t ldr, int n_rows,
                      const int32_t* inverse, const float* topk_w, void* y, int y_dtype,
                      int64_t ldy, int T, int top_k, int H, void* hip_stream) {
    if (!routing_ok(T, top_k) || H < 0 || H > kMaxDim || n_rows < 0 || ldr < H || ldy < H) return SEEDMM_EINVAL;
    if (!float_type(r_dtype) || !float_type(y_dtype)) return SEEDMM_EINVAL;
    if (T == 0 || H == 0) return SEEDMM_OK;
    if (!inverse || !y || (n_rows > 0 && !rows)) return SEEDMM_EINVAL;
    if (off_type(rows, r_dtype) || off_type(y, y_dtype) || off4(inverse) || off4(topk_w)) return SEEDMM_EALIGN;
    UnsortArgs a = {rows, inverse, topk_w, y, nullptr, nullptr, nullptr, ldr, ldy, 0, T, (uint32_t)n_rows,
                    top_k, H, y_dtype == SEEDMM_BF16};
    hipStream_t st = (hipStream_t)hip_stream;
    const bool f = r_dtype == SEEDMM_F32;
    if (H <= 512) f ? launch_unsort<64, SEEDMM_F32>(a, st) : launch_unsort<64, SEEDMM_BF16>(a, st);
    else f ? launch_unsort<256, SEEDMM_F32>(a, st) : launch_unsort<256, SEEDMM_BF16>(a, st);
    return launch_status();
}

int seedmm_moe_unsort_grad(const void* dy, int dy_dtype, int64_t ldd, const void* rows, int r_dtype,
                           int64_t ldr, int n_rows, const int32_t* inverse, const float* topk_w,
                           void* drows, int64_t ldg, float* dw, int T, int top_k, int H,
                           void* hip_stream) {
    if (!routing_ok(T, top_k) || H < 0 || H > kMaxDim || n_rows < 0 || ldd < H) return SEEDMM_EINVAL;
    if (!float_type(dy_dtype) || !float_type(r_dtype)) return SEEDMM_EINVAL;
    if ((dw && ldr < H) || (drows && ldg < H) || (drows && drows == rows && ldg != ldr)) return SEEDMM_EINVAL;
    if (T == 0 || (H == 0 && !dw)) return SEEDMM_OK;
    if (!inverse || !topk_w || (!drows && !dw) || (H > 0 && !dy) || (dw && H > 0 && n_rows > 0 && !rows)) return SEEDMM_EINVAL;
    if (off_type(dy, dy_dtype) || off_type(rows, r_dtype) || off_type(drows, r_dtype) || off4(inverse) ||
        off4(topk_w) || off4(dw))
        return SEEDMM_EALIGN;
    UnsortArgs a = {rows, inverse, topk_w, nullptr, dy, drows, dw, ldr, ldd, ldg, T, (uint32_t)n_rows, top_k, H, 0};
    hipStream_t st = (hipStream_t)hip_stream;
    const bool yf = dy_dtype == SEEDMM_F32, rf = r_dtype == SEEDMM_F32;
    if (yf) rf ? launch_grad<SEEDMM_F32, SEEDMM_F32>(a, st) : launch_grad<SEEDMM_F32, SEEDMM_BF16>(a, st);
    else rf ? launch_grad<SEEDMM_BF16, SEEDMM_F32>(a, st) : launch_grad<SEEDMM_BF16, SEEDMM_BF16>(a, st);
    return launch_status();
}

int seedmm_swiglu(const void* gate_up, int g_dtype, int64_t ldg, void* out, int out_dtype,
                  int64_t ldo, float* scale, const int32_t* count, int N, int I, void* hip_stream) {
    if (N < 0 || I < 0 || I > kMaxDim / 2 || ldg < 2 * (int64_t)I || ldo < I) return SEEDMM_EINVAL;
    if (!float_type(g_dtype) || (!float_type(out_dtype) && out_dtype != SEEDMM_I8)) return SEEDMM_EINVAL;
    if (N == 0 || I == 0) return SEEDMM_OK;
    if ((out_dtype == SEEDMM_I8) != (scale != nullptr) || !gate_up || !out) return SEEDMM_EINVAL;
    if (off_type(gate_up, g_dtype) || off_type(out, out_dtype) || off4(scale) || off4(count)) return SEEDMM_EALIGN;
    const SwigluArgs a = {gate_up, out, scale, count, ldg, ldo, 0, N, I, out_dtype};
    hipStream_t st = (hipStream_t)hip_stream;
    const bool f32 = g_dtype == SEEDMM_F32;
    out_dtype == SEEDMM_I8 ? launch_swiglu<true>(a, f32, st) : launch_swiglu<false>(a, f32, st);
    return launch_status();
}

// Scratch of one layer call: the order, the sorted rows, gate and up (whose room the down
// product's rows take later), and the SwiGLU rows.  Gate and up and the down product's rows are bf16: of
// the layer's error against 64 bits, 2.041% of y, 2.034 remain with fp32 rows behind the down product,
// nearly all of it from the 8-bit rows of the SwiGLU; they would take 495 us for 439 at 4096 tokens (8 of
// 100 experts of 2048 x 1024).
struct LayerPlan {
    size_t offsets, inverse, rows, row_scale, gu, h, h_scale, total;
};
static bool layer_plan(int T, int top_k, int E, int H, int I, LayerPlan* p) {
    if (!routing_ok(T, top_k) || E < 1 || E > kMaxExperts || H < 1 || I < 1 || H > 131071 || I > 131071) return false;
    const size_t P = (size_t)T * (size_t)top_k;
    if (P > (size_t)kMaxDim) return false;
    p->offsets = align_up(seedmm_moe_sort_workspace_bytes(T, top_k, E));
    p->inverse = p->offsets + align_up((size_t)(E + 1) * 4);
    p->rows = p->inverse + align_up(P * 4);
    p->row_scale = p->rows + align_up(P * (size_t)H);
    p->gu = p->row_scale + align_up(P * 4);
    p->h = p->gu + align_up(P * (size_t)(2 * I > H ? 2 * I : H) * 2);
    p->h_scale = p->h + align_up(P * (size_t)I);
    p->total = p->h_scale + align_up(P * 4);
    return true;
}

size_t seedmm_moe_i8_workspace_bytes(int T, int top_k, int E, int H, int I) {
    LayerPlan p;
    return layer_plan(T, top_k, E, H, I, &p) ? p.total : 0;
}

int seedmm_moe_i8(const int32_t* topk_ids, const float* topk_w, int T, int top_k, const int8_t* x,
                  const float* x_scale, float* y, int E, int H, int I, seedmm_i8mat gate_up,
                  seedmm_i8mat down, void* workspace, size_t workspace_bytes, void* hip_stream) {
    LayerPlan p;
    if (!layer_plan(T, top_k, E, H, I, &p)) return SEEDMM_EINVAL;
    if (!float_type(gate_up.s_dtype) || !float_type(down.s_dtype)) return SEEDMM_EINVAL;
    if (T == 0) return SEEDMM_OK;
    if (!topk_ids || !topk_w || !x || !x_scale || !y || !gate_up.weight || !gate_up.scales || !down.weight || !down.scales)
        return SEEDMM_EINVAL;
    if (off4(topk_ids) || off4(topk_w) || off4(x_scale) || off4(y) || off_type(gate_up.scales, gate_up.s_dtype) ||
        off_type(down.scales, down.s_dtype))
        return SEEDMM_EALIGN;
    if (!workspace || workspace_bytes < p.total) return SEEDMM_EWORKSPACE;
    if (!aligned16(workspace)) return SEEDMM_EALIGN;
    char* ws = (char*)workspace;
    int32_t *offsets = (int32_t*)(ws + p.offsets), *inverse = (int32_t*)(ws + p.inverse);
    int8_t *rows = (int8_t*)(ws + p.rows), *h = (int8_t*)(ws + p.h);
    float *row_scale = (float*)(ws + p.row_scale), *h_scale = (float*)(ws + p.h_scale);
    const int P = T * top_k;
    int e = seedmm_moe_sort(topk_ids, T, top_k, E, x, SEEDMM_I8, H, x_scale, rows, H, row_scale, H, offsets,
                            inverse, ws, p.offsets, hip_stream);
    if (!e)
        e = seedmm_i8_gemv(gate_up.weight, gate_up.scales, gate_up.s_dtype, E, offsets, rows, H, row_scale,
                           ws + p.gu, SEEDMM_BF16, 2 * (int64_t)I, 2 * I, H, P, hip_stream);
    if (!e)
        e = seedmm_swiglu(ws + p.gu, SEEDMM_BF16, 2 * (int64_t)I, h, SEEDMM_I8, I, h_scale, offsets + E, P, I, hip_stream);
    if (!e)
        e = seedmm_i8_gemv(down.weight, down.scales, down.s_dtype, E, offsets, h, I, h_scale, ws + p.gu,
                           SEEDMM_BF16, H, H, I, P, hip_stream);
    if (!e)
        e = seedmm_moe_unsort(ws + p.gu, SEEDMM_BF16, H, P, inverse, topk_w, y, SEEDMM_F32, H, T, top_k, H, hip_stream);
    return e;
}

}  // extern "C"
