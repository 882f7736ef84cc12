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
// a count over ids, so no pair waits for another and the order is always the same.  Batches
// of up to kSortOnce pairs count over all ids in the workgroup that moves the token (one
// launch).  Larger ones are cut into chunks: k_sort_count has each chunk's experts counted,
// k_sort_scan sums the chunks in front, and k_sort counts inside the chunk only.
// ----------------------------------------------------------------------------------
constexpr int kSortOnce = 2048;      // pairs
constexpr int kSortChunk = 1024;     // pairs of a chunk, rounded down to whole tokens

struct SortArgs {
    const int32_t* ids;     // [T][k]
    const char* x;          // rows of row_bytes, ldx bytes apart
    const float* xs;        // null: no scales
    char* rows;
    float* rs;
    int32_t* offsets;       // [E + 1]
    int32_t* inverse;       // [T][k]
    int32_t* start;         // [chunks][E]: pairs of the expert in the chunks in front
    int32_t* total;         // [E]
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
    for (int i = threadIdx.x; i < n; i += 256) {
        const uint32_t e = (uint32_t)a.ids[p0 + i];
        if (e < (uint32_t)a.E) atomicAdd(&hist[e], 1);   // whole numbers: any order, one sum
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += 256) a.start[c * a.E + e] = hist[e];
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
        for (int64_t c = c0; c < c1; ++c) sum += a.start[c * a.E + e];
    part[run][col] = sum;
    __syncthreads();
    int32_t front = 0;
    for (int r = 0; r < run; ++r) front += part[r][col];
    if (e >= a.E) return;
    for (int64_t c = c0; c < c1; ++c) {
        const int32_t v = a.start[c * a.E + e];
        a.start[c * a.E + e] = front;
        front += v;
    }
    if (run == 15) a.total[e] = front;
}

// offsets[0 .. E] by one workgroup of 256 threads
template <bool CHUNKED>
__device__ void sort_offsets(const SortArgs& a, int32_t* hist) {
    __shared__ int32_t wave_sums[4];
    const int tid = threadIdx.x;
    if constexpr (CHUNKED) {
        for (int e = tid; e < a.E; e += 256) hist[e] = a.total[e];
    } else {
        for (int e = tid; e < a.E; e += 256) hist[e] = 0;
        __syncthreads();
        const int n = a.T * a.k;
        for (int i = tid; i < n; i += 256) {
            const uint32_t e = (uint32_t)a.ids[i];
            if (e < (uint32_t)a.E) atomicAdd(&hist[e], 1);
        }
    }
    __syncthreads();
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

// Workgroup 0 of the first part writes the offsets; each other one places a token's pairs and
// moves its row: the wave w counts for the slots w, w + 4, ... (a ballot counts 64 ids), then
// all threads read the row once and write it to every place.
template <bool CHUNKED>
__global__ __launch_bounds__(256) void k_sort(const SortArgs a, int64_t first) {
    extern __shared__ int32_t lds[];
    __shared__ int32_t place[kMaxTopK];
    const int64_t b = first + blockIdx.x;
    if (b == 0) return sort_offsets<CHUNKED>(a, lds);
    const int64_t t = b - 1;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t chunk = CHUNKED ? t / a.tokens : 0;
    const int64_t q0 = chunk * a.tokens * a.k;
    const int p0 = (int)(t * a.k - q0);                          // the token's pairs in the chunk
    const int n = CHUNKED ? p0 + a.k : a.T * a.k;                // pairs that count
    const int full = (n + 255) & ~255;                           // behind n: no expert
    for (int i = tid; i < full; i += 256) lds[i] = i < n ? a.ids[q0 + i] : -1;
    __syncthreads();
    for (int s = wave; s < a.k; s += 4) {
        const uint32_t e = (uint32_t)__builtin_amdgcn_readfirstlane(lds[p0 + s]);
        int32_t at = -1;
        if (e < (uint32_t)a.E) {
            uint32_t count = 0;
            if constexpr (CHUNKED) {
                uint32_t below = 0;
                for (int i = lane; i < (int)e; i += 64) below += (uint32_t)a.total[i];
                count = wave_usum(below) + (uint32_t)a.start[chunk * a.E + e];
            }
            for (int i0 = 0; i0 < n; i0 += 256) {
#pragma unroll
                for (int i = i0 + lane; i < i0 + 256; i += 64) {
                    const uint32_t q = (uint32_t)lds[i];
                    const bool in_front = (q == e && i < p0 + s) || (!CHUNKED && q < e);
                    count += (uint32_t)__popcll(__ballot(in_front));
                }
            }
            at = (int32_t)count;
        }
        if (lane == 0) {
            place[s] = at;
            a.inverse[t * a.k + s] = at;
            if (a.xs && at >= 0) a.rs[at] = a.xs[t];
        }
    }
    __syncthreads();
    const char* src = a.x + t * a.ldx;
    const int64_t nv = a.row_bytes / 16;
    // Short rows: several slots at a time (`per` threads a slot)
    const int per = nv >= 256 ? 256 : nv > 128 ? 256 : nv > 64 ? 128 : 64;
    const int g = tid / per, groups = 256 / per;
    for (int64_t v = tid % per; v < nv; v += per) {
        u32x4 w;
        __builtin_memcpy(&w, src + v * 16, 16);
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
// seedmm_moe_unsort and its gradients: TPR threads a token, 8 columns a thread and pass.  A
// token's places and weights are uniform over a wave; the rows of 8 slots are in flight at once.
// ----------------------------------------------------------------------------------
struct UnsortArgs {
    const void* rows;         // [n_rows][ldr]
    const int32_t* inverse;   // [T][k]
    const float* w;           // [T][k] or null
    void* y;                  // [T][ldy]
    const void* dy;           // [T][ldy] (gradients)
    void* drows;              // [n_rows][ldg] or null
    float* dw;                // [T][k] or null
    int64_t ldr, ldy, ldg, t0, T;   // tokens from t0 on
    uint32_t n_rows;
    int k, H, y_bf16;
};

constexpr int kSlots = 8;     // slots in flight

template <int TPR, int RT>
__global__ __launch_bounds__(256) void k_unsort(const UnsortArgs a) {
    const int tid = threadIdx.x;
    const int64_t t = a.t0 + (int64_t)blockIdx.x * (256 / TPR) + __builtin_amdgcn_readfirstlane(tid / TPR);
    if (t >= a.T) return;
    const int32_t* inv = a.inverse + t * a.k;
    const float* w = a.w ? a.w + t * a.k : nullptr;
    for (int c = tid % TPR * 8; c < a.H; c += TPR * 8) {
        const int n = a.H - c;
        float sum[8] = {};
        for (int s0 = 0; s0 < a.k; s0 += kSlots) {
            Eight<RT> r[kSlots];
            bool has[kSlots];
#pragma unroll
            for (int s = 0; s < kSlots; ++s) {
                const uint32_t at = s0 + s < a.k ? (uint32_t)inv[s0 + s] : 0xFFFFFFFFu;
                has[s] = at < a.n_rows;
                if (has[s]) r[s].load(a.rows, at * a.ldr + c, n);
            }
#pragma unroll
            for (int s = 0; s < kSlots; ++s) {
                if (!has[s]) continue;
                const float f = w ? w[s0 + s] : 1.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] = __builtin_fmaf(f, r[s].get(j), sum[j]);
            }
        }
        if (a.y_bf16) store8<SEEDMM_BF16>(a.y, t * a.ldy + c, n, sum);
        else store8<SEEDMM_F32>(a.y, t * a.ldy + c, n, sum);
    }
}

template <int TPR, int YT, int RT>
__global__ __launch_bounds__(256) void k_unsort_grad(const UnsortArgs a) {
    __shared__ float red[4][kSlots];
    const int tid = threadIdx.x;
    const int64_t t = a.t0 + (int64_t)blockIdx.x * (256 / TPR) + __builtin_amdgcn_readfirstlane(tid / TPR);
    if (TPR < 256 && t >= a.T) return;          // no barrier below for these
    const int32_t* inv = a.inverse + t * a.k;
    for (int s0 = 0; s0 < a.k; s0 += kSlots) {
        uint32_t at[kSlots];
        float f[kSlots], dot[kSlots];
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            at[s] = s0 + s < a.k ? (uint32_t)inv[s0 + s] : 0xFFFFFFFFu;
            f[s] = at[s] < a.n_rows ? a.w[t * a.k + s0 + s] : 0.f;
            dot[s] = 0.f;
        }
        for (int c = tid % TPR * 8; c < a.H; c += TPR * 8) {
            const int n = a.H - c;
            Eight<YT> d;
            Eight<RT> r[kSlots];
            d.load(a.dy, t * a.ldy + c, n);
            if (a.dw) {
#pragma unroll
                for (int s = 0; s < kSlots; ++s)
                    if (at[s] < a.n_rows) r[s].load(a.rows, at[s] * a.ldr + c, n);
            }
#pragma unroll
            for (int s = 0; s < kSlots; ++s) {
                if (at[s] >= a.n_rows) continue;
                if (a.dw) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) dot[s] = __builtin_fmaf(d.get(j), r[s].get(j), dot[s]);
                }
                if (a.drows) {
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = f[s] * d.get(j);
                    store8<RT>(a.drows, at[s] * a.ldg + c, n, v);
                }
            }
        }
        if (!a.dw) continue;
#pragma unroll
        for (int s = 0; s < kSlots; ++s) dot[s] = wave_sum(dot[s]);
        if constexpr (TPR > 64) {
            if (s0) __syncthreads();
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

// ----------------------------------------------------------------------------------
// seedmm_swiglu.  TPR threads a row, NP pieces of 8 columns a thread held in registers; for 8
// bits the row's largest |h| is found before the codes are written.
// ----------------------------------------------------------------------------------
struct SwigluArgs {
    const void* gu;           // [N][ldg]
    void* out;                // [N][ldo]
    float* scale;             // [N] with 8-bit codes
    const int32_t* count;     // null: all rows
    int64_t ldg, ldo, n0, N;  // rows from n0 on
    int I, out_dt;
};

// exp of -|g| cannot overflow: silu(g) = g / (1 + e) or, for g < 0, g e / (1 + e)
__device__ __forceinline__ float swiglu(float g, float u) {
    const float e = expf(-fabsf(g));
    return (g < 0.f ? g * e : g) / (1.f + e) * u;
}

// the larger, a NaN above everything
__device__ __forceinline__ float max_or_nan(float a, float b) { return a != a ? a : b != b ? b : fmaxf(a, b); }

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

template <int NW>     // waves that share a row
__device__ __forceinline__ float row_top(float top, float* red) {
    const uint32_t u = wave_umax(__float_as_uint(top));      // not negative: ordered as whole numbers, NaN on top
    if constexpr (NW == 1) return __uint_as_float(u);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = __uint_as_float(u);
    __syncthreads();
    float m = red[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) m = max_or_nan(m, red[i]);
    return m;
}

template <int TPR, int NP, int GT>
__global__ __launch_bounds__(256) void k_swiglu(const SwigluArgs a) {
    __shared__ float red[4];
    const int tid = threadIdx.x;
    const int64_t n = a.n0 + (int64_t)blockIdx.x * (256 / TPR) + __builtin_amdgcn_readfirstlane(tid / TPR);
    if (n >= a.N || (a.count && n >= *a.count)) return;     // a whole workgroup where waves share a row
    float h[NP][8], top = 0.f;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int c = (p * TPR + tid % TPR) * 8, cnt = a.I - c;
        if (cnt <= 0) continue;
        Eight<GT> g, u;
        g.load(a.gu, n * a.ldg + c, cnt);
        u.load(a.gu, n * a.ldg + a.I + c, cnt);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            h[p][j] = swiglu(g.get(j), u.get(j));
            top = max_or_nan(top, fabsf(h[p][j]));
        }
    }
    float inv = 0.f;
    if (a.out_dt == SEEDMM_I8) {
        const CodeScale o = code_scale(row_top<TPR / 64>(top, red));
        if (tid % TPR == 0) a.scale[n] = o.sc;
        inv = o.inv;
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int c = (p * TPR + tid % TPR) * 8, cnt = a.I - c;
        if (cnt <= 0) continue;
        if (a.out_dt == SEEDMM_I8) {
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
template <int GT>
__global__ __launch_bounds__(1024) void k_swiglu_long(const SwigluArgs a) {
    __shared__ float red[16];
    const int64_t n = a.n0 + blockIdx.x;
    if (a.count && n >= *a.count) return;
    auto piece = [&](int64_t c, float (&h)[8]) {
        Eight<GT> g, u;
        const int cnt = (int)(a.I - c < 8 ? a.I - c : 8);
        g.load(a.gu, n * a.ldg + c, cnt);
        u.load(a.gu, n * a.ldg + a.I + c, cnt);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = swiglu(g.get(j), u.get(j));
        return cnt;
    };
    float inv = 0.f;
    if (a.out_dt == SEEDMM_I8) {
        float top = 0.f;
        for (int64_t c = threadIdx.x * 8; c < a.I; c += 8192) {
            float h[8];
            piece(c, h);
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max_or_nan(top, fabsf(h[j]));
        }
        const CodeScale o = code_scale(row_top<16>(top, red));
        if (threadIdx.x == 0) a.scale[n] = o.sc;
        inv = o.inv;
    }
    for (int64_t c = threadIdx.x * 8; c < a.I; c += 8192) {
        float h[8];
        const int cnt = piece(c, h);
        if (a.out_dt == SEEDMM_I8) {
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

template <int TPR, int RT>
void launch_unsort(const UnsortArgs& a, hipStream_t st) {
    launch_parts(k_unsort<TPR, RT>, a, &UnsortArgs::t0, a.T, TPR, 256, st);
}

template <int TPR, int YT, int RT>
void launch_grad(const UnsortArgs& a, hipStream_t st) {
    launch_parts(k_unsort_grad<TPR, YT, RT>, a, &UnsortArgs::t0, a.T, TPR, 256, st);
}

template <int YT, int RT>
void launch_grad(const UnsortArgs& a, hipStream_t st) {
    if (a.H <= 512) launch_grad<64, YT, RT>(a, st);
    else launch_grad<256, YT, RT>(a, st);
}

template <int TPR, int NP, int GT>
void launch_swiglu(const SwigluArgs& a, hipStream_t st) {
    launch_parts(k_swiglu<TPR, NP, GT>, a, &SwigluArgs::n0, a.N, TPR, 256, st);
}

template <int GT>
void launch_swiglu(const SwigluArgs& a, hipStream_t st) {
    if (a.I <= 512) launch_swiglu<64, 1, GT>(a, st);
    else if (a.I <= 2048) launch_swiglu<256, 1, GT>(a, st);
    else if (a.I <= 4096) launch_swiglu<256, 2, GT>(a, st);
    else if (a.I <= 8192) launch_swiglu<256, 4, GT>(a, st);
    else launch_parts(k_swiglu_long<GT>, a, &SwigluArgs::n0, a.N, 1024, 1024, st);
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
    const bool chunked = need != 0;
    if (chunked) {
        a.total = (int32_t*)workspace;
        a.start = a.total + E;
        hipLaunchKernelGGL(k_sort_count, dim3((unsigned)a.chunks), dim3(256), (size_t)E * 4, st, a);
        hipLaunchKernelGGL(k_sort_scan, dim3((unsigned)((E + 15) / 16)), dim3(256), 0, st, a);
    }
    const int held = chunked ? kSortChunk : (T * top_k + 255) & ~255;
    const size_t lds = 4 * (size_t)(E > held ? E : held);
    constexpr int64_t most = kLaunchThreads / 256;
    for (int64_t b0 = 0; b0 < (int64_t)T + 1; b0 += most) {     // the offsets, then a token a workgroup
        const int64_t n = (int64_t)T + 1 - b0 < most ? (int64_t)T + 1 - b0 : most;
        if (chunked) hipLaunchKernelGGL((k_sort<true>), dim3((unsigned)n), dim3(256), lds, st, a, b0);
        else hipLaunchKernelGGL((k_sort<false>), dim3((unsigned)n), dim3(256), lds, st, a, b0);
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
    UnsortArgs a = {rows, inverse, topk_w, y, nullptr, nullptr, nullptr, ldr, ldy, 0, 0, T, (uint32_t)n_rows,
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
    UnsortArgs a = {rows, inverse, topk_w, nullptr, dy, drows, dw, ldr, ldd, ldg, 0, T, (uint32_t)n_rows, top_k, H, 0};
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
    g_dtype == SEEDMM_F32 ? launch_swiglu<SEEDMM_F32>(a, st) : launch_swiglu<SEEDMM_BF16>(a, st);
    return launch_status();
}

// Scratch of one layer call: the order, the sorted rows, gate and up (whose room the down
// product's rows take later), and the SwiGLU rows.
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
