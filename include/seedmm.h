/*
 * seedmm.h -- C ABI of the SeedLM seed-decoding matrix products for AMD MI355X (gfx950).
 *
 * What the library computes.  A weight matrix W[M][K] is stored as blocks of 8
 * consecutive weights along K (block b = m*(K/8) + k/8).  Each block holds a 16-bit
 * LFSR seed, P (3 or 4) signed int4 coefficients and a 4-bit exponent code; each
 * matrix holds one int32 exp_bias (model card "K2-Horizon-MoVA-36B-A4B - NanoSeedLM
 * p4mx-q4v", section "This upload": NAME.seeds U16, NAME.coefs U16, NAME.codes U8,
 * NAME.exp_bias I32).  The kernels regenerate each block inside the product and never
 * write W back (NanoSeedLM README, "Highlights"; barnson.org post, "What I changed:
 * September 2026", never decompress):
 *
 *     w_i = 2^(code + exp_bias - 15) * sum_{j<P} c_j * (s_{iP+j+1} - 32768),  i = 0..7
 *
 * where s_1, s_2, ... are the states after steps 1, 2, ... of a 16-bit Fibonacci
 * register started at the seed (shift left, new bit = parity(state & 0xB400)), the
 * basis is filled row-major, c_j = (q ^ 8) - 8 for nibble q (barnson.org post, "LFSR is
 * free"), and the power of two multiplies (barnson.org post, "Attempt one").
 *
 * Stream layout of one matrix (all little-endian):
 *   seeds  uint16[M*K/8]              one seed per block;
 *   coefs  uint16[ceil(M*K/8*P/4)]    one nibble stream, P nibbles per block, nibble
 *                                     n = b*P + j at word n>>2, bits 4*(n&3);
 *   codes  uint8 [ceil(M*K/16)]       two 4-bit codes per byte, even block in the low nibble.
 * Stacked experts ([E] matrices of equal shape) are the E single-matrix streams
 * concatenated; this requires (M*K/8)*P % 4 == 0 and (M*K/8) % 2 == 0.  The weights
 * are exact in fp32: |sum| <= 2^20 and the scale is a power of two.
 *
 * Conventions for every entry point:
 *   - All array pointers are DEVICE pointers owned by the caller (e.g. PyTorch tensors).
 *     The library allocates no memory and keeps no mutable global state: no streams,
 *     events or tables of its own.  Scratch memory (the layer's workspace, the encoder's
 *     table, a second stream and its events) comes from the caller, so calls are
 *     reentrant and calls from several host threads are independent as long as they do
 *     not share a workspace, a table being prepared or a seedmm_side.
 *   - Work is enqueued asynchronously on `hip_stream` (a hipStream_t; NULL = the
 *     default stream).  Results are valid after the stream is synchronised.
 *   - Arguments are validated before anything is launched; an error returns a negative
 *     status and launches nothing.  SEEDMM_EHIP reports a failed kernel launch
 *     (hipGetLastError); faults during execution surface at the next synchronisation.
 *   - Limits: K % 8 == 0; P in {3, 4}; exp_bias in [-100, 100] (keeps every weight a
 *     normal fp32); activation rows 16-byte aligned (x pointer 16-byte aligned, ldx a
 *     multiple of 8 elements for bf16 and of 4 for fp32).  Seed streams that are 16-byte
 *     aligned with K % 64 == 0 take the vector-load path; other layouts take a per-block
 *     path with the same results.
 */
#ifndef SEEDMM_H
#define SEEDMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
    SEEDMM_OK = 0,
    SEEDMM_EINVAL = -1,     /* null pointer, bad size, bad P / dtype / exp_bias / ld   */
    SEEDMM_EALIGN = -2,     /* activation or output pointer / leading dim misaligned  */
    SEEDMM_EWORKSPACE = -3, /* workspace missing or smaller than seedmm_moe_workspace_bytes */
    SEEDMM_EHIP = -4,       /* the HIP runtime reported a launch failure              */
    SEEDMM_ECAPACITY = -5,  /* an expert cache call routes to more distinct experts
                               than the cache has slots                               */
    SEEDMM_ESCRATCH = -6    /* seedmm_moe_noalloc: the batch needs more scratch than
                               SEEDMM_NOALLOC_SCRATCH_BYTES                           */
};

enum { SEEDMM_F32 = 0, SEEDMM_BF16 = 1, SEEDMM_I8 = 2 /* dense operators only */ };
enum { SEEDMM_SOFTMAX = 0, SEEDMM_SIGMOID = 1 };   /* scores of seedmm_route */

/* One seed-coded matrix, or E stacked matrices of one shape (streams concatenated). */
typedef struct seedmm_mat {
    const uint16_t *seeds;    /* NAME.seeds                                     */
    const uint16_t *coefs;    /* NAME.coefs (nibble stream)                     */
    const uint8_t *codes;     /* NAME.codes (two codes per byte)                */
    const int32_t *exp_bias;  /* NAME.exp_bias, int32[E] in device memory      */
} seedmm_mat;

/*
 * seedmm_gemv -- y = W x for one fp32 activation vector (the decode matrix-vector
 * product of the SeedLM pages: NanoSeedLM README "How it works").
 *   seeds/coefs/codes: one [M][K] matrix;  exp_bias: its bias (by value);
 *   x: fp32[K];  y: fp32[M] (overwritten).  Runs on the default stream.
 *   Accumulates in fp32 with exact fp32 weights.
 * Errors: SEEDMM_EINVAL (null pointer, M < 0, K < 0, K % 8 != 0, P not 3/4, exp_bias
 * out of range), SEEDMM_EALIGN (x not 16-byte aligned), SEEDMM_EHIP.
 */
int seedmm_gemv(const uint16_t *seeds, const uint16_t *coefs, const uint8_t *codes,
                int32_t exp_bias, const float *x, float *y, int M, int K, int P);

/*
 * seedmm_gemv_ex -- Y[n] = W X[n] for N activation rows: the product of seedmm_gemv for a
 * batch of rows that share each regenerated block (barnson.org post, "What I changed:
 * September 2026": the weights are rebuilt inside the product, never stored).
 *   x: row-major [N][ldx] of dtype x_dtype (SEEDMM_F32 or SEEDMM_BF16 raw bits);
 *   y: fp32 row-major [N][ldy], overwritten (ldy >= M).
 *   fp32 x: fp32 products and sums with exact weights.  bf16 x: the block weights are
 *   rounded to bf16 (nearest even) and multiplied on the matrix cores with fp32
 *   accumulation.
 * Errors: as seedmm_gemv, plus SEEDMM_EINVAL for N < 0, ldx < K, ldy < M, bad dtype;
 * SEEDMM_EALIGN for a misaligned x or ldx.
 */
int seedmm_gemv_ex(const uint16_t *seeds, const uint16_t *coefs, const uint8_t *codes,
                   int32_t exp_bias, const void *x, int x_dtype, int ldx, float *y, int ldy,
                   int M, int K, int P, int N, void *hip_stream);

/*
 * seedmm_reconstruct -- write W[M][K] row-major: fp32 (exact) or bf16 (round to nearest
 * even of the exact fp32).  The reference point for bit-exact checks against a scalar C
 * reference (barnson.org post, "What I changed: September 2026": every GPU path is held
 * to a plain C function); the products above never materialise W.  A seed of 0 is
 * decoded like any other (every state is 0, every basis value -32768).
 * Errors: SEEDMM_EINVAL (null pointer, bad size, P, dtype or exp_bias), SEEDMM_EHIP.
 */
int seedmm_reconstruct(const uint16_t *seeds, const uint16_t *coefs, const uint8_t *codes,
                       int32_t exp_bias, void *W, int w_dtype, int M, int K, int P,
                       void *hip_stream);

/*
 * seedmm_moe_dispatch -- group the (token, slot) pairs of a routed batch by expert (the
 * routed experts of a layer, K2-Horizon card "This upload": 100 routed experts per
 * layer, top-8; each expert's matrices are then read once for all its tokens).
 *   topk_ids: int32[T][top_k], each in [0, E) and distinct within a token.
 *   counts: int32[E] (out) -- number of pairs routed to each expert;
 *   lists:  int32[E][T] (out) -- expert e's pair indices p = t*top_k + slot, in
 *           increasing order, in lists[e*T .. e*T + counts[e]).  Entries past counts[e]
 *           are not written.
 * Deterministic.  Ids outside [0, E) are counted nowhere (the caller validates ids).
 * Errors: SEEDMM_EINVAL (null pointer, T < 0, top_k < 1, E < 1, T*top_k >= 2^31),
 * SEEDMM_EHIP.
 */
int seedmm_moe_dispatch(const int32_t *topk_ids, int T, int top_k, int E, int32_t *counts,
                        int32_t *lists, void *hip_stream);

/* Bytes of scratch memory seedmm_moe (and _ex, _timed, _mixed, seedmm_cache_moe) needs
 * for a batch of T tokens routed to top_k of E experts of hidden size H and intermediate
 * size I (0 on bad args, T*top_k >= 2^31 among them): expert counts int32[E], pair lists int32[E][T], the SwiGLU rows
 * bf16 [T*top_k][I] and the per-slot outputs fp32 [T*top_k][H], each 256-byte aligned,
 * plus per-tile counts int32[ceil(T*top_k/8192)][E] above 8,192 pairs.  H and I enter
 * because the SwiGLU rows and the per-slot outputs dominate the size.  (Routed layer of
 * the K2-Horizon card, "This upload".) */
size_t seedmm_moe_workspace_bytes(int T, int top_k, int E, int H, int I);

/*
 * seedmm_moe -- one routed mixture-of-experts layer of SwiGLU experts whose weights
 * are seeds (K2-Horizon card "This upload": routed FFN experts are SeedLM P=4):
 *     y[t] = sum_{s < top_k} topk_w[t][s] * down_e( silu(gate_e x[t]) * (up_e x[t]) ),
 *     e = topk_ids[t][s],  silu(z) = z / (1 + exp(-z)).
 *   (The pages do not spell out the expert FFN; SwiGLU experts with softmax-weighted
 *   top-k slots are this library's reading.)
 *   x: bf16 [T][H] (raw bits), y: fp32 [T][H] (overwritten);
 *   gate, up: E stacked [I][H] matrices; down: E stacked [H][I] matrices;
 *   topk_ids: int32[T][top_k], each in [0, E) and distinct within a token (the caller
 *   validates them; a token that breaks this gets undefined y);
 *   workspace: device scratch of at least seedmm_moe_workspace_bytes(T, top_k, E, H, I)
 *   bytes, 16-byte aligned; its contents need not be initialised.  Calls that overlap
 *   in time must use different workspaces.
 *   Expert products run on the matrix cores with bf16 weights and fp32 accumulation;
 *   the SwiGLU output h is rounded to bf16 (nearest even) before the down product, in
 *   the decode and the prefill kernels alike; the slots of a token are summed in slot
 *   order, so results are bit-reproducible and a token's output does not depend on the
 *   other tokens of the batch.  All work runs on hip_stream (seedmm_moe_ex splits it
 *   over a second stream of the caller's).
 * Errors: SEEDMM_EINVAL (null pointer, T < 0, top_k outside [1, min(E, 64)], T*top_k
 * >= 2^31 (pair indices are int32), E < 1 or > 4096, H or I not a multiple of 8, P not 3/4, stacked streams not whole words),
 * SEEDMM_EALIGN (x not 16-byte aligned or H % 8 != 0), SEEDMM_EWORKSPACE, SEEDMM_EHIP.
 */
int seedmm_moe(const int32_t *topk_ids, const float *topk_w, int T, int top_k,
               const void *x, float *y, int E, int H, int I, int P,
               seedmm_mat gate, seedmm_mat up, seedmm_mat down,
               void *workspace, size_t workspace_bytes, void *hip_stream);

/*
 * seedmm_moe_ex -- the routed layer of seedmm_moe (one P) or seedmm_moe_mixed (P = 0 and
 * p4mask), with a second stream from the caller.  The layer runs as two independent
 * halves: for one P, the experts e < E/2 on hip_stream and the others on side->stream;
 * for mixed packs, the P = 4 launches on hip_stream and the P = 3 launches on
 * side->stream.  side->fork is recorded on hip_stream after the dispatch and waited for
 * by side->stream; side->join is recorded on side->stream after its launches and waited
 * for by hip_stream before the combine.  So all the work still completes in hip_stream's
 * order, and graph capture on hip_stream records the fork and the join as dependencies.
 * The two halves' workgroups fill each other's partly empty last rounds (each expert
 * kernel leaves part of the chip idle at its tail).  The output bits equal seedmm_moe's.
 *   side: NULL or side->stream NULL = everything on hip_stream.  Otherwise side->stream
 *   is a stream of hip_stream's device other than hip_stream, and side->fork and
 *   side->join are events (hipEventDisableTiming is enough), all created and owned by
 *   the caller.  Calls that may overlap in time must not share a seedmm_side.  One-token
 *   batches run on hip_stream alone (splitting their slots over two streams measured
 *   slower: the cross-stream edges cost more than the overlap gains).
 * Errors: as seedmm_moe; SEEDMM_EINVAL also for P = 0 without p4mask, a p4mask with
 * P = 3 or 4, or a side stream given without both events or equal to hip_stream.  If the
 * fork cannot be recorded the call runs on hip_stream alone; if the join cannot be
 * recorded it returns SEEDMM_EHIP without launching the combine (y is then not valid).
 */
typedef struct seedmm_side {
    void *stream;   /* hipStream_t */
    void *fork;     /* hipEvent_t  */
    void *join;     /* hipEvent_t  */
} seedmm_side;

int seedmm_moe_ex(const int32_t *topk_ids, const float *topk_w, int T, int top_k,
                  const void *x, float *y, int E, int H, int I, int P, const uint32_t *p4mask,
                  seedmm_mat gate, seedmm_mat up, seedmm_mat down,
                  void *workspace, size_t workspace_bytes, void *hip_stream,
                  const seedmm_side *side);

/*
 * seedmm_moe_noalloc -- seedmm_moe without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc).  Its scratch memory is a static device array of the library,
 * SEEDMM_NOALLOC_SCRATCH_BYTES (8 MiB) on every device it runs on, held until the process
 * ends; the call allocates nothing (no hipMalloc, no hipFree, no allocating library
 * routine).  The first call on a device looks up that device's copy of the array
 * (hipGetSymbolAddress) with the device current; make it outside graph capture.
 *   Arguments, results and errors as seedmm_moe (one stream), plus SEEDMM_ESCRATCH when
 *   seedmm_moe_workspace_bytes(T, top_k, E, H, I) exceeds SEEDMM_NOALLOC_SCRATCH_BYTES
 *   (for 100 experts 2048 -> 1024 -> 2048, top-8: up to 96 tokens), checked before
 *   anything runs, and SEEDMM_EINVAL when hip_stream belongs to another device than the
 *   current one (the array used is the current device's).
 *   Every call on one device shares that device's array: calls that overlap in time on
 *   one device race (serialise them on one stream), and the array keeps the last call's
 *   contents, which no call reads before writing them.
 */
#define SEEDMM_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)
int seedmm_moe_noalloc(const int32_t *topk_ids, const float *topk_w, int T, int top_k,
                       const void *x, float *y, int E, int H, int I, int P,
                       seedmm_mat gate, seedmm_mat up, seedmm_mat down, void *hip_stream);

/*
 * seedmm_moe_timed -- seedmm_moe that also records caller-created hipEvent_t handles on
 * hip_stream between its kernels, for measuring each stage in place (the pages time
 * their engines stage by stage: NanoSeedLM documentation index, "Results"):
 *   events[0] before the dispatch, events[1] after it, events[2] after the gate/up
 *   kernel, events[3] after the down kernel, events[4] after the combine.  A one-token
 *   batch (T = 1) runs no dispatch kernel (its top_k ids name the experts directly), so
 *   events[0] and events[1] are recorded back to back; with one P, vector layouts and
 *   2 <= top_k <= 8 it runs no combine kernel either (its down kernel adds the slots,
 *   same bits), so events[3] and events[4] are back to back too.
 * `events` may be NULL and any entry may be NULL.  Same arguments, results and errors
 * as seedmm_moe; no event is recorded when the arguments are rejected.  When `events`
 * is not NULL every kernel runs on hip_stream (no side stream), so the recorded stage
 * times are those of single launches over all experts.
 */
int seedmm_moe_timed(const int32_t *topk_ids, const float *topk_w, int T, int top_k,
                     const void *x, float *y, int E, int H, int I, int P,
                     seedmm_mat gate, seedmm_mat up, seedmm_mat down,
                     void *workspace, size_t workspace_bytes, void *hip_stream,
                     void *const *events);

/*
 * seedmm_moe_mixed -- seedmm_moe for mixed packs: P chosen per expert (NanoSeedLM
 * documentation index: "Results", hybrid P3 / P4 seed packs with a third of the experts
 * in P4; "Plans", a P4 tier for the hot experts and P3 for the rest).
 *   p4mask: device uint32[ceil(E/32)], bit e (word e/32, bit e%32) set when expert e has
 *   P = 4, clear when it has P = 3.
 *   Stacked streams: seeds and codes at the same per-expert strides as seedmm_moe;
 *   expert e's coefficient stream starts at word (I*H/8/4) * (3e + number of P = 4
 *   experts before e), i.e. the experts' own streams concatenated in expert order.
 *   Requires (I*H/8) % 4 == 0.  Other arguments, results and errors as seedmm_moe
 *   (SEEDMM_EINVAL also for a NULL p4mask).  Each expert kernel runs once per P; a
 *   launch serves only the experts of its P.  All work runs on hip_stream
 *   (seedmm_moe_ex with P = 0 runs the P = 3 launches on a second stream).
 */
int seedmm_moe_mixed(const int32_t *topk_ids, const float *topk_w, int T, int top_k,
                     const void *x, float *y, int E, int H, int I, const uint32_t *p4mask,
                     seedmm_mat gate, seedmm_mat up, seedmm_mat down,
                     void *workspace, size_t workspace_bytes, void *hip_stream);

/*
 * seedmm_search -- encode W [M][K] into a seed-coded matrix by the exhaustive seed search
 * (Qwen3.8-Flash-Next-NanoSeedLM-P4 card, "How it works": every one of the 65,535 seeds
 * is tried for every block; barnson.org post, "GPU search == CPU search").  For each
 * block of 8 weights w (with importances d, all ones when colw is NULL) and every seed:
 *   U_ij = s_{iP+j+1} - 32768 (the states the products regenerate);
 *   alpha solves A alpha = r, A_jk = sum_i (d_i U_ij) U_ik, r_j = sum_i (d_i U_ij) w_i, by
 *   Gaussian elimination with partial pivoting (a pivot below 1e-300 skips the seed);
 *   for every code 0..15: c_j = clamp(round_half_even(alpha_j / 2^(code+exp_bias-15)),
 *   -8, 7), err = sum_i d_i (w_i - 2^(code+exp_bias-15) sum_j U_ij c_j)^2;
 * and keeps the smallest (err, seed, code).  Every step is an IEEE double operation in
 * that order (sums in increasing i, no contraction), so the result equals a CPU
 * evaluation of the same definition bit for bit.
 *   W: fp32 row-major [M][ldw] (ldw >= K), K % 8 == 0;  colw: fp32 [K] importances of
 *   the columns (activation weighting) or NULL;  outputs in the layout the products
 *   read: seeds uint16[M*K/8], coefs uint16[ceil(M*K/8*P/4)], codes uint8[ceil(M*K/16)],
 *   err: float64[M*K/8] squared error of each block (may be NULL).  A block for which
 *   no seed gives a solvable system gets seed 0, zero coefficients and err = +inf.
 *   Pairs (block, seed) that provably cannot win are skipped (a least-squares bound and,
 *   at P = 4, a bound of every code's error, each with a safe margin); the result is the
 *   same as evaluating them all.
 *   table: without importances (colw NULL), device memory of at least
 *   seedmm_search_table_bytes(P) bytes, 256-byte aligned, filled for this P by
 *   seedmm_search_prepare on hip_stream or before it in stream order (a table filled for
 *   the other P, or not filled, gives undefined results); with importances it is not
 *   read and may be NULL.  The call only launches kernels (no host wait), so it can be
 *   captured into a graph.  Calls may share a prepared table and overlap on different
 *   streams.
 * Errors: SEEDMM_EINVAL (null pointer, a NULL table without importances, bad size, P not
 * 3/4, exp_bias outside [-100, 100], ldw < K), SEEDMM_EALIGN (table not 256-byte
 * aligned), SEEDMM_EHIP.
 */
int seedmm_search(const float *W, int ldw, const float *colw, int M, int K, int P,
                  int32_t exp_bias, uint16_t *seeds, uint16_t *coefs, uint8_t *codes,
                  double *err, const void *table, void *hip_stream);

/*
 * The encoder's per-seed table for one P (barnson.org post, "LFSR is free": the pages'
 * encoder and decoder precompute per-seed streams; here the search precomputes, once per
 * P, each seed's basis rows along the register's cycle, its normal matrix, the matrix's
 * Cholesky factor and a certified bound of its smallest eigenvalue): about 16.5 MB
 * (P = 4) or 12.3 MB (P = 3) of caller-owned device memory.
 * seedmm_search_table_bytes returns the size (0 for P not 3/4).  seedmm_search_prepare
 * fills `table` on hip_stream with kernels only (no host wait; capturable).
 * Errors: SEEDMM_EINVAL (P not 3/4, NULL table, table_bytes too small), SEEDMM_EALIGN
 * (table not 256-byte aligned), SEEDMM_EHIP.
 */
size_t seedmm_search_table_bytes(int P);
int seedmm_search_prepare(int P, void *table, size_t table_bytes, void *hip_stream);

/*
 * Expert cache: routed experts resident in host memory, the recently used ones in device
 * memory (NanoSeedLM README, "Highlights": the engine can keep the routed experts in
 * RAM with a VRAM cache of the recently used ones, and "With the engine": a cache sized
 * with --expert-cache-gb; documentation index, "Results": LRU beats LFU and a fixed hot
 * set as the eviction policy).
 *
 * One cache serves one layer of E experts (gate/up [I][H], down [H][I], one P) with S
 * device slots.  An expert is one RECORD of its nine streams, in the order gate.seeds,
 * gate.coefs, gate.codes, up.seeds, ..., down.codes, each stream (the expert's own
 * streams as in seedmm_moe: n*2, ceil(n*P/4)*2 and ceil(n/2) bytes, n = I*H/8) starting
 * at a multiple of 256 bytes from the record start; seedmm_cache_record_layout gives the
 * offsets and the record size (a multiple of 256).  Loading an expert copies its record.
 * All memory is the caller's:
 *   state      host memory of seedmm_cache_state_bytes(E, S) bytes, 8-byte aligned: the
 *              bookkeeping (which expert sits in which slot, last use of each slot,
 *              counters); it is the cache handle, used only by the calls below;
 *   device     device memory of seedmm_cache_device_bytes(E, H, I, P, S) bytes,
 *              256-byte aligned: S records and the device expert -> slot map;
 *   host_pack  PINNED host memory (hipHostMalloc) of E records, expert e at byte
 *              e * record; read by host-to-device copies only;
 *   exp_bias   device int32[3][E]: the exp_bias of gate, up and down of every expert
 *              (stays resident).
 * Calls on one cache must not overlap (one host thread at a time), and their device work
 * must run in call order: a call's record copies can overwrite slots that the previous
 * call's kernels still read, so pass one stream to every call on a cache, or make the
 * new call's stream wait for the previous call's.  The host pack must stay unchanged
 * while the cache is in use (seedmm_cache_reset after changing it).
 */
typedef struct seedmm_cache seedmm_cache;

/* Record size in bytes, and the nine stream offsets into `offsets` (may be NULL); 0 for
 * an invalid shape. */
size_t seedmm_cache_record_layout(int H, int I, int P, size_t offsets[9]);
size_t seedmm_cache_state_bytes(int E, int S);
size_t seedmm_cache_device_bytes(int E, int H, int I, int P, int S);

/* Initialise `state` as an empty cache.  Host only (no HIP call).  Requires E in
 * [1, 4096], S in [1, E], P in {3, 4} and the layer shapes of seedmm_moe (H, I > 0,
 * multiples of 8, with the stacking conditions on n = I*H/8: n*P % 4 == 0, n % 2 == 0).
 * Errors: SEEDMM_EINVAL (null pointer, bad size, state_bytes or device_bytes too small),
 * SEEDMM_EALIGN (state not 8-byte or device not 256-byte aligned). */
int seedmm_cache_init(void *state, size_t state_bytes, int E, int H, int I, int P, int S,
                      const void *host_pack, const int32_t *exp_bias, void *device,
                      size_t device_bytes);

/* Empty the cache and zero its counters (every expert is loaded again on its next use).
 * Host only. */
int seedmm_cache_reset(seedmm_cache *cache);

/* The host half of one call, on its own: marks the distinct experts of topk_ids_host
 * [T][top_k] used and assigns a slot to each that is not resident.  Resident experts are
 * hits; each miss takes, in increasing expert order, the lowest free slot, else the slot
 * whose expert was used longest ago (ties: lowest slot) among those this call does not
 * use.  loads: host int32[2*S] receiving (expert, slot) pairs in that order (may be
 * NULL); *n_loads their count.  Host only; the state changes only on success.
 * Errors: SEEDMM_EINVAL (id outside [0, E), bad T / top_k), SEEDMM_ECAPACITY (more
 * distinct experts than slots). */
int seedmm_cache_plan(seedmm_cache *cache, const int32_t *topk_ids_host, int T, int top_k,
                      int32_t *loads, int *n_loads);

/* One routed layer call through the cache: seedmm_cache_plan on topk_ids_host, then on
 * hip_stream one host-to-device copy of every loaded expert's record into its slot, the
 * update of the device slot map, and the layer of seedmm_moe reading the experts from
 * their slots.  topk_ids (device) must hold the same ids as topk_ids_host; the other
 * arguments, results and errors are seedmm_moe's, plus SEEDMM_ECAPACITY; argument errors
 * leave the state unchanged.  The output equals seedmm_moe's on the resident layer bit
 * for bit.  If a copy or launch fails the cache is emptied and SEEDMM_EHIP returned. */
int seedmm_cache_moe(seedmm_cache *cache, const int32_t *topk_ids_host,
                     const int32_t *topk_ids, const float *topk_w, int T, int top_k,
                     const void *x, float *y, void *workspace, size_t workspace_bytes,
                     void *hip_stream);

/* Counters since init or reset: out[0] calls, out[1] expert uses (distinct experts per
 * call, summed), out[2] hits, out[3] misses (= records copied), out[4] bytes copied
 * host-to-device. */
int seedmm_cache_stats(const seedmm_cache *cache, uint64_t out[5]);

/*
 * Dense operators around the routed layer.  A pack keeps everything but its routed experts
 * in affine 4 bits (Qwen3.8-Flash-Next-NanoSeedLM-P4 card, "Files", and K2-Horizon card,
 * "This upload": NAME.weight, NAME.scales, NAME.biases in groups of 32 or 64), normalises
 * the residual stream before each layer and chooses the experts with a router.
 *
 * seedmm_q4_gemv -- Y[n] = W X[n] for N activation rows, with W[m][k] = s q + b:
 *     y[n][m] = x_scale[n] * sum_g ( s[m][g] sum_{k in g} q[m][k] x[n][k]
 *                                    + b[m][g] sum_{k in g} x[n][k] )
 *   weight: uint32[M][K/8], code q of column k in word k/8, bits 4*(k%8);
 *   scales, biases: [M][K/group] of s_dtype (SEEDMM_F32 or SEEDMM_BF16); group 32, 64 or
 *   128; columns g*group .. g*group + group - 1 form group g;
 *   x: [N][ldx] of x_dtype (SEEDMM_F32, SEEDMM_BF16 or SEEDMM_I8);  x_scale: fp32[N] with
 *   SEEDMM_I8 (the value of a code c of row n is c * x_scale[n]), NULL otherwise;
 *   y: [N][ldy] of y_dtype (SEEDMM_F32 or SEEDMM_BF16), overwritten; columns M .. ldy - 1
 *   are left as they were.
 *   Weights are not rounded to the activations' type: the codes enter the matrix
 *   instructions as integers, code times activation is exact, sums are fp32 (exact inside a
 *   group for SEEDMM_I8), the scales and biases multiply the groups' sums in fp32 (with fp32
 *   biases and laid-out rows a group's b X is off by less than 2^-21 of it), and y is
 *   rounded once.  15 sum_{k in g} |x[n][k]| of a group has to be an fp32 number, and what an
 *   fp32 x has below 2^-133 is dropped.  The sums run in a fixed order that depends on the
 *   sizes and types only: the same call gives the same bits.  A row of x with an infinity or
 *   NaN gives a row of y without finite meaning and leaves the other rows alone.
 * Errors: SEEDMM_EINVAL (null pointer, M, K or N < 0, M or K above 2^30, N above 2^30 - 64,
 * another group, K % group != 0, ldx < K, ldy < M, bad dtype, x_scale missing or given without
 * SEEDMM_I8), SEEDMM_EALIGN (weight, x or the workspace not 16-byte aligned, ldx not a
 * multiple of 16 bytes where N > 1, another pointer not aligned to its type),
 * SEEDMM_EWORKSPACE (workspace missing or smaller than seedmm_q4_workspace_bytes),
 * SEEDMM_EHIP.  M = 0 or N = 0 is an empty success; K = 0 writes zeros.
 */
int seedmm_q4_gemv(const uint32_t *weight, const void *scales, const void *biases, int s_dtype,
                   int group, const void *x, int x_dtype, int ldx, const float *x_scale, void *y,
                   int y_dtype, int ldy, int M, int K, int N, void *workspace,
                   size_t workspace_bytes, void *hip_stream);
/* Bytes of device scratch (16-byte aligned, contents need not be initialised) that a product
 * of these sizes needs: 0 for few rows (up to 16; 5 with fp32 x); else the activation rows in
 * the operands' order, where a launch lays them out (fp32 x, and large products), and the
 * partial sums, where K is split over workgroups; 0 too where neither is so.  Where it is 0,
 * workspace may be NULL.  0 on bad arguments.  Calls that overlap in time use different
 * workspaces. */
size_t seedmm_q4_workspace_bytes(int x_dtype, int group, int M, int K, int N);

/*
 * seedmm_add_norm -- the residual's addition and the root-mean-square norm before a layer
 * (the stream that seedmm_moe's fp32 output is added to):
 *     r = x + delta;   out = r / sqrt(mean_h r^2 + eps) * weight
 *   x: [N][ldx] fp32 or bf16;  delta: [N][ldd] fp32 or bf16, or NULL (r = x);
 *   weight: [H] fp32 or bf16, or NULL (ones);
 *   residual: [N][ldr] of x's type receiving r, or NULL; it may be x itself, with ldr = ldx.
 *   Outputs overlap inputs in no other way.
 *   out: [N][ldo] of out_dtype.  SEEDMM_F32, SEEDMM_BF16: the value, rounded once.
 *   SEEDMM_I8: codes round(value / scale[n]) in [-127, 127] with scale[n] = max_h |value| /
 *   127 (at least 2^-126); a row that holds an infinity or NaN gets scale NaN and codes 0.
 *   scale: fp32[N] with SEEDMM_I8, NULL otherwise.
 *   r is an fp32 sum, not rounded further before the norm (only where it is stored as bf16).
 *   Squares are summed in fp32, of a row taken times a power of two where fp32 does not hold
 *   them, so finite rows of any size have their norm; r times weight has to be an fp32 number,
 *   and a row of zeros with eps = 0 has no value (0/0).  Rows of any ld
 *   and alignment are taken; rows that start on 16 bytes are faster.  Elements past H are
 *   left as they were.
 * Errors: SEEDMM_EINVAL (null pointer, N or H < 0, ld < H, x as residual with another ld, bad
 * dtype, eps negative or not finite, scale missing or given without SEEDMM_I8), SEEDMM_EALIGN (a pointer not aligned
 * to its type), SEEDMM_EHIP.  N = 0 or H = 0 is an empty success.
 */
int seedmm_add_norm(const void *x, int x_dtype, int64_t ldx, const void *delta, int delta_dtype,
                    int64_t ldd, const void *weight, int w_dtype, float eps, void *residual,
                    int64_t ldr, void *out, int out_dtype, int64_t ldo, float *scale, int N, int H,
                    void *hip_stream);

/*
 * seedmm_route -- the routing that seedmm_moe takes (barnson.org post, "Why
 * K2-Horizon-MoVA": sigmoid routers whose bias only selects experts; softmax over the
 * chosen logits is this library's reading for the others):
 *   SEEDMM_SOFTMAX: the top_k largest logits of a token; weights = softmax over those.
 *   SEEDMM_SIGMOID: the top_k largest sigmoid(logit) + bias (bias fp32[E] or NULL; compared
 *   in 64 bits); weights = sigmoid(logit) over their sum, without the bias.  Sigmoids are
 *   64-bit numbers: where every chosen logit is below -709 they are 0, and so are the weights.
 *   logits: [T][ldl] fp32 or bf16;  ids: int32[T][top_k], w: fp32[T][top_k], in falling
 *   order of score; equal scores go to the lower expert first.
 *   A logit of -inf or NaN (and a bias of -inf or NaN) masks its expert.  Where fewer than
 *   top_k experts are left the slots that remain name masked experts, lowest first, with
 *   weight 0, so the ids of a token are always distinct and in [0, E).
 * Errors: SEEDMM_EINVAL (null pointer, T < 0, E outside [1, 4096], top_k outside
 * [1, min(E, 64)], T*top_k >= 2^31, ldl < E, bad dtype or score, a bias with
 * SEEDMM_SOFTMAX), SEEDMM_EALIGN (a pointer not aligned to its type), SEEDMM_EHIP.
 */
int seedmm_route(const void *logits, int l_dtype, int64_t ldl, const float *bias, int score, int T,
                 int E, int top_k, int32_t *ids, float *w, void *hip_stream);

/*
 * seedmm_moe_block -- one routed layer with its norm and its router on the residual
 * stream (the routed layer of the K2-Horizon card, "This upload"):
 *     r += delta;  x = bf16(r / sqrt(mean r^2 + eps) * norm_weight);
 *     ids, w = route(router x);  y = seedmm_moe(ids, w, x)
 * by the calls seedmm_add_norm, seedmm_q4_gemv, seedmm_route and seedmm_moe_ex, with their
 * results.  y is the next layer's delta.
 *   block: host struct; device pointers inside.  The router is an [E][H] matrix in affine
 *   4 bits; P = 3 or 4, or 0 with p4mask (mixed packs).
 *   r: [T][H] fp32 or bf16, updated in place if delta is not NULL;  delta: [T][H] fp32 or
 *   bf16, or NULL; it may not overlap r or y;  y: fp32[T][H];  ids: int32[T][top_k] and
 *   w: fp32[T][top_k] receive the routing (each may be NULL);
 *   workspace: device scratch of seedmm_moe_block_workspace_bytes(block, T) bytes; overlapping
 *   calls use different ones.  side: as for seedmm_moe_ex.
 * Errors: those of the four calls, before anything runs (but for SEEDMM_EHIP, of a launch that
 * HIP refuses); r, delta, y, norm_weight and the router's arrays 16-byte aligned.
 */
typedef struct seedmm_block {
    const void *norm_weight;         /* [H] or NULL                                   */
    const uint32_t *router_weight;   /* [E][H/8]                                      */
    const void *router_scales;       /* [E][H/group]                                  */
    const void *router_biases;
    const float *router_bias;        /* selection bias fp32[E] or NULL (SIGMOID only) */
    const uint32_t *p4mask;          /* mixed packs, else NULL                        */
    seedmm_mat gate, up, down;
    float eps;
    int norm_dtype, router_dtype, group, score, top_k, E, H, I, P;
} seedmm_block;

size_t seedmm_moe_block_workspace_bytes(const seedmm_block *block, int T);
int seedmm_moe_block(const seedmm_block *block, void *r, int r_dtype, const void *delta,
                     int delta_dtype, float *y, int32_t *ids, float *w, int T, void *workspace,
                     size_t workspace_bytes, void *hip_stream, const seedmm_side *side);

/*
 * Routed experts in 8-bit integers.  Not every expert of a pack is a seed (K2-Horizon card,
 * "This upload": 64 value experts, top 4, and the dense layers stay affine): these operators
 * serve the ones that are kept as 8-bit integers with a scale a channel.  seedmm_moe_sort puts
 * a routed batch's rows in the order of their experts, seedmm_i8_gemv multiplies each run of
 * rows with its expert's matrix, seedmm_swiglu joins gate and up, seedmm_moe_unsort returns
 * the weighted sum of each token's rows, and seedmm_moe_i8 is the routed layer made of them.
 * Rows of any leading dimension and alignment (of their type) are taken; rows that start on 16
 * bytes are faster.  No result depends on the order in which anything runs: the same call
 * gives the same bits, and a token's result does not depend on the batch around it.  Outputs
 * overlap neither inputs nor each other, but where a call says so.  Gradients are there for the
 * moves of rows (sort, unsort); the products, the SwiGLU step and the layer have none.
 *
 * seedmm_i8_gemv -- Y[n] = W X[n] for N rows of 8-bit integers with a scale a row, W in 8-bit
 * integers with a scale a channel, for one matrix or one an expert:
 *     y[n][m] = ( sum_k x[n][k] weight[e][m][k] ) * x_scale[n] * scales[e][m]
 *   weight: int8[E][M][K];  scales: [E][M] of s_dtype (SEEDMM_F32 or SEEDMM_BF16);
 *   offsets: NULL (E = 1, all rows), or device int32[E + 1], not decreasing, from 0 to at most
 *   N: rows offsets[e] .. offsets[e + 1] - 1 belong to expert e (seedmm_moe_sort writes them).
 *   Rows of y from offsets[E] on are left as they were.  Values outside of [0, N] are taken as
 *   the nearer end, so a wrong array gives wrong rows, never an access outside of x and y.
 *   Of rows that do not start on 4 bytes the aligned words of 4 bytes are read that hold them: up
 *   to 3 bytes in front of and behind weight and x, in words with bytes of theirs.  No result
 *   depends on these bytes.
 *   x: int8 [N][ldx];  x_scale: fp32[N];  y: [N][ldy] of y_dtype (SEEDMM_F32, SEEDMM_BF16),
 *   overwritten; columns M .. ldy - 1 are left as they were.
 *   The sums are exact (int32; all 256 codes); one is converted to fp32, multiplied by the row's
 *   scale and then by the channel's, each rounded to fp32, and y rounded once: sum * x_scale
 *   has to be an fp32 number.  A scale of NaN gives a row or a column of NaN.
 * Errors: SEEDMM_EINVAL (null pointer, M, K or N < 0, M or N above 2^30, K above 131,071 (the
 * sums would leave int32), E outside [1, 4096], E != 1 without offsets, ldx < K, ldy < M, bad
 * dtype), SEEDMM_EALIGN (a pointer not aligned to its type), SEEDMM_EHIP.  M = 0 or N = 0 is an
 * empty success; with K = 0 the sums are 0 (weight and x may be NULL).
 */
int seedmm_i8_gemv(const int8_t *weight, const void *scales, int s_dtype, int E,
                   const int32_t *offsets, const int8_t *x, int64_t ldx, const float *x_scale,
                   void *y, int y_dtype, int64_t ldy, int M, int K, int N, void *hip_stream);

/*
 * seedmm_moe_sort -- the rows of a routed batch in the order of their experts (the grouping
 * of seedmm_moe_dispatch as rows in memory).  Pair p = t*top_k + s is token t's slot s:
 *     the pairs with topk_ids[p] in [0, E) are ordered by (topk_ids[p], p);
 *     inverse[p] = the pair's place in that order, or -1 for any other id;
 *     offsets[e] = number of pairs with an id in [0, e), e = 0 .. E;
 *     rows[inverse[p]] = x[t],  row_scale[inverse[p]] = x_scale[t].
 *   topk_ids: int32[T][top_k]; an id outside of [0, E) drops its slot (an expert of another
 *   device, a padding token); a token may name an expert twice.
 *   x: [T][ldx] of x_dtype (SEEDMM_F32, SEEDMM_BF16 or SEEDMM_I8);  x_scale: fp32[T] or NULL;
 *   rows: [T*top_k][ldr] of x_dtype; rows from offsets[E] on and columns H .. ldr - 1 are left
 *   as they were;  row_scale: fp32[T*top_k], given with x_scale;  offsets: int32[E + 1];
 *   inverse: int32[T][top_k].  H = 0 writes the order alone (x and rows may be NULL).
 *   The gradient of rows with respect to x is seedmm_moe_unsort without weights.
 *   workspace: device scratch of seedmm_moe_sort_workspace_bytes(T, top_k, E) bytes, 16-byte
 *   aligned, contents need not be initialised; NULL where that is 0 (small batches).  Calls
 *   that overlap in time use different ones.
 * Errors: SEEDMM_EINVAL (null pointer, T or H < 0, H above 2^30, top_k outside [1, 64], T*top_k
 * >= 2^31, E outside [1, 4096], ldx or ldr < H, bad dtype, one scale without the other),
 * SEEDMM_EALIGN (a pointer not aligned to its type, the workspace not 16-byte aligned),
 * SEEDMM_EWORKSPACE, SEEDMM_EHIP.  T = 0 writes offsets of 0.
 */
int seedmm_moe_sort(const int32_t *topk_ids, int T, int top_k, int E, const void *x, int x_dtype,
                    int64_t ldx, const float *x_scale, void *rows, int64_t ldr, float *row_scale,
                    int H, int32_t *offsets, int32_t *inverse, void *workspace,
                    size_t workspace_bytes, void *hip_stream);
size_t seedmm_moe_sort_workspace_bytes(int T, int top_k, int E);

/*
 * seedmm_moe_unsort -- sorted rows back to their tokens, weighted and summed:
 *     y[t] = sum_s topk_w[t][s] * rows[inverse[t][s]]   over the slots with a row
 *   rows: [n_rows][ldr] of r_dtype (SEEDMM_F32 or SEEDMM_BF16);  inverse: int32[T][top_k] of
 *   seedmm_moe_sort; a value outside of [0, n_rows) is a slot without a row: neither a row nor
 *   its weight enters;  topk_w: fp32[T][top_k], or NULL (ones: the gradient of seedmm_moe_sort);
 *   y: [T][ldy] of y_dtype (SEEDMM_F32 or SEEDMM_BF16), overwritten (0 for a token without
 *   rows); columns H .. ldy - 1 are left as they were.
 *   Summed in fp32 in slot order, rounded once.
 * seedmm_moe_unsort_grad -- its gradients for dy = d loss / d y (what a routed expert's row and
 * its weight mean to a loss; the experts that matter most are the ones to keep in more bits):
 *     drows[inverse[t][s]] = topk_w[t][s] * dy[t];   dw[t][s] = sum_h dy[t][h] rows[inverse[t][s]][h]
 *   dy: [T][ldd] fp32 or bf16;  drows: [n_rows][ldg] of r_dtype, or NULL; rows that no slot
 *   names are left as they were;  dw: fp32[T][top_k], 0 for slots without a row, or NULL (rows
 *   may then be NULL).  Sums in fp32 in a fixed order; no atomics.  The inverse names each row
 *   at most once.  drows may be rows itself with ldg = ldr; outputs overlap inputs in no other
 *   way.
 * Errors: SEEDMM_EINVAL (null pointer, T, H or n_rows < 0, H above 2^30, top_k outside [1, 64],
 * T*top_k >= 2^31, a leading dimension < H, bad dtype, rows as drows with another ld),
 * SEEDMM_EALIGN (a pointer not aligned to its type), SEEDMM_EHIP.  T = 0 is an empty success,
 * and so is H = 0 but for dw, which is then 0.
 */
int seedmm_moe_unsort(const void *rows, int r_dtype, int64_t ldr, int n_rows,
                      const int32_t *inverse, const float *topk_w, void *y, int y_dtype,
                      int64_t ldy, int T, int top_k, int H, void *hip_stream);
int seedmm_moe_unsort_grad(const void *dy, int dy_dtype, int64_t ldd, const void *rows, int r_dtype,
                           int64_t ldr, int n_rows, const int32_t *inverse, const float *topk_w,
                           void *drows, int64_t ldg, float *dw, int T, int top_k, int H,
                           void *hip_stream);

/*
 * seedmm_swiglu -- h = silu(gate) * up of the rows of a gate-and-up product (the SwiGLU of
 * seedmm_moe as an operator of its own), in a float type or as rows for the next product:
 *     h[n][i] = g / (1 + exp(-g)) * u,  g = gate_up[n][i],  u = gate_up[n][I + i]
 *   gate_up: [N][ldg] of g_dtype (SEEDMM_F32 or SEEDMM_BF16), ldg >= 2 I;
 *   out: [N][ldo] of out_dtype.  SEEDMM_F32, SEEDMM_BF16: h, computed in fp32, rounded once.
 *   (Below g = -87 exp(g) is no normal fp32 number: h is off by up to 2^-149 (4 + |g|)(1 + |u|) more,
 *   which a u of 1e30 makes visible; g = -infinity gives NaN, as the formula does.)
 *   SEEDMM_I8: codes round(h / scale[n]) in [-127, 127] with scale[n] = max_i |h| / 127 (at
 *   least 2^-126); a row that holds an infinity or NaN gets scale NaN and codes 0 (as
 *   seedmm_add_norm's).  scale: fp32[N] with SEEDMM_I8, NULL otherwise.
 *   count: NULL, or device int32[1]: only the first count[0] rows exist (the offsets[E] of
 *   seedmm_moe_sort); rows and scales behind are left as they were and not read.
 * Errors: SEEDMM_EINVAL (null pointer, N or I < 0, I above 2^29, ldg < 2 I, ldo < I, bad dtype,
 * scale missing or given without SEEDMM_I8), SEEDMM_EALIGN (a pointer not aligned to its type),
 * SEEDMM_EHIP.  N = 0 or I = 0 is an empty success.
 */
int seedmm_swiglu(const void *gate_up, int g_dtype, int64_t ldg, void *out, int out_dtype,
                  int64_t ldo, float *scale, const int32_t *count, int N, int I, void *hip_stream);

/*
 * seedmm_moe_i8 -- one routed layer of SwiGLU experts in 8-bit integers:
 *     y[t] = sum_s topk_w[t][s] * down_e h,  h = i8( silu(gate_e x[t]) * (up_e x[t]) ),
 *     e = topk_ids[t][s]
 *   by seedmm_moe_sort, seedmm_i8_gemv (gate and up at once, bf16 rows), seedmm_swiglu (8-bit
 *   rows), seedmm_i8_gemv (bf16 rows) and seedmm_moe_unsort, with their results: an id outside
 *   of [0, E) drops its slot, a token without slots gets 0.  The rows between are bf16, each
 *   value off by 2^-8 of itself at most, sums are fp32.  What gate and up give is rounded to 8 bits
 *   next, by up to 1/254 of a row's largest; the down product's rows carry that error, some 2% of their
 *   length, and bf16 adds 0.1 to 0.2% to it: against 64 bits the layer is off by 2.041% of y, by
 *   2.034% with fp32 rows behind the down product (64 tokens, 8 of 100 experts of 2048 x 1024),
 *   which take 495 us for 439 at 4096 tokens.  A caller who wants them makes the five calls, with
 *   y_dtype SEEDMM_F32 for the second product.
 *   x: int8 [T][H] with x_scale fp32[T] (seedmm_add_norm writes them);  gate_up: E matrices
 *   [2 I][H], gate rows 0 .. I - 1, up rows I .. 2 I - 1;  down: E matrices [H][I];
 *   y: fp32 [T][H], overwritten: seedmm_add_norm's delta.
 *   workspace: device scratch of seedmm_moe_i8_workspace_bytes(T, top_k, E, H, I) bytes, 16-byte
 *   aligned; overlapping calls use different ones.
 * Errors: those of the calls, before anything runs (but for SEEDMM_EHIP), SEEDMM_EINVAL also for
 * H or I < 1 or above 131,071 and T*top_k above 2^30, SEEDMM_EWORKSPACE, SEEDMM_EALIGN (the
 * workspace not 16-byte aligned).
 */
typedef struct seedmm_i8mat {
    const int8_t *weight;   /* [E][M][K]                    */
    const void *scales;     /* [E][M]                       */
    int s_dtype;            /* SEEDMM_F32 or SEEDMM_BF16    */
} seedmm_i8mat;

size_t seedmm_moe_i8_workspace_bytes(int T, int top_k, int E, int H, int I);
int seedmm_moe_i8(const int32_t *topk_ids, const float *topk_w, int T, int top_k, const int8_t *x,
                  const float *x_scale, float *y, int E, int H, int I, seedmm_i8mat gate_up,
                  seedmm_i8mat down, void *workspace, size_t workspace_bytes, void *hip_stream);

/* Static description of a status code (the C engine's error convention: a plain C99
 * interface, NanoSeedLM README "How it works"). */
const char *seedmm_strerror(int status);

/* Library ABI version (major * 100 + minor); 200 = caller-owned side streams and
 * encoder tables. */
int seedmm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SEEDMM_H */
