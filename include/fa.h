/*
 * fa.h -- C ABI of the GB300 (sm_103a) exact-attention library (libfa.so).
 *
 * Operation.  Per (b,h) head, with Q, K, V, O of shape [L, D]:
 *     S = scale * Q K^T   (S_ij = -inf for j > i when causal)
 *     P = softmax(S) row by row,  O = P V,  LSE_i = log(sum_j exp(S_ij))
 * computed the tiled, streaming way: Q in 128-row tiles kept on chip, K/V streamed in 128-key
 * tiles, a running row max and row sum with the partial output rescaled as tiles arrive, and
 * only O and the per-row log-sum-exp written ("FlashAttention data-flow optimisation: MI50
 * memory and bandwidth bottlenecks", section 2.2, first and second layers;
 * "FlashAttention principles and engineering practice", section 2.1 for the plain
 * definition attn = softmax(q k^T * scale) v).  The backward pass recomputes P from the saved
 * LSE instead of storing the L x L matrix (data-flow page, section 2.2, third layer).
 *
 * Conventions shared by every entry point:
 *  - Tensors are DEVICE pointers to row-major [B, H, L, D] arrays (LSE: [B, H, L] fp32), each
 *    16-byte aligned: contiguous for fa_fwd / fa_bwd, strided (fa_strides) for fa_fwd_ex /
 *    fa_bwd_ex.  q, k, v, o, dO, dq, dk, dv all have the dtype `dtype`.
 *  - Supported: D in {64, 128}; B, H, L >= 0 (an empty problem returns FA_OK and launches
 *    nothing); causal in {0, 1} (query i sees key j iff j <= i); scale finite, of either sign
 *    or zero ("FlashAttention principles and engineering practice", section 2.1: the scale
 *    multiplies q k^T before the softmax), with scale * (q . k) inside the fp32 range.
 *  - The caller allocates and owns every buffer, including the backward workspace; the
 *    library never allocates or frees device memory in these calls.  The one exception is
 *    fa_bwd_noalloc's fixed scratch array, which is compiled into the library.
 *  - Calls are asynchronous: they validate, enqueue on `stream` (a cudaStream_t; NULL is the
 *    legacy default stream) and return without synchronising.  Argument errors are reported
 *    before anything is enqueued and leave every output untouched.  A non-OK status from a
 *    launch leaves outputs undefined.  Kernels never spin without bound: a wait that exceeds
 *    its time limit records FA_ERR_TIMEOUT in a device status word, read by
 *    fa_get_device_status().
 *  - Outputs must not overlap inputs.  fa_bwd overwrites dq, dk, dv (it does not accumulate).
 *  - The library keeps no per-call state.  It caches the driver entry point used to build TMA
 *    descriptors and, per device index, the address of its status word, the address of
 *    fa_bwd_noalloc's scratch array and the SM count.  Those addresses belong to the device's
 *    primary context: after cudaDeviceReset (or anything else that destroys that context) the
 *    cached addresses are stale, so do not call into the library on that device again in the
 *    same process.
 */
#ifndef FA_H
#define FA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FA_OK = 0,
    FA_ERR_INVALID_ARG = 1, /* null/misaligned/overlapping pointer, bad size, bad flag */
    FA_ERR_UNSUPPORTED = 2, /* valid request outside what the kernels implement (e.g. D) */
    FA_ERR_CUDA = 3,        /* a CUDA runtime/driver call or a launch failed */
    FA_ERR_TIMEOUT = 4      /* a device-side bounded wait ran out (see fa_get_device_status) */
} fa_status;

typedef enum { FA_BF16 = 0, FA_FP16 = 1 } fa_dtype;

/*
 * Element strides of one [B, H, L, D] operand whose D elements are contiguous.  The layouts of
 * the flash_attn_func interface ("FlashAttention data-flow optimisation", section 4.1, step 3:
 * [B, L, H, D]) and of flash_attn_qkvpacked_func ("AIInfra notes 01: from TFLOPS to
 * FlashAttention", sections 4.2-4.3: [B, L, 3, H, D]) are both of this form:
 *     contiguous [B,H,L,D]:   {H*L*D, L*D,  D}
 *     [B,L,H,D]:              {L*H*D, D,    H*D}
 *     q/k/v of [B,L,3,H,D]:   {3*L*H*D, D,  3*H*D}, bases at +0, +H*D, +2*H*D elements.
 * Every stride is a positive multiple of 8 elements (16 bytes: the tensor-copy unit's rule) and
 * below 2^39; a stride of 0 is accepted for a dimension of size 1.
 */
typedef struct {
    int64_t batch, head, row;
} fa_strides;

/*
 * Forward.  Writes o [B,H,L,D] (dtype) and lse [B,H,L] (fp32, natural log).
 * Data-flow page, section 2.2 (tiling, streaming softmax, statistics kept for backward).
 */
fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                 int L, int D, float scale, int causal, int dtype, void* stream);

/*
 * Forward with general layouts and lengths: q [B,H,Lq,D], k and v [B,H,Lk,D], o [B,H,Lq,D], each
 * addressed through its own strides (strides[0..3] = q, k, v, o); lse is contiguous [B,H,Lq].
 * Lq may differ from Lk.  Under the causal mask the queries are the last Lq positions of the
 * key sequence (a block of new tokens after Lk - Lq earlier ones): query i sees key j iff
 * j <= i + Lk - Lq.  A query row that sees no key (only when Lq > Lk) gets O = 0 and
 * LSE = -inf.  Lq = 0 returns FA_OK with nothing to do; Lk = 0 with Lq > 0 returns
 * FA_ERR_UNSUPPORTED.  Extents (first to last element) of the outputs must not overlap those of
 * the inputs or each other.  fa_fwd(..., L, ...) is fa_fwd_ex with Lq = Lk = L, contiguous
 * strides and no dropout.
 *
 * Dropout on P (flash_attn_func's dropout_p, data-flow page, section 4.1, step 3):
 * dropout_p in [0, 1) (NaN or outside: FA_ERR_INVALID_ARG); 0 runs the kernels without
 * dropout.  O = (P o Z) V with Z_ij = 0 for a dropped entry and 1 / (1 - dropout_p) for a kept
 * one; LSE stays that of P itself.  Entry (i, j) of head bh = b * H + h (query row i, key j) is
 * kept iff word j % 4 of the Philox-4x32-10 block (Salmon et al., "Parallel random numbers: as
 * easy as 1, 2, 3", SC 2011) at counter (j / 4, i, bh, 0) under key (seed & 0xffffffff,
 * seed >> 32) is at least floor(dropout_p * 2^32).  The pages fix no generator; this one is
 * counter-based, so the backward regenerates the mask from (dropout_p, seed) instead of storing
 * it.
 */
fa_status fa_fwd_ex(const void* q, const void* k, const void* v, void* o, float* lse,
                    const fa_strides* strides, int B, int H, int Lq, int Lk, int D, float scale,
                    int causal, double dropout_p, uint64_t seed, int dtype, void* stream);

/*
 * Bytes of device workspace fa_bwd needs for this shape: two fp32 vectors per head padded to
 * a whole number of 128-row tiles (-LSE * log2(e) and Delta = rowsum(dO * O)), then 16 bytes
 * of work counters for the persistent passes.  Returns 0 for an empty problem or invalid sizes.
 * The pages have no such call: they keep the row maximum and the sum of exponentials for the
 * backward (data-flow page, section 2.2, third layer) without saying where the per-row
 * vectors the backward derives from them live.  Here the caller owns that memory, so the
 * library reports how much it needs.
 */
size_t fa_bwd_workspace_bytes(int B, int H, int L, int D);

/*
 * Bytes of device workspace fa_bwd_ex needs for q of [B, H, Lq, D] and the given
 * `deterministic` flag (0 or 1; else 0 is returned): with deterministic = 0 at D = 64 the
 * backward reduces dQ into an fp32 accumulator [B*H, Lqpad, D] kept in the workspace after the
 * two per-row vectors (Lqpad = Lq rounded up to a multiple of 128; the work counters follow
 * it).  A workspace of this size
 * also serves the same shape with dropout (which always takes the deterministic path).
 * fa_bwd_workspace_bytes(B, H, L, D) = fa_bwd_workspace_bytes_ex(B, H, L, D, 1).
 * Pages: silent (as for fa_bwd_workspace_bytes).
 */
size_t fa_bwd_workspace_bytes_ex(int B, int H, int Lq, int D, int deterministic);

/*
 * Backward.  Given q, k, v, the forward's o and lse, and the output gradient dout, writes
 * dq, dk, dv [B,H,L,D] (dtype).  `workspace` is a device buffer of at least
 * fa_bwd_workspace_bytes(B,H,L,D) bytes, 16-byte aligned, owned by the caller; its contents
 * on entry do not matter.  Three kernels are enqueued on `stream`: the Delta/LSE preprocess,
 * the dK/dV pass (one CTA per key tile, or, when key tiles are seen by at most 32 query tiles
 * on average, one persistent CTA per SM) and the dQ pass (likewise per query tile, persistent
 * when query tiles see at most 32 key tiles on average); persistent CTAs take the next tile of
 * a heaviest-first order from a counter in the workspace whenever they are ready for one.  The
 * results are the same either way.
 * Data-flow page, section 2.2, third layer (recompute P from the saved statistics).
 */
fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout,
                 const float* lse, void* dq, void* dk, void* dv, void* workspace,
                 size_t workspace_bytes, int B, int H, int L, int D, float scale, int causal,
                 int dtype, void* stream);

/*
 * Backward with general layouts and lengths (see fa_fwd_ex): strides[0..7] = q, k, v, o, dout,
 * dq, dk, dv; dq has the shape of q, dk and dv that of k.  The workspace is
 * fa_bwd_workspace_bytes(B, H, Lq, D).  Rows that see no key get dQ = 0.  Lq = Lk = 0 returns
 * FA_OK; only one of them 0 returns FA_ERR_UNSUPPORTED.  dq, dk and dv may be the three
 * interleaved parts of one packed [B,L,3,H,D] gradient (Lq = Lk, equal strides, the heads of a
 * row together, each part's heads ending before the next part's begin); otherwise no two
 * outputs' extents may overlap, and no output may overlap an input.  fa_bwd is fa_bwd_ex with
 * Lq = Lk = L, contiguous strides, no dropout and deterministic = 1.  dropout_p and seed must
 * be those of the forward that produced o and lse (the same mask is regenerated):
 * dV = (P o Z)^T dO and dS = P o ((dO V^T) o Z - Delta), Delta = rowsum(dO o O); the backward
 * under dropout always runs one CTA per tile.
 *
 * deterministic (0 or 1, else FA_ERR_INVALID_ARG): 1 computes dQ in its own pass, one CTA (or
 * persistent CTA) per query tile summing its key tiles in a fixed order, so every call gives
 * the same bits.  0 allows dQ to be computed inside the dK/dV pass ("dQ by atomics or a
 * separate pass", the method's two options): at D = 64 without dropout each (key tile, query
 * tile) pair adds its dS K into an fp32 accumulator in the workspace with vector reductions
 * (additions in arrival order: the result may differ in the last bits between calls) and a
 * third kernel converts it to dq; elsewhere 0 takes the deterministic path.  The workspace is
 * then fa_bwd_workspace_bytes_ex(B, H, Lq, D, 0) bytes.
 */
fa_status fa_bwd_ex(const void* q, const void* k, const void* v, const void* o, const void* dout,
                    const float* lse, void* dq, void* dk, void* dv, void* workspace,
                    size_t workspace_bytes, const fa_strides* strides, int B, int H, int Lq,
                    int Lk, int D, float scale, int causal, double dropout_p, uint64_t seed,
                    int deterministic, int dtype, void* stream);

/* Size of the fixed device scratch array behind fa_bwd_noalloc: 16 MiB for the per-row
 * vectors and 256 bytes for the work counters. */
#define FA_BWD_NOALLOC_SCRATCH_BYTES (((size_t)16 << 20) + 256)

/*
 * Backward for callers that cannot allocate device memory.  The pages describe no such entry
 * point; it has no counterpart in the method and exists only for callers that must not call
 * cudaMalloc themselves (for example a plugin whose host framework owns all device memory and
 * passes it only inputs and outputs, or a running latency-critical loop where an allocation
 * could synchronise the device at an unbounded cost).
 *
 * Same arguments, results and checks as fa_bwd, minus the workspace: the scratch fa_bwd would
 * take from `workspace` comes from a file-scope device array of FA_BWD_NOALLOC_SCRATCH_BYTES
 * compiled into the library, which every GPU that loads the library's code holds until the
 * process exits.  The limit: fa_bwd_workspace_bytes(B,H,L,D) = 8*B*H*ceil(L/128)*128 + 16
 * bytes must not exceed FA_BWD_NOALLOC_SCRATCH_BYTES (B*H*ceil(L/128)*128 <= 2^21 rows, e.g.
 * B*H = 256 heads at L = 8192); larger problems return FA_ERR_UNSUPPORTED before anything is
 * enqueued.  The call allocates nothing (no cudaMalloc, cudaFree or allocating library call).
 *
 * The first call on each device looks up the array's device address (cudaGetSymbolAddress,
 * with that device current); make that first call before any stream capture.  Every call on
 * a device shares the one array, so calls whose kernels overlap on the GPU (on different
 * streams, or from different threads) race on it and give undefined results: serialise them.
 * Nothing in the array needs clearing between calls; each call's first kernel overwrites
 * everything its later kernels read.  Checks run in fa_bwd's order (sizes and flags, then null
 * pointers), then the scratch limit, then fa_bwd's remaining checks; every outcome consumes a
 * trace arming made with fa_trace_next_call.
 */
fa_status fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o,
                         const void* dout, const float* lse, void* dq, void* dk, void* dv, int B,
                         int H, int L, int D, float scale, int causal, int dtype, void* stream);

/* Tokens per page of the paged key/value cache of fa_decode_paged. */
#define FA_PAGE_TOKENS 16

/*
 * Bytes of device workspace fa_decode_paged needs for this shape: 0 when every (sequence, head)
 * pair is one CTA, else room for the per-split partial results (fp32).  0 for invalid sizes.
 */
size_t fa_decode_workspace_bytes(int B, int H, int D, int max_pages);

/*
 * One decode step over a paged key/value cache ("FlashAttention principles and engineering
 * practice", section 4.2: serving with PagedAttention, block_size 16, continuous batching).
 * Sequence b adds one token; its query rows q[b, h, :] attend to all seq_lens[b] tokens cached
 * for it (the new token's key and value already written to the cache by the caller):
 *     O[b,h] = softmax(scale * q[b,h] K_bh^T) V_bh,   LSE[b,h] = log sum_t exp(scale q.k_t),
 * with token t of sequence b in physical page block_tables[b*max_pages + t/16], slot t % 16.
 *   q, o:             [B, H, D] 16-bit (dtype), contiguous, 16-byte aligned;
 *   k_cache, v_cache: [num_pages, H, FA_PAGE_TOKENS, D] 16-bit, contiguous, 16-byte aligned
 *                     (the 16 tokens of one head in one page are contiguous);
 *   block_tables:     [B, max_pages] int32, device; entries past a sequence's pages are unread;
 *   seq_lens:         [B] int32, device, 0 <= seq_lens[b] <= 16 * max_pages;
 *   lse:              [B, H] fp32; workspace: fa_decode_workspace_bytes(B, H, D, max_pages).
 * A sequence with no cached token gets O = 0 and LSE = -inf.  Slots past a sequence's end may hold
 * anything.  A row with a NaN score gets NaN in O and LSE.  Host-side argument errors return
 * before anything is enqueued; a page index outside [0, num_pages) or a length outside its range
 * (device data, checked by the kernel before any copy) is skipped and reported by
 * fa_get_device_status() as FA_ERR_INVALID_ARG, with the outputs of that call undefined.
 */
fa_status fa_decode_paged(const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* block_tables, const int32_t* seq_lens, void* o,
                          float* lse, void* workspace, size_t workspace_bytes, int B, int H, int D,
                          int num_pages, int max_pages, float scale, int dtype, void* stream);

/*
 * Rotary positions.  The pages attend to queries and keys as given; a model that marks positions
 * by rotation turns them first.  In row l of sequence b, at position m, every pair (x1, x2) of
 * the first rotary_dim elements of a head becomes
 *     y1 = mscale * (x1 cos(m theta_i) - x2 sin(m theta_i)),
 *     y2 = mscale * (x2 cos(m theta_i) + x1 sin(m theta_i)),      i = 0 .. rotary_dim/2 - 1,
 * the pairs being elements (i, i + rotary_dim/2), or (2i, 2i+1) with interleaved = 1; elements
 * past rotary_dim are copied.  Computed in fp32 and rounded once.  inverse = 1 turns by the
 * negative angle: the gradient of the inputs from the gradient of the outputs.
 *   q, q_out: [B, Hq, L, D], k, k_out: [B, Hk, L, D] views (strides[0..3] = q, k, q_out, k_out;
 *             Hk = 0 or Hq = 0: that operand is absent and its pointers are ignored);
 *             D in {64, 128}; an output may be its own input (same pointer and strides), or
 *             interleave with another operand as a part of one packed tensor (of equal strides,
 *             the parts at any place among its dimensions); no other overlap;
 *   positions: [B, L] int32, device, rows position_stride elements apart (0: one row for all
 *             sequences; negative positions turn backwards), or null: position l;
 *   freqs:    [rotary_dim / 2] int64, device: theta_i as a fraction of a turn, theta_i / (2 pi)
 *             * 2^64, as fa_rotary_freqs makes it (angles are reduced exactly at any position);
 *   rotary_dim: even, 2 .. D.  B * L < 2^31.
 */
fa_status fa_rotary(const void* q, const void* k, void* q_out, void* k_out,
                    const fa_strides* strides, const int32_t* positions, int64_t position_stride,
                    const int64_t* freqs, int rotary_dim, float mscale, int interleaved,
                    int inverse, int B, int Hq, int Hk, int L, int D, int dtype, void* stream);

/*
 * Frequencies for fa_rotary, on the host: fills freqs[0 .. rotary_dim/2) and *mscale.
 *   FA_ROTARY_PLAIN   theta_i = base^(-2i / rotary_dim)
 *   FA_ROTARY_LINEAR  theta_i / factor (positions interpolated)
 *   FA_ROTARY_NTK     base * factor^(rotary_dim / (rotary_dim - 2)) in the place of base: the
 *                     highest frequency stays, the lowest is divided by factor
 *   FA_ROTARY_YARN    by parts (Peng et al., "YaRN", 2023): a frequency that turns 32 times or more
 *                     within original_len positions stays, one that turns once or less is divided
 *                     by factor, a linear ramp between; mscale = 0.1 ln(factor) + 1
 * mscale is 1 otherwise.  base >= 1, factor >= 1; original_len > 0 (YaRN only).
 */
typedef enum {
    FA_ROTARY_PLAIN = 0,
    FA_ROTARY_LINEAR = 1,
    FA_ROTARY_NTK = 2,
    FA_ROTARY_YARN = 3
} fa_rotary_scaling;
fa_status fa_rotary_freqs(int rotary_dim, double base, int scaling, double factor,
                          double original_len, int64_t* freqs, float* mscale);

/*
 * What a paged cache holds.  FA_CACHE_16BIT: rows of the call's dtype, as fa_decode_paged reads
 * them.  FA_CACHE_E4M3: a row x of D values as D e4m3 bytes, e4m3(x_i * 2^-e), and one byte e + 127
 * in k_exp / v_exp, e being the smallest integer in [-127, 127] with max|x| <= 448 * 2^e (values
 * rounded to nearest even; the scaling is exact).  A row with an infinity or a NaN gets the byte
 * 255 and reads back as NaN.
 */
typedef enum { FA_CACHE_16BIT = 0, FA_CACHE_E4M3 = 1 } fa_cache_dtype;

/*
 * Writes new keys and values into a paged cache.  Sequence b adds new_lens[b] rows (rows
 * 0 .. new_lens[b]-1 of k[b], v[b]), which become its last tokens seq_lens[b] - new_lens[b] ..
 * seq_lens[b] - 1; rows of k and v behind them count for nothing, other slots keep what they hold.
 *   k, v:        [B, H, L, D] views of dtype (strides[0..1]);
 *   k_cache, v_cache: [num_pages, H, FA_PAGE_TOKENS, D], k_exp, v_exp: [num_pages, H,
 *                FA_PAGE_TOKENS] bytes (ignored for a 16-bit cache), 16-byte aligned, contiguous;
 *   block_tables [B, max_pages], seq_lens [B], new_lens [B]: int32, device.  new_lens null: every
 *                sequence adds L rows, one of length 0 (an unused place of the batch) none;
 *   rotary_dim > 0 rotates each key by its token index (fa_rotary's freqs, mscale, interleaved)
 *                in fp32 before it is rounded or quantised; 0 writes the keys as they are.
 * A token must have one owner: pages that two sequences of the batch share may be read by both,
 * but not written in one call.  A bad length or page index (device data) is reported by
 * fa_get_device_status() as FA_ERR_INVALID_ARG; the sequence's rows with it are not written.
 */
fa_status fa_cache_append(const void* k, const void* v, const fa_strides* strides, void* k_cache,
                          void* v_cache, void* k_exp, void* v_exp, const int32_t* block_tables,
                          const int32_t* seq_lens, const int32_t* new_lens, const int64_t* freqs,
                          int rotary_dim, float mscale, int interleaved, int B, int H, int L, int D,
                          int num_pages, int max_pages, int dtype, int cache_dtype, void* stream);

/*
 * Reads a paged cache back: rows 0 .. L-1 of every sequence as dense k, v [B, H, L, D] views of
 * dtype (strides[0..1]); rows at or past seq_lens[b] are written as zeros.  An e4m3 row is
 * its values times 2^e, rounded to dtype (exact in bf16, but for a value that quantising rounded up
 * to 2^128).  k and v may be parts of one packed tensor, as in fa_rotary.  For a prompt that continues behind
 * cached tokens: the dense rows are the keys and values of fa_fwd_ex with Lk > Lq.  Bad device data
 * is reported as for fa_cache_append; those rows are written as zeros.
 */
fa_status fa_cache_read(const void* k_cache, const void* v_cache, const void* k_exp,
                        const void* v_exp, const int32_t* block_tables, const int32_t* seq_lens,
                        void* k, void* v, const fa_strides* strides, int B, int H, int L, int D,
                        int num_pages, int max_pages, int dtype, int cache_dtype, void* stream);

/* Bytes of device workspace fa_decode_paged_ex needs (the parts of rows whose pages are
 * split, fp32: at D = 128 at most 2.5 MB, from 2048 (sequence, cache head) pairs on 7.5 MB, for every
 * query head of a group up to 16).  Calls that may
 * overlap on the GPU need a workspace each.  0 for invalid sizes. */
size_t fa_decode_workspace_bytes_ex(int B, int Hq, int Hk, int D, int max_pages);

/*
 * fa_decode_paged with grouped heads and either kind of cache: q, o [B, Hq, D] and lse [B, Hq],
 * caches [num_pages, Hk, FA_PAGE_TOKENS, D] of dtype (FA_CACHE_16BIT) or e4m3 bytes with k_exp, v_exp
 * [num_pages, Hk, FA_PAGE_TOKENS] (FA_CACHE_E4M3; ignored otherwise).  Hq is a multiple of Hk and
 * query head h reads cache head h / (Hq / Hk).  Everything else is as for fa_decode_paged: empty
 * sequences get O = 0, LSE = -inf, slots past a sequence's end may hold anything, a bad length or
 * page index is reported by fa_get_device_status().  Enqueues one kernel for a short step (few
 * sequences and cache heads, tables of up to 256 pages, groups of up to 8), else two for every 1024
 * sequences (the second may start before the first has finished).  B * max_pages, B * Hq and num_pages * Hk
 * are below 2^31.
 */
fa_status fa_decode_paged_ex(const void* q, const void* k_cache, const void* v_cache,
                             const void* k_exp, const void* v_exp, const int32_t* block_tables,
                             const int32_t* seq_lens, void* o, float* lse, void* workspace,
                             size_t workspace_bytes, int B, int Hq, int Hk, int D, int num_pages,
                             int max_pages, float scale, int dtype, int cache_dtype, void* stream);

/* Bytes of device workspace fa_decode_shared_prefix needs: fa_decode_paged_ex's and fp32 parts of
 * every query row.  0 for invalid sizes. */
size_t fa_shared_prefix_workspace_bytes(int B, int Hq, int Hk, int D, int prefix_len,
                                        int max_pages);

/*
 * One decode step of a batch whose sequences all begin with the same prefix_len tokens (a system
 * prompt, a document), which lie once in the cache: token t of the prefix in page
 * prefix_table[t / 16] at slot t % 16, and sequence b's own seq_lens[b] tokens behind it in the pages
 * of block_tables[b], from that table's first slot on (a prefix that ends inside a page leaves the
 * rest of that page unused).  O[b,h] and LSE[b,h] are those of fa_decode_paged_ex over the prefix's
 * tokens followed by the sequence's own.  The prefix is read once per cache head for all B * Hq / Hk
 * query rows of it (tensor-core kernel), the own tokens as by fa_decode_paged_ex, and a third
 * kernel joins the parts.
 *   caches of dtype (16-bit), Hq a multiple of Hk with Hq / Hk <= 128; prefix_len >= 0 (a host
 *   integer; 0: no prefix), prefix_table int32, device, ceil(prefix_len / 16) entries; max_pages 0:
 *   no sequence has tokens of its own.  A row with no token at all gets O = 0, LSE = -inf.
 * Bad page indexes and lengths are reported as for fa_decode_paged_ex.  Enqueues three kernels (without
 * a prefix those of fa_decode_paged_ex; two more for every further 1024 sequences); each may start before the one in
 * front has finished.
 */
fa_status fa_decode_shared_prefix(const void* q, const void* k_cache, const void* v_cache,
                                  const int32_t* prefix_table, int prefix_len,
                                  const int32_t* block_tables, const int32_t* seq_lens, void* o,
                                  float* lse, void* workspace, size_t workspace_bytes, int B, int Hq,
                                  int Hk, int D, int num_pages, int max_pages, float scale,
                                  int dtype, void* stream);

/*
 * Synchronises `stream`, then reads and clears the current device's status word.  Returns
 * FA_OK, FA_ERR_TIMEOUT if a kernel gave up on a bounded wait since the last call,
 * FA_ERR_INVALID_ARG if a decode kernel found a page index or sequence length out of range, or
 * FA_ERR_CUDA if synchronisation itself failed or a kernel refused to run (its dynamic shared
 * memory was not 1024-byte aligned; it then wrote nothing).
 * The pages are silent on failure detection; this call is the library's own way of making a
 * stalled kernel visible without faulting the GPU (every device-side wait is bounded).
 */
fa_status fa_get_device_status(void* stream);

/*
 * Selects the forward kernel at D = 128 without dropout: mode 1 runs it on CTA pairs (one
 * tensor-core contraction of 256 query rows over two SMs, tcgen05 cta_group::2, each CTA
 * loading half of every K and V tile), mode 0 (the default) on single CTAs.  The two give the
 * same results up to the order of nothing: every row's arithmetic is the same, so O and LSE are
 * bit for bit equal.  Process-wide; other head sizes and dropout always use single CTAs.
 * FA_ERR_INVALID_ARG for other modes.  The pages have no counterpart (TFLOPS page, sections
 * 3.2-3.3 size tiles for one SM).
 */
fa_status fa_set_forward_pair(int mode);

/* Time limit of every device-side wait, in nanoseconds (default 4e9).  0 restores the
 * default.  Applies to launches made after the call; returns FA_OK. */
fa_status fa_set_wait_timeout_ns(uint64_t timeout_ns);

/*
 * Self-test of the bounded-wait machinery: enqueues one tiny kernel that waits on a barrier
 * nothing will ever complete, with the given limit.  The kernel gives up, records
 * FA_ERR_TIMEOUT in the status word and returns, so the following fa_get_device_status()
 * reports FA_ERR_TIMEOUT and the context stays usable.
 */
fa_status fa_selftest_wait_timeout(uint64_t timeout_ns, void* stream);

/*
 * Kernel timing trace (the CUDA-event measurement the TFLOP/s figures rest on, per kernel).
 * Arms the next forward or backward call made by this host thread: the i-th kernel that call
 * enqueues is bracketed by cudaEventRecord(events[2*i], stream) and
 * cudaEventRecord(events[2*i+1], stream).  `events` holds n_pairs pairs of cudaEvent_t created
 * by the caller (with timing enabled); kernels beyond n_pairs are not traced.  The next call
 * consumes the arming.  A forward enqueues 1 kernel (2 under the causal mask with Lq > Lk: the
 * second writes the rows that see no key), a backward 3 (preprocess, dK/dV, dQ).
 */
fa_status fa_trace_next_call(void* const* events, int n_pairs);

/* Number of kernels this library has enqueued in this process so far. */
uint64_t fa_launch_count(void);

/* Static, human-readable name of a status code.  The pages have no counterpart (they
 * define no C interface); it names the fa_status values above. */
const char* fa_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* FA_H */
