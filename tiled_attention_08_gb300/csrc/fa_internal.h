// fa_internal.h -- launch parameters shared between the C-ABI layer and the kernel units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace fa {

// Status codes a kernel records in the device status word (first error wins).
enum DeviceError : int {
    kDevOk = 0,
    kDevBadShared = 3,  // dynamic shared memory not 1024-byte aligned (kernel did nothing)
    kDevTimeout = 4,    // a bounded wait ran out
    kDevBadArg = 5,     // device-side argument out of range (a page index or sequence length)
};

// Tile geometry shared by every kernel: 128 query rows x 128 keys per tile; operands are
// staged in shared memory as 128-row x 64-element boxes with the 128-byte swizzle.
constexpr int kTileRows = 128;
constexpr int kChunkElems = 64;
constexpr int kChunkBytes = kTileRows * kChunkElems * 2;  // 16 KiB per box

// Tile schedule shared by the attention kernels.  Heads are taken in groups of `group`
// (chosen on the host so that a group's streamed operands fit in L2 with room to spare);
// inside a group, tiles go heaviest first across all of the group's heads.  Returns the head
// and the tile's rank by weight (0 = heaviest: the last query tile, or key tile 0, under the
// causal mask).
__host__ __device__ __forceinline__ void tile_coords(int tile_id, int BH, int n_tiles, int group,
                                                     int& bh, int& rank) {
    const int span = group * n_tiles;
    const int g = tile_id / span;
    const int r = tile_id - g * span;
    const int heads = (BH - g * group) < group ? (BH - g * group) : group;
    rank = r / heads;
    bh = g * group + (r - rank * heads);
}

// Element strides of a [B, H, L, D] view whose D elements are contiguous (a row): contiguous
// [B,H,L,D], [B,L,H,D] and the q/k/v parts of a packed [B,L,3,H,D] tensor are all of this form.
struct Strides {
    long long b, h, l;
};

// Byte offset of row `row` of head `bh` (= b*H + h) of a 16-bit tensor with strides `s`.
__host__ __device__ __forceinline__ size_t row_offset(const Strides& s, int bh, int H, int row) {
    const int b = bh / H, h = bh - b * H;
    return (size_t)((long long)b * s.b + (long long)h * s.h + (long long)row * s.l) * 2u;
}

// Dropout on P: entry (bh, i, j) is dropped iff word j % 4 of Philox-4x32-10 at counter
// (j / 4, i, bh, 0) under the key (seed_lo, seed_hi) is below `threshold` = floor(p * 2^32); kept
// entries count 1/(1-p) (`keep_scale`).  threshold = 0: no dropout.
struct Dropout {
    uint32_t threshold, seed_lo, seed_hi;
    float keep_scale;
};

struct FwdParams {
    CUtensorMap tm_q, tm_k, tm_v;  // 16-bit {D, L, H, B} (strided), box {64, 128, 1, 1}
    CUtensorMap tm_k_half;         // K with box {64, 64, 1, 1} (CTA-pair forward only)
    void* o;                       // [B, H, Lq, D] 16-bit, strides so
    Strides so;
    float* lse;                    // [B*H, Lq] natural-log LSE (contiguous)
    int Lq, Lk, H, BH;
    int n_qtiles, n_ktiles;  // ceil(Lq / 128), ceil(Lk / 128)
    int group;          // heads per schedule group (tile_coords)
    float scale_log2;   // |scale| * log2(e)
    uint32_t s_negate;  // kIdescNegateA when scale < 0 (S is computed as -Q K^T), else 0
    Dropout drop;
    int* status;        // device status word
    uint64_t timeout_ns;
};

struct BwdPreParams {
    const void* o;       // [B, H, Lq, D], strides so
    const void* dout;    // [B, H, Lq, D], strides sdo
    void* dq;            // [B, H, Lq, D], strides sdq: rows that see no key are zeroed here
    Strides so, sdo, sdq;
    const float* lse;    // [BH, Lq]
    float* nlse2_pad;    // [BH, Lqpad]: -LSE * log2(e), zero past Lq
    float* delta_pad;    // [BH, Lqpad]: rowsum(dO * O), zero past Lq
    float* dq_acc;       // [BH, Lqpad, D] fp32, zeroed here (dQ by reduction), or null
    int* sched;          // work counters of the persistent passes, zeroed here
    int Lq, Lqpad, H, BH, D;
    int first_seen_row;  // rows below this see no key (causal with Lq > Lk), else 0
    int bf16;
};

// Work counters of the persistent backward passes at the end of the backward workspace.
constexpr int kSchedCounters = 4;
constexpr size_t kSchedBytes = kSchedCounters * sizeof(int);

// Decode over a paged key/value cache: tokens per page.
constexpr int kPageTokens = 16;

struct DecodeParams {
    const void* q;             // [B, H, D] 16-bit: the new token's query rows
    const void* k_cache;       // [num_pages, H, kPageTokens, D] 16-bit
    const void* v_cache;       // [num_pages, H, kPageTokens, D] 16-bit
    const int* block_tables;   // [B, max_pages]: physical page of each sequence's page
    const int* seq_lens;       // [B]: cached tokens per sequence (the new one included)
    void* o;                   // [B, H, D] 16-bit
    float* lse;                // [B, H] natural log
    float* part_o;             // [B*H*splits, D] fp32 (splits > 1)
    float* part_lse;           // [B*H*splits] log2 domain (splits > 1)
    int B, H, num_pages, max_pages, splits, pages_per_split;
    float scale_log2;          // scale * log2(e), either sign
    int* status;
    uint64_t timeout_ns;
};

struct BwdParams {
    CUtensorMap tm_q, tm_k, tm_v, tm_do;  // 16-bit {D, L, H, B} (strided), box {64, 128, 1, 1}
    const void* dout;                     // rows staged into TMEM by the dQ pass
    Strides sdo;
    const float* nlse2_pad;               // [BH, Lqpad]: -LSE * log2(e)
    const float* delta_pad;               // [BH, Lqpad]
    void* dq;                             // [B, H, Lq, D]
    void* dk;                             // [B, H, Lk, D]
    void* dv;                             // [B, H, Lk, D]
    Strides sdq, sdk, sdv;
    int Lq, Lk, Lqpad, H, BH, n_qtiles, n_ktiles;
    int group;          // heads per schedule group (tile_coords)
    float scale;        // softmax scale (applied to dQ and dK)
    float scale_log2;   // scale * log2(e)
    Dropout drop;
    float* dq_acc;      // [BH, Lqpad, D] fp32: dQ by reduction in the dK/dV pass, or null
    int* sched;         // [kSchedCounters] work counters: [0] dK/dV pass, [1] dQ pass
    int* status;
    uint64_t timeout_ns;
};

// Rotary positions (fa_rotary): one operand of the launch, a [B, H, L, D] view.
struct RotaryOperand {
    const void* x;
    void* y;  // may be x itself (same strides)
    Strides sx, sy;
    int H;
};

// The rotation shared by fa_rotary and fa_cache_append.
struct RotaryParams {
    const long long* freqs;  // [rotary_dim / 2] turns per position, fixed point (2^64 = one turn)
    int rotary_dim;          // even; 0: no rotation
    float mscale;            // factor on cos and sin
    int interleaved;         // pairs (2i, 2i+1) instead of (i, i + rotary_dim/2)
};

struct RotaryLaunch {
    RotaryOperand op[2];     // queries, keys (op[1].H = 0 when there is no second operand)
    RotaryParams rot;
    const int* positions;    // [B, L] with batch stride pos_stride, or null: the row index
    long long pos_stride;
    int B, L, D;
    int inverse;             // rotate by the negative angle (the gradient)
    int copy_rest;           // elements past rotary_dim are copied (some output is not in place)
};

// Writing rows into a paged cache (fa_cache_append) and reading them back (fa_cache_read).
struct CacheAppendParams {
    const void *k, *v;        // [B, H, L, D] 16-bit views
    Strides sk, sv;
    void *k_cache, *v_cache;  // [num_pages, H, 16, D] 16-bit, or e4m3 bytes
    uint8_t *k_exp, *v_exp;   // [num_pages, H, 16] biased exponents (e4m3 caches), else null
    const int* block_tables;  // [B, max_pages]
    const int* seq_lens;      // [B] lengths with the new rows
    const int* new_lens;      // [B] rows that each sequence adds, or null: L (0 when empty)
    RotaryParams rot;         // applied to the keys
    int B, H, L, D, num_pages, max_pages;
    int* status;
};

struct CacheReadParams {
    const void *k_cache, *v_cache;
    const uint8_t *k_exp, *v_exp;
    const int* block_tables;
    const int* seq_lens;
    void *k, *v;  // [B, H, L, D] 16-bit views
    Strides sk, sv;
    int B, H, L, D, num_pages, max_pages;
    int* status;
};

// One decode step with grouped heads over a paged cache (fa_decode_gqa.cu).  B is at most
// kGqaMaxSequences (a longer batch takes several launches).
constexpr int kGqaMaxSequences = 1024;

struct GqaParams {
    CUtensorMap tm_k, tm_v;    // {D, 16, num_pages * Hk}: one box is a page's rows of one head
    const void* q;             // [B, Hq, D] 16-bit
    const uint8_t *k_exp, *v_exp;  // [num_pages, Hk, 16] (e4m3 caches)
    const int* block_tables;   // [B, max_pages]
    const int* seq_lens;       // [B]
    void* o;                   // [B, Hq, D] 16-bit
    float* lse;                // [B, Hq] natural log
    int2* unit_parts;          // [B, units of a sequence] written: first warp with its pages, and how many
    float* slot_o;             // [2 * warps * rounds, slot_rows, D] fp32: parts of units that are cut
    float* slot_lse;           // [2 * warps * rounds, slot_rows] log2 domain
    float *full_o, *full_lse;  // [B * Hq, D], [B * Hq]: whole units when parts_only
    int rounds;                // of the split, 1 or 3
    int slot_rows;             // rows of a slot: the group, at most 8 or (above 8) 16
    int parts_only;            // rows have other parts (a shared prefix): o, lse are the merge's
    int short_step;            // a cluster per unit and no merge (gqa_short)
    int early;                 // launched before the kernel in front of it has finished
    int warps;                 // of a round, a multiple of 4
    int B, Hq, Hk, group, q_blocks, num_pages, max_pages;
    float scale_log2;          // scale * log2(e), either sign
    int* status;
    uint64_t timeout_ns;
};

// Joins the parts of the rows of a decode step (fa_decode_gqa.cu).
struct MergeParams {
    const float *prefix_o, *prefix_lse;  // [rows, n_prefix, D], [rows, n_prefix]; LSE = -inf: absent
    int n_prefix;
    const float *slot_o, *slot_lse, *full_o, *full_lse;  // as in GqaParams
    const int2* unit_parts;
    void* o;     // [rows, D] 16-bit
    float* lse;  // [rows] natural log
    int rows, B, Hq, Hk, group, q_rows, q_blocks, slot_rows;
    int workers;  // warps that may have left parts, over all rounds
};

// Attention of all query rows of a batch to one shared prefix (fa_prefix.cu).  A work unit is one
// 128-key tile of one pair of 128-row query tiles of one cache head; CTA c takes the units
// c * units / grid .. of the order (head, pair, key tile), so a pair's key tiles are one part per
// CTA that has any of them.
struct PrefixParams {
    CUtensorMap tm_q;          // {D, Hq, B}, box {64, group, rows_b}
    CUtensorMap tm_k, tm_v;    // {D, 16, num_pages * Hk}, box {64, 16, 1}
    CUtensorMap tm_k_tail, tm_v_tail;  // the same with the last page's rows only
    const int* table;          // [ceil(prefix_len / 16)]
    float* part_o;             // [B*Hq, max_segments, D] fp32
    float* part_lse;           // [B*Hq, max_segments] log2 domain
    int max_segments;
    int prefix_len, num_pages;
    int B, Hq, Hk, group;
    int rows_b;                // sequences per query tile (group * rows_b <= 128 rows)
    int n_tiles, n_pairs, key_tiles;
    int grid;
    float scale_log2;          // |scale| * log2(e)
    uint32_t s_negate;
    int* status;
    uint64_t timeout_ns;
};

// Host-side helpers of the C-ABI layer shared with the other entry-point units.
// Consumes the fa_trace_next_call arming of the calling thread (every public call ends so).
void trace_disarm();
// Number of SMs of the current device (looked up once per device index); 0 if unknown.
int sm_count();
// fa_bwd's checks of sizes, flags and null pointers (the workspace excepted), in fa_bwd's
// order; on FA_OK (an int fa_status) *ws_need is the workspace the shape needs (0: empty).
int bwd_check_args(const void* q, const void* k, const void* v, const void* o, const void* dout,
                   const float* lse, const void* dq, const void* dk, const void* dv, int B, int H,
                   int L, int D, float scale, int causal, int dtype, size_t* ws_need);

// Enqueues kern<<<grid, block, smem, s>>>(args...) and returns the status of that launch alone.
// (cudaGetLastError after a <<<>>> launch would also report a stale error left on the calling
// thread by any earlier runtime call, for example by a framework's set-up of its own threads.)
template <typename... KArgs, typename... Args>
cudaError_t launch_kernel(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                          cudaStream_t s, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<Args&&>(args)...);
}

// The same, allowed to start before the previous kernel of the stream has finished: `kern` calls
// griddepcontrol.wait before it touches anything that kernel writes.
template <typename... KArgs, typename... Args>
cudaError_t launch_kernel_early(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                cudaStream_t s, Args&&... args) {
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<Args&&>(args)...);
}

// A launch in clusters of `ctas` neighbouring CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_kernel_cluster(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, int ctas,
                                  cudaStream_t s, Args&&... args) {
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<Args&&>(args)...);
}

// Launchers (one per kernel unit).  Return the launch error, if any.
cudaError_t launch_fwd(const FwdParams& p, int D, bool bf16, bool causal, bool drop,
                       cudaStream_t s);
// The forward at D = 128 on CTA pairs (fa_fwd_pair.cu); needs p.tm_k_half.
cudaError_t launch_fwd_pair(const FwdParams& p, bool bf16, bool causal, cudaStream_t s);
cudaError_t launch_fwd_empty_rows(const FwdParams& p, int D, int rows, cudaStream_t s);
cudaError_t launch_bwd_pre(const BwdPreParams& p, cudaStream_t s);
cudaError_t launch_bwd_dkdv(const BwdParams& p, int D, bool bf16, bool causal, bool drop,
                            cudaStream_t s);
// The dK/dV pass that also reduces dQ = dS K into p.dq_acc (D = 64, no dropout), then the
// conversion of p.dq_acc (times the scale) into p.dq.
cudaError_t launch_bwd_dkdv_dq_reduce(const BwdParams& p, bool bf16, bool causal, cudaStream_t s);
cudaError_t launch_bwd_dq_convert(const BwdParams& p, int D, bool bf16, cudaStream_t s);
cudaError_t launch_bwd_dq(const BwdParams& p, int D, bool bf16, bool causal, bool drop,
                          cudaStream_t s);
cudaError_t launch_wait_selftest(int* status, uint64_t timeout_ns, cudaStream_t s);
cudaError_t launch_decode(const DecodeParams& p, int D, bool bf16, cudaStream_t s);
cudaError_t launch_rotary(const RotaryLaunch& p, bool bf16, cudaStream_t s);
cudaError_t launch_cache_append(const CacheAppendParams& p, bool bf16, bool q8, cudaStream_t s);
cudaError_t launch_cache_read(const CacheReadParams& p, bool bf16, bool q8, cudaStream_t s);
// q8: an e4m3 cache; else one of q's type (bf16 or fp16).
cudaError_t launch_decode_gqa(const GqaParams& p, int D, bool bf16, bool q8, cudaStream_t s);
cudaError_t launch_prefix(const PrefixParams& p, int D, bool bf16, cudaStream_t s);
// The work split of a shared prefix: fills rows_b, n_tiles, n_pairs, key_tiles, grid, max_segments.
void prefix_plan(int B, int Hk, int group, int prefix_len, PrefixParams* p);
cudaError_t launch_merge(const MergeParams& p, int D, bool bf16, cudaStream_t s);
// Query rows of a block (8 or 16), the most warps that a step may launch (workspace), and those it
// does (busy_sms: SMs that an earlier kernel still holds).
int gqa_q_rows(int group);
int gqa_warps(int B, int Hk, int group, int max_pages);
int gqa_rounds(int B, int Hk, int group);
// Whether a step takes a cluster per unit (and no merge).
bool gqa_short(int B, int Hk, int group, int max_pages, int D, bool q8);
int gqa_launched_warps(int B, int Hk, int group, int max_pages, int D, bool q8, int busy_sms);
// Splits of the page range per (sequence, head) for a decode step of this shape.
int decode_splits(int B, int H, int max_pages);

}  // namespace fa
