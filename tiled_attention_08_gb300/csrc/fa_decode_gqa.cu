// fa_decode_gqa.cu -- one decode step with grouped heads over a 16-bit or e4m3 paged cache (sm_103a).
//
// Query rows q[b, h], h = hk * G .. hk * G + G - 1, share the cache head hk:
//     O[b,h] = softmax(scale * q[b,h] K^T) V,  LSE[b,h] = log sum exp(scale * q[b,h] . k_t),
// over the seq_lens[b] tokens of the sequence, token t in page block_tables[b][t / 16] at slot
// t % 16.  A cached e4m3 row is its values times a power of two (fa_e4m3.cuh).
//
// Bound by HBM: every cached row is read once per cache head and used by G query rows (up to 16: a
// larger group is cut into blocks of 16, each of which reads the rows again), 4 G D FLOPs for 2 D or
// 4 D bytes.  On the FMA pipes the products alone would cost G instructions per value
// and lane, over the issue rate from G = 4 on, so they run on the tensor cores.  tcgen05's
// smallest tile has 64 rows and reads its operands from shared memory, where e4m3 rows would
// first have to be written back as 16-bit; mma.sync m16n8k16 takes its operands from registers,
// where the conversion costs one instruction per two values, and its 8 columns are the group.
// The keys are its 16 rows: S^T = K Q^T (16 keys = one page, 8 queries) and O^T += V^T P^T.  At
// the rate HBM delivers the tensor pipe is under a fifth busy.
//
// Work split.  A unit is one (sequence, cache head, block of 8 or 16 queries); its pages, unit
// after unit, form one line of P pages, of which every warp takes an equal stretch: whatever the
// sequences' lengths, all warps finish together, and no grid of splits has to be chosen.  P is known
// on the device only, so each CTA first sums the sequences' pages (a scan over seq_lens in
// shared memory).  A warp is a worker of its own: it has a ring of page slots filled by TMA
// (one lane issues, an mbarrier per slot) that runs on from unit to unit; 32 lanes look 32 pages'
// addresses up at once.  A unit that lies whole in one warp's stretch is written as O and LSE; of
// a cut one each warp leaves a part (at most two a warp: one that began before it, one that
// ends behind it), and fa_merge_kernel joins them.  Operand layouts, with
// lane = 4 g + t as the mma defines them:
//  * K, A operand (rows g, g+8 = keys): the contraction runs over D in any order that Q follows,
//    so a lane reads whole 16-byte units of its two rows, units 2t and 2t+1 of each 128-byte row;
//  * S^T comes out with its columns (queries 2t, 2t+1) in the lane that also holds O^T's columns,
//    so each lane keeps the running statistics of its own two queries;
//  * P^T, B operand: S^T's 8 x 8 blocks transposed in registers (movmatrix);
//  * V^T, A operand (rows = elements, contraction over keys 2t, 2t+1, 2t+8, 2t+9): a lane reads unit
//    g of its four keys; bytes (or halves) of two keys are paired by byte permutes.
// The TMA's 128-byte (64-byte) swizzle spreads these reads over all banks.
//
// Short steps.  With few units and short tables (gqa_short) the split above is mostly overhead: the
// scan, a search per page, parts through memory and a second kernel.  There a cluster of eight CTAs takes
// one unit, its 32 warps an equal share of the unit's pages each, and the parts are joined through
// distributed shared memory: CTA r joins query row r, and writes O and LSE.  One sequence of 512 tokens, 8
// cache heads, group 4, e4m3: 8.2 -> 6.6 us; 17 sequences of 500, 4 heads: 11.3 -> 8.8; a sequence of 4096
// among eight of 16: 15.1 -> 12.1.  It loses where the clusters do not all fit at once (72 fit with
// four CTAs per SM and 48 with three; 76 and 52 took 9.1 -> 11.6 and 10.4 -> 12.0 us), where a few
// units are long (one unit of 4096 tokens: 10.4 -> 11.8 us; 32 units of 8192, all but one head's short: 16.7 ->
// 17.8), and with groups above 8 (three CTAs per SM: 14.7 -> 22.0 us for 52 units).  Tables' width, in pages,
// all sequences that long, group 4, line against cluster: 8 units over e4m3, heads of 128, of 128 pages 11.4 and
// 9.6 us, 192 11.9 and 11.4, 256 12.4 and 12.7, 512 14.7 and 18.6; 32 units 256 17.6 and 14.9, 384 21.7 and 18.2,
// 512 23.7 and 21.4 (lengths spread from a quarter up: 20.6 and 20.6).  So 128 for fewer than 32 units, else
// 256.  Both are careful: 16-bit caches still gain there (8 units of 256 pages, heads of 64: 10.4 and 9.9).
//
// Softmax in the log2 domain.  The reference of a column is only raised when a score exceeds it
// by more than 2^8 (a warp vote), so the maximum over the lanes is rarely taken.  An e4m3 cache
// needs a second one: the sum of weights takes p_j = 2^(y_j - m); the products take
// a_j = 2^((y_j - m) + (ev_j - eo)) with the value row's exponent ev_j, so that a weight times its
// row's scale neither overflows nor is lost in fp16, whatever the rows' magnitudes.  (eo is relative
// to m: added to y_j itself, ev_j would be lost behind a large score.)  P is rounded to the
// cache's 16-bit type (fp16 for e4m3: 2^-12), as in the prefill kernels; sums stay fp32.  The reference
// of weights in fp16 stays 2^7 below the largest, which with the 2^8 keeps them below 2^15: fp16's range
// of normal numbers then begins 2^-21 below the largest instead of 2^-14, and many small weights behind a
// large one, which the sum of weights has in full, are not rounded away in the products.
//
// Measured.  256 sequences of 1..4096 tokens, 32 heads of 128, e4m3: 620 us (6.9 TB/s); 16-bit
// caches of long batches 6.8 to 7.0 TB/s.  48 sequences of 1..16384, 64 queries on 8 cache heads of 128,
// e4m3: 140 us (5.8 TB/s; no SM idle until the first stretches end).  Heads of 64, e4m3: 4.0 to 4.6
// TB/s: an SM turns over 10 to 12 pages per us whatever their size, with 377 instructions a page and warp
// and 16 warps' registers.
// 32 sequences of 8192, 4 cache heads, groups of 8, 16, 32, 64: heads of 128 e4m3 62, 74, 128, 234 us,
// 16-bit 97, 105, 181, 343; heads of 64 e4m3 43, 53, 88, 159, 16-bit 59, 59, 97, 178.  Two query blocks at
// heads of 128 spill 36 words of 168 registers.
#include <atomic>
#include <type_traits>

#include "fa_e4m3.cuh"
#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRaise = 8.0f;  // log2 headroom of the references
constexpr float kLift = 7.0f;   // a reference of fp16 weights stays this far below the largest score
constexpr int kWarps = 4;
constexpr int kGqaSms = 152;     // the grid is sized for this many SMs on any device, so that the
                                 // workspace does not depend on it
constexpr int kGqaMinPages = 4;  // pages of a warp's stretch at least ...
constexpr int kGqaFewPages = 1024;  // ... where there are more than this many
constexpr int kClusterCtas = 8;  // of a unit in a short step
constexpr int kGqaManyUnits = 2048;  // from so many on the line is dealt out in three rounds

// The split of the line of `total` pages.  One round: `workers` warps take equal stretches.  Not
// all SMs get the same share of the memory's bandwidth, so equal stretches end up to 15% apart;
// with three rounds the line's first 52/64 are dealt out like that, the next 8/64 and the last 4/64
// again in stretches so much shorter, to CTAs that start as earlier ones end (735 -> 641 us for 256
// sequences of 1..4096 tokens, 32 heads of 128, e4m3; borders at 40/56 to 60/62 of 64 take 603 to 634 us
// there, and 52/60 is within 1% of the best of them over four other batches of 2048 and more units).  Short
// stretches cut long units into many
// parts and each begins with an empty ring, so three rounds need kGqaManyUnits: with 2048 to 4096
// units they took -12% to +1% over e4m3 and 16-bit caches, heads of 64 and 128, groups of 1 to 4; with
// 1024 (groups of 8) +1% to +18%, with 384 +3% to +25% (142 -> 158 us for 48 sequences of up to
// 16384 tokens, e4m3, heads of 128).
struct GqaSplit {
    long long second, third, total;  // first pages of rounds 1 and 2 (total: there is none), the end
    int workers, rounds;
    __device__ __forceinline__ long long at(int r) const {
        return r == 0 ? 0 : r == 1 ? second : r == 2 ? third : total;
    }
    __device__ __forceinline__ long long start(int r, int i) const {
        return at(r) + (at(r + 1) - at(r)) * i / workers;
    }
    __device__ __forceinline__ int worker_of(long long x) const {  // the one that has page x
        const int r = x >= third ? 2 : x >= second ? 1 : 0;
        return r * workers + (int)(((x - at(r) + 1) * workers - 1) / (at(r + 1) - at(r)));
    }
};
// A page for each warp while there are few (latency is all: 13.1 -> 10.1 us for a token written and
// attended to behind 333, 8 cache heads, with this split), else at least kGqaMinPages; and a unit is cut
// into no more than 128 parts on average, which one CTA joins.  Limits of 32, 64, 128, 256, 512 for
// one unit, groups of 8: of 16384 tokens (e4m3, heads of 128) 32, 21, 16, 16, 19 us; two of 32768 (16-bit, heads of
// 64) 34, 21, 16, 17, 20; longer units would gain from 256 (one of 65536, e4m3: 109, 58, 34, 25, 25).
__device__ __forceinline__ GqaSplit gqa_split(long long total, int warps, int rounds, int units) {
    const long long a = total <= kGqaFewPages ? total : total / kGqaMinPages, b = 128LL * units;
    const long long m = a < b ? a : b;
    GqaSplit s;
    s.workers = m < 1 ? 1 : m < warps ? (int)m : warps;
    s.rounds = total >= 16LL * s.workers ? rounds : 1;
    s.second = s.rounds > 1 ? total / 64 * 52 : total;
    s.third = s.rounds > 1 ? total / 64 * 60 : total;
    s.total = total;
    return s;
}

// cudaFuncSetAttribute once per kernel and device (the calls below repeat every few microseconds).
template <int D, bool Q8, bool BF16, int NT, bool SHORT>
struct kGqaKernelId {};
template <typename Id, typename K>
cudaError_t allow_shared(K kern, int bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (done.load() >> dev & 1)) return cudaSuccess;
    const cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (r == cudaSuccess && dev < 64) done.fetch_or(uint64_t(1) << dev);
    return r;
}

// Q8: an e4m3 cache.
template <int D, bool Q8>
struct GqaCfg {
    static constexpr int kRowBytes = (D * (Q8 ? 1 : 2)) < 128 ? 64 : 128;  // of one TMA box
    static constexpr int kBoxes = D * (Q8 ? 1 : 2) / kRowBytes;
    static constexpr int kBoxBytes = kPageTokens * kRowBytes;
    static constexpr int kPageBytes = kBoxes * kBoxBytes;
    static constexpr int kSteps = D / 16;   // contraction steps of S^T
    static constexpr int kTiles = D / 16;   // 16-element row tiles of O^T
    // Page slots per warp.  Small rings and more CTAs per SM win: the serving batch of 256
    // sequences of 1..4096 tokens, 32 heads of 128, e4m3, takes 646 us with 3 slots, 653 with 2,
    // 726 with 4 (fewer CTAs fit), 926 with 6.
    static constexpr int kStages = Q8 ? (D == 128 ? 3 : 4) : (D == 128 ? 2 : 3);
    static constexpr int kRingBytes = kWarps * kStages * (2 * kPageBytes + (Q8 ? 32 : 0));
};
// CTAs per SM that fit (registers and shared memory); the grid is that many times 152 SMs.
constexpr int gqa_occupancy(int D, bool q8, int nt) { return nt == 2 || (D == 128 && !q8) ? 3 : 4; }

// A page's rows of one head; the line goes out of L2 first (each is read once).
__device__ __forceinline__ void tma_load_page(void* dst, const CUtensorMap* map, uint64_t* bar, int x,
                                              int page_head, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(0), "r"(page_head), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}
__device__ __forceinline__ uint64_t policy_evict_first() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Maximum over the lanes that hold the same column (lanes with the same t).
__device__ __forceinline__ float column_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
__device__ __forceinline__ float column_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 4);
    v += __shfl_xor_sync(0xffffffffu, v, 8);
    return v + __shfl_xor_sync(0xffffffffu, v, 16);
}

// A reference before any score: below every finite one, and finite, so that no difference of it is
// a NaN (a masked -inf minus it is -inf).
constexpr float kNoRef = -3.4028234663852886e38f;  // -FLT_MAX

// Raises a reference to the column's maximum less `lift`; returns the factor of what was summed under it.
__device__ __forceinline__ float raise(float& ref, float top, float lift) {
    const float next = fmaxf(ref, column_max(top) - lift);
    const float f = ex2_approx(ref - next);
    ref = next;
    return f;
}

// Pages of one warp, 32 at a time: lane i knows the i-th.
struct Batch {
    int page_head;  // page * Hk + head in the cache
    int b, unit;    // sequence, and (cache head, query block) in it
    int flags;      // tokens that count (1..16) | first page of its unit << 8 | last << 9
};
constexpr int kFirst = 1 << 8, kLast = 1 << 9;

// Thread-block clusters of short steps: the value at shared::cta address `addr` of CTA `rank`.
__device__ __forceinline__ float lds_cluster(uint32_t addr, uint32_t rank) {
    float v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
        : "=f"(v)
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}

// BF16: the type of q and o (and of a 16-bit cache).  NT: blocks of 8 queries.  SHORT: a cluster per
// unit, whose warps share the unit's pages and join their parts through distributed shared memory.
template <int D, bool Q8, bool BF16, int NT, bool SHORT>
__global__ void __launch_bounds__(kWarps * 32, gqa_occupancy(D, Q8, NT))
    fa_decode_gqa_kernel(const __grid_constant__ GqaParams p) {
    using C = GqaCfg<D, Q8>;
    constexpr bool kMmaBf16 = BF16 && !Q8;  // e4m3 values are exact in fp16
    constexpr float kLiftM = Q8 || BF16 ? 0.0f : kLift;  // (over e4m3 m is the reference of the sum alone)
    constexpr int stages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    __shared__ uint64_t bar_full[kWarps][stages];
    __shared__ int warp_sum[kWarps];
    int* cum = reinterpret_cast<int*>(smem + C::kRingBytes);  // [B + 1] pages before sequence b
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

    const int per_seq = p.Hk * p.q_blocks;  // units of a sequence
    const int unit_id = (int)blockIdx.x / kClusterCtas, short_b = unit_id / per_seq;  // (SHORT)
    const int short_unit = unit_id - short_b * per_seq, rank = (int)blockIdx.x % kClusterCtas;
    pdl_launch_dependents();
    // The queries into L2 (they are read when a warp begins a unit, behind the stream of pages).
    for (size_t at = ((size_t)blockIdx.x * (kWarps * 32) + threadIdx.x) * 128;
         !SHORT && at < (size_t)p.B * p.Hq * D * 2; at += (size_t)gridDim.x * (kWarps * 32) * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint8_t*>(p.q) + at));
    if (threadIdx.x == 0 && p.num_pages > 0) {
        tma_prefetch_desc(&p.tm_k);
        tma_prefetch_desc(&p.tm_v);
    }
    if (lane < stages) mbar_init(&bar_full[warp][lane], 1);
    mbar_fence_init();
    // ---- pages before each sequence: every thread sums a run of sequences ----
    const int n_seqs = SHORT ? 0 : p.B;
    const int run = (p.B + kWarps * 32 - 1) / (kWarps * 32);
    const int s0 = min((int)threadIdx.x * run, n_seqs), s1 = min(s0 + run, n_seqs);
    auto pages_of = [&](int b) {
        const int n = p.seq_lens[b];
        if (n < 0 || n > (long long)p.max_pages * kPageTokens || (n > 0 && p.num_pages == 0)) {
            if (SHORT || blockIdx.x == 0) atomicCAS(p.status, 0, (int)kDevBadArg);
            return 0;  // counts as empty
        }
        return (n + kPageTokens - 1) / kPageTokens;
    };
    GqaSplit split;
    int w = 0, mine = 0;  // this worker, and its pages x0 .. x0 + mine - 1 of the line (SHORT: of the unit)
    long long x0 = 0, total = 0;
    if constexpr (SHORT) {
        const int n_pages = pages_of(short_b), i = warp * kClusterCtas + rank;  // neighbours on different SMs
        constexpr int kWorkers = kClusterCtas * kWarps;
        x0 = n_pages * (long long)i / kWorkers;
        mine = (int)(n_pages * (long long)(i + 1) / kWorkers - x0);
        __syncthreads();  // (the barriers are initialised)
    } else {
        int sum = 0;
        for (int b = s0; b < s1; ++b) sum += pages_of(b);
        int scan = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, scan, off);
            if (lane >= off) scan += v;
        }
        if (lane == 31) warp_sum[warp] = scan;
        __syncthreads();
        int before = scan - sum;
        for (int w = 0; w < warp; ++w) before += warp_sum[w];
        for (int b = s0; b < s1; ++b) {
            cum[b] = before;
            before += pages_of(b);
        }
        if (threadIdx.x == kWarps * 32 - 1) cum[p.B] = before;
        __syncthreads();
        for (int b = blockIdx.x; b < p.B; b += gridDim.x)
            if (cum[b] == cum[b + 1])
                for (int i = threadIdx.x; i < per_seq; i += kWarps * 32)
                    p.unit_parts[(size_t)b * per_seq + i] = make_int2(0, 0);  // no key, no part
        total = (long long)cum[p.B] * per_seq;
        split = gqa_split(total, p.warps, p.rounds, p.B * per_seq);
        const int ctas = p.warps / kWarps;  // of a round
        const int r = (int)blockIdx.x / ctas;
        const int wi = warp * ctas + (int)blockIdx.x - r * ctas;  // neighbours on different SMs
        const bool works = r < split.rounds && wi < split.workers;
        w = r * split.workers + wi;
        x0 = works ? split.start(r, wi) : 0;
        mine = works ? (int)(split.start(r, wi + 1) - x0) : 0;
    }

    uint8_t* ring = smem + (size_t)warp * stages * (2 * C::kPageBytes);
    uint8_t* exps = smem + (size_t)kWarps * stages * (2 * C::kPageBytes) + warp * stages * 32;
    auto lookup = [&](int first) {  // pages first .. first + 31 of this warp
        Batch r = {0, 0, 0, 0};
        if (SHORT && first + lane < mine) {
            const int pg = (int)x0 + first + lane;
            int page = p.block_tables[(size_t)short_b * p.max_pages + pg];
            if (page < 0 || page >= p.num_pages) {  // as below
                atomicCAS(p.status, 0, (int)kDevBadArg);
                page = 0;
            }
            r.page_head = page * p.Hk + short_unit / p.q_blocks;
            r.flags = min(p.seq_lens[short_b] - pg * kPageTokens, kPageTokens);
        } else if (!SHORT && first + lane < mine) {
            const long long x = x0 + first + lane;
            // (64-bit quotients cost ten times 32-bit ones)
            const bool small = total <= 0x7fffffffLL;
            const int at = small ? (int)((uint32_t)x / (uint32_t)per_seq) : (int)(x / per_seq);
            int lo = 0, hi = p.B;  // the sequence with cum[b] <= at < cum[b + 1]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cum[mid] <= at) lo = mid;
                else hi = mid;
            }
            const int n_pages = cum[lo + 1] - cum[lo];
            const long long rest = x - (long long)cum[lo] * per_seq;
            r.b = lo;
            r.unit = small ? (int)((uint32_t)rest / (uint32_t)n_pages) : (int)(rest / n_pages);
            const int pg = (int)(rest - (long long)r.unit * n_pages);
            int page = p.block_tables[(size_t)lo * p.max_pages + pg];
            if (page < 0 || page >= p.num_pages) {
                // Reported; page 0 is read instead: nothing outside the cache is touched.
                atomicCAS(p.status, 0, (int)kDevBadArg);
                page = 0;
            }
            r.page_head = page * p.Hk + r.unit / p.q_blocks;
            r.flags = min(p.seq_lens[lo] - pg * kPageTokens, kPageTokens) | (pg == 0 ? kFirst : 0) |
                      (pg == n_pages - 1 ? kLast : 0);
        }
        return r;
    };
    const uint64_t policy = policy_evict_first();
    Batch prod = lookup(0), cons = prod, next = lookup(32);
    auto issue = [&](int i, int st) {  // page i of this warp into slot st = i % stages; the whole warp calls it
        if (i > 0 && (i & 31) == 0) {
            prod = next;
            next = lookup(i + 32);
        }
        const int ph = __shfl_sync(0xffffffffu, prod.page_head, i & 31);
        if (lane == 0) {
            uint64_t* bar = &bar_full[warp][st];
            uint8_t* dst = ring + st * (2 * C::kPageBytes);
            mbar_arrive_expect_tx(bar, 2 * C::kPageBytes + (Q8 ? 32 : 0));
#pragma unroll
            for (int x = 0; x < C::kBoxes; ++x)
                tma_load_page(dst + x * C::kBoxBytes, &p.tm_k, bar, x * 64, ph, policy);
            if constexpr (Q8) {
                bulk_load(exps + st * 32, p.k_exp + (size_t)ph * kPageTokens, 16, bar);
                bulk_load(exps + st * 32 + 16, p.v_exp + (size_t)ph * kPageTokens, 16, bar);
            }
#pragma unroll
            for (int x = 0; x < C::kBoxes; ++x)
                tma_load_page(dst + C::kPageBytes + x * C::kBoxBytes, &p.tm_v, bar, x * 64, ph, policy);
        }
    };
    for (int i = 0; i < min(stages, mine); ++i) issue(i, i);

    // Q fragments (B operand).  Step s of lane t covers elements elem(s) .. + 3: the order in
    // which the K rows are read below.
    uint32_t qf[C::kSteps][NT][2];
    float q_factor[NT][2];  // factor of S^T's columns 2t, 2t+1: scale * log2(e), and for e4m3 the
                            // power of two that brought the query row into fp16's range
    auto load_q = [&](size_t row0, int n_q) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int qi = nt * 8 + g;
            const uint8_t* src = static_cast<const uint8_t*>(p.q) + (row0 + qi) * D * 2;
            uint32_t w[C::kSteps][2];
#pragma unroll
            for (int s = 0; s < C::kSteps; ++s) {
                const int e = Q8 ? (D / 4) * t + 4 * s : 64 * (s >> 2) + 16 * t + 4 * (s & 3);
                uint2 u = make_uint2(0u, 0u);
                if (qi < n_q) u = *reinterpret_cast<const uint2*>(src + e * 2);
                w[s][0] = u.x;
                w[s][1] = u.y;
            }
            float f = 1.0f;  // the row's power of two
            if constexpr (Q8 && BF16) {
                uint32_t mx = 0;
#pragma unroll
                for (int s = 0; s < C::kSteps; ++s)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        mx = max(mx, max((w[s][j] << 16) & 0x7fff0000u, w[s][j] & 0x7fff0000u));
                mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                // Largest magnitude to [2^14, 2^15); 2^100 at most (rows below 2^-86 lose nothing
                // that a score could show).
                const int ex = (int)(mx >> 23) - 127;
                if (mx != 0 && mx < 0x7f800000u) f = __uint_as_float((uint32_t)(127 + min(14 - ex, 100)) << 23);
#pragma unroll
                for (int s = 0; s < C::kSteps; ++s)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float2 v = unpack2<true>(w[s][j]);
                        w[s][j] = pack2<false>(v.x * f, v.y * f);
                    }
            }
#pragma unroll
            for (int s = 0; s < C::kSteps; ++s) {
                qf[s][nt][0] = w[s][0];
                qf[s][nt][1] = w[s][1];
            }
            const float back = p.scale_log2 / f;
            q_factor[nt][0] = __shfl_sync(0xffffffffu, back, 8 * t);      // lane of g = 2t
            q_factor[nt][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);  // lane of g = 2t + 1
        }
    };

    float acc[C::kTiles][NT][4];
    float m[NT][2], eo[NT][2], l[NT][2];
    size_t row0 = 0;       // first query row of the unit
    int n_q = 0;           // queries of its block
    bool cut = false;      // the unit began in an earlier warp's stretch
    bool ok = true;
    int done = 0, st = 0;  // pages behind this one, and this one's slot
    uint32_t parity = 0;   // of the slot's phase
    for (; done < mine; ++done) {
        if (done > 0 && (done & 31) == 0) cons = prod;  // (the ring is less than a batch ahead)
        const int flags = __shfl_sync(0xffffffffu, cons.flags, done & 31);
        if (done == 0 || (flags & kFirst)) {  // a new unit
            const int b = SHORT ? short_b : __shfl_sync(0xffffffffu, cons.b, done & 31);
            const int unit = SHORT ? short_unit : __shfl_sync(0xffffffffu, cons.unit, done & 31);
            const int hk = unit / p.q_blocks, q0 = (unit - hk * p.q_blocks) * (NT * 8);
            n_q = min(NT * 8, p.group - q0);
            row0 = (size_t)b * p.Hq + (size_t)hk * p.group + q0;
            cut = !(flags & kFirst);
            load_q(row0, n_q);
            if (!SHORT && !cut && lane == 0) {  // for the merge: the warps that have the unit's pages
                const long long last = x0 + done + (cum[b + 1] - cum[b]) - 1;
                const int n = done + (cum[b + 1] - cum[b]) <= mine ? 1 : split.worker_of(last) - w + 1;
                p.unit_parts[(size_t)b * per_seq + unit] = make_int2(w, n);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    m[nt][j] = eo[nt][j] = kNoRef;
                    l[nt][j] = 0.0f;
                }
#pragma unroll
                for (int i = 0; i < C::kTiles; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][nt][j] = 0.0f;
            }
        }
        ok = wait_warp(&bar_full[warp][st], parity, nullptr, p.timeout_ns);
        if (!ok) break;
        const uint8_t* kp = ring + st * (2 * C::kPageBytes);
        const uint8_t* vp = kp + C::kPageBytes;
        const uint32_t ks = smem_u32(kp), vs = smem_u32(vp);
        constexpr bool kSmall = Q8 && D == 64;  // 64-byte rows
        // ---- S^T = K Q^T: rows g and g + 8 of the page, even and odd steps apart ----
        // (One accumulator where two query blocks already take turns.)
        constexpr bool kTwo = NT == 1;
        float c[NT][4], c2[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) c[nt][j] = c2[nt][j] = 0.0f;
        if constexpr (!Q8) {
            uint4 lo[C::kBoxes][2], hi[C::kBoxes][2];
#pragma unroll
            for (int x = 0; x < C::kBoxes; ++x)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const uint32_t u = ks + x * C::kBoxBytes + (uint32_t)((2 * t + hf) ^ g) * 16;
                    lo[x][hf] = lds_u32x4(u + g * 128);
                    hi[x][hf] = lds_u32x4(u + (g + 8) * 128);
                }
#pragma unroll
            for (int x = 0; x < C::kBoxes; ++x)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const int s = 4 * x + 2 * hf;
                        const uint4 &a = lo[x][hf], &b = hi[x][hf];
                        mma16816<kMmaBf16>(c[nt], a.x, b.x, a.y, b.y, qf[s][nt][0], qf[s][nt][1]);
                        mma16816<kMmaBf16>(kTwo ? c2[nt] : c[nt], a.z, b.z, a.w, b.w, qf[s + 1][nt][0],
                                           qf[s + 1][nt][1]);
                    }
        } else {
            constexpr int kUnits = D / 64;  // 16-byte units of a row per lane
            uint4 lo[kUnits], hi[kUnits];
#pragma unroll
            for (int hf = 0; hf < kUnits; ++hf) {
                // (64-byte rows: unit index XOR (row / 2) % 4)
                const uint32_t u = D == 128 ? ks + g * 128 + (uint32_t)((2 * t + hf) ^ g) * 16
                                            : ks + g * 64 + (uint32_t)(t ^ ((g >> 1) & 3)) * 16;
                lo[hf] = lds_u32x4(u);
                hi[hf] = lds_u32x4(u + 8 * C::kRowBytes);
            }
#pragma unroll
            for (int hf = 0; hf < kUnits; ++hf) {
                const uint32_t wl[4] = {lo[hf].x, lo[hf].y, lo[hf].z, lo[hf].w};
                const uint32_t wh[4] = {hi[hf].x, hi[hf].y, hi[hf].z, hi[hf].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a0 = e4m3x2_to_f16x2(wl[i] & 0xffffu), a2 = e4m3x2_to_f16x2(wl[i] >> 16);
                    const uint32_t a1 = e4m3x2_to_f16x2(wh[i] & 0xffffu), a3 = e4m3x2_to_f16x2(wh[i] >> 16);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816<false>(kTwo && (i & 1) ? c2[nt] : c[nt], a0, a1, a2, a3, qf[4 * hf + i][nt][0],
                                        qf[4 * hf + i][nt][1]);
                }
            }
        }
        // ---- V into registers, the slot to the page `stages` further on ----
        // Unit g of keys 2t, 2t+1, 2t+8, 2t+9 (64-byte rows: half a unit).  Two query blocks leave no
        // registers for that: they read V below, and free the slot after it.
        // Slots past the sequence's end hold anything: their values count as zeros (their weights
        // are zero, but zero times a NaN is not).
        constexpr bool kEarly = NT == 1 && !Q8;
        const int left = flags & 31;  // tokens of this page
        const bool partial = left < kPageTokens;
        uint4 vq[kSmall ? 1 : C::kBoxes][4];
        uint2 vh[4];
        auto read_v = [&](int x) __attribute__((always_inline)) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int key = 2 * t + (k & 1) + 8 * (k >> 1);
                const bool there = !partial || key < left;
                if constexpr (kSmall) {
                    vh[k] = lds_u32x2(vs + key * 64 + (uint32_t)((g >> 1) ^ ((key >> 1) & 3)) * 16 + (g & 1) * 8);
                    if (!there) vh[k] = make_uint2(0u, 0u);
                } else {
                    vq[x][k] = lds_u32x4(vs + x * C::kBoxBytes + key * 128 + (uint32_t)(g ^ (key & 7)) * 16);
                    if (!there) vq[x][k] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
        };
        auto release = [&]() __attribute__((always_inline)) {
            __syncwarp();  // every lane has read the slot
            if (done + stages < mine) issue(done + stages, st);
        };
        float fk[2] = {1.0f, 1.0f}, ev[2] = {0.0f, 0.0f};  // rows g, g + 8: factor of K, exponent of V
        if constexpr (Q8) {
            const uint8_t* ex = exps + st * 32;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                fk[r] = row_scale(ex[g + 8 * r]);
                const uint32_t E = ex[16 + g + 8 * r];
                ev[r] = E == kExpNan ? __uint_as_float(0x7fc00000u) : (float)((int)E - 127);
            }
        }
        if constexpr (kEarly) {
#pragma unroll
            for (int x = 0; x < (kSmall ? 1 : C::kBoxes); ++x) read_v(x);
            release();
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) c[nt][j] += c2[nt][j];
        // ---- online softmax over the page ----
        bool up = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 4; ++j) c[nt][j] *= Q8 ? fk[j >> 1] * q_factor[nt][j & 1] : q_factor[nt][j & 1];
        }
        if (partial) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                if (g + 8 * r < left) continue;
                ev[r] = 0.0f;  // (a slot's byte may be anything)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) c[nt][2 * r] = c[nt][2 * r + 1] = -INFINITY;
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                up |= fmaxf(c[nt][j], c[nt][j + 2]) > m[nt][j] + (kRaise + kLiftM);
                if constexpr (Q8)
                    up |= fmaxf(c[nt][j] - m[nt][j] + ev[0], c[nt][j + 2] - m[nt][j] + ev[1]) >
                          eo[nt][j] + (kRaise + kLift);
            }
        }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float old = m[nt][j];
                    const float f = raise(m[nt][j], fmaxf(c[nt][j], c[nt][j + 2]), kLiftM);
                    l[nt][j] *= f;
                    float fo = f;
                    if constexpr (Q8) {
                        eo[nt][j] = fmaxf(eo[nt][j] + (old - m[nt][j]), kNoRef);  // under the new m
                        fo = raise(eo[nt][j], fmaxf(c[nt][j] - m[nt][j] + ev[0], c[nt][j + 2] - m[nt][j] + ev[1]),
                                   kLift);
                    }
#pragma unroll
                    for (int i = 0; i < C::kTiles; ++i) {
                        acc[i][nt][j] *= fo;
                        acc[i][nt][j + 2] *= fo;
                    }
                }
            }
        }
        uint32_t pf[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float a[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float d = c[nt][j] - m[nt][j & 1];
                const float pj = ex2_approx(d);
                l[nt][j & 1] += pj;
                a[j] = Q8 ? ex2_approx(d + (ev[j >> 1] - eo[nt][j & 1])) : pj;
            }
            pf[nt][0] = transpose8x8(pack2<kMmaBf16>(a[0], a[1]));
            pf[nt][1] = transpose8x8(pack2<kMmaBf16>(a[2], a[3]));
        }
        // ---- O^T += V^T P^T: keys 2t, 2t+1, 2t+8, 2t+9 of the page ----
        // Words of the four keys: pairs of keys side by side are an operand register.
        auto pv8 = [&](int tile, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {  // 4 elements, e4m3
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const uint32_t lo = __byte_perm(w0, w1, hf ? 0x7362 : 0x5140);
                const uint32_t hi = __byte_perm(w2, w3, hf ? 0x7362 : 0x5140);
                const uint32_t a0 = e4m3x2_to_f16x2(lo & 0xffffu), a1 = e4m3x2_to_f16x2(lo >> 16);
                const uint32_t a2 = e4m3x2_to_f16x2(hi & 0xffffu), a3 = e4m3x2_to_f16x2(hi >> 16);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma16816<false>(acc[tile + hf][nt], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
            }
        };
        auto pv16 = [&](int tile, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {  // 2 elements
            const uint32_t a0 = __byte_perm(w0, w1, 0x5410), a1 = __byte_perm(w0, w1, 0x7632);
            const uint32_t a2 = __byte_perm(w2, w3, 0x5410), a3 = __byte_perm(w2, w3, 0x7632);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                mma16816<kMmaBf16>(acc[tile][nt], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
        };
        if constexpr (kSmall) {
            if constexpr (!kEarly) read_v(0);
            pv8(0, vh[0].x, vh[1].x, vh[2].x, vh[3].x);
            pv8(2, vh[0].y, vh[1].y, vh[2].y, vh[3].y);
        } else {
#pragma unroll
            for (int x = 0; x < C::kBoxes; ++x) {
                if constexpr (!kEarly) read_v(x);
                const uint4(&v)[4] = vq[x];
                if constexpr (Q8) {
                    pv8(0, v[0].x, v[1].x, v[2].x, v[3].x);
                    pv8(2, v[0].y, v[1].y, v[2].y, v[3].y);
                    pv8(4, v[0].z, v[1].z, v[2].z, v[3].z);
                    pv8(6, v[0].w, v[1].w, v[2].w, v[3].w);
                } else {
                    pv16(4 * x, v[0].x, v[1].x, v[2].x, v[3].x);
                    pv16(4 * x + 1, v[0].y, v[1].y, v[2].y, v[3].y);
                    pv16(4 * x + 2, v[0].z, v[1].z, v[2].z, v[3].z);
                    pv16(4 * x + 3, v[0].w, v[1].w, v[2].w, v[3].w);
                }
            }
        }
        if constexpr (!kEarly) release();
        if (++st == stages) {
            st = 0;
            parity ^= 1u;
        }
        const bool ends = (flags & kLast) != 0;
        if (!ends && done + 1 < mine) continue;
        // ---- the unit, or this warp's part of it, is done ----
        // Lane (g, t) holds, for queries 2t and 2t+1, whole runs of elements: e4m3 D/8 from
        // D/8 g on, 16-bit 8 from 64 x + 8 g on for each box x.
        const bool whole = !SHORT && !cut && ends && !p.parts_only;
        float* part_o = nullptr;
        float* part_lse = nullptr;
        if constexpr (SHORT) {  // into this warp's ring, which is empty now
            part_o = reinterpret_cast<float*>(ring);
            part_lse = part_o + NT * 8 * D;
        } else if (!whole) {
            const size_t slot = (cut || !ends) ? 2 * (size_t)w + (cut ? 0 : 1) : 0;
            if (!cut && ends) {  // a whole unit of a row that has other parts
                part_o = p.full_o + row0 * D;
                part_lse = p.full_lse + row0;
            } else {
                part_o = p.slot_o + slot * p.slot_rows * D;
                part_lse = p.slot_lse + slot * p.slot_rows;
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float L = column_sum(l[nt][j]);
                const int qi = nt * 8 + 2 * t + j;
                if (qi >= n_q) continue;
                // (L = 0: every score is -inf, as if the row saw no key.)  2^eo in two steps: alone it
                // may be below fp32's range.
                const float f = L == 0.0f ? 0.0f : 1.0f / L;
                const float hop = Q8 ? ex2_approx(0.5f * eo[nt][j]) : 1.0f;
                const float lse2 = m[nt][j] + log2f(L);
                if (g == 0) {
                    if (whole) p.lse[row0 + qi] = lse2 * kLn2;
                    else part_lse[qi] = lse2;
                }
                constexpr int kRun = Q8 ? C::kTiles : 4;  // tiles of one run
#pragma unroll
                for (int x = 0; x < C::kTiles / kRun; ++x) {
                    const int e = Q8 ? (D / 8) * g : 64 * x + 8 * g;
                    float v[2 * kRun];
#pragma unroll
                    for (int i = 0; i < kRun; ++i) {
                        v[2 * i] = acc[x * kRun + i][nt][j] * f * hop * hop;
                        v[2 * i + 1] = acc[x * kRun + i][nt][j + 2] * f * hop * hop;
                    }
                    if (whole) {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + (row0 + qi) * D + e);
#pragma unroll
                        for (int i = 0; i < kRun / 4; ++i)
                            dst[i] = make_uint4(pack2<BF16>(v[8 * i], v[8 * i + 1]),
                                                pack2<BF16>(v[8 * i + 2], v[8 * i + 3]),
                                                pack2<BF16>(v[8 * i + 4], v[8 * i + 5]),
                                                pack2<BF16>(v[8 * i + 6], v[8 * i + 7]));
                    } else {
                        float4* dst = reinterpret_cast<float4*>(part_o + (size_t)qi * D + e);
#pragma unroll
                        for (int i = 0; i < kRun / 2; ++i)
                            dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    }
                }
            }
        }
    }
    if (!ok) {
        if (lane == 0) atomicCAS(p.status, 0, (int)kDevTimeout);
        // No copy may still be landing when the CTA exits.
        for (int i = done; i < min(mine, done + stages); ++i)
            wait_bounded(&bar_full[warp][i % stages], (uint32_t)(i / stages) & 1u, nullptr, p.timeout_ns);
    }
    if constexpr (SHORT) {
        static_assert((NT * 8 * (D + 1)) * 4 <= stages * 2 * C::kPageBytes, "a warp's part in its ring");
        if ((mine == 0 || !ok) && lane < NT * 8) reinterpret_cast<float*>(ring)[NT * 8 * D + lane] = -INFINITY;
        cluster_sync();
        const int hk = short_unit / p.q_blocks, q0 = (short_unit - hk * p.q_blocks) * (NT * 8);
        const int rows = min(NT * 8, p.group - q0);
        const size_t row = (size_t)short_b * p.Hq + (size_t)hk * p.group + q0;
        const uint32_t part0 = smem_u32(smem);
        constexpr uint32_t kPart = stages * 2 * C::kPageBytes;  // between two warps' parts
        for (int qi = rank; qi < rows; qi += kClusterCtas) {
            // Lane i: part i, of warp i % 4 in CTA i / 4.
            const float y = lds_cluster(part0 + lane % kWarps * kPart + (NT * 8 * D + qi) * 4, lane / kWarps);
            const uint32_t there = __ballot_sync(0xffffffffu, y != -INFINITY);  // (else nothing was written)
            float top = y;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float wi = y == -INFINITY ? 0.0f : ex2_approx(y - top);
            float sum = wi;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            float x = 0.0f;
#pragma unroll 8
            for (int i = 0; i < 32; ++i) {
                const float wv = __shfl_sync(0xffffffffu, wi, i);
                if (threadIdx.x < D && (there >> i & 1u))
                    x = fmaf(wv,
                             lds_cluster(part0 + i % kWarps * kPart + (qi * D + threadIdx.x) * 4, i / kWarps),
                             x);
            }
            const bool any = sum != 0.0f;  // (true of a NaN)
            if (threadIdx.x < D)
                static_cast<uint16_t*>(p.o)[(row + qi) * D + threadIdx.x] =
                    any ? (uint16_t)pack2<BF16>(x / sum, 0.0f) : (uint16_t)0;
            if (threadIdx.x == 0) p.lse[row + qi] = any ? (top + log2f(sum)) * kLn2 : -INFINITY;
        }
        cluster_sync();  // the parts have been read
        return;
    }
    // Launched early behind a kernel that writes other parts of the same rows, this grid ends only
    // after that one (one CTA waits; the others make room), so that the merge waits for both by
    // waiting for this one.
    if (blockIdx.x == 0) pdl_wait();
}

// Joins the parts of each query row: O = sum w_i O_i / sum w_i, LSE = log sum exp(LSE_i), with
// w_i = 2^(LSE2_i - max).  Parts 0 .. n_prefix-1 are a shared prefix's, then those that the warps of
// fa_decode_gqa_kernel left of the row's unit (or the whole unit, in full_o).  WPR warps per row
// take every WPR-th group of four parts and meet in shared memory.  A row that the decode kernel has
// written itself is left alone; one without any key gets O = 0, LSE = -inf.
template <int D, bool BF16, int WPR>
__global__ void __launch_bounds__(256) fa_merge_kernel(const MergeParams p) {
    constexpr int kPer = D / 32, kAhead = 8;  // parts whose loads are in flight together
    using Vec = typename std::conditional<kPer == 4, float4, float2>::type;
    __shared__ float red[WPR > 1 ? WPR : 1][D + 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = WPR > 1 ? (int)blockIdx.x : (int)blockIdx.x * 8 + warp;
    const int sub = WPR > 1 ? warp : 0;
    pdl_wait();
    if (row >= p.rows) return;
    const int b = row / p.Hq, h = row - b * p.Hq;
    const int hk = h / p.group, gi = h - hk * p.group;
    const int qb = gi / p.q_rows, qi = gi - qb * p.q_rows;
    const int2 own = p.unit_parts[((size_t)b * p.Hk + hk) * p.q_blocks + qb];
    // (A kernel that gave up on a wait may have left an entry as it found it: no part, then.)
    const bool there = own.x >= 0 && own.y >= 0 && own.x < p.workers && own.y <= p.workers - own.x;
    const int w_first = own.x, n_own = there ? own.y : 0;
    const int n_parts = p.n_prefix + n_own;
    if (p.n_prefix == 0 && n_own == 1) return;  // written whole
    const float* pre_o = p.prefix_o + (size_t)row * p.n_prefix * D;
    const float* pre_lse = p.prefix_lse + (size_t)row * p.n_prefix;
    auto locate = [&](int i, const float*& o, const float*& lse2) {
        if (i < p.n_prefix) {
            o = pre_o + (size_t)i * D;
            lse2 = pre_lse + i;
        } else if (n_own == 1) {
            o = p.full_o + (size_t)row * D;
            lse2 = p.full_lse + row;
        } else {
            const int k = i - p.n_prefix;
            const size_t at = (2 * (size_t)(w_first + k) + (k == 0 ? 1 : 0)) * p.slot_rows + qi;
            o = p.slot_o + at * D;
            lse2 = p.slot_lse + at;
        }
    };
    float top = -INFINITY, sum = 0.0f, x[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) x[e] = 0.0f;
    for (int i0 = sub * kAhead; i0 < n_parts; i0 += WPR * kAhead) {
        Vec v[kAhead];
        float y[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            y[j] = -INFINITY;
            if (i0 + j < n_parts) {
                const float *o, *l2;
                locate(i0 + j, o, l2);
                y[j] = *l2;
                v[j] = *reinterpret_cast<const Vec*>(o + lane * kPer);
            }
        }
        float next = top;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) next = fmaxf(next, y[j]);
        const float base = next == -INFINITY ? 0.0f : next;
        const float f = ex2_approx(top - base);  // (0 at first: top = -inf)
        sum *= f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) x[e] *= f;
        top = next;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (y[j] == -INFINITY) continue;  // no key: its values were not written
            const float wj = ex2_approx(y[j] - base);
            sum += wj;
            const float* vf = reinterpret_cast<const float*>(&v[j]);
#pragma unroll
            for (int e = 0; e < kPer; ++e) x[e] = fmaf(wj, vf[e], x[e]);
        }
    }
    if constexpr (WPR > 1) {
        if (lane == 0) {
            red[warp][D] = top;
            red[warp][D + 1] = sum;
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) red[warp][lane * kPer + e] = x[e];
        __syncthreads();
        if (warp != 0) return;
        float all = -INFINITY;
#pragma unroll
        for (int k = 0; k < WPR; ++k) all = fmaxf(all, red[k][D]);
        sum = 0.0f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) x[e] = 0.0f;
#pragma unroll
        for (int k = 0; k < WPR; ++k) {
            // (a warp without parts has a sum of 0; one with a NaN part keeps its NaN)
            const float f = red[k][D] == -INFINITY ? 1.0f : ex2_approx(red[k][D] - all);
            sum = fmaf(red[k][D + 1], f, sum);
#pragma unroll
            for (int e = 0; e < kPer; ++e) x[e] = fmaf(red[k][lane * kPer + e], f, x[e]);
        }
        top = all;
    }
    const bool any = sum != 0.0f;  // (true of a NaN)
    const float f = any ? 1.0f / sum : 0.0f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + (size_t)row * D + lane * kPer);
#pragma unroll
    for (int e = 0; e < kPer; e += 2) dst[e / 2] = any ? pack2<BF16>(x[e] * f, x[e + 1] * f) : 0u;
    if (lane == 0) p.lse[row] = any ? (top + log2f(sum)) * kLn2 : -INFINITY;
}

template <int D, bool Q8, bool BF16, int NT, bool SHORT>
cudaError_t launch_t(const GqaParams& p, cudaStream_t s) {
    using C = GqaCfg<D, Q8>;
    auto kern = fa_decode_gqa_kernel<D, Q8, BF16, NT, SHORT>;
    const int smem = C::kRingBytes + 1024 + (kGqaMaxSequences + 1) * 4;
    const cudaError_t e = allow_shared<kGqaKernelId<D, Q8, BF16, NT, SHORT>>(kern, smem);
    if (e != cudaSuccess) return e;
    if constexpr (SHORT)
        return launch_kernel_cluster(kern, dim3((unsigned)(p.B * p.Hk * p.q_blocks * kClusterCtas)),
                                     dim3(kWarps * 32), (size_t)C::kRingBytes + 1024, kClusterCtas, s, p);
    const int here = C::kRingBytes + 1024 + (p.B + 1) * 4;
    const dim3 grid((unsigned)(p.warps / kWarps * p.rounds));
    return p.early ? launch_kernel_early(kern, grid, dim3(kWarps * 32), (size_t)here, s, p)
                   : launch_kernel(kern, grid, dim3(kWarps * 32), (size_t)here, s, p);
}

template <int D, bool Q8, bool BF16>
cudaError_t launch_n(const GqaParams& p, cudaStream_t s) {
    if (p.short_step) return launch_t<D, Q8, BF16, 1, true>(p, s);
    return p.group <= 8 ? launch_t<D, Q8, BF16, 1, false>(p, s) : launch_t<D, Q8, BF16, 2, false>(p, s);
}

template <int D>
cudaError_t launch_d(const GqaParams& p, bool bf16, bool q8, cudaStream_t s) {
    if (q8) return bf16 ? launch_n<D, true, true>(p, s) : launch_n<D, true, false>(p, s);
    return bf16 ? launch_n<D, false, true>(p, s) : launch_n<D, false, false>(p, s);
}

template <int D, bool BF16>
cudaError_t launch_m(const MergeParams& p, cudaStream_t s) {
    // Eight warps per row while a wave of CTAs holds the rows, else a warp per row.
    if (p.rows <= 4 * kGqaSms)
        return launch_kernel_early(fa_merge_kernel<D, BF16, 8>, dim3((unsigned)p.rows), dim3(256), 0, s, p);
    return launch_kernel_early(fa_merge_kernel<D, BF16, 1>, dim3((unsigned)((p.rows + 7) / 8)), dim3(256), 0,
                               s, p);
}

}  // namespace

int gqa_q_rows(int group) { return group <= 8 ? 8 : 16; }

int gqa_warps(int B, int Hk, int group, int max_pages) {
    const long long q_blocks = (group + gqa_q_rows(group) - 1) / gqa_q_rows(group);
    const long long ctas = ((long long)B * Hk * q_blocks * max_pages + kWarps - 1) /
                           kWarps;
    return kWarps * (int)(ctas < 1 ? 1 : ctas < 4 * kGqaSms ? ctas : 4 * kGqaSms);
}

bool gqa_short(int B, int Hk, int group, int max_pages, int D, bool q8) {
    if (group > 8) return false;
    const long long units = (long long)B * Hk;
    return units <= (gqa_occupancy(D, q8, 1) == 4 ? 72 : 48) && max_pages <= (units < 32 ? 128 : 256);
}

int gqa_rounds(int B, int Hk, int group) {
    const long long units = (long long)B * Hk * ((group + gqa_q_rows(group) - 1) / gqa_q_rows(group));
    return units >= kGqaManyUnits ? 3 : 1;
}

int gqa_launched_warps(int B, int Hk, int group, int max_pages, int D, bool q8, int busy_sms) {
    const int per_sm = gqa_occupancy(D, q8, group <= 8 ? 1 : 2) * kWarps;
    const int warps = gqa_warps(B, Hk, group, max_pages);
    // Beside a kernel that holds busy_sms SMs: the warps that find room at once, if the step is so
    // short (16 pages a warp at most) that a second wave behind that kernel would be its tail
    // (28.5 -> 24.5 us for 64 sequences of up to 512 tokens beside a prefix of 4096 on 64 SMs).  All SMs
    // against those left, 64 sequences, 8 cache heads of 128, group 4: beside 4096 tokens, sequences of up to
    // 256 24.5 and 22.2 us, 512 29.5 and 27.7, 768 (over the limit) 34.3 and 33.9, 2048 56.0 and 58.3; beside
    // 8192, which leaves 24 SMs (most over the limit), 128 29.3 and 28.0, 256 31.1 and 40.9, 512 36.0 and 60.6.
    const int beside = (kGqaSms - busy_sms) * per_sm;
    const long long q_blocks = (group + gqa_q_rows(group) - 1) / gqa_q_rows(group);
    if (busy_sms > 0 && beside > 0 && (long long)B * Hk * q_blocks * max_pages <= 16LL * beside)
        return warps < beside ? warps : beside;
    return warps < kGqaSms * per_sm ? warps : kGqaSms * per_sm;
}

cudaError_t launch_decode_gqa(const GqaParams& p, int D, bool bf16, bool q8, cudaStream_t s) {
    return D == 64 ? launch_d<64>(p, bf16, q8, s) : launch_d<128>(p, bf16, q8, s);
}

cudaError_t launch_merge(const MergeParams& p, int D, bool bf16, cudaStream_t s) {
    if (D == 64) return bf16 ? launch_m<64, true>(p, s) : launch_m<64, false>(p, s);
    return bf16 ? launch_m<128, true>(p, s) : launch_m<128, false>(p, s);
}

}  // namespace fa
