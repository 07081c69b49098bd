// fa_host.h -- host-side helpers shared by the units that implement C entry points.
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/fa.h"
#include "fa_internal.h"
#include "fa_overlap.h"

namespace fa {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};
inline Range range(const void* p, size_t bytes) {
    uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + bytes};
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

// Device address of the status word of the current device (looked up once per device).
int* status_ptr();

// The limit of device-side waits (fa_set_wait_timeout_ns).
uint64_t wait_timeout_ns();

// Makes the current device's primary context current on the calling thread.
bool bind_context();

// A caller's strides, checked for the 16-byte rules (positive multiples of 8 elements, below
// 2^39 elements); a stride of 0 is accepted for a dimension of size 1 and replaced by 8.
bool take_strides(const fa_strides& in, int B, int H, Strides* out);

// Bytes from the first to one past the last element of a strided [B, H, L, D] 16-bit operand.
Range extent(const void* p, const Strides& s, int B, int H, int L, int D);

// The same layout: equal strides of the dimensions that have more than one entry.
inline bool same(const Strides& a, const Strides& b, int B, int H, int L) {
    return (B <= 1 || a.b == b.b) && (H <= 1 || a.h == b.h) && (L <= 1 || a.l == b.l);
}
// Parts of one packed tensor: the same layout, extents that overlap, no element in common.
inline bool packed_parts(const void* a, const Strides& sa, int Ha, const void* b, const Strides& sb, int Hb, int B,
                         int L, int D) {
    const intptr_t pa = reinterpret_cast<intptr_t>(a), pb = reinterpret_cast<intptr_t>(b);
    if (!same(sa, sb, B, Ha < Hb ? Ha : Hb, L)) return false;
    const long long h = Ha > 1 ? sa.h : sb.h;
    return pa < pb ? interleave_apart((pb - pa) / 2, B, Ha, Hb, L, D, sa.b, h, sa.l)
                   : interleave_apart((pa - pb) / 2, B, Hb, Ha, L, D, sa.b, h, sa.l);
}

// Tiled tensor map of up to 5 dimensions: sizes and box in elements, strides (of dimensions 1..)
// in bytes; elements past the sizes read as zeros.
bool make_tiled_map(CUtensorMap* m, CUtensorMapDataType type, const void* ptr, int rank,
                    const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                    CUtensorMapSwizzle swizzle);

// The armed trace events (fa_trace_next_call) around the index-th kernel of a call, and the
// process-wide launch counter.
cudaError_t trace_before(int index, cudaStream_t s);
cudaError_t trace_after(int index, cudaStream_t s);

// Enqueues one kernel through `launch`, bracketed by the armed trace events (if any).
template <typename F>
cudaError_t traced_launch(int index, cudaStream_t s, F&& launch) {
    cudaError_t e = trace_before(index, s);
    if (e != cudaSuccess) return e;
    e = launch();
    if (e != cudaSuccess) return e;
    return trace_after(index, s);
}

// Consumes the trace arming at the end of a public call, whatever its outcome.
struct TraceDisarm {
    ~TraceDisarm() { trace_disarm(); }
};

}  // namespace fa
