// fa_window_sched.h -- which key tiles see which query tiles under a sliding window with first
// tokens that stay visible (host and device).
//
// A query at position t sees key j iff 0 <= j <= t and (j > t - window or j < sinks).
#pragma once

namespace fa {

__host__ __device__ __forceinline__ int imin(int a, int b) { return a < b ? a : b; }
__host__ __device__ __forceinline__ int imax(int a, int b) { return a > b ? a : b; }

// Key tiles of 128 that some query at positions first .. last sees: 0 .. lead - 1 (first tokens) and
// lo .. hi - 1 (the window), lead <= lo <= hi.  The j-th of them is tile(j).
struct KeyTiles {
    int lead, lo, hi;
    __host__ __device__ __forceinline__ int count() const { return lead + hi - lo; }
    __host__ __device__ __forceinline__ int tile(int j) const { return j < lead ? j : lo + (j - lead); }
    __host__ __device__ __forceinline__ bool has(int kt) const { return kt < hi && (kt >= lo || kt < lead); }
};
// 1 <= window <= Lk, 0 <= sinks <= Lk, and Lq + Lk < 2^31 - 1024: no sum below passes 31 bits.
__host__ __device__ __forceinline__ KeyTiles key_tiles(int first, int last, int window, int sinks) {
    KeyTiles k = {0, 0, 0};
    if (last < 0) return k;
    k.hi = last / 128 + 1;
    k.lo = imax(first - window + 1, 0) / 128;
    k.lead = imin((sinks + 127) / 128, k.lo);
    return k;
}

// Whether some of the keys key0 .. key0 + n - 1 is hidden from some of the positions first .. last:
// behind one of them, or in front of its window and no first token.
__host__ __device__ __forceinline__ bool hides_later(int key0, int n, int first) {
    return key0 + n - 1 > first;
}
__host__ __device__ __forceinline__ bool hides_earlier(int key0, int n, int last, int window, int sinks) {
    return imax(key0, sinks) <= imin(last - window, key0 + n - 1);
}
// Whether all of them are hidden from all of the positions.
__host__ __device__ __forceinline__ bool hides_all(int key0, int n, int first, int last, int window, int sinks) {
    return key0 > last || (key0 + n - 1 <= first - window && key0 >= sinks);
}

// Query tiles lo .. hi - 1 of 128 rows (row i at position i + off, Lq rows) that see a key of key tile kt.
struct QueryTiles {
    int lo, hi;
};
__host__ __device__ __forceinline__ QueryTiles query_tiles(int kt, int Lq, int off, int window, int sinks) {
    const int first = imax(kt * 128 - off, 0);  // first row that sees the tile's first key
    int last = Lq - 1;
    if (kt * 128 >= sinks) last = imin(last, kt * 128 + 126 + window - off);
    QueryTiles q = {first / 128, 0};
    q.hi = last >= first ? last / 128 + 1 : q.lo;
    return q;
}

}  // namespace fa
