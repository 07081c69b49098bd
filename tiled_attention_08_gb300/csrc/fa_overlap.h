// fa_overlap.h -- whether strided operands share an element (host code, no CUDA).
#pragma once

#include <cstdint>

namespace fa {

// Two operands [B, Ha, L, D] and [B, Hb, L, D] of one packed tensor: contiguous rows of D, the same
// element strides b, h, l (> 0; of a dimension of size 1 they mean nothing), the second starting
// `delta` >= 0 elements behind the first.  True only if they have no element in common: their inner
// dimensions, up to some level, lie one behind the other in each step of the dimensions outside it,
// which are nested (each steps over all of the one inside it, so that two of their points are at
// least the innermost step apart).  Covers [B, L, parts, H, D] as well as [B, parts, H, L, D].
inline bool interleave_apart(long long delta, int B, int Ha, int Hb, int L, int D, long long b, long long h,
                             long long l) {
    struct Dim {
        long long stride;
        int first, second;
    } d[3] = {{b, B, B}, {h, Ha, Hb}, {l, L, L}}, t;
    int n = 0;
    for (int i = 0; i < 3; ++i)  // those that count, innermost first
        if (d[i].first > 1 || d[i].second > 1) {
            int at = n++;
            t = d[i];
            for (; at > 0 && d[at - 1].stride > t.stride; --at) d[at] = d[at - 1];
            d[at] = t;
        }
    long long first = D, second = D;  // elements from the first to behind the last, dimensions below k
    for (int k = 0; k <= n; ++k) {
        bool nested = true;
        for (int i = k; i + 1 < n; ++i) {
            const int most = d[i].first > d[i].second ? d[i].first : d[i].second;
            nested = nested && d[i + 1].stride / most >= d[i].stride;
        }
        if (nested && delta >= first && (k == n || delta + second <= d[k].stride)) return true;
        if (k < n) {
            first += (d[k].first - 1) * d[k].stride;
            second += (d[k].second - 1) * d[k].stride;
        }
    }
    return false;
}

}  // namespace fa
