// Which tiles see which under a sliding window with first tokens, against the mask itself entry by entry.
#define __host__
#define __device__
#define __forceinline__ inline
#include "../../tiled_attention_08_gb300/csrc/fa_window_sched.h"

#include <cstdio>
#include <vector>

using namespace fa;

static bool sees(int t, int j, int w, int s) { return j >= 0 && j <= t && (j > t - w || j < s); }

int main() {
    long long checked = 0;
    const int lens[] = {1, 2, 127, 128, 129, 255, 256, 300, 513, 700};
    const int windows[] = {1, 2, 63, 127, 128, 129, 130, 255, 256, 257, 600, 1 << 30};
    const int sinks[] = {0, 1, 64, 127, 128, 129, 256, 400, 700};
    for (int Lq : lens)
        for (int Lk : lens)
            for (int w0 : windows)
                for (int s0 : sinks) {
                    const int off = Lk - Lq, s = s0 < Lk ? s0 : Lk, w = w0 < Lk ? w0 : Lk;
                    const int nq = (Lq + 127) / 128, nk = (Lk + 127) / 128;
                    std::vector<char> seen(nq * nk, 0);
                    for (int i = 0; i < Lq; ++i)
                        for (int j = 0; j < Lk; ++j)
                            if (sees(i + off, j, w, s)) seen[(i / 128) * nk + j / 128] = 1;
                    for (int qt = 0; qt < nq; ++qt) {
                        const int first = qt * 128 + off, last = (qt * 128 + 127 < Lq - 1 ? qt * 128 + 127 : Lq - 1) + off;
                        const KeyTiles k = key_tiles(first, last, w, s);
                        std::vector<int> times(nk, 0);
                        for (int j = 0; j < k.count(); ++j) {
                            const int kt = k.tile(j);
                            if (kt < 0 || kt >= nk || !k.has(kt) || ++times[kt] > 1)
                                return std::printf("key tile %d out of place\n", kt), 1;
                        }
                        for (int kt = 0; kt < nk; ++kt) {
                            if (k.has(kt) != (times[kt] == 1)) return std::printf("has(%d)\n", kt), 1;
                            if (seen[qt * nk + kt] && !times[kt]) return std::printf("key tile %d missing\n", kt), 1;
                            const QueryTiles q = query_tiles(kt, Lq, off, w, s);
                            if (q.lo < 0 || q.hi > nq || q.lo > q.hi) return std::printf("query range\n"), 1;
                            if (seen[qt * nk + kt] && !(q.lo <= qt && qt < q.hi))
                                return std::printf("query tile %d of key tile %d missing\n", qt, kt), 1;
                            // No tile without a visible entry but at the ragged ends of the lengths.
                            if (!seen[qt * nk + kt] && times[kt] && first >= 0 && kt < nk - 1 && kt >= k.lo)
                                return std::printf("key tile %d for nothing\n", kt), 1;
                            // The three questions about blocks of 32 keys and 32 positions.
                            for (int kb = 0; kb < 4; ++kb)
                                for (int qb = 0; qb < 4; ++qb) {
                                    const int j0 = kt * 128 + kb * 32, t0 = first + qb * 32;
                                    bool later = false, earlier = false, any = false;
                                    for (int j = j0; j < j0 + 32; ++j)
                                        for (int t = t0; t < t0 + 32; ++t) {
                                            later |= j > t;
                                            earlier |= j <= t - w && j >= s;
                                            any |= j <= t && (j > t - w || j < s);
                                        }
                                    if (later != hides_later(j0, 32, t0) ||
                                        earlier != hides_earlier(j0, 32, t0 + 31, w, s))
                                        return std::printf("edges at %d %d\n", j0, t0), 1;
                                    if (any && hides_all(j0, 32, t0, t0 + 31, w, s))
                                        return std::printf("hidden at %d %d\n", j0, t0), 1;
                                    ++checked;
                                }
                        }
                        // Two consecutive tiles together: nothing missing, each one's tiles among them.
                        if (qt + 1 < nq) {
                            const int last2 = (qt * 128 + 255 < Lq - 1 ? qt * 128 + 255 : Lq - 1) + off;
                            const KeyTiles u = key_tiles(first, last2, w, s), b = key_tiles(first + 128, last2, w, s);
                            for (int kt = 0; kt < nk; ++kt)
                                if ((k.has(kt) || b.has(kt)) != u.has(kt) && (k.count() > 0 || b.count() > 0) &&
                                    !(first < 0))
                                    return std::printf("pair: tile %d\n", kt), 1;
                            for (int kt = 0; kt < nk; ++kt)
                                if ((k.has(kt) || b.has(kt)) && !u.has(kt)) return std::printf("pair: %d lost\n", kt), 1;
                        }
                    }
                }
    std::printf("ok %lld\n", checked);
    return 0;
}
