// Host check of interleave_apart against the elements themselves: layouts of packed tensors, which it
// must accept, and random sizes and strides, where it must never accept two operands that meet.
#include <cstdio>
#include <random>
#include <unordered_set>

#include "fa_overlap.h"

namespace {
using ll = long long;

bool meet(ll delta, int B, int Ha, int Hb, int L, int D, ll b, ll h, ll l) {
    std::unordered_set<ll> seen;
    for (int pass = 0; pass < 2; ++pass)
        for (int i = 0; i < B; ++i)
            for (int j = 0; j < (pass ? Hb : Ha); ++j)
                for (int k = 0; k < L; ++k)
                    for (int e = 0; e < D; ++e) {
                        const ll at = (pass ? delta : 0) + i * b + j * h + k * l + e;
                        if (!pass) seen.insert(at);
                        else if (seen.count(at)) return true;
                    }
    return false;
}
int fails = 0, apart = 0;
void expect(bool want, ll delta, int B, int Ha, int Hb, int L, int D, ll b, ll h, ll l) {
    if (fa::interleave_apart(delta, B, Ha, Hb, L, D, b, h, l) != want) {
        std::printf("expected %d: delta %lld, B %d, H %d and %d, L %d, D %d, strides %lld %lld %lld\n", want, delta, B,
                    Ha, Hb, L, D, b, h, l);
        ++fails;
    }
}
}  // namespace

int main() {
    const int D = 8, H = 3, L = 5, B = 2;
    for (int B1 : {1, B})
        for (int L1 : {1, L})
            for (int part : {1, 2}) {
                expect(true, part * H * D, B1, H, H, L1, D, 3 * L1 * H * D, D, 3 * H * D);      // [B,L,3,H,D]
                expect(true, part * H * L1 * D, B1, H, H, L1, D, 3 * H * L1 * D, L1 * D, D);    // [B,3,H,L,D]
                expect(true, part * L1 * H * D, B1, H, H, L1, D, 3 * L1 * H * D, D, H * D);     // [B,3,L,H,D]
                expect(true, part * B1 * H * L1 * D, B1, H, H, L1, D, H * L1 * D, L1 * D, D);   // [3,B,H,L,D]
                expect(true, part * D, B1, H, H, L1, D, L1 * H * 3 * D, 3 * D, H * 3 * D);      // [B,L,H,3,D]
            }
    expect(true, 4 * D, B, 4, 1, L, D, L * 6 * D, D, 6 * D);  // grouped heads of one row
    expect(true, 4 * D, B, 4, 1, 1, D, 6 * D, D, 1);          // a single row: its stride means nothing
    expect(false, 4 * D, B, 4, 3, L, D, L * 6 * D, D, 6 * D);  // ... that reach into the next row
    expect(false, 0, B, H, H, L, D, L * H * D, D, H * D);
    expect(false, H * D, B, H, H, L, D, L * H * D, D, H * D);  // shifted by one row
    std::mt19937 rng(7);
    auto in = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
    for (int i = 0; i < 300000; ++i) {
        const int b = in(1, 3), ha = in(1, 3), hb = in(1, 3), l = in(1, 3), d = in(1, 4);
        const ll sb = in(1, 40), sh = in(1, 40), sl = in(1, 40), delta = in(0, 60);
        if (!fa::interleave_apart(delta, b, ha, hb, l, d, sb, sh, sl)) continue;
        ++apart;
        if (meet(delta, b, ha, hb, l, d, sb, sh, sl)) {
            std::printf("accepted, but they meet: delta %lld, B %d, H %d and %d, L %d, D %d, strides %lld %lld %lld\n",
                        delta, b, ha, hb, l, d, sb, sh, sl);
            if (++fails > 10) break;
        }
    }
    if (apart < 10000) ++fails;
    std::printf("%d accepted of the random ones\n%s\n", apart, fails ? "FAILED" : "OK");
    return fails != 0;
}
