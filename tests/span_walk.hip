// The walk of a tile over the sequences of a packed or dense batch (csrc/gdn2_layer.h), run on the
// host over tables read from stdin. Per line of input: seqlen total tile n, and with seqlen < 0 the
// n + 1 offsets. Prints every span as: tile i first end lo hi starts ends, and "." after a table.
#include <cstdio>
#include <vector>

#include "gdn2_layer.h"

int main() {
    int seqlen, total, tile, n;
    while (std::scanf("%d %d %d %d", &seqlen, &total, &tile, &n) == 4) {
        std::vector<int32_t> cu(n + 1);
        if (seqlen < 0)
            for (int32_t &v : cu)
                if (std::scanf("%d", &v) != 1) return 1;
        const gdn2::SeqMap m{seqlen < 0 ? cu.data() : nullptr, n, seqlen < 0 ? 0 : seqlen, total};
        for (int t0 = 0; t0 < total || t0 == 0; t0 += tile) {
            const int t1 = total - t0 < tile ? total : t0 + tile;
            const int i = gdn2::seq_search(m, t0, [&](int lo, int step, int hi) {
                int c = 0;
                for (int64_t l = 0; l < 64; ++l)
                    c += lo + l * step < hi && gdn2::seq_begin(m, static_cast<int>(lo + l * step)) < t0;
                return c;
            });
            gdn2::walk_spans(m, t0, t1, i, [&](const gdn2::Span &s) {
                std::printf("%d %d %d %d %d %d %d %d\n", t0 / tile, s.i, s.first, s.end, s.lo, s.hi,
                            s.starts, s.ends);
            });
        }
        std::printf(".\n");
    }
    return 0;
}
