// CPU replay of csrc/seq_index.h: reads lines
//   n_seq T len seq_start[0] .. seq_start[n_seq]
// and prints, for every tile number of the launch (T / len + n_seq of them),
// the rows [first, last) the tile works on as "seq first last" (empty tiles
// print nothing), then "ends", the same for tiles that are not a sequence's
// last (numbered without gaps), with their number in the scan's workspace, and
// "end".
#include <cstdio>
#include <vector>

#include "seq_index.h"

int main() {
    int n, T, len;
    while (scanf("%d %d %d", &n, &T, &len) == 3) {
        std::vector<int> start(n + 1);
        for (int &s : start)
            if (scanf("%d", &s) != 1) return 1;
        const dl::SeqIdx q{start.data(), nullptr, nullptr, n, T, n};
        for (int tile = 0; tile < T / len + n; ++tile) {
            int in_seq = 0, s0, rows;
            const int i = dl::seq_of_tile(q, tile, len, in_seq);
            if (i < 0 || !dl::seq_range(q, i, s0, rows) || in_seq >= (rows + len - 1) / len) continue;
            const int t0 = in_seq * len, t1 = t0 + len < rows ? t0 + len : rows;
            printf("%d %d %d\n", i, s0 + t0, s0 + t1);
        }
        printf("ends\n");
        for (int tile = 0; tile < T / len; ++tile) {
            int in_seq = 0, s0, rows;
            const int i = dl::seq_of_tile(q, tile, len, in_seq, 0);
            if (i < 0 || !dl::seq_range(q, i, s0, rows) || in_seq >= dl::segs_of(rows, len) - 1) continue;
            printf("%d %d %d %d\n", i, s0 + in_seq * len, s0 + in_seq * len + len, dl::seg_base(s0, len) + in_seq);
        }
        printf("end %lld\n", dl::seg_count(T, len));
    }
    return 0;
}
