// CPU replay of csrc/seq_index.h: reads lines
//   n_seq T len seq_start[0] .. seq_start[n_seq]
// and prints, for every tile number of the launch (T / len + n_seq of them),
// the rows [first, last) the tile works on as "seq first last" (empty tiles
// print nothing), then "end" after each line of input.
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
        printf("end\n");
    }
    return 0;
}
