// Index arithmetic of calls over ragged sequences and pool slots. Host-callable,
// so that the CPU tests replay what the kernels compute.
#pragma once

#ifndef DL_HD
#ifdef __CUDACC__
#define DL_HD __host__ __device__
#else
#define DL_HD
#endif
#endif

namespace dl {

// Which rows a call works on: sequences seq_start[i] .. seq_start[i + 1] of T
// rows (prompts), or row i alone (seq_start == nullptr: one token each), and
// the pool slot of each (slot == nullptr: slot i).
struct SeqIdx {
    const int *seq_start;
    const int *slot;
    int *status;
    int n_seq, T, P;
};

// Slot of sequence i, or -1.
DL_HD inline int seq_slot(const SeqIdx &q, int i) {
    const int s = q.slot ? q.slot[i] : i;
    return s >= 0 && s < q.P ? s : -1;
}
// First row and length of sequence i; false (and n = 0) if its bounds are bad.
DL_HD inline bool seq_range(const SeqIdx &q, int i, int &s0, int &n) {
    s0 = q.seq_start[i];
    const int s1 = q.seq_start[i + 1];
    const bool good = s0 >= 0 && s0 <= s1 && s1 <= q.T;
    n = good ? s1 - s0 : 0;
    return good;
}
// Ragged sequences cut into tiles of `len` rows, each from its own start, as
// one grid: sequence i takes tile numbers from seq_start[i] / len + i on. The
// next sequence's first number is at least ceil(n / len) further, so numbers
// never collide, and n_seq + T / len of them cover every sequence without the
// host knowing the lengths. Finds the sequence of a tile number and the tile
// in it; -1 for none.
DL_HD inline int seq_tile_base(const SeqIdx &q, int i, int len, int gap) {
    const int s = q.seq_start[i];
    return (s > 0 ? s : 0) / len + gap * i;
}
// gap 1: as above. gap 0: the numbers of tiles that are not a sequence's last
// (ceil(n / len) - 1 <= floor(n / len) of them, T / len in all): sequences of one
// tile share a number with the next one, which the search prefers.
DL_HD inline int seq_of_tile(const SeqIdx &q, int tile, int len, int &in_seq, int gap = 1) {
    int lo = -1, hi = q.n_seq - 1;
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (seq_tile_base(q, mid, len, gap) <= tile)
            lo = mid;
        else
            hi = mid - 1;
    }
    if (lo >= 0) in_seq = tile - seq_tile_base(q, lo, len, gap);
    return lo;
}

// Segments of `len` rows of a sequence that has more than one: their numbers in
// the scan's workspace start here. A sequence of n > len rows has at most
// 2 n / len of them, so numbers never collide, and 2 T / len + 1 suffice.
DL_HD inline int seg_base(int s0, int len) { return (int)((2LL * s0 + len - 1) / len); }
DL_HD inline long long seg_count(int T, int len) { return 2LL * T / len + 1; }
DL_HD inline int segs_of(int n, int len) { return (int)(((long long)n + len - 1) / len); }
// Tokens of a segment (a multiple of `chunk`), or 0 where sequences are not
// split. `units` blocks (of at most `sms` at a time, one per SM) walk a
// sequence's chunks in order, so few or uneven sequences leave the GPU idle;
// split, each segment's end state comes first (about 0.4 of a chunk's time
// each), then the segments run side by side. One sequence: as many segments as
// fill the GPU. Several, whose lengths the host does not know: segments of twice
// an SM's even share, which only a sequence well above it exceeds. Both
// need at least 4 chunks a segment, and to beat the longest sequence there can
// be, unsplit, by more than the two launches they cost (about 8 chunks).
DL_HD inline int seg_len_for(int T, int n_seq, long long units, int chunk, int sms) {
    const long long chunks = ((long long)T + chunk - 1) / chunk;
    long long len;
    if (n_seq == 1) {
        long long n = sms / units;
        if (n > chunks / 4) n = chunks / 4;
        if (n < 2) return 0;
        len = (chunks + n - 1) / n;
    } else {
        len = (2 * chunks * units + sms - 1) / sms;
        if (len < 4) len = 4;
    }
    if (10 * chunks <= 14 * len + 80) return 0;
    return (int)(len * chunk);
}

}  // namespace dl
