// Replays the tcgen05 scan's layout (ssm_tc_layout.h) on the CPU: every region of
// shared memory lies inside the block's request and apart from the others,
// swizzled tiles start where their pattern does, the swizzles are one-to-one, and
// the tensor-memory columns of the state, scores, outputs and addends are apart.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "ssm_tc_layout.h"

using namespace dl::stc;

static int failures = 0;
static void check(bool good, const char *what, int a, int b) {
    if (good) return;
    std::printf("%s (%d, %d)\n", what, a, b);
    ++failures;
}

struct Map {
    std::vector<char> used;
    explicit Map(int n) : used(n, 0) {}
    void take(int at, int bytes, int align, const char *what) {
        check(at >= 0 && at + bytes <= (int)used.size(), what, at, bytes);
        check(at % align == 0, "alignment", at, align);
        for (int i = at < 0 ? 0 : at; i < at + bytes && i < (int)used.size(); ++i) {
            if (used[i]) return check(false, what, at, i);
            used[i] = 1;
        }
    }
};

template <int DK, int NH, bool GATE>
static void scan() {
    using LY = Layout<DK, NH, GATE>;
    check(LY::REQUEST <= SMEM_LIMIT && LY::BYTES + 1023 <= LY::REQUEST, "request", LY::REQUEST, LY::BYTES);
    Map m(LY::BYTES);
    m.take(LY::C, LY::CTILE, 1024, "c");
    for (int i = 0; i < 2; ++i) m.take(LY::b(i), LY::CTILE, 1024, "b");
    m.take(LY::S, LY::STILE, 1024, "state");
    for (int i = 0; i < LY::NXQ; ++i) m.take(LY::x(i), XQ, 1024, "x");
    for (int w = 0; GATE && w < 8; ++w)
        for (int i = 0; i < LY::NZ; ++i) m.take(LY::z(w, i), LY::ZBLOCK, 256, "gate");
    for (int i = 0; i < 2; ++i)
        for (int h = 0; h < NH; ++h) m.take(LY::scal(i, h), Scal::FLOATS * 4, 16, "scalars");
    m.take(LY::NF, LY::NF_CHUNKS * 4 * Q / 8, 16, "masks");
    m.take(LY::BAR, 8 * LY::N_BAR, 8, "barriers");
    m.take(LY::TSLOT, 4, 4, "tensor-memory address");
    m.take(LY::ABORT, 4, 4, "abort");
    // a chunk's quarters are held together, and the next chunk's first with them
    check(LY::NXQ >= 5, "x places", LY::NXQ, 0);
}

template <int DK, int NH>
static void ends() {
    using LY = EndLayout<DK, NH>;
    check(LY::REQUEST <= SMEM_LIMIT && LY::BYTES + 1023 <= LY::REQUEST, "request", LY::REQUEST, LY::BYTES);
    Map m(LY::BYTES);
    for (int i = 0; i < LY::ST; ++i) {
        m.take(LY::b(i), LY::CTILE, 1024, "b");
        for (int q = 0; q < 4; ++q) m.take(LY::x(i, q), XQ, 1024, "x");
    }
    for (int i = 0; i < 2; ++i)
        for (int h = 0; h < NH; ++h) m.take(LY::scal(i, h), Q * 4, 16, "weights");
    m.take(LY::BAR, 8 * LY::N_BAR, 8, "barriers");
    m.take(LY::TSLOT, 4, 4, "tensor-memory address");
    m.take(LY::ABORT, 4, 4, "abort");
}

int main() {
    scan<64, 1, false>(), scan<64, 1, true>(), scan<64, 2, false>(), scan<64, 2, true>();
    scan<128, 1, false>(), scan<128, 1, true>(), scan<128, 2, false>(), scan<128, 2, true>();
    ends<64, 1>(), ends<64, 2>(), ends<128, 1>(), ends<128, 2>();
    {
        Map tile(2 * PANEL), quarter(XQ), gate(1024);
        for (int r = 0; r < Q; ++r)
            for (int p = 0; p < 16; ++p) tile.take(tile_off(r, p), 16, 16, "tile");
        for (int r = 0; r < 32; ++r) {
            for (int p = 0; p < 16; ++p) quarter.take(xq_off(r, p), 16, 16, "quarter of x");
            for (int p = 0; p < 2; ++p) gate.take(gate_off(r, p), 16, 16, "gate block");
        }
        // a quarter's rows lie as the same rows of a whole tile do (one 128-byte row each, 8-row pattern)
        for (int r = 0; r < Q; ++r)
            for (int p = 0; p < 8; ++p) check(tile_off(r, p) % 4096 == xq_off(r & 31, p), "row", r, p);
    }
    {
        Map t(T_COLS);
        t.take(T_S, 128, 1, "state");
        t.take(T_G, Q, 1, "scores");
        t.take(T_Y, R, 1, "outputs");
        for (int i = 0; i < W_PLACES; ++i) t.take(T_W + W_PLACE * i, W_PLACE, 1, "addends");
        Map p(Q);  // decayed scores over the scores they come from: 16 columns' worth each, both heads
        for (int k = 0; k < 8; ++k)
            for (int h = 0; h < 2; ++h) {
                p.take(p_col(k, h) - T_G, 8, 8, "decayed scores");
                check((p_col(k, h) - T_G) / 16 == k, "decayed scores of other tokens", k, h);
            }
        Map e(T_COLS);  // the kernel of end states
        e.take(T_S, 128, 1, "state");
        for (int i = 0; i < 8; ++i) e.take(256 + W_PLACE * i, W_PLACE, 1, "addends of end states");
    }
    std::printf(failures ? "%d failures\n" : "ok\n", failures);
    return failures != 0;
}
