// Shared-memory and tensor-memory layout of the tensor-core scan (ssm_tc.cu),
// host-callable so that a CPU program can replay its addresses.
#pragma once

#include <stdint.h>

#ifndef DL_HD
#ifdef __CUDACC__
#define DL_HD __host__ __device__
#else
#define DL_HD
#endif
#endif

namespace dl {
namespace stc {

constexpr int Q = 128;        // tokens of a chunk: the rows of every token operand
constexpr int R = 128;        // value rows of a block: one head's, or two heads' of 64
constexpr int PANEL = Q * 128;  // 128 rows of 64 bf16 under 128-byte swizzle
constexpr int THREADS = 768;
constexpr int SMEM_LIMIT = 227 * 1024;

// Byte of (row, 16-byte piece) of a tile of 64-column panels.
DL_HD inline constexpr int tile_off(int row, int piece) {
    return (piece >> 3) * PANEL + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
}

// x is held by quarters of a chunk: 32 tokens, two panels of 64 columns.
constexpr int XQ = 2 * 32 * 128;
DL_HD inline constexpr int xq_off(int row, int piece) {
    return (piece >> 3) * (XQ / 2) + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
}

// Byte of (row, 16-byte piece) of a warp's gate block: 32 rows of 16 columns under 32-byte swizzle.
DL_HD inline constexpr int gate_off(int row, int piece) { return row * 32 + ((piece ^ ((row >> 2) & 1)) << 4); }

// Per chunk and head, from the step sizes (floats): the base-2 log decay from
// the start of a token's 32 through token t, l; u = 2^(l at the end of its 32 tokens
// - l) dt; dt; w = exp(log decay behind the token, within the chunk) dt; the base-2
// log decays between blocks of 32 tokens; exp of the whole chunk's log decay.
// Sums over 32 tokens only, so that steps which forget all leave the weak steps
// of other blocks their accuracy.
struct Scal {
    static constexpr int L = 0, U = Q, DT = 2 * Q, W = 3 * Q, RB = 4 * Q, E = RB + 16, FLOATS = RB + 20;
    // Place of the log decay of the blocks behind block j and in front of block i > j,
    DL_HD static constexpr int between(int i, int j) { return RB + 4 * i + j; }
    // and of all blocks of the chunk in front of block i.
    DL_HD static constexpr int before(int i) { return RB + 5 * i; }
};

template <int DK, int NH, bool GATE>
struct Layout {
    static constexpr int KP = DK / 64;          // panels of b, c and the state
    static constexpr int CTILE = KP * PANEL, STILE = KP * PANEL;
    static constexpr int NXQ = GATE ? 8 : 11;  // quarters of x held: what fits at DK = 128
    static constexpr int C = 0, B = C + CTILE, S = B + 2 * CTILE, X = S + STILE, Z = X + NXQ * XQ;
    static constexpr int NF_CHUNKS = 3;
    static constexpr int NZ = 3, ZBLOCK = 32 * 32;  // gate blocks in flight for each of 8 warps
    static constexpr int SCAL = Z + (GATE ? 8 * NZ * ZBLOCK : 0);
    static constexpr int SCAL_BYTES = Scal::FLOATS * 4;                 // one head of one chunk
    static constexpr int NF = SCAL + 2 * NH * SCAL_BYTES;               // masks of tokens with no number: [chunks][4 warps][Q bits]
    static constexpr int BAR = NF + NF_CHUNKS * 16 * 4;
    static constexpr int N_BAR = 53 + 2 * NXQ;
    static constexpr int TSLOT = BAR + 8 * N_BAR, ABORT = TSLOT + 4, BYTES = ABORT + 12;
    static constexpr int REQUEST = BYTES + 1024;  // the kernel aligns its base to 1024
    static_assert(REQUEST <= SMEM_LIMIT, "shared memory of a block");
    static_assert(SCAL_BYTES % 16 == 0 && NF % 16 == 0 && BAR % 8 == 0, "alignment");
    DL_HD static constexpr int b(int i) { return B + i * CTILE; }
    DL_HD static constexpr int x(int i) { return X + i * XQ; }
    DL_HD static constexpr int z(int warp, int i) { return Z + (warp * NZ + i) * ZBLOCK; }
    DL_HD static constexpr int scal(int i, int h) { return SCAL + (i * NH + h) * SCAL_BYTES; }
};

// The kernel of segments' end states: three chunks of b and x, two of weights.
template <int DK, int NH>
struct EndLayout {
    static constexpr int KP = DK / 64, CTILE = KP * PANEL;
    static constexpr int ST = 3;  // chunks of b and x in flight
    static constexpr int B = 0, X = ST * CTILE, SCAL = X + ST * 4 * XQ, SCAL_BYTES = Q * 4;
    static constexpr int BAR = SCAL + 2 * NH * SCAL_BYTES, N_BAR = 30;
    static constexpr int TSLOT = BAR + 8 * N_BAR, ABORT = TSLOT + 4, BYTES = ABORT + 12;
    static constexpr int REQUEST = BYTES + 1024;
    static_assert(REQUEST <= SMEM_LIMIT, "shared memory of a block");
    DL_HD static constexpr int b(int i) { return B + i * CTILE; }
    DL_HD static constexpr int x(int i, int q) { return X + (4 * i + q) * XQ; }
    DL_HD static constexpr int scal(int i, int h) { return SCAL + (i * NH + h) * SCAL_BYTES; }
};

// Tensor-memory columns (fp32 words): the state [R x DK]; the scores C B^T
// [Q x Q], overwritten 16 columns at a time by the decayed scores as bf16
// pairs (8 columns of each of one or two heads); the outputs [Q x R]; the
// decayed addends of 16 tokens [R x 16] as bf16 pairs in up to three parts of 8
// columns, in five places used in turn (the kernel of end states, which has
// neither scores nor outputs, has eight from column 256 on).
constexpr int T_S = 0, T_G = 128, T_Y = 256, T_W = 384, T_COLS = 512, W_PLACE = 24, W_PLACES = 5;
// Columns of head h's decayed scores of tokens 16 k .. 16 k + 15.
DL_HD inline constexpr int p_col(int k, int h) { return T_G + 16 * k + 8 * h; }

}  // namespace stc
}  // namespace dl
