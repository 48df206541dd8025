// Selective state space scan over prompts on the tcgen05 tensor cores
// (bfloat16 inputs), in chunks of Q = 128 tokens.
//
// With l_t the log decay from a chunk's start through token t (a sum of dt A),
// the recurrence S <- exp(dt A) S + dt x b^T, y = S c is, over one chunk,
//
//   y_t   = sum_{s <= t} (c_t . b_s) exp(l_t - l_s) dt_s x_s  +  exp(l_t) S c_t
//   S'    = exp(l_end) S + sum_s (exp(l_end - l_s) dt_s x_s) b_s^T
//
// four matrix products of 128-row tiles, three of them per head:
//   G  = C B^T           [tokens x tokens], K = d_k
//   Y  = (C S^T) scaled by exp(l_t), + P X with P = G o decay, K = d_k and tokens
//   S' = exp(l_end) S + W^T B, W = X o weights, K = tokens
//
// What is rounded: x, b and c are bfloat16 and enter as they are. P and the
// state read by C S^T are rounded to bfloat16 once (at most 2^-8 of each term, as
// y itself): they are operands of a bf16 product, and y's own rounding hides most
// of it (y's mean error grows by an eighth). The addends W go in as three bfloat16
// parts (at most 2^-26 left), so that the state, accumulated and kept in fp32,
// keeps fp32's accuracy; two parts (2^-17) where the state is stored as bfloat16.
// Every exponent is <= 0: between blocks of 32 tokens the decay is split at the end
// of the earlier token's block, inside a block it is taken directly, and sums of
// log decays run over no more than a block (see Scal). The weights' exponents are
// sums from the chunk's end backwards, so a token's weight is as accurate as its
// own exponent is small.
//
// One block per (sequence, 128 value rows): one head's, or two heads' of 64
// that share b and c. It walks the chunks in order with S in tensor memory:
//   warps 0-3, 16-19  P from G, then y: read Y, + D x, gate, store (thread =
//                token row), half of the columns each
//   warps 4-7    S: to bfloat16 for C S^T and scaled in place for the next
//                update (thread = value row); then Y's scaling (thread = token)
//   warps 8-15   W from X, 16 tokens at a time, two sets of four warps in turn
//   warp 20      TMA: x two chunks ahead, b and c one
//   warp 21      issues the products: G, W^T B by 16 tokens, C S^T between them, P X
//   warps 22-23  step sizes and decays of a chunk (one head each), one ahead
// Each product's time at d_k = 128 is 512 cycles of the tensor pipe, W^T B three
// times that: 3100 a chunk in all. What the other warps issue is as much, so
// their loops are short (unrolled over a tile they waited for instructions five
// cycles for each one issued: 320 us where the loops took 234 us, before other
// changes). With every SM at work a chunk takes 6450 cycles (3.4 us; 3.7 in long
// runs, in which the clock falls to 1.73 GHz), bound by the chain from G over P to
// P X with y's epilogue behind it and by the issue slots; 10600 with a gate, 8700
// for two heads of 64, 12000 for two with a gate. 8 ragged prompts of 16263 tokens
// on 32 heads of 128 x 128, the longest of 40 chunks, take 153 us, where moving
// their bytes takes 47: 40 chunks, and 15 us for the first loads and the last stores.
// The kernels of end states and join, which find nothing to do there, are 12 more.
//
// What is not a number stays where the recurrence has it: products would
// spread it, as a weight of zero times NaN is NaN. Rows behind the segment are
// zeroed in X and B (after G, in which they reach only rows of y that are not
// stored); an x that is no finite number is zeroed in X (after W has
// taken it) and its row flagged, and y's owners of later rows add it back from
// global memory.
//
// Every wait is bounded (about 2 s, fault bit 0).
#include "launch.h"
#include "ssm_tc_layout.h"
#include "tc_scan.cuh"
#include "tensor_map.h"

namespace dl {

// Fault word of the tensor-core scan (bit 0: a bounded wait ran out).
__device__ unsigned int g_ssm_faults = 0;

namespace {

using namespace stc;


struct Args {
    SsmParams p;
    SeqIdx q;
    int seg_len;       // tokens of a segment (a multiple of Q)
    int units;         // blocks per segment
    // sequences of several segments, [segments, H, d_v, d_k] and [segments, H]: a
    // segment's own end state and log decay, then the state in front of it
    float *seg_state, *seg_decay;
};

enum Bar {
    C_FULL, C_FREE, B_FULL, B_FREE = B_FULL + 2, SC_FULL = B_FREE + 2,
    SC_FREE = SC_FULL + 2, Z_FULL = SC_FREE + 2, W_FULL = Z_FULL + 24, W_FREE = W_FULL + W_PLACES,
    S_READY = W_FREE + W_PLACES, G_DONE, P_READY, Y2_DONE, YS_READY, Y_DONE, Y_FREE, ST_DONE, DRAIN, X_FULL  // (then x's places' X_FREE)
};

__device__ __forceinline__ uint64_t globaltimer() {
    uint64_t t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}
// Wait for the phase of `bar` with parity `par`; gives up after about two
// seconds, or once another role has (*abort set). The long wait is a call: the
// roles' loops have to stay in the instruction caches together.
__device__ __noinline__ bool wait_long(uint64_t *bar, uint32_t par, volatile int *abort) {
    const uint64_t t0 = globaltimer();
    for (;;) {
        // (suspended for up to 20 us at a time, rather than spinning beside the other roles)
        if (tc::mbar_try_wait_for(bar, par, 20000u)) return true;
        if (*abort) return false;
        if (globaltimer() - t0 > 2000000000ull) {
            *abort = 1;
            atomicOr(&g_ssm_faults, 1u);
            return false;
        }
    }
}
__device__ __forceinline__ bool wait1(uint64_t *bar, uint32_t par, volatile int *abort) {
    return tc::mbar_try_wait(bar, par) || wait_long(bar, par, abort);
}
// The same for a whole warp, which leaves together.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t par, volatile int *abort) {
    return __all_sync(0xffffffffu, wait1(bar, par, abort));
}
// After giving up: wait (a tenth of a second at most) for copies or products in flight.
__device__ __forceinline__ void drain(uint64_t *bar, uint32_t par) {
    const uint64_t t0 = globaltimer();
    while (!tc::mbar_try_wait(bar, par) && globaltimer() - t0 < 100000000ull) {
    }
}

// Value rows of one block.
struct Rows {
    int h0, g, r0, col0;  // first head, its group, first row in the head, first column of x
    bool two;             // (heads of 64) the second head exists
};
template <int NH>
__device__ __forceinline__ Rows rows_of(const SsmParams &p, int u) {
    const int per = p.H / p.G;
    if constexpr (NH == 1) {
        const int tiles = p.dv / R, h = u / tiles, r0 = (u - h * tiles) * R;
        return {h, h / per, r0, h * p.dv + r0, false};
    } else {
        const int pairs = (per + 1) / 2, g = u / pairs, j = 2 * (u - g * pairs);
        return {g * per + j, g, 0, (g * per + j) * p.dv, j + 1 < per};
    }
}

// The lowest n bits of a word (none for n <= 0, all from 32 on).
__device__ __forceinline__ uint32_t low_bits(int n) {
    uint32_t r;
    asm("shl.b32 %0, %1, %2;" : "=r"(r) : "r"(0xffffffffu), "r"(max(n, 0)));  // (shifts clamp at 32)
    return ~r;
}
// 16 floats (bits) times f.
__device__ __forceinline__ void scale16(uint32_t (&v)[16], float f) {
    const uint64_t ff = pair(f, f);
#pragma unroll
    for (int j = 0; j < 16; j += 2) unpair(mul2(pair(v[j], v[j + 1]), ff), v[j], v[j + 1]);
}

// Four 8 x 8 tiles of 16-bit elements from shared memory, transposed.
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// 16 lanes x 8 columns: register 2 n holds lane (thread / 4), column 4 n + thread % 4,
// register 2 n + 1 the same of lane + 8.
__device__ __forceinline__ void tmem_st_16x8(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3])
                 : "memory");
}
// Folds a pair of bfloat16 into `acc`, which turns NaN if one of them is no finite number.
__device__ __forceinline__ void watch(uint32_t &acc, uint32_t pair) {
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(pair), "r"(0u));
}
__device__ __forceinline__ bool saw_no_number(uint32_t acc) { return (acc & 0x7fff7fffu) != 0; }

// W of a warp's 32 value rows and 16 tokens to tensor memory at `at`: x from its
// rows of a quarter (xt: the first of the tokens), the tokens' weights w. Each of
// the TERMS parts, 8 columns, holds the leading 8 bits of what the parts before
// it leave; CLEAN drops parts behind the first that are no finite numbers.
template <int TERMS, bool CLEAN>
__device__ __forceinline__ void convert_w(uint32_t at, uint32_t xt, const float *w, int quad, int lane, uint32_t &acc) {
    // this lane's row of the transposing loads: token (lane & 7) + 8 (lane >> 4),
    // 8 value rows (lane >> 3) & 1 of 16
    const int mtok = (lane & 7) + ((lane >> 4) << 3), mpiece = 4 * quad + ((lane >> 3) & 1);
    uint32_t xr[2][4];
#pragma unroll
    for (int half = 0; half < 2; ++half) ldmatrix4_trans(xr[half], xt + xq_off(mtok, mpiece + 2 * half));  // 16 value rows
    uint64_t ws[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) ws[j] = *reinterpret_cast<const uint64_t *>(w + 8 * j + 2 * (lane & 3));  // this lane's pair of 8 tokens
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t part[TERMS][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 2; ++q) {  // value rows lane / 4 and + 8
                uint64_t f = mul2(pair_bf(xr[half][2 * j + q]), ws[j]);
#pragma unroll
                for (int i = 0; i < TERMS; ++i) {
                    const uint32_t word = pack_bf2(f);
                    part[i][2 * j + q] = word;
                    if (i == 0) watch(acc, word);
                    if (i + 1 < TERMS) f = fma2(pair_bf(word), pair(-1.f, -1.f), f);
                    if constexpr (CLEAN) {
                        float f0, f1;
                        unpair(f, f0, f1);
                        f = pair(fabsf(f0) <= 3.4e38f ? f0 : 0.f, fabsf(f1) <= 3.4e38f ? f1 : 0.f);
                    }
                }
            }
#pragma unroll
        for (int i = 0; i < TERMS; ++i) tmem_st_16x8(at + ((uint32_t)(16 * half) << 16) + 8 * i, part[i]);
    }
}

// 16 columns of a state row.
__device__ __forceinline__ void store_row16(float *p, const uint32_t (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; i += 4) *reinterpret_cast<uint4 *>(p + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
__device__ __forceinline__ uint4 pack8(const uint32_t *v) {  // floats' bits
    const float *f = reinterpret_cast<const float *>(v);
    return make_uint4(pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3]), pack_bf2(f[4], f[5]), pack_bf2(f[6], f[7]));
}
__device__ __forceinline__ void store_row16(bf16 *p, const uint32_t (&v)[16]) {
    reinterpret_cast<uint4 *>(p)[0] = pack8(v);
    reinterpret_cast<uint4 *>(p)[1] = pack8(v + 8);
}

// Tile k of at most 32 sequences taken from the longest to the shortest (by a
// whole warp): its sequence, or -1, and the segment in it. Blocks start in this
// order, so the short ones fill in behind the long ones. (Prompts of 17 to 5000
// tokens on 32 heads: 153 us; 182 in the sequences' own order.)
__device__ __forceinline__ int tile_by_length(const SeqIdx &q, int k, int len, int lane, int &seg) {
    int s0, n = -1, first = 0;
    if (lane < q.n_seq) seq_range(q, lane, s0, n);
    const int segs = n > 0 ? segs_of(n, len) : 0;
    for (int j = 0; j < q.n_seq; ++j) {
        const int n_j = __shfl_sync(0xffffffffu, n, j), segs_j = __shfl_sync(0xffffffffu, segs, j);
        if (n_j > n || (n_j == n && j < lane)) first += segs_j;
    }
    const unsigned mine = __ballot_sync(0xffffffffu, first <= k && k < first + segs);
    if (!mine) return -1;
    const int i = __ffs(mine) - 1;
    seg = k - __shfl_sync(0xffffffffu, first, i);
    return i;
}

// Step sizes and decays of a chunk of one head, by one warp: lane = token of each 32.
struct Steps {
    // dt_raw of tokens lane, 32 + lane, ..: this chunk's, and the next one's on its way (as
    // loaded: a conversion would wait for it)
    float raw[4];
    unsigned short ahead[4];
    // Rows row0 + ..; tokens at or behind `m` get no step.
    __device__ __forceinline__ void fetch(const dl_ssm &in, long long row0, int h, int lane, int m) {
#pragma unroll
        for (int j = 0; j < 4; ++j) raw[j] = bf_lo(ahead[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            ahead[j] = 32 * j + lane < m ? static_cast<const unsigned short *>(in.dt)[(row0 + 32 * j + lane) * in.dt_stride + h] : 0;
    }
    // Every value of the chunk, before the place for it is free.
    float dt[4], l[4], u[4], w[4], end;
    // `behind`: log decay behind the chunk that the weights take in as well.
    __device__ __forceinline__ void compute(float bias, float A, int lane, int m, float behind) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = 32 * j + lane < m;  // (no decay behind the segment: 0 A is no number for an A of -inf)
            dt[j] = in ? softplus_f(raw[j] + bias) : 0.f;
            // (a step of e^-128 is 0 in fp32 as any stronger one is; kept there, sums over 32
            // tokens stay within 4096, and the exponential of a difference of two is off by
            // at most 2^-10 behind any number of such steps: a quarter of a bf16 rounding)
            l[j] = w[j] = in ? max_nan(dt[j] * A, -128.f) : 0.f;
        }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1)
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // sums over the 32 tokens from the front (l) and from behind (w)
                const float a = __shfl_up_sync(0xffffffffu, l[j], off), b = __shfl_down_sync(0xffffffffu, w[j], off);
                if (lane >= off) l[j] += a;
                if (lane + off < 32) w[j] += b;
            }
        end = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float all = __shfl_sync(0xffffffffu, l[j], 31);
            u[j] = expf(all - l[j]) * dt[j];
            end += all;
        }
#pragma unroll
        for (int j = 3; j >= 0; --j) {  // behind: of the 32 tokens
            const float own = __shfl_down_sync(0xffffffffu, w[j], 1), all = __shfl_sync(0xffffffffu, w[j], 0);
            w[j] = expf(lane < 31 ? own + behind : behind) * dt[j];
            behind += all;
        }
    }
    __device__ __forceinline__ void write(float *sc, int lane) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sc[Scal::DT + 32 * j + lane] = dt[j];
            sc[Scal::L + 32 * j + lane] = l[j] * LOG2E;
            sc[Scal::U + 32 * j + lane] = u[j];
            sc[Scal::W + 32 * j + lane] = w[j];
        }
        // lane 4 i + j: blocks behind j and in front of i; lane 5 i: all in front of i
        const int i = lane >> 2, j = lane % 4 == i ? -1 : lane & 3;
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const float all = __shfl_sync(0xffffffffu, l[k], 31);
            if (k > j && k < i) sum += all;
        }
        if (lane < 16) sc[Scal::RB + lane] = sum * LOG2E;
        if (lane == 31) sc[Scal::E] = expf(end);
    }
};

// Adds to row t of y what flagged rows s <= t of x that hold no finite numbers
// make of it (see the top); rare, so from global memory.
__device__ __noinline__ void add_no_numbers(const SsmParams &p, long long row0, int t, const uint32_t *masks, const float *sc,
                                            int h, int g, int r0, int cols) {
    const dl_ssm &in = p.in;
    const bf16 *x = static_cast<const bf16 *>(in.x) + (long long)h * p.dv + r0;
    const bf16 *c = static_cast<const bf16 *>(in.c) + (row0 + t) * in.c_stride + (long long)g * p.dk;
    bf16 *y = static_cast<bf16 *>(p.y) + ((row0 + t) * p.H + h) * p.dv + r0;
    for (int s = 0; s <= t; ++s) {
        uint32_t any = 0;
        for (int w = 0; w < 4; ++w) any |= masks[4 * w + (s >> 5)];
        if (!((any >> (s & 31)) & 1)) continue;
        const bf16 *b = static_cast<const bf16 *>(in.b) + (row0 + s) * in.b_stride + (long long)g * p.dk;
        float f = 0.f;
        for (int e = 0; e < p.dk; ++e) f = fmaf(to_f(c[e]), to_f(b[e]), f);
        float l = sc[Scal::L + t] - sc[Scal::L + s];
        if ((t ^ s) >> 5) l += sc[Scal::between(t >> 5, s >> 5)] + sc[Scal::L + (s | 31)];  // of different 32 tokens
        f *= exp2f(l) * sc[Scal::DT + s];
        if (s == t && in.D) f += in.D[h];
        for (int e = 0; e < cols; ++e) {
            const float v = to_f(x[(row0 + s) * in.x_stride + e]);
            if (fabsf(v) <= 3.4e38f) continue;
            float add = f * v;
            if (in.z) add *= silu_f<bf16>(to_f(static_cast<const bf16 *>(in.z)[(row0 + t) * in.z_stride + (long long)h * p.dv + r0 + e]));
            y[e] = __float2bfloat16_rn(to_f(y[e]) + add);
        }
    }
}

template <class ST, int DK, int NH, bool GATE>
__global__ void __launch_bounds__(THREADS, 1)
ssm_tc_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_b,
              const __grid_constant__ CUtensorMap map_c, const __grid_constant__ CUtensorMap map_y,
              const __grid_constant__ CUtensorMap map_z, const __grid_constant__ Args a) {
    using LY = Layout<DK, NH, GATE>;
    constexpr int X_FREE = X_FULL + LY::NXQ, BARS = X_FREE + LY::NXQ;
    static_assert(LY::N_BAR == BARS && BARS <= 128, "barriers");
    // parts of the addends: 24 bits under an fp32 state, 16 under a bfloat16 one
    constexpr int TERMS = sizeof(ST) == 4 ? 3 : 2;
    extern __shared__ uint8_t smem_raw[];
    // (aligned by an offset: a pointer made from an integer would be read with generic loads)
    uint8_t *sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + LY::BAR);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + LY::TSLOT);
    volatile int *abort = reinterpret_cast<volatile int *>(sm + LY::ABORT);
    // (from a shuffle, so that the compiler knows them alike in a warp: a product
    // whose operands it must first move to uniform registers takes 120 cycles to
    // issue instead of its 64)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const SsmParams &p = a.p;
    const dl_ssm &in = p.in;

    const long long gid = (long long)blockIdx.x * THREADS + tid;
    if (gid < a.q.n_seq) seq_check(a.q, (int)gid);
    // the block's segment and value rows
    const int tile = (int)(blockIdx.x / (unsigned)a.units);
    const Rows rw = rows_of<NH>(p, (int)(blockIdx.x - (unsigned)tile * a.units));
    int seg = 0, s0, n;
    const int i = a.q.n_seq <= 32 ? tile_by_length(a.q, tile, a.seg_len, lane, seg) : seq_of_tile(a.q, tile, a.seg_len, seg);
    if (i < 0 || !seq_range(a.q, i, s0, n)) return;
    const int slot = seq_slot(a.q, i);
    const int segs = segs_of(n, a.seg_len);
    if (slot < 0 || seg >= segs) return;
    const int len = min(a.seg_len, n - seg * a.seg_len);  // this segment's tokens, from row0
    const int row0 = s0 + seg * a.seg_len, chunks = (len + Q - 1) / Q;

    if (tid < BARS) {  // (a thread each, and each once: a second init of a live barrier is undefined)
        const int b = tid;
        const bool four = b == S_READY || b == YS_READY || (b >= W_FULL && b < W_FREE), eight = b == P_READY || b == Y_FREE;
        const bool sc_full = b >= SC_FULL && b < SC_FREE, sc_free = b >= SC_FREE && b < Z_FULL, two = b == Y_DONE || b >= X_FREE;
        tc::mbar_init(&bars[b], four ? 4 : eight ? 8 : sc_full ? NH : sc_free ? 20 : two ? 2 : 1);
        if (b == 0) *abort = 0;
        tc::mbar_init_fence();
    }
    if (warp == 21) {
        tc::tmem_alloc(tslot, T_COLS);
        tc::tmem_relinquish();
    }
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tb = __shfl_sync(0xffffffffu, *tslot, 0);
    // the state in front of the segment, DK / 4 columns of a row a thread of the first 16 warps
    if (warp < 16) {
        const int r = 32 * (warp & 3) + lane, h = NH == 2 ? r >> 6 : 0, col = (warp >> 2) * (DK / 4);
        const long long srow = (long long)(rw.h0 + h) * p.dv + rw.r0 + (NH == 2 ? r & 63 : r);
        float f[DK / 4];
#pragma unroll
        for (int j = 0; j < DK / 4; ++j) f[j] = 0.f;
        if (h == 0 || rw.two) {
            if (segs > 1)
                load_vec<DK / 4>(a.seg_state + ((long long)(seg_base(s0, a.seg_len) + seg) * p.H * p.dv + srow) * DK + col, f);
            else
                load_vec<DK / 4>(static_cast<const ST *>(p.S) + ((long long)slot * p.H * p.dv + srow) * DK + col, f);
        }
#pragma unroll
        for (int k = 0; k < DK / 64; ++k) {
            uint32_t v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(f[16 * k + j]);
            tc::tmem_st16(tb + ((uint32_t)(32 * (warp & 3)) << 16) + T_S + col + 16 * k, v);
        }
        tc::tmem_wait_st();
        tc::tc_fence_before();
    }
    __syncthreads();
    tc::tc_fence_after();
    auto scal = [&](int c, int h) { return reinterpret_cast<float *>(sm + LY::scal(c & 1, h)); };
    auto arrive = [&](int b) {  // once per warp, after every lane's writes
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars[b]);
    };

    if (warp < 4 || (warp >= 16 && warp < 20)) {
        // ------------------------------------------------ P from G, and y (thread = token row t), half of the columns
        const int quad = warp & 3, half = warp >> 4, t = 32 * quad + lane;
        const uint32_t trow = tb + ((uint32_t)(32 * quad) << 16);
        const int yh = rw.h0 + (NH == 2 ? half : 0), ycol = rw.r0 + (NH == 2 ? 0 : 64 * half);  // head and column of this half
        const bool live = NH == 1 || half == 0 || rw.two;
        const float D = in.D && live ? in.D[yh] : 0.f;
        const uint64_t DD = pair(D, D);
        // the gate of the warp's rows: blocks of 16 columns, four a chunk, three in flight
        int nz = 0;
        const int zslot = 4 * half + quad;
        auto load_z = [&]() {
            if (GATE && lane == 0 && nz < 4 * chunks) {
                uint64_t *full = &bars[Z_FULL + 3 * zslot + nz % 3];
                tc::mbar_arrive_expect_tx(full, LY::ZBLOCK);
                tc::tma_load_2d(sm + LY::z(zslot, nz % 3), &map_z, rw.col0 + 64 * half + 16 * (nz & 3),
                                row0 + (nz >> 2) * Q + 32 * quad, full);
                ++nz;
            }
        };
        if constexpr (GATE)
            for (int k = 0; k < 3; ++k) load_z();
        for (int c = 0; c < chunks; ++c) {
            const uint32_t par = c & 1, par2 = (c >> 1) & 1;
            if (!wait_warp(&bars[SC_FULL + par], par2, abort)) break;
            if (!wait_warp(&bars[G_DONE], par, abort)) break;
            tc::tc_fence_after();
            uint32_t r0[16], r1[16];  // 16 columns each, one being loaded
            tc::tmem_ld16(trow + T_G + 16 * half, r0);
            float lth[NH];
#pragma unroll
            for (int h = 0; h < NH; ++h) lth[h] = scal(c, h)[Scal::L + t];
            // P of tokens 16 k .. 16 k + 15 from their scores
            auto decayed = [&](int k, const uint32_t (&g)[16], bool diagonal) {
                uint32_t pw[8];
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const float *sc = scal(c, h);
                    const float lt = lth[h];
                    if (!diagonal) {
                        const float v = ex2_ftz(lt + sc[Scal::between(quad, k >> 1)]);
                        const uint64_t vv = pair(v, v);
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(sc + Scal::U + 16 * k + e);
                            pw[e / 2] = pack_bf2(mul2(pair(g[e], g[e + 1]), mul2(u.x, vv)));
                            pw[e / 2 + 1] = pack_bf2(mul2(pair(g[e + 2], g[e + 3]), mul2(u.y, vv)));
                        }
                    } else {  // tokens up to t: those bits of the packed words
                        const int upto = 16 * (t + 1 - 16 * k);
                        const uint64_t ll = pair(lt, lt);
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            float x0, x1;
                            unpair(fma2(*reinterpret_cast<const uint64_t *>(sc + Scal::L + 16 * k + e), pair(-1.f, -1.f), ll), x0, x1);
                            const uint64_t f = mul2(pair(ex2_ftz(x0), ex2_ftz(x1)),
                                                    *reinterpret_cast<const uint64_t *>(sc + Scal::DT + 16 * k + e));
                            pw[e / 2] = pack_bf2(mul2(pair(g[e], g[e + 1]), f)) & low_bits(upto - 16 * e);
                        }
                    }
                    tc::tmem_st8(trow + p_col(k, h), pw);
                }
            };
            // (of each 32 tokens, the 16 of this half)
#pragma unroll 1
            for (int kb = 0; kb <= quad; kb += 2) {
                tc::tmem_wait_ld();
                if (kb < quad) tc::tmem_ld16(trow + T_G + 32 * kb + 32 + 16 * half, r1);
                decayed(2 * kb + half, r0, kb == quad);
                if (kb == quad) break;
                tc::tmem_wait_ld();
                if (kb + 1 < quad) tc::tmem_ld16(trow + T_G + 32 * kb + 64 + 16 * half, r0);
                decayed(2 * kb + 2 + half, r1, kb + 1 == quad);
            }
#pragma unroll 1
            for (int k = 2 * quad + 2 + half; k < 8; k += 2) {  // tokens behind every t of the warp
                uint32_t zero[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
                for (int h = 0; h < NH; ++h) tc::tmem_st8(trow + p_col(k, h), zero);
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
            arrive(P_READY);
            if (c > 0) {  // the previous chunk's stores have read x's place: it may be loaded again
                if (lane == 0) tc::bulk_wait_read<0>();
                arrive(X_FREE + (4 * (c - 1) + quad) % LY::NXQ);
            }

            // y of row t: Y + D x, gated; through x's place in shared memory to
            // HBM by TMA, or straight from registers where the warp's 32 rows
            // reach behind the segment (or x holds what is no number)
            const int m = min(Q, len - c * Q);
            const long long row = (long long)row0 + c * Q + t;
            // z / (1 + exp(-z)) of 16 value columns; the first before Y is there
            uint64_t gate[GATE ? 8 : 1];
            auto load_gate = [&](int k) {
                const int zi = 4 * c + k;
                if (!wait_warp(&bars[Z_FULL + 3 * zslot + zi % 3], (zi / 3) & 1, abort)) return false;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint4 z = *reinterpret_cast<const uint4 *>(sm + LY::z(zslot, zi % 3) + gate_off(lane, j));
                    const uint32_t zw[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) gate[GATE ? 4 * j + e : 0] = silu2<bf16>(pair_bf(zw[e]));
                }
                __syncwarp();
                load_z();
                return true;
            };
            if (GATE && !load_gate(0)) break;
            if (!wait_warp(&bars[Y_DONE], par, abort)) break;
            tc::tc_fence_after();
            tc::tmem_ld16(trow + T_Y + 64 * half, r0);
            const uint4 *nf = reinterpret_cast<const uint4 *>(sm + LY::NF) + 4 * (c % LY::NF_CHUNKS);
            uint32_t any = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) any |= nf[j].x | nf[j].y | nf[j].z | nf[j].w;
            const bool direct = any || 32 * quad + 32 > m;
            uint8_t *xp = sm + LY::x((4 * c + quad) % LY::NXQ) + half * (XQ / 2);  // the warp's 32 rows of x
            const uint32_t swz = (t & 7) << 4;
            auto x_at = [&](int k, int j) {  // 8 of 16 value columns
                return reinterpret_cast<uint4 *>(xp + lane * 128 + ((32 * k + 16 * j) ^ swz));
            };
            auto columns = [&](int k, const uint32_t (&y)[16], const uint4 &x0, const uint4 &x1) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint4 xv = j ? x1 : x0;
                    const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
                    uint32_t ow[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint64_t o = fma2(DD, pair_bf(xw[e]), pair(y[8 * j + 2 * e], y[8 * j + 2 * e + 1]));
                        if constexpr (GATE) o = mul2(o, gate[4 * j + e]);
                        ow[e] = pack_bf2(o);
                    }
                    const uint4 out = make_uint4(ow[0], ow[1], ow[2], ow[3]);
                    if (!direct)
                        *x_at(k, j) = out;
                    else if (t < m && live)
                        reinterpret_cast<uint4 *>(static_cast<bf16 *>(p.y) + (row * p.H + yh) * p.dv + ycol)[2 * k + j] = out;
                }
            };
            if constexpr (GATE) {
                bool ok = true;
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {  // 16 value columns each
                    const uint4 xa = *x_at(k, 0), xb = *x_at(k, 1);
                    tc::tmem_wait_ld();
                    columns(k, r0, xa, xb);
                    if (k == 3) break;
                    tc::tmem_ld16(trow + T_Y + 64 * half + 16 * k + 16, r0);
                    if (!(ok = load_gate(k + 1))) break;
                }
                if (!ok) break;
            } else {
#pragma unroll 1
                for (int k = 0; k < 4; k += 2) {
                    const uint4 xa = *x_at(k, 0), xb = *x_at(k, 1), xc = *x_at(k + 1, 0), xd = *x_at(k + 1, 1);
                    tc::tmem_wait_ld();
                    tc::tmem_ld16(trow + T_Y + 64 * half + 16 * k + 16, r1);
                    columns(k, r0, xa, xb);
                    tc::tmem_wait_ld();
                    if (k == 0) tc::tmem_ld16(trow + T_Y + 64 * half + 32, r0);
                    columns(k + 1, r1, xc, xd);
                }
            }
            tc::tc_fence_before();
            arrive(Y_FREE);
            if (!direct) {
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0 && live) {
                    tc::tma_store_2d(&map_y, rw.col0 + 64 * half, row0 + c * Q + 32 * quad, xp);
                    tc::bulk_commit();
                }
            } else if (any && t < m && live) {
                add_no_numbers(p, (long long)row0 + c * Q, t, reinterpret_cast<const uint32_t *>(nf), scal(c, NH == 2 ? half : 0), yh,
                               rw.g, ycol, 64);
            }
            arrive(SC_FREE + par);
        }
        if (lane == 0) {  // the warp's last copies have landed
            tc::bulk_wait_all();
            for (int k = 0; GATE && k < 3; ++k) {
                const int n = (nz + 2 - k) / 3;
                if (n) drain(&bars[Z_FULL + 3 * zslot + k], (n - 1) & 1);
            }
        }
    } else if (warp < 8) {
        // ------------------------------------------------ S (thread = value row r), and Y's scaling (thread = token row r)
        const int quad = warp & 3, r = 32 * quad + lane, h = NH == 2 ? r >> 6 : 0;
        const uint32_t trow = tb + ((uint32_t)(32 * quad) << 16);
        const bool live = h == 0 || rw.two;
        const long long srow = (long long)(rw.h0 + h) * p.dv + rw.r0 + (NH == 2 ? r & 63 : r);
        ST *S = static_cast<ST *>(p.S) + ((long long)slot * p.H * p.dv + srow) * DK;
        bool ok = true;
        for (int c = 0; c < chunks; ++c) {
            const uint32_t par = c & 1, par2 = (c >> 1) & 1;
            if (!(ok = wait_warp(&bars[SC_FULL + par], par2, abort))) break;
            const float e = scal(c, h)[Scal::E];
            if (c > 0) {
                if (!(ok = wait_warp(&bars[ST_DONE], (c - 1) & 1, abort))) break;
                tc::tc_fence_after();
            }
            uint32_t r0[16], r1[16];  // 16 columns each, one being loaded
            // 16 key columns: rounded for C S^T, and decayed by this chunk
            auto advance = [&](int k, uint32_t (&v)[16]) {
                uint8_t *dst = sm + LY::S + (k >> 2) * PANEL + r * 128;
                *reinterpret_cast<uint4 *>(dst + (((32 * k) & 127) ^ ((r & 7) << 4))) = pack8(v);
                *reinterpret_cast<uint4 *>(dst + (((32 * k + 16) & 127) ^ ((r & 7) << 4))) = pack8(v + 8);
                scale16(v, e);
                tc::tmem_st16(trow + T_S + 16 * k, v);
            };
            tc::tmem_ld16(trow + T_S, r0);
#pragma unroll 1
            for (int k = 0; k < DK / 16; k += 2) {
                tc::tmem_wait_ld();
                tc::tmem_ld16(trow + T_S + 16 * k + 16, r1);
                advance(k, r0);
                tc::tmem_wait_ld();
                if (k + 2 < DK / 16) tc::tmem_ld16(trow + T_S + 16 * k + 32, r0);
                advance(k + 1, r1);
            }
            tc::fence_async_smem();
            tc::tmem_wait_st();
            tc::tc_fence_before();
            arrive(S_READY);

            float ex[NH];
#pragma unroll
            for (int k = 0; k < NH; ++k)  // (from r: an index kept in a register of its own spilled others, 161 -> 174 us)
                ex[k] = ex2_ftz(scal(c, k)[Scal::L + r] + scal(c, k)[Scal::before(r >> 5)]);
            arrive(SC_FREE + par);
            if (!(ok = wait_warp(&bars[Y2_DONE], par, abort))) break;
            tc::tc_fence_after();
            tc::tmem_ld16(trow + T_Y, r0);
            auto scale = [&](int k, uint32_t (&v)[16]) {
                scale16(v, NH == 2 && k >= 4 ? ex[NH - 1] : ex[0]);
                tc::tmem_st16(trow + T_Y + 16 * k, v);
            };
#pragma unroll 1
            for (int k = 0; k < 8; k += 2) {
                tc::tmem_wait_ld();
                tc::tmem_ld16(trow + T_Y + 16 * k + 16, r1);
                scale(k, r0);
                tc::tmem_wait_ld();
                if (k + 2 < 8) tc::tmem_ld16(trow + T_Y + 16 * k + 32, r0);
                scale(k + 1, r1);
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
            arrive(YS_READY);
        }
        if (ok && wait_warp(&bars[ST_DONE], (chunks - 1) & 1, abort) && seg == segs - 1) {
            tc::tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < DK / 16; ++k) {
                uint32_t v[16];
                tc::tmem_ld16(trow + T_S + 16 * k, v);
                tc::tmem_wait_ld();
                if (live) store_row16(S + 16 * k, v);
            }
            tc::tc_fence_before();
        }
    } else if (warp < 16) {
        // ------------------------------------------------ W from X (a warp's 32 value rows), every other 16 tokens
        const int quad = warp & 3, set = (warp - 8) >> 2, r = 32 * quad + lane, h = NH == 2 ? r >> 6 : 0;
        const uint32_t trow = tb + ((uint32_t)(32 * quad) << 16);
        uint16_t *nf = reinterpret_cast<uint16_t *>(sm + LY::NF) + 8 * quad;
        bool ok = true;
        for (int c = 0; ok && c < chunks; ++c) {
            const uint32_t par = c & 1, par2 = (c >> 1) & 1;
            const int m = min(Q, len - c * Q);
            if (!wait_warp(&bars[SC_FULL + par], par2, abort)) break;
            // (the last chunk: b has come, and the scores have been formed from it, before its rows behind the segment are zeroed)
            if (m < Q && !(wait_warp(&bars[B_FULL + par], par2, abort) && wait_warp(&bars[G_DONE], par, abort))) break;
            const float *w = scal(c, h) + Scal::W;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {  // 32 tokens, this set's 16 of them
                const int nx = 4 * c + q, nw = 2 * nx + set, place = nw % W_PLACES, first = 32 * q + 16 * set;
                uint8_t *xt = sm + LY::x(nx % LY::NXQ);
                if (!(ok = wait_warp(&bars[X_FULL + nx % LY::NXQ], (uint32_t)(nx / LY::NXQ) & 1, abort))) break;
                if (first + 16 > m) {  // (the last chunk) zeros behind the segment, in X and B
                    constexpr int BP = DK / 32;  // pieces of a row of b for each warp
                    for (int k = lane; k < 16 * (4 + BP); k += 32) {
                        const int row = first + k / (4 + BP), pc = k % (4 + BP);
                        uint8_t *dst = pc < 4 ? xt + xq_off(row & 31, 4 * quad + pc) : sm + LY::b(par) + tile_off(row, BP * quad + pc - 4);
                        if (row >= m) *reinterpret_cast<uint4 *>(dst) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    tc::fence_async_smem();
                    __syncwarp();
                }
                if (nw >= W_PLACES) {  // the update that used this place has read it
                    if (!(ok = wait_warp(&bars[W_FREE + place], (uint32_t)(nw / W_PLACES - 1) & 1, abort))) break;
                    tc::tc_fence_after();
                }
                uint32_t acc = 0u, mask = 0u;
                const uint32_t at = trow + T_W + W_PLACE * place, x16 = tc::smem_u32(xt) + 16 * 128 * set;
                convert_w<TERMS, false>(at, x16, w + first, quad, lane, acc);
                if (__any_sync(0xffffffffu, saw_no_number(acc))) {
                    // again, without later parts that are no numbers; then x's own zeroed
                    convert_w<TERMS, true>(at, x16, w + first, quad, lane, acc);
                    for (int s = 0; s < 16; ++s) {
                        bf16 *xp = reinterpret_cast<bf16 *>(xt + xq_off(16 * set + s, r >> 3) + (r & 7) * 2);
                        if (!(fabsf(to_f(*xp)) <= 3.4e38f)) {
                            *xp = __float2bfloat16_rn(0.f);
                            mask |= 1u << s;
                        }
                    }
                    mask = __reduce_or_sync(0xffffffffu, mask);
                    tc::fence_async_smem();
                }
                if (lane == 0) nf[32 * (c % LY::NF_CHUNKS) + 2 * q + set] = (uint16_t)mask;
                if (q == 3) arrive(SC_FREE + par);
                tc::tmem_wait_st();
                tc::tc_fence_before();
                arrive(W_FULL + place);
            }
        }
    } else if (warp == 20) {
        // ------------------------------------------------ loads
        if (lane == 0) {
            tc::tma_prefetch_desc(&map_x);
            tc::tma_prefetch_desc(&map_b);
            tc::tma_prefetch_desc(&map_c);
            auto load = [&](const CUtensorMap *map, int off, int panels, int bytes, int col, int row, uint64_t *full) {
                tc::mbar_arrive_expect_tx(full, panels * bytes);
                for (int k = 0; k < panels; ++k) tc::tma_load_2d(sm + off + k * bytes, map, col + 64 * k, row, full);
            };
            // whatever has a free place, b first; given up on as the waits are
            int nb = 0, nx = 0, nc = 0;  // copies issued
            uint64_t t0 = globaltimer();
            while (nb < chunks || nc < chunks || nx < 4 * chunks) {
                const int before = nb + nc + nx;
                if (nb < chunks && (nb < 2 || tc::mbar_try_wait(&bars[B_FREE + (nb & 1)], (uint32_t)((nb >> 1) - 1) & 1))) {
                    load(&map_b, LY::b(nb & 1), LY::KP, PANEL, rw.g * DK, row0 + nb * Q, &bars[B_FULL + (nb & 1)]);
                    ++nb;
                }
                if (nc < chunks && (nc < 1 || tc::mbar_try_wait(&bars[C_FREE], (uint32_t)(nc - 1) & 1))) {
                    load(&map_c, LY::C, LY::KP, PANEL, rw.g * DK, row0 + nc * Q, &bars[C_FULL]);
                    ++nc;
                }
                const int xp = nx % LY::NXQ;
                if (nx < 4 * chunks && (nx < LY::NXQ || tc::mbar_try_wait(&bars[X_FREE + xp], (uint32_t)(nx / LY::NXQ - 1) & 1))) {
                    load(&map_x, LY::x(xp), R / 64, XQ / 2, rw.col0, row0 + nx * 32, &bars[X_FULL + xp]);
                    ++nx;
                }
                const uint64_t now = globaltimer();
                if (nb + nc + nx > before) {
                    t0 = now;
                } else if (*abort || now - t0 > 2000000000ull) {
                    if (!*abort) atomicOr(&g_ssm_faults, 1u);
                    *abort = 1;
                    break;
                } else {
                    __nanosleep(40);
                }
            }
            // every copy has landed before the block may leave
            if (nb) drain(&bars[B_FULL + ((nb - 1) & 1)], (uint32_t)((nb - 1) >> 1) & 1);
            if (nb > 1) drain(&bars[B_FULL + (nb & 1)], (uint32_t)((nb - 2) >> 1) & 1);
            if (nc) drain(&bars[C_FULL], (uint32_t)(nc - 1) & 1);
            for (int k = 0; k < LY::NXQ; ++k) {
                const int x = (nx + LY::NXQ - 1 - k) / LY::NXQ;  // copies into place k
                if (x) drain(&bars[X_FULL + k], (x - 1) & 1);
            }
        }
        __syncwarp();
    } else if (warp == 21) {
        // ------------------------------------------------ products
        {
            const uint32_t lead = tc::elect_one() ? 1u : 0u;
            const int n_chunks = __shfl_sync(0xffffffffu, chunks, 0);
            constexpr uint32_t ID_G = tc::instr_desc(tc::FMT_BF16, false, false, Q, Q);
            constexpr uint32_t ID_Y2 = tc::instr_desc(tc::FMT_BF16, false, false, Q, R);
            constexpr uint32_t ID_Y1 = tc::instr_desc(tc::FMT_BF16, false, true, Q, R / NH);
            constexpr uint32_t ID_S = tc::instr_desc(tc::FMT_BF16, false, true, R, DK);
            // descriptors of the tiles' first 16 columns (K along the columns: the
            // tile's rows are the product's rows or columns), and of the first 16
            // rows (K along the rows: its columns are the product's columns); those
            // of the others differ by a constant (in 16-byte units)
            auto kmajor = [&](int off) { return tc::smem_desc(tc::smem_u32(sm + off), 16, 1024, tc::SWZ_128); };
            auto nmajor = [&](int off, int panel) { return tc::smem_desc(tc::smem_u32(sm + off), panel, 1024, tc::SWZ_128); };
            constexpr uint64_t COLS = 32 / 16, PANELS = PANEL / 16, ROWS = 16 * 128 / 16;
            const uint64_t ck = kmajor(LY::C), sk = kmajor(LY::S);
            const uint64_t bk = kmajor(LY::B), bn = nmajor(LY::B, PANEL), xn = nmajor(LY::X, XQ / 2);
            constexpr uint64_t NEXT_B = LY::CTILE / 16, NEXT_X = XQ / 16;
            bool ok = true;
            for (int c = 0; c < n_chunks; ++c) {
                const uint32_t par = c & 1, par2 = (c >> 1) & 1;
                // A B^T over DK columns of two tiles
                auto over_columns = [&](uint32_t d, uint64_t ad, uint64_t bd, uint32_t id) {
#pragma unroll
                    for (int pn = 0; pn < LY::KP; ++pn)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc::mma_ss_f16_by(lead, d, ad + pn * PANELS + k * COLS, bd + pn * PANELS + k * COLS, id, pn + k > 0);
                };
                // S' of 16 tokens g ..
                auto update = [&](int from, int to) {
#pragma unroll 1
                    for (int g = from; g < to; ++g) {
                        const int nw = 8 * c + g, place = nw % W_PLACES;
                        if (!wait_warp(&bars[W_FULL + place], (uint32_t)(nw / W_PLACES) & 1, abort)) return false;
                        tc::tc_fence_after();
#pragma unroll
                        for (int i = 0; i < TERMS; ++i)
                            tc::mma_ts_f16_by(lead, tb + T_S, tb + T_W + W_PLACE * place + 8 * i, bn + par * NEXT_B + g * ROWS, ID_S, true);
                        tc::mma_commit_by(lead, &bars[W_FREE + place]);
                    }
                    return true;
                };
                if (!(ok = wait_warp(&bars[C_FULL], par, abort) && wait_warp(&bars[B_FULL + par], par2, abort))) break;
                // the previous chunk's P X has read P, which lies in G's columns: products with
                // different accumulators are not ordered by their issue (they share one pipe: no time lost)
                if (!(ok = c == 0 || wait_warp(&bars[Y_DONE], (c - 1) & 1, abort))) break;
                tc::tc_fence_after();
                over_columns(tb + T_G, ck, bk + par * NEXT_B, ID_G);
                tc::mma_commit_by(lead, &bars[G_DONE]);
                if (!(ok = wait_warp(&bars[S_READY], par, abort) && update(0, W_PLACES))) break;
                if (!(ok = c == 0 || wait_warp(&bars[Y_FREE], (c - 1) & 1, abort))) break;
                tc::tc_fence_after();
                over_columns(tb + T_Y, ck, sk, ID_Y2);
                tc::mma_commit_by(lead, &bars[Y2_DONE]);
                tc::mma_commit_by(lead, &bars[C_FREE]);
                if (!(ok = update(W_PLACES, 8))) break;
                tc::mma_commit_by(lead, &bars[ST_DONE]);
                tc::mma_commit_by(lead, &bars[B_FREE + par]);
                // (a commit speaks for products only: this arrival passes on x and its flags, of
                // which the addends' barriers told, to the warps that wait for y)
                tc::mbar_arrive_by(lead, &bars[Y_DONE]);
                if (!(ok = wait_warp(&bars[P_READY], par, abort) && wait_warp(&bars[YS_READY], par, abort))) break;
                tc::tc_fence_after();
#pragma unroll
                for (int q = 0; q < 4; ++q) {  // (32 tokens of x)
                    const uint64_t xd = xn + (uint64_t)((4 * c + q) % LY::NXQ) * NEXT_X;
#pragma unroll
                    for (int h = 0; h < NH; ++h)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            tc::mma_ts_f16_by(lead, tb + T_Y + (R / NH) * h, tb + p_col(2 * q + k, h), xd + h * (XQ / 32) + k * ROWS, ID_Y1,
                                           true);
                }
                tc::mma_commit_by(lead, &bars[Y_DONE]);
            }
            if (!ok) {  // products in flight have completed before tensor memory is freed
                tc::mma_commit_by(lead, &bars[DRAIN]);
                drain(&bars[DRAIN], 0);
            }
        }
        __syncwarp();
    } else if (warp >= 22 && warp < 22 + NH) {
        // ------------------------------------------------ step sizes and decays of head h
        const int h = warp - 22;
        const bool live = h == 0 || rw.two;
        const float A = live ? in.A[rw.h0 + h] : 0.f, bias = live && in.dt_bias ? in.dt_bias[rw.h0 + h] : 0.f;
        Steps st;
        st.fetch(in, row0, rw.h0 + h, lane, live ? len : 0);
        for (int c = 0; c < chunks; ++c) {
            const int m = live ? len - c * Q : 0;
            st.fetch(in, (long long)row0 + (c + 1) * Q, rw.h0 + h, lane, m - Q);
            st.compute(bias, A, lane, m, 0.f);
            if (c >= 2 && !wait_warp(&bars[SC_FREE + (c & 1)], (uint32_t)((c >> 1) - 1) & 1, abort)) break;
            st.write(scal(c, h), lane);
            arrive(SC_FULL + (c & 1));
        }
    }
    __syncthreads();
    if (warp == 21) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tb, T_COLS);
    }
}

// The end state of every segment but a sequence's last, from a state of zero,
// and its log decay: the scan's state products alone, over the chunks from the
// last to the first, so that each token's weight takes in the decay behind its
// chunk and the state needs no scaling. Three parts always: what is summed here
// reaches the last state.
constexpr int END_THREADS = 640;  // 16 warps on W, three chunks ahead of the products: what bounds this is W

template <int DK, int NH>
__global__ void __launch_bounds__(END_THREADS, 1)
ssm_tc_ends_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ Args a) {
    using LY = EndLayout<DK, NH>;
    constexpr int TERMS = 3;
    enum { B_FULL, FREE = B_FULL + LY::ST, X_FULL = FREE + LY::ST, SC_FULL = X_FULL + LY::ST, SC_FREE = SC_FULL + 2, W_FULL = SC_FREE + 2,
           W_FREE = W_FULL + 8, DONE = W_FREE + 8, BARS };  // (a place of W for each 16 tokens of a chunk)
    constexpr int T_W8 = 256;
    static_assert(LY::N_BAR == BARS && BARS <= 128, "barriers");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + LY::BAR);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + LY::TSLOT);
    volatile int *abort = reinterpret_cast<volatile int *>(sm + LY::ABORT);
    // (from a shuffle, so that the compiler knows them alike in a warp: a product
    // whose operands it must first move to uniform registers takes 120 cycles to
    // issue instead of its 64)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const SsmParams &p = a.p;
    const dl_ssm &in = p.in;

    const int tile = (int)(blockIdx.x / (unsigned)a.units);
    const Rows rw = rows_of<NH>(p, (int)(blockIdx.x - (unsigned)tile * a.units));
    int seg = 0, s0, n;
    const int i = seq_of_tile(a.q, tile, a.seg_len, seg, 0);
    if (i < 0 || !seq_range(a.q, i, s0, n)) return;
    if (seq_slot(a.q, i) < 0 || seg >= segs_of(n, a.seg_len) - 1) return;
    const int row0 = s0 + seg * a.seg_len, chunks = a.seg_len / Q;
    const long long out = (long long)seg_base(s0, a.seg_len) + seg;

    if (tid < BARS) {
        const int b = tid;
        const bool sc_full = b >= SC_FULL && b < SC_FREE, sc_free = b >= SC_FREE && b < W_FULL, w_full = b >= W_FULL && b < W_FREE;
        tc::mbar_init(&bars[b], sc_full ? NH : sc_free ? 16 : w_full ? 4 : b >= FREE && b < X_FULL ? 2 : 1);
        if (b == 0) *abort = 0;
        tc::mbar_init_fence();
    }
    if (warp == 17) {
        tc::tmem_alloc(tslot, T_COLS);
        tc::tmem_relinquish();
    }
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tb = __shfl_sync(0xffffffffu, *tslot, 0);
    auto weights = [&](int c, int h) { return reinterpret_cast<float *>(sm + LY::scal(c & 1, h)); };
    auto arrive = [&](int b) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars[b]);
    };

    if (warp < 16) {
        // ------------------------------------------------ W, 16 of each 64 tokens; the end state (thread = value row r)
        const int quad = warp & 3, set = warp >> 2, r = 32 * quad + lane, h = NH == 2 ? r >> 6 : 0;
        const uint32_t trow = tb + ((uint32_t)(32 * quad) << 16);
        bool ok = true;
        for (int c = 0; ok && c < chunks; ++c) {
            const uint32_t par = c & 1, par2 = (c >> 1) & 1;
            const int k = c % LY::ST;
            if (!(ok = wait_warp(&bars[X_FULL + k], (uint32_t)(c / LY::ST) & 1, abort) && wait_warp(&bars[SC_FULL + par], par2, abort)))
                break;
            const float *w = weights(c, h);
#pragma unroll 1
            for (int g = set; g < 8; g += 4) {  // 16 tokens
                if (c > 0) {
                    if (!(ok = wait_warp(&bars[W_FREE + g], (uint32_t)(c - 1) & 1, abort))) break;
                    tc::tc_fence_after();
                }
                uint32_t acc = 0u;
                const uint32_t at = trow + T_W8 + W_PLACE * g, x16 = tc::smem_u32(sm + LY::x(k, g >> 1)) + 16 * 128 * (g & 1);
                convert_w<TERMS, false>(at, x16, w + 16 * g, quad, lane, acc);
                if (__any_sync(0xffffffffu, saw_no_number(acc))) convert_w<TERMS, true>(at, x16, w + 16 * g, quad, lane, acc);
                if (g >= 4) arrive(SC_FREE + par);
                tc::tmem_wait_st();
                tc::tc_fence_before();
                arrive(W_FULL + g);
            }
        }
        if (ok && set == 0 && wait_warp(&bars[DONE], 0, abort) && (h == 0 || rw.two)) {
            tc::tc_fence_after();
            const long long srow = (long long)(rw.h0 + h) * p.dv + rw.r0 + (NH == 2 ? r & 63 : r);
            float *dst = a.seg_state + (out * p.H * p.dv + srow) * DK;
#pragma unroll 1
            for (int k = 0; k < DK / 16; ++k) {
                uint32_t v[16];
                tc::tmem_ld16(trow + T_S + 16 * k, v);
                tc::tmem_wait_ld();
                store_row16(dst + 16 * k, v);
            }
            tc::tc_fence_before();
        }
    } else if (warp == 16) {
        // ------------------------------------------------ loads, from the last chunk
        if (lane == 0) {
            tc::tma_prefetch_desc(&map_x);
            tc::tma_prefetch_desc(&map_b);
            int issued = 0;
            for (int c = 0; c < chunks; ++c) {
                const int k = c % LY::ST, row = row0 + (chunks - 1 - c) * Q;
                if (c >= LY::ST && !wait1(&bars[FREE + k], (uint32_t)(c / LY::ST - 1) & 1, abort)) break;
                tc::mbar_arrive_expect_tx(&bars[X_FULL + k], 4 * XQ);
                for (int q = 0; q < 4; ++q)
                    for (int j = 0; j < R / 64; ++j)
                        tc::tma_load_2d(sm + LY::x(k, q) + j * (XQ / 2), &map_x, rw.col0 + 64 * j, row + 32 * q, &bars[X_FULL + k]);
                tc::mbar_arrive_expect_tx(&bars[B_FULL + k], LY::CTILE);
                for (int j = 0; j < LY::KP; ++j)
                    tc::tma_load_2d(sm + LY::b(k) + j * PANEL, &map_b, rw.g * DK + 64 * j, row, &bars[B_FULL + k]);
                ++issued;
            }
            for (int k = 0; k < LY::ST; ++k) {
                const int m = (issued + LY::ST - 1 - k) / LY::ST;
                if (m) {
                    drain(&bars[B_FULL + k], (m - 1) & 1);
                    drain(&bars[X_FULL + k], (m - 1) & 1);
                }
            }
        }
        __syncwarp();
    } else if (warp == 17) {
        // ------------------------------------------------ products
        {
            const uint32_t lead = tc::elect_one() ? 1u : 0u;
            const int n_chunks = __shfl_sync(0xffffffffu, chunks, 0);
            constexpr uint32_t ID_S = tc::instr_desc(tc::FMT_BF16, false, true, R, DK);
            constexpr uint64_t ROWS = 16 * 128 / 16;
            bool ok = true;
            for (int c = 0; ok && c < n_chunks; ++c) {
                const uint32_t par = c & 1, k = c % LY::ST;
                const uint64_t bd = tc::smem_desc(tc::smem_u32(sm + LY::b(k)), PANEL, 1024, tc::SWZ_128);
                if (!(ok = wait_warp(&bars[B_FULL + k], (uint32_t)(c / LY::ST) & 1, abort))) break;
#pragma unroll 1
                for (int g = 0; g < 8; ++g) {
                    if (!(ok = wait_warp(&bars[W_FULL + g], par, abort))) break;
                    tc::tc_fence_after();
#pragma unroll
                    for (int i = 0; i < TERMS; ++i)
                        tc::mma_ts_f16_by(lead, tb + T_S, tb + T_W8 + W_PLACE * g + 8 * i, bd + g * ROWS, ID_S, c + g + i > 0);
                    tc::mma_commit_by(lead, &bars[W_FREE + g]);
                }
                if (ok) {
                    tc::mma_commit_by(lead, &bars[FREE + k]);
                    tc::mbar_arrive_by(lead, &bars[FREE + k]);  // (W of the chunk has been made, so x has been read too)
                }
            }
            tc::mma_commit_by(lead, &bars[DONE]);
            if (!ok) drain(&bars[DONE], 0);
        }
        __syncwarp();
    } else if (warp - 18 < NH) {
        // ------------------------------------------------ weights of head h, from the last chunk
        const int h = warp - 18;
        const bool live = h == 0 || rw.two;
        const float A = live ? in.A[rw.h0 + h] : 0.f, bias = live && in.dt_bias ? in.dt_bias[rw.h0 + h] : 0.f;
        const int m = live ? Q : 0;
        float behind = 0.f;
        Steps st;
        st.fetch(in, (long long)row0 + (chunks - 1) * Q, rw.h0 + h, lane, m);
        bool ok = true;
        for (int c = 0; c < chunks; ++c) {
            st.fetch(in, (long long)row0 + (chunks - 2 - c) * Q, rw.h0 + h, lane, c + 1 < chunks ? m : 0);
            st.compute(bias, A, lane, m, behind);
            behind += st.end;
            if (c >= 2 && !(ok = wait_warp(&bars[SC_FREE + (c & 1)], (uint32_t)((c >> 1) - 1) & 1, abort))) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) weights(c, h)[32 * j + lane] = st.w[j];
            arrive(SC_FULL + (c & 1));
        }
        if (ok && live && rw.r0 == 0 && lane == 0) a.seg_decay[out * p.H + rw.h0 + h] = behind;
    }
    __syncthreads();
    if (warp == 17) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tb, T_COLS);
    }
}

// Segments' own end states -> the states in front of them, in place: a thread
// takes four elements of one sequence's state through its segments.
template <class ST>
__global__ void __launch_bounds__(256) ssm_join_kernel(const SsmParams p, const SeqIdx q, const SsmSegs g, long long quads_per_seq) {
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    int seg = 0, s0, n;
    const int i = seq_of_tile(q, (int)blockIdx.y, g.len, seg, 0);
    if (i < 0 || seg != 0 || id >= quads_per_seq) return;
    const int slot = seq_slot(q, i);
    if (!seq_range(q, i, s0, n) || slot < 0) return;
    const int segs = segs_of(n, g.len);
    if (segs < 2) return;
    const long long at = id * 4, per = quads_per_seq * 4;
    const int h = (int)(at / ((long long)p.dv * p.dk));
    const long long base = seg_base(s0, g.len);
    float s[4];
    load_vec<4>(static_cast<const ST *>(p.S) + slot * per + at, s);
    float4 *e = reinterpret_cast<float4 *>(g.state + base * per + at);
    const float *dec = g.decay + base * p.H + h;
    constexpr int AHEAD = 6;  // segments whose loads are in flight
    for (int j0 = 0; j0 < segs; j0 += AHEAD) {
        float4 own[AHEAD];
        float d[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (j0 + j + 1 < segs) {
                own[j] = e[(j0 + j) * (per / 4)];
                d[j] = dec[(long long)(j0 + j) * p.H];
            }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            if (j0 + j >= segs) break;
            e[(j0 + j) * (per / 4)] = make_float4(s[0], s[1], s[2], s[3]);
            if (j0 + j + 1 == segs) break;
            const float f = expf(d[j]);
            s[0] = fmaf(s[0], f, own[j].x);
            s[1] = fmaf(s[1], f, own[j].y);
            s[2] = fmaf(s[2], f, own[j].z);
            s[3] = fmaf(s[3], f, own[j].w);
        }
    }
}

// A [rows, cols] bfloat16 matrix with a row stride, in boxes of box_rows rows of
// box_cols columns (64 with 128-byte swizzle, 16 with 32-byte).
cudaError_t row_map(CUtensorMap *m, const void *base, long long cols, long long rows, long long stride, int box_rows = Q, int box_cols = 64) {
    tc::EncodeTiledFn fn = tc::encoder();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    const cuuint32_t es[2] = {1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_32B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <class ST, int DK, int NH, bool GATE>
cudaError_t launch_typed(const SsmParams &p, const SeqIdx &q, const SsmSegs &g, bool split, cudaStream_t st) {
    using LY = Layout<DK, NH, GATE>;
    auto kern = ssm_tc_kernel<ST, DK, NH, GATE>;
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(kern), LY::REQUEST);
    if (e != cudaSuccess) return e;
    CUtensorMap mx, mb, mc, my, mz;
    const dl_ssm &in = p.in;
    if ((e = row_map(&mx, in.x, (long long)p.H * p.dv, q.T, in.x_stride, 32)) != cudaSuccess) return e;
    if ((e = row_map(&mb, in.b, (long long)p.G * DK, q.T, in.b_stride)) != cudaSuccess) return e;
    if ((e = row_map(&mc, in.c, (long long)p.G * DK, q.T, in.c_stride)) != cudaSuccess) return e;
    const long long yw = (long long)p.H * p.dv;
    if ((e = row_map(&my, p.y, yw, q.T, yw, 32)) != cudaSuccess) return e;
    mz = my;  // (not read without a gate)
    if (GATE && (e = row_map(&mz, in.z, yw, q.T, in.z_stride, 32, 16)) != cudaSuccess) return e;
    const int per = p.H / p.G;
    Args a{p, q, g.len, NH == 2 ? p.G * ((per + 1) / 2) : p.H * (p.dv / R), g.state, g.decay};
    const long long blocks = ((long long)q.T / a.seg_len + q.n_seq) * a.units;
    if (split) {
        using LE = EndLayout<DK, NH>;
        auto ends = ssm_tc_ends_kernel<DK, NH>;
        if ((e = allow_smem(reinterpret_cast<const void *>(ends), LE::REQUEST)) != cudaSuccess) return e;
        ends<<<(unsigned)(q.T / g.len) * (unsigned)a.units, END_THREADS, LE::REQUEST, st>>>(mx, mb, a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if ((e = launch_ssm_join(p, q, g, st)) != cudaSuccess) return e;
    }
    kern<<<(unsigned)blocks, THREADS, LY::REQUEST, st>>>(mx, mb, mc, my, mz, a);
    return cudaGetLastError();
}

}  // namespace

size_t ssm_work_bytes(int T, int n_seq, int H, int dk, int dv) {
    const int len = ssm_seg_len(T, n_seq, H, dv);
    return len ? (size_t)seg_count(T, len) * H * ((size_t)dv * dk + 1) * sizeof(float) : 0;
}

cudaError_t launch_ssm_join(const SsmParams &p, const SeqIdx &q, const SsmSegs &g, cudaStream_t st) {
    const long long quads = (long long)p.H * p.dv * p.dk / 4;
    const dim3 grid((unsigned)((quads + 255) / 256), (unsigned)(q.T / g.len));
    if (p.s_dt == DL_BF16)
        ssm_join_kernel<bf16><<<grid, 256, 0, st>>>(p, q, g, quads);
    else
        ssm_join_kernel<float><<<grid, 256, 0, st>>>(p, q, g, quads);
    return cudaGetLastError();
}

bool ssm_tc_supported(const SsmParams &p) { return p.in.dtype == DL_BF16 && tc::encoder() != nullptr; }

cudaError_t launch_ssm_tc(const SsmParams &p, const SeqIdx &q, const SsmSegs &g, bool split, cudaStream_t st) {
    auto with_nh = [&](auto s, auto dk) -> cudaError_t {
        using ST = decltype(s);
        constexpr int DK = decltype(dk)::value;
        if (p.in.z) return p.dv == 64 ? launch_typed<ST, DK, 2, true>(p, q, g, split, st) : launch_typed<ST, DK, 1, true>(p, q, g, split, st);
        return p.dv == 64 ? launch_typed<ST, DK, 2, false>(p, q, g, split, st) : launch_typed<ST, DK, 1, false>(p, q, g, split, st);
    };
    auto with_dk = [&](auto s) -> cudaError_t {
        return p.dk == 64 ? with_nh(s, std::integral_constant<int, 64>{}) : with_nh(s, std::integral_constant<int, 128>{});
    };
    return p.s_dt == DL_BF16 ? with_dk(bf16{}) : with_dk(float{});
}

cudaError_t read_ssm_faults(unsigned int *out, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_ssm_faults, sizeof(unsigned int));
    if (e == cudaSuccess && clear) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_ssm_faults, &zero, sizeof(unsigned int));
    }
    return e;
}

}  // namespace dl
