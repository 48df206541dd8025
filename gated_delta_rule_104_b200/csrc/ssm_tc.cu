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
// state read by C S^T are rounded to bfloat16 once (2^-9 of each term, where y
// itself is rounded to 2^-9); the addends W go in as a high and a low bfloat16
// part (2^-18 of each term), so that the state, accumulated and kept in fp32,
// keeps fp32's accuracy. Every exponent is <= 0: between 32-token blocks the
// decay is split at the end of the earlier token's block, inside a block it is
// taken directly. The weights' exponents are sums from the chunk's end
// backwards, so a token's weight is as accurate as its own exponent is small.
//
// One block per (sequence, 128 value rows): one head's, or two heads' of 64
// that share b and c. It walks the chunks in order with S in tensor memory:
//   warps 0-3    P from G (thread = token row), then y: read Y, + D x, gate, store
//   warps 4-7    S: to bfloat16 for C S^T and scaled in place for the next
//                update (thread = value row); then Y's scaling (thread = token)
//   warps 8-11   W from X (thread = value row; x is read down a column)
//   warp 12      TMA: b and x two chunks ahead, c one
//   warp 13      issues the products: G, C S^T, W^T B, P X
//   warps 14-15  step sizes and decays of a chunk (one head each), one ahead
// Each product's time at d_k = 128 is 512 cycles of the tensor pipe, W^T B twice
// that: 2560 a chunk.
//
// What is not a number stays where the recurrence has it: products would
// spread it, as a weight of zero times NaN is NaN. Rows behind the segment are
// zeroed in X and B; an x that is no finite number is zeroed in X (after W has
// taken it) and its row flagged, and y's owners of later rows add it back from
// global memory.
//
// Every wait is bounded (about 2 s, fault bit 0).
#include "launch.h"
#include "ssm_tc_layout.h"
#include "tc.cuh"

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
    float *seg_state;  // [segments, H, d_v, d_k]: state in front of each segment (sequences of several)
};

enum Bar {
    C_FULL, C_FREE, B_FULL, B_FREE = B_FULL + 2, X_FULL = B_FREE + 2, X_FREE = X_FULL + 2, SC_FULL = X_FREE + 2,
    SC_FREE = SC_FULL + 2, S_READY = SC_FREE + 2, W_READY, G_DONE, P_READY, Y2_DONE, YS_READY, Y_DONE, Y_FREE, ST_DONE,
    ZEROED, DRAIN, BARS
};

__device__ __forceinline__ uint64_t globaltimer() {
    uint64_t t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}
// Wait for the phase of `bar` with parity `par`; gives up after about two
// seconds, or once another role has (*abort set).
__device__ __forceinline__ bool wait1(uint64_t *bar, uint32_t par, volatile int *abort) {
    if (tc::mbar_try_wait(bar, par)) return true;
    const uint64_t t0 = globaltimer();
    for (uint32_t i = 0;; ++i) {
        if (tc::mbar_try_wait(bar, par)) return true;
        if ((i & 63u) == 63u) {
            if (*abort) return false;
            if (globaltimer() - t0 > 2000000000ull) {
                *abort = 1;
                atomicOr(&g_ssm_faults, 1u);
                return false;
            }
        }
    }
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

__device__ __forceinline__ void load_row32(const float *p, float (&v)[32]) { load_vec<32>(p, v); }
__device__ __forceinline__ void load_row32(const bf16 *p, float (&v)[32]) { load_vec<32>(p, v); }
__device__ __forceinline__ void store_row32(float *p, const uint32_t (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 32; i += 4) *reinterpret_cast<uint4 *>(p + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
__device__ __forceinline__ void store_row32(bf16 *p, const uint32_t (&v)[32]) {
    const float *f = reinterpret_cast<const float *>(v);
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        *reinterpret_cast<uint4 *>(p + i) = make_uint4(pack_bf2(f[i], f[i + 1]), pack_bf2(f[i + 2], f[i + 3]),
                                                       pack_bf2(f[i + 4], f[i + 5]), pack_bf2(f[i + 6], f[i + 7]));
}

// Step sizes and decays of chunk tokens 4 lane .. 4 lane + 3 of one head, by one warp.
struct Steps {
    float raw[4];
    // dt_raw of rows row0 + 4 lane ..; tokens at or behind `m` get no step.
    __device__ __forceinline__ void fetch(const dl_ssm &in, long long row0, int h, int lane, int m) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            raw[j] = 4 * lane + j < m ? to_f(static_cast<const bf16 *>(in.dt)[(row0 + 4 * lane + j) * in.dt_stride + h]) : 0.f;
    }
    __device__ __forceinline__ void write(float *sc, float bias, float A, int lane, int m) const {
        float dt[4], l[4], w[4], sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            dt[j] = 4 * lane + j < m ? softplus_f(raw[j] + bias) : 0.f;
            sum += dt[j] * A;
            l[j] = sum;
        }
        // sums over the lanes before and behind this one
        float before = sum, behind = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const float a = __shfl_up_sync(0xffffffffu, before, off), b = __shfl_down_sync(0xffffffffu, behind, off);
            if (lane >= off) before += a;
            if (lane + off < 32) behind += b;
        }
        before = __shfl_up_sync(0xffffffffu, before, 1);
        behind = __shfl_down_sync(0xffffffffu, behind, 1);
        if (lane == 0) before = 0.f;
        if (lane == 31) behind = 0.f;
#pragma unroll
        for (int j = 3; j >= 0; --j) {
            w[j] = expf(behind) * dt[j];
            behind += dt[j] * A;
            l[j] += before;
        }
        const float end = __shfl_sync(0xffffffffu, l[3], lane | 7);  // l at the end of the lane's 32 tokens
        *reinterpret_cast<float4 *>(sc + Scal::L + 4 * lane) = make_float4(l[0], l[1], l[2], l[3]);
        *reinterpret_cast<float4 *>(sc + Scal::U + 4 * lane) =
            make_float4(expf(end - l[0]) * dt[0], expf(end - l[1]) * dt[1], expf(end - l[2]) * dt[2], expf(end - l[3]) * dt[3]);
        *reinterpret_cast<float4 *>(sc + Scal::DT + 4 * lane) = make_float4(dt[0], dt[1], dt[2], dt[3]);
        *reinterpret_cast<float4 *>(sc + Scal::W + 4 * lane) = make_float4(w[0], w[1], w[2], w[3]);
        if ((lane & 7) == 7) sc[Scal::RB + (lane >> 3)] = l[3];
        if (lane == 31) sc[Scal::E] = expf(l[3]);
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
        f *= expf(sc[Scal::L + t] - sc[Scal::L + s]) * sc[Scal::DT + s];
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

template <class ST, int DK, int NH>
__global__ void __launch_bounds__(THREADS, 1)
ssm_tc_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_b,
              const __grid_constant__ CUtensorMap map_c, const __grid_constant__ Args a) {
    using LY = Layout<DK, NH>;
    static_assert(LY::N_BAR == BARS, "barriers");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + LY::BAR);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + LY::TSLOT);
    volatile int *abort = reinterpret_cast<volatile int *>(sm + LY::ABORT);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const SsmParams &p = a.p;
    const dl_ssm &in = p.in;

    const long long gid = (long long)blockIdx.x * THREADS + tid;
    if (gid < a.q.n_seq) seq_check(a.q, (int)gid);
    // the block's segment and value rows
    const int tile = (int)(blockIdx.x / (unsigned)a.units);
    const Rows rw = rows_of<NH>(p, (int)(blockIdx.x - (unsigned)tile * a.units));
    int seg = 0, s0, n;
    const int i = seq_of_tile(a.q, tile, a.seg_len, seg);
    if (i < 0 || !seq_range(a.q, i, s0, n)) return;
    const int slot = seq_slot(a.q, i);
    const int segs = (int)(((long long)n + a.seg_len - 1) / a.seg_len);
    if (slot < 0 || seg >= segs) return;
    const int len = min(a.seg_len, n - seg * a.seg_len);  // this segment's tokens, from row0
    const int row0 = s0 + seg * a.seg_len, chunks = (len + Q - 1) / Q;

    if (tid == 0) {
        auto init = [&](int b, int count) { tc::mbar_init(&bars[b], count); };
        for (int b = 0; b < BARS; ++b) init(b, 1);
        for (int b : {(int)S_READY, (int)W_READY, (int)P_READY, (int)YS_READY, (int)Y_FREE, (int)ZEROED}) init(b, 4);
        for (int k = 0; k < 2; ++k) {
            init(X_FREE + k, 4);
            init(SC_FULL + k, NH);
            init(SC_FREE + k, 12);
        }
        *abort = 0;
        tc::mbar_init_fence();
    }
    if (warp == 13) {
        tc::tmem_alloc(tslot, T_COLS);
        tc::tmem_relinquish();
    }
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tb = *tslot;
    auto scal = [&](int c, int h) { return reinterpret_cast<float *>(sm + LY::scal(c & 1, h)); };
    auto arrive = [&](int b) {  // once per warp, after every lane's writes
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars[b]);
    };

    if (warp < 4) {
        // ------------------------------------------------ P from G, and y (thread = token row t)
        const int quad = warp, t = 32 * quad + lane;
        const uint32_t trow = tb + ((uint32_t)(32 * quad) << 16);
        for (int c = 0; c < chunks; ++c) {
            const uint32_t par = c & 1, par2 = (c >> 1) & 1;
            if (!wait_warp(&bars[SC_FULL + par], par2, abort)) break;
            if (!wait_warp(&bars[G_DONE], par, abort)) break;
            tc::tc_fence_after();
#pragma unroll 1
            for (int kb = 0; kb < 4; ++kb) {
                uint32_t pw[NH][16];
                if (kb <= quad) {
                    uint32_t gr[32];
                    tc::tmem_ld32(trow + T_G + 32 * kb, gr);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        const float *sc = scal(c, h);
                        const float lt = sc[Scal::L + t];
                        if (kb < quad) {
                            const float v = __expf(lt - sc[Scal::RB + kb]);
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float4 u = *reinterpret_cast<const float4 *>(sc + Scal::U + 32 * kb + e);
                                pw[h][e / 2] = pack_bf2(__uint_as_float(gr[e]) * (u.x * v), __uint_as_float(gr[e + 1]) * (u.y * v));
                                pw[h][e / 2 + 1] =
                                    pack_bf2(__uint_as_float(gr[e + 2]) * (u.z * v), __uint_as_float(gr[e + 3]) * (u.w * v));
                            }
                        } else {  // the block on the diagonal: tokens up to t
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float4 l = *reinterpret_cast<const float4 *>(sc + Scal::L + 32 * kb + e);
                                const float4 d = *reinterpret_cast<const float4 *>(sc + Scal::DT + 32 * kb + e);
                                const float f0 = e <= lane ? __uint_as_float(gr[e]) * (__expf(lt - l.x) * d.x) : 0.f;
                                const float f1 = e + 1 <= lane ? __uint_as_float(gr[e + 1]) * (__expf(lt - l.y) * d.y) : 0.f;
                                const float f2 = e + 2 <= lane ? __uint_as_float(gr[e + 2]) * (__expf(lt - l.z) * d.z) : 0.f;
                                const float f3 = e + 3 <= lane ? __uint_as_float(gr[e + 3]) * (__expf(lt - l.w) * d.w) : 0.f;
                                pw[h][e / 2] = pack_bf2(f0, f1);
                                pw[h][e / 2 + 1] = pack_bf2(f2, f3);
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < NH; ++h)
#pragma unroll
                        for (int e = 0; e < 16; ++e) pw[h][e] = 0u;
                }
#pragma unroll
                for (int h = 0; h < NH; ++h) tc::tmem_st16(trow + p_col(2 * kb, h), pw[h]);
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
            arrive(P_READY);

            // y of row t: Y + D x, gated
            const int m = min(Q, len - c * Q);
            const long long row = (long long)row0 + c * Q + t;
            if (!wait_warp(&bars[Y_DONE], par, abort)) break;
            tc::tc_fence_after();
            const uint8_t *xt = sm + LY::x(par);
#pragma unroll 1
            for (int cb = 0; cb < 4; ++cb) {
                const int h = NH == 2 ? cb >> 1 : 0, col = rw.r0 + (NH == 2 ? (cb & 1) * 32 : cb * 32);
                const bool live = t < m && (h == 0 || rw.two);
                uint4 zr[4];
                if (in.z && live) {
                    const uint4 *z = reinterpret_cast<const uint4 *>(static_cast<const bf16 *>(in.z) + row * in.z_stride +
                                                                     (long long)(rw.h0 + h) * p.dv + col);
#pragma unroll
                    for (int j = 0; j < 4; ++j) zr[j] = z[j];
                }
                uint32_t yr[32];
                tc::tmem_ld32(trow + T_Y + 32 * cb, yr);
                tc::tmem_wait_ld();
                if (!live) continue;
                const float D = in.D ? in.D[rw.h0 + h] : 0.f;
                uint4 *y = reinterpret_cast<uint4 *>(static_cast<bf16 *>(p.y) + (row * p.H + rw.h0 + h) * p.dv + col);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float x[8], o[8];
                    StateVec<bf16>::unpack(*reinterpret_cast<const uint4 *>(xt + tile_off(t, 4 * cb + j)), x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = fmaf(D, x[e], __uint_as_float(yr[8 * j + e]));
                    if (in.z) {
                        float z[8];
                        StateVec<bf16>::unpack(zr[j], z);
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] *= silu_f<bf16>(z[e]);
                    }
                    y[j] = StateVec<bf16>::pack(o);
                }
            }
            tc::tc_fence_before();
            arrive(Y_FREE);
            const uint32_t *nf = reinterpret_cast<const uint32_t *>(sm + LY::NF) + 16 * par;
            uint32_t any = 0;
#pragma unroll
            for (int j = 0; j < 16; ++j) any |= nf[j];
            if (any && t < m)
                for (int h = 0; h < NH; ++h)
                    if (h == 0 || rw.two)
                        add_no_numbers(p, (long long)row0 + c * Q, t, nf, scal(c, h), rw.h0 + h, rw.g, rw.r0, R / NH);
            arrive(X_FREE + par);
            arrive(SC_FREE + par);
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
#pragma unroll
            for (int cb = 0; cb < DK / 32; ++cb) {
                uint32_t v[32];
                if (c > 0) {
                    tc::tmem_ld32(trow + T_S + 32 * cb, v);
                    tc::tmem_wait_ld();
                } else {
                    float f[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) f[j] = 0.f;
                    if (live) {
                        if (segs > 1)
                            load_row32(a.seg_state + ((long long)(seg_base(s0, a.seg_len) + seg) * p.H * p.dv + srow) * DK + 32 * cb, f);
                        else
                            load_row32(S + 32 * cb, f);
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(f[j]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float *f = reinterpret_cast<const float *>(v) + 8 * j;
                    *reinterpret_cast<uint4 *>(sm + LY::S + tile_off(r, 4 * cb + j)) = make_uint4(
                        pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3]), pack_bf2(f[4], f[5]), pack_bf2(f[6], f[7]));
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * e);
                tc::tmem_st32(trow + T_S + 32 * cb, v);
            }
            tc::fence_async_smem();
            tc::tmem_wait_st();
            tc::tc_fence_before();
            arrive(S_READY);

            float ex[NH];
#pragma unroll
            for (int k = 0; k < NH; ++k) ex[k] = __expf(scal(c, k)[Scal::L + r]);
            arrive(SC_FREE + par);
            if (!(ok = wait_warp(&bars[Y2_DONE], par, abort))) break;
            tc::tc_fence_after();
#pragma unroll
            for (int cb = 0; cb < 4; ++cb) {
                uint32_t v[32];
                tc::tmem_ld32(trow + T_Y + 32 * cb, v);
                tc::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * ex[NH == 2 ? cb >> 1 : 0]);
                tc::tmem_st32(trow + T_Y + 32 * cb, v);
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
            arrive(YS_READY);
        }
        if (ok && wait_warp(&bars[ST_DONE], (chunks - 1) & 1, abort) && seg == segs - 1) {
            tc::tc_fence_after();
#pragma unroll
            for (int cb = 0; cb < DK / 32; ++cb) {
                uint32_t v[32];
                tc::tmem_ld32(trow + T_S + 32 * cb, v);
                tc::tmem_wait_ld();
                if (live) store_row32(S + 32 * cb, v);
            }
            tc::tc_fence_before();
        }
    } else if (warp < 12) {
        // ------------------------------------------------ W from X (thread = value row r)
        const int quad = warp & 3, r = 32 * quad + lane, h = NH == 2 ? r >> 6 : 0;
        const uint32_t trow = tb + ((uint32_t)(32 * quad) << 16);
        const int piece = r >> 3, in_piece = (r & 7) * 2;
        uint32_t *nf = reinterpret_cast<uint32_t *>(sm + LY::NF) + 4 * quad;
        for (int c = 0; c < chunks; ++c) {
            const uint32_t par = c & 1, par2 = (c >> 1) & 1;
            const int m = min(Q, len - c * Q);
            uint8_t *xt = sm + LY::x(par);
            if (!wait_warp(&bars[X_FULL + par], par2, abort)) break;
            if (!wait_warp(&bars[SC_FULL + par], par2, abort)) break;
            if (m < Q) {  // (the last chunk) zeros behind the segment, in X and B
                if (!wait_warp(&bars[B_FULL + par], par2, abort)) break;
                constexpr int XP = R / 8, BP = DK / 8;
                for (int k = tid - 256; k < (Q - m) * (XP + BP); k += 128) {
                    const int row = m + k / (XP + BP), pc = k % (XP + BP);
                    uint8_t *dst = pc < XP ? xt + tile_off(row, pc) : sm + LY::b(par) + tile_off(row, pc - XP);
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(0u, 0u, 0u, 0u);
                }
                tc::fence_async_smem();
                arrive(ZEROED);
                if (!wait_warp(&bars[ZEROED], 0, abort)) break;
            }
            const float *w = scal(c, h) + Scal::W;
            float no_number = 0.f;  // NaN once an x is no finite number
            bool ok = true;
#pragma unroll 1
            for (int kb = 0; kb < 4; ++kb) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 w4 = *reinterpret_cast<const float4 *>(w + 32 * kb + e);
                    const float ws[4] = {w4.x, w4.y, w4.z, w4.w};
                    float f[4], rest[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int s = e + k;  // (row 32 kb + s: the same position in its 8 rows)
                        const float x = to_f(*reinterpret_cast<const bf16 *>(
                            xt + (piece >> 3) * PANEL + (32 * kb + s) * 128 + (((piece & 7) ^ (s & 7)) << 4) + in_piece));
                        no_number = fmaf(x, 0.f, no_number);
                        f[k] = x * ws[k];
                    }
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        const uint32_t hw = pack_bf2(f[k], f[k + 1]);
                        rest[k] = f[k] - bf_lo(hw);
                        rest[k + 1] = f[k + 1] - bf_hi(hw);
                        if (!(fabsf(rest[k]) <= 3.4e38f)) rest[k] = 0.f;
                        if (!(fabsf(rest[k + 1]) <= 3.4e38f)) rest[k + 1] = 0.f;
                        hi[(e + k) / 2] = hw;
                        lo[(e + k) / 2] = pack_bf2(rest[k], rest[k + 1]);
                    }
                }
                if (kb == 0 && c > 0) {  // the previous update has read W
                    if (!(ok = wait_warp(&bars[ST_DONE], (c - 1) & 1, abort))) break;
                    tc::tc_fence_after();
                }
                tc::tmem_st16(trow + T_W + 16 * kb, hi);
                tc::tmem_st16(trow + T_WLO + 16 * kb, lo);
            }
            if (!ok) break;
            arrive(SC_FREE + par);
            uint32_t mask[4] = {0u, 0u, 0u, 0u};
            if (__any_sync(0xffffffffu, !(no_number == 0.f))) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    for (int s = 0; s < 32; ++s) {
                        bf16 *xp = reinterpret_cast<bf16 *>(xt + tile_off(32 * j + s, piece) + in_piece);
                        if (!(fabsf(to_f(*xp)) <= 3.4e38f)) {
                            *xp = __float2bfloat16_rn(0.f);
                            mask[j] |= 1u << s;
                        }
                    }
                    mask[j] = __reduce_or_sync(0xffffffffu, mask[j]);
                }
                tc::fence_async_smem();
            }
            if (lane == 0) {
#pragma unroll
                for (int j = 0; j < 4; ++j) nf[16 * par + j] = mask[j];
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
            arrive(W_READY);
        }
    } else if (warp == 12) {
        // ------------------------------------------------ loads
        if (lane == 0) {
            tc::tma_prefetch_desc(&map_x);
            tc::tma_prefetch_desc(&map_b);
            tc::tma_prefetch_desc(&map_c);
            auto load = [&](const CUtensorMap *map, int off, int panels, int col, int row, uint64_t *full) {
                tc::mbar_arrive_expect_tx(full, panels * PANEL);
                for (int k = 0; k < panels; ++k) tc::tma_load_2d(sm + off + k * PANEL, map, col + 64 * k, row, full);
            };
            int nb = 0, nx = 0, nc = 0;  // copies issued
            for (int c = 0; c < chunks; ++c) {
                const int k = c & 1, row = row0 + c * Q;
                const uint32_t old = (uint32_t)((c >> 1) - 1) & 1;
                if (c >= 2 && !wait1(&bars[B_FREE + k], old, abort)) break;
                load(&map_b, LY::b(k), LY::KP, rw.g * DK, row, &bars[B_FULL + k]);
                ++nb;
                if (c == 0) {
                    load(&map_c, LY::C, LY::KP, rw.g * DK, row, &bars[C_FULL]);
                    ++nc;
                }
                if (c >= 2 && !wait1(&bars[X_FREE + k], old, abort)) break;
                load(&map_x, LY::x(k), R / 64, rw.col0, row, &bars[X_FULL + k]);
                ++nx;
                if (c > 0) {
                    if (!wait1(&bars[C_FREE], (c - 1) & 1, abort)) break;
                    load(&map_c, LY::C, LY::KP, rw.g * DK, row, &bars[C_FULL]);
                    ++nc;
                }
            }
            // every copy has landed before the block may leave
            for (int k = 0; k < 2; ++k) {
                const int b = (nb + 1 - k) / 2, x = (nx + 1 - k) / 2;  // copies into buffer k
                if (b) drain(&bars[B_FULL + k], (b - 1) & 1);
                if (x) drain(&bars[X_FULL + k], (x - 1) & 1);
            }
            if (nc) drain(&bars[C_FULL], (nc - 1) & 1);
        }
        __syncwarp();
    } else if (warp == 13) {
        // ------------------------------------------------ products
        if (lane == 0) {
            constexpr uint32_t ID_G = tc::instr_desc(tc::FMT_BF16, false, false, Q, Q);
            constexpr uint32_t ID_Y2 = tc::instr_desc(tc::FMT_BF16, false, false, Q, R);
            constexpr uint32_t ID_Y1 = tc::instr_desc(tc::FMT_BF16, false, true, Q, R / NH);
            constexpr uint32_t ID_S = tc::instr_desc(tc::FMT_BF16, false, true, R, DK);
            const uint32_t ct = tc::smem_u32(sm + LY::C), st = tc::smem_u32(sm + LY::S);
            // 16 columns of K of a tile whose rows are the product's rows or columns
            auto kmajor = [](uint32_t tile, int k) {
                return tc::smem_desc(tile + (k >> 2) * PANEL + (k & 3) * 32, 16, 1024, tc::SWZ_128);
            };
            // 16 rows of K of a tile whose columns are the product's columns
            auto nmajor = [](uint32_t tile, int k) { return tc::smem_desc(tile + k * 2048, PANEL, 1024, tc::SWZ_128); };
            bool ok = true;
            for (int c = 0; c < chunks; ++c) {
                const uint32_t par = c & 1, par2 = (c >> 1) & 1;
                const uint32_t bt = tc::smem_u32(sm + LY::b(par)), xt = tc::smem_u32(sm + LY::x(par));
                if (!(ok = wait1(&bars[C_FULL], par, abort) && wait1(&bars[B_FULL + par], par2, abort))) break;
                tc::tc_fence_after();
#pragma unroll
                for (int k = 0; k < DK / 16; ++k) tc::mma_ss_f16(tb + T_G, kmajor(ct, k), kmajor(bt, k), ID_G, k > 0);
                tc::mma_commit(&bars[G_DONE]);
                if (!(ok = wait1(&bars[S_READY], par, abort) && (c == 0 || wait1(&bars[Y_FREE], (c - 1) & 1, abort)))) break;
                tc::tc_fence_after();
#pragma unroll
                for (int k = 0; k < DK / 16; ++k) tc::mma_ss_f16(tb + T_Y, kmajor(ct, k), kmajor(st, k), ID_Y2, k > 0);
                tc::mma_commit(&bars[Y2_DONE]);
                tc::mma_commit(&bars[C_FREE]);
                if (!(ok = wait1(&bars[W_READY], par, abort))) break;
                tc::tc_fence_after();
#pragma unroll
                for (int k = 0; k < Q / 16; ++k) tc::mma_ts_f16(tb + T_S, tb + T_W + 8 * k, nmajor(bt, k), ID_S, true);
#pragma unroll
                for (int k = 0; k < Q / 16; ++k) tc::mma_ts_f16(tb + T_S, tb + T_WLO + 8 * k, nmajor(bt, k), ID_S, true);
                tc::mma_commit(&bars[ST_DONE]);
                tc::mma_commit(&bars[B_FREE + par]);
                if (!(ok = wait1(&bars[P_READY], par, abort) && wait1(&bars[YS_READY], par, abort))) break;
                tc::tc_fence_after();
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int k = 0; k < Q / 16; ++k)
                        tc::mma_ts_f16(tb + T_Y + (R / NH) * h, tb + p_col(k, h), nmajor(xt + h * PANEL, k), ID_Y1, true);
                tc::mma_commit(&bars[Y_DONE]);
            }
            if (!ok) {  // products in flight have completed before tensor memory is freed
                tc::mma_commit(&bars[DRAIN]);
                drain(&bars[DRAIN], 0);
            }
        }
        __syncwarp();
    } else if (warp - 14 < NH) {
        // ------------------------------------------------ step sizes and decays of head h
        const int h = warp - 14;
        const bool live = h == 0 || rw.two;
        const float A = live ? in.A[rw.h0 + h] : 0.f, bias = live && in.dt_bias ? in.dt_bias[rw.h0 + h] : 0.f;
        Steps next;
        next.fetch(in, row0, rw.h0 + h, lane, live ? len : 0);
        for (int c = 0; c < chunks; ++c) {
            const Steps now = next;
            const int m = live ? len - c * Q : 0;
            next.fetch(in, (long long)row0 + (c + 1) * Q, rw.h0 + h, lane, m - Q);
            if (c >= 2 && !wait_warp(&bars[SC_FREE + (c & 1)], (uint32_t)((c >> 1) - 1) & 1, abort)) break;
            now.write(scal(c, h), bias, A, lane, m);
            arrive(SC_FULL + (c & 1));
        }
    }
    __syncthreads();
    if (warp == 13) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tb, T_COLS);
    }
}

// A [rows, cols] bfloat16 matrix with a row stride, in boxes of Q rows of 64 columns.
cudaError_t row_map(CUtensorMap *m, const void *base, long long cols, long long rows, long long stride) {
    tc::EncodeTiledFn fn = tc::encoder();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)Q};
    const cuuint32_t es[2] = {1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <class ST, int DK, int NH>
cudaError_t launch_typed(const SsmParams &p, const SeqIdx &q, cudaStream_t st) {
    using LY = Layout<DK, NH>;
    auto kern = ssm_tc_kernel<ST, DK, NH>;
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(kern), LY::REQUEST);
    if (e != cudaSuccess) return e;
    CUtensorMap mx, mb, mc;
    const dl_ssm &in = p.in;
    if ((e = row_map(&mx, in.x, (long long)p.H * p.dv, q.T, in.x_stride)) != cudaSuccess) return e;
    if ((e = row_map(&mb, in.b, (long long)p.G * DK, q.T, in.b_stride)) != cudaSuccess) return e;
    if ((e = row_map(&mc, in.c, (long long)p.G * DK, q.T, in.c_stride)) != cudaSuccess) return e;
    const int per = p.H / p.G;
    Args a{p, q, (q.T + Q - 1) / Q * Q, NH == 2 ? p.G * ((per + 1) / 2) : p.H * (p.dv / R), nullptr};
    const long long blocks = ((long long)q.T / a.seg_len + q.n_seq) * a.units;
    kern<<<(unsigned)blocks, THREADS, LY::REQUEST, st>>>(mx, mb, mc, a);
    return cudaGetLastError();
}

}  // namespace

bool ssm_tc_supported(const SsmParams &p) { return p.in.dtype == DL_BF16 && tc::encoder() != nullptr; }

cudaError_t launch_ssm_tc(const SsmParams &p, const SeqIdx &q, cudaStream_t st) {
    auto with_nh = [&](auto s, auto dk) -> cudaError_t {
        using ST = decltype(s);
        constexpr int DK = decltype(dk)::value;
        return p.dv == 64 ? launch_typed<ST, DK, 2>(p, q, st) : launch_typed<ST, DK, 1>(p, q, st);
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
