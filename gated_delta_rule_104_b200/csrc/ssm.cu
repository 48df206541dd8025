// Selective state space scan with one decay per head, for single tokens and
// (token by token) for prompts. Per head, with S in R^{d_v x d_k}:
//
//   dt = softplus(dt_raw + dt_bias),  S <- exp(dt A) S + dt x b^T,
//   y = S c + D x  (times z / (1 + exp(-z)))
//
// which is the head-wise decay of the eager step with k = b, q = c, v = dt x and
// no delta correction; the state has the steps' layout.
#include "launch.h"

namespace dl {

namespace {

// dt and exp(dt A) of (row, head).
template <class IT>
__device__ __forceinline__ void step_size(const dl_ssm &in, long long row, int h, float &dt, float &da) {
    dt = softplus_f(to_f(static_cast<const IT *>(in.dt)[row * in.dt_stride + h]) + (in.dt_bias ? in.dt_bias[h] : 0.f));
    da = expf(dt * in.A[h]);
}

constexpr int STEP_R = 8;  // state loads a lane has in flight

// One token per sequence. HBM-bound on the state like the eager step, and laid
// out as that is: a state row over a group of lanes, 16 bytes each, R rows'
// loads in flight per lane before any arithmetic, a shuffle sum per row, no
// shared memory. A lane holds x, z and y of one of the unit's rows, which keeps a
// float32 state's kernel within the 64 registers of four blocks an SM (256
// sequences of 32 heads of 128 x 128: 166 us of the 164 that the state's bytes take;
// 198 with each row's x loaded by its lanes and three blocks, 177 with four rows'
// loads in flight; all three a pass through the binding).
template <class ST, class IT, int DK>
__global__ void __launch_bounds__(256, sizeof(ST) == 4 ? 4 : 3) ssm_step_kernel(const SsmParams p, const SeqIdx q, long long num_units) {
    constexpr int VEC = StateVec<ST>::N, G = DK / VEC, RPW = 32 / G, R = STEP_R, UNIT = R * RPW;
    const long long gid = (long long)blockIdx.x * 256 + threadIdx.x;
    if (gid < q.n_seq) seq_check(q, (int)gid);
    const int lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (unit >= num_units) return;  // whole warps leave together
    const int upr = p.H * (p.dv / UNIT);  // units of a batch row
    const long long b = unit / upr;
    const int in_row = (int)(unit - b * upr), h = in_row / (p.dv / UNIT);
    const int r0 = (in_row - h * (p.dv / UNIT)) * UNIT;
    const int slot = seq_slot(q, (int)b);
    if (slot < 0) return;
    const int sub = lane / G, col = (lane % G) * VEC;
    ST *srow = static_cast<ST *>(p.S) + (((long long)slot * p.H + h) * p.dv + r0 + sub) * DK + col;
    uint4 raw[R];
#pragma unroll
    for (int r = 0; r < R; ++r) raw[r] = ld_stream(srow + (long long)r * RPW * DK);

    const dl_ssm &in = p.in;
    const int g = h / (p.H / p.G);
    float bb[VEC], cc[VEC], xl = 0.f, zl = 0.f, yl = 0.f, dt, da;
    load_vec<VEC>(static_cast<const IT *>(in.b) + b * in.b_stride + g * DK + col, bb);
    load_vec<VEC>(static_cast<const IT *>(in.c) + b * in.c_stride + g * DK + col, cc);
    // x, z and y of the unit's row `lane`
    const bool own = lane < UNIT;
    const long long at = (long long)h * p.dv + r0 + lane;
    if (own) xl = to_f(static_cast<const IT *>(in.x)[b * in.x_stride + at]);
    if (own && in.z) zl = to_f(static_cast<const IT *>(in.z)[b * in.z_stride + at]);
    step_size<IT>(in, b, h, dt, da);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float s[VEC], y = 0.f;
        StateVec<ST>::unpack(raw[r], s);
        const float dx = dt * __shfl_sync(0xffffffffu, xl, r * RPW + sub);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            s[e] = fmaf(s[e], da, dx * bb[e]);
            y = fmaf(s[e], cc[e], y);
        }
        st_stream(srow + (long long)r * RPW * DK, StateVec<ST>::pack(s));
        y = __shfl_sync(0xffffffffu, group_sum<G>(y), (lane % RPW) * G);
        if (lane / RPW == r) yl = y;
    }
    if (in.D) yl = fmaf(in.D[h], xl, yl);
    if (in.z) yl *= silu_f<IT>(zl);
    if (own) store_f(static_cast<IT *>(p.y) + b * p.H * p.dv + at, yl);
}

// Prompts, token by token: a block keeps ROWS rows of one head's state in
// registers (8 columns of RPT rows a thread) for the whole segment, so the state
// moves once; the operands of 16 tokens are staged as floats, the next 16
// tokens' loads in flight meanwhile. Tokens behind the segment are staged as
// steps of zero, so every stage runs whole. Bound by its instructions (three
// products of pairs per pair of state elements and token) and by their latency:
// two tokens at a time, each row's sum over its lanes with the rows exchanged on
// the way. 16 rows a block where 64 would leave SMs without one (257 and 40
// tokens, 16 heads of 64: 94 us by 64 rows a block and a token at a time, 47 us
// now).
//
// ENDS: the end state of a segment from a state of zero, and its log decay, for
// sequences of several segments (see ssm_tc.cu); no outputs.
constexpr int SCAN_TOK = 16;

__device__ __forceinline__ void store_state8(float *p, const uint64_t (&s)[4]) {
    reinterpret_cast<ulonglong2 *>(p)[0] = make_ulonglong2(s[0], s[1]);
    reinterpret_cast<ulonglong2 *>(p)[1] = make_ulonglong2(s[2], s[3]);
}
__device__ __forceinline__ void store_state8(bf16 *p, const uint64_t (&s)[4]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf2(s[0]), pack_bf2(s[1]), pack_bf2(s[2]), pack_bf2(s[3]));
}
__device__ __forceinline__ void store4(float *p, const float (&y)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(y[0], y[1], y[2], y[3]);
}
__device__ __forceinline__ void store4(bf16 *p, const float (&y)[4]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3]));
}

// The sum over lanes 0 .. 15, for lane 0.
__device__ __forceinline__ float group_sum16(float x) {
#pragma unroll
    for (int off = 8; off >= 1; off /= 2) x += __shfl_down_sync(0xffffu, x, off);
    return x;
}

template <class ST, class IT, int DK, int ROWS, bool ENDS>
__global__ void __launch_bounds__(4 * ROWS) ssm_scan_kernel(const SsmParams p, const SeqIdx q, const SsmSegs g) {
    constexpr int NT = 4 * ROWS, LPR = DK / 8, RPT = ROWS * LPR / NT;  // threads, lanes a row, rows a thread
    constexpr int BE = SCAN_TOK * DK / NT, BV = BE < 8 ? BE : 8;       // b (and c) elements a thread stages, at a time
    static_assert(RPT == 2 || RPT == 4, "rows a thread");
    __shared__ alignas(16) float xs[SCAN_TOK][ROWS], ys[ENDS ? 1 : SCAN_TOK][ROWS], bs[SCAN_TOK][DK], cs[ENDS ? 1 : SCAN_TOK][DK];
    __shared__ float2 steps[SCAN_TOK];  // dt, exp(dt A)
    const int tid = threadIdx.x;
    const long long gid = (long long)blockIdx.x * NT + tid;
    if (!ENDS && gid < q.n_seq) seq_check(q, (int)gid);
    const int tiles = p.dv / ROWS;
    const int tile = (int)(blockIdx.x / (unsigned)(p.H * tiles)), rest = (int)(blockIdx.x - (unsigned)tile * (p.H * tiles));
    const int h = rest / tiles, r0 = (rest - h * tiles) * ROWS;
    int seg = 0, s0, len;
    const int i = seq_of_tile(q, tile, g.len, seg, ENDS ? 0 : 1);
    if (i < 0 || !seq_range(q, i, s0, len)) return;
    const int slot = seq_slot(q, i), segs = segs_of(len, g.len);
    if (slot < 0 || seg >= (ENDS ? segs - 1 : segs)) return;
    const long long place = ((long long)(segs > 1 ? seg_base(s0, g.len) + seg : 0) * p.H + h) * p.dv + r0;  // row in the workspace
    const int n = min(g.len, len - seg * g.len), row0 = s0 + seg * g.len;
    const dl_ssm &in = p.in;
    const int gr = h / (p.H / p.G);
    const IT *x = static_cast<const IT *>(in.x) + (long long)row0 * in.x_stride + (long long)h * p.dv + r0;
    const IT *z = in.z ? static_cast<const IT *>(in.z) + (long long)row0 * in.z_stride + (long long)h * p.dv + r0 : nullptr;
    const IT *b = static_cast<const IT *>(in.b) + (long long)row0 * in.b_stride + gr * DK;
    const IT *c = static_cast<const IT *>(in.c) + (long long)row0 * in.c_stride + gr * DK;
    IT *y = static_cast<IT *>(p.y) + ((long long)row0 * p.H + h) * p.dv + r0;
    const float D = in.D ? in.D[h] : 0.f, bias = in.dt_bias ? in.dt_bias[h] : 0.f, A = in.A[h];

    // staging: thread t takes 4 x of one token and BE elements of b and c of one
    const int xt = tid / (ROWS / 4), xc = (tid % (ROWS / 4)) * 4, bt = tid * BE / DK, bc = tid * BE % DK;
    float rx[4], rb[BE], rc[BE], rdt = 0.f;
    auto fetch = [&](int t0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) rx[e] = 0.f;
#pragma unroll
        for (int e = 0; e < BE; ++e) rb[e] = rc[e] = 0.f;
        if (t0 + xt < n) load_vec<4>(x + (long long)(t0 + xt) * in.x_stride + xc, rx);
        if (t0 + bt < n) {
#pragma unroll
            for (int e = 0; e < BE; e += BV) {
                float v[BV];
                load_vec<BV>(b + (long long)(t0 + bt) * in.b_stride + bc + e, v);
#pragma unroll
                for (int k = 0; k < BV; ++k) rb[e + k] = v[k];
                if constexpr (!ENDS) {
                    load_vec<BV>(c + (long long)(t0 + bt) * in.c_stride + bc + e, v);
#pragma unroll
                    for (int k = 0; k < BV; ++k) rc[e + k] = v[k];
                }
            }
        }
        if (tid < SCAN_TOK && t0 + tid < n) rdt = to_f(static_cast<const IT *>(in.dt)[((long long)row0 + t0 + tid) * in.dt_stride + h]);
    };
    fetch(0);

    const int rg = tid / LPR, lr = tid % LPR, col = lr * 8;
    const long long srow = ((long long)slot * p.H + h) * p.dv + r0;
    uint64_t s[RPT][4];
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (ENDS) {
        } else if (segs > 1) {
            load_vec<8>(g.state + (place + rg * RPT + r) * DK + col, f);
        } else {
            load_vec<8>(static_cast<const ST *>(p.S) + (srow + rg * RPT + r) * DK + col, f);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[r][e] = pair(f[2 * e], f[2 * e + 1]);
    }
    float decay = 0.f;  // (thread < SCAN_TOK) the log decay of its tokens

    for (int t0 = 0; t0 < n; t0 += SCAN_TOK) {
        __syncthreads();  // the previous tokens' operands and outputs have been read
#pragma unroll
        for (int e = 0; e < 4; ++e) xs[xt][xc + e] = rx[e];
#pragma unroll
        for (int e = 0; e < BE; ++e) {
            bs[bt][bc + e] = rb[e];
            if constexpr (!ENDS) cs[bt][bc + e] = rc[e];
        }
        if (tid < SCAN_TOK) {
            const bool in = t0 + tid < n;  // (no decay behind the segment: 0 A is no number for an A of -inf)
            const float dt = in ? softplus_f(rdt + bias) : 0.f, ld = in ? dt * A : 0.f;
            steps[tid] = make_float2(dt, expf(ld));
            decay += ld;
        }
        __syncthreads();
        fetch(t0 + SCAN_TOK);
#pragma unroll 4
        for (int t = 0; t < SCAN_TOK; ++t) {
            const float2 st = steps[t];
            const uint64_t da = pair(st.y, st.y);
            const ulonglong2 b0 = *reinterpret_cast<const ulonglong2 *>(&bs[t][col]), b1 = *reinterpret_cast<const ulonglong2 *>(&bs[t][col + 4]);
            const uint64_t bb[4] = {b0.x, b0.y, b1.x, b1.y};
            float xv[RPT], dot[RPT];
            load_vec<RPT>(&xs[t][rg * RPT], xv);
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                const float dx = st.x * xv[r];
                const uint64_t d = pair(dx, dx);
#pragma unroll
                for (int e = 0; e < 4; ++e) s[r][e] = fma2(s[r][e], da, mul2(d, bb[e]));
            }
            if constexpr (!ENDS) {
                const ulonglong2 c0 = *reinterpret_cast<const ulonglong2 *>(&cs[t][col]), c1 = *reinterpret_cast<const ulonglong2 *>(&cs[t][col + 4]);
#pragma unroll
                for (int r = 0; r < RPT; ++r) {
                    const uint64_t a = fma2(s[r][3], c1.y, fma2(s[r][2], c1.x, fma2(s[r][1], c0.y, mul2(s[r][0], c0.x))));
                    float a0, a1;
                    unpair(a, a0, a1);
                    dot[r] = a0 + a1;
                }
                // over the row's lanes; half of the rows stay with each half of them
#pragma unroll
                for (int m = RPT / 2, off = LPR / 2; m >= 1; m /= 2, off /= 2) {
                    const bool upper = (lr & off) != 0;
#pragma unroll
                    for (int r = 0; r < m; ++r) {
                        const float keep = upper ? dot[r + m] : dot[r], send = upper ? dot[r] : dot[r + m];
                        dot[r] = keep + __shfl_xor_sync(0xffffffffu, send, off);
                    }
                }
#pragma unroll
                for (int off = LPR / RPT / 2; off >= 1; off /= 2) dot[0] += __shfl_xor_sync(0xffffffffu, dot[0], off);
                if (lr % (LPR / RPT) == 0) ys[t][rg * RPT + lr / (LPR / RPT)] = dot[0];
            }
        }
        if constexpr (!ENDS) {
            __syncthreads();
            if (t0 + xt < n) {
                float o[4], zz[4] = {0.f, 0.f, 0.f, 0.f};
                if (z) load_vec<4>(z + (long long)(t0 + xt) * in.z_stride + xc, zz);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    o[e] = fmaf(D, xs[xt][xc + e], ys[xt][xc + e]);
                    if (z) o[e] *= silu_f<IT>(zz[e]);
                }
                store4(y + (long long)(t0 + xt) * p.H * p.dv + xc, o);
            }
        }
    }
    if (ENDS) {
#pragma unroll
        for (int r = 0; r < RPT; ++r) store_state8(g.state + (place + rg * RPT + r) * DK + col, s[r]);
        if (tid < SCAN_TOK) {
            decay = group_sum16(decay);
            if (tid == 0 && r0 == 0) g.decay[place / p.dv] = decay;
        }
    } else if (seg == segs - 1) {
#pragma unroll
        for (int r = 0; r < RPT; ++r) store_state8(static_cast<ST *>(p.S) + (srow + rg * RPT + r) * DK + col, s[r]);
    }
}

// f(ST{}, IT{}, DK constant)
template <class F>
cudaError_t dispatch_ssm(const SsmParams &p, F &&f) {
    auto with_dk = [&](auto st, auto it) -> cudaError_t {
        if (p.dk == 64) return f(st, it, std::integral_constant<int, 64>{});
        return f(st, it, std::integral_constant<int, 128>{});
    };
    auto with_it = [&](auto st) -> cudaError_t {
        return p.in.dtype == DL_BF16 ? with_dk(st, bf16{}) : with_dk(st, float{});
    };
    return p.s_dt == DL_BF16 ? with_it(bf16{}) : with_it(float{});
}

}  // namespace

cudaError_t launch_ssm_step(const SsmParams &p, const SeqIdx &q, cudaStream_t st) {
    return dispatch_ssm(p, [&](auto s, auto t, auto dk) -> cudaError_t {
        using ST = decltype(s);
        using IT = decltype(t);
        constexpr int DK = decltype(dk)::value, UNIT = STEP_R * 32 / (DK / StateVec<ST>::N);
        static_assert(64 % UNIT == 0, "a unit is rows of one head");
        const long long units = (long long)q.n_seq * p.H * (p.dv / UNIT);
        ssm_step_kernel<ST, IT, DK><<<(unsigned)((units + 7) / 8), 256, 0, st>>>(p, q, units);
        return cudaGetLastError();
    });
}

cudaError_t launch_ssm_prompt(const SsmParams &p, const SeqIdx &q, void *work, cudaStream_t st) {
    SsmSegs g;
    g.len = ssm_seg_len(q.T, q.n_seq, p.H, p.dv);
    const bool split = g.len != 0;
    if (split) {
        g.state = static_cast<float *>(work);
        g.decay = g.state + seg_count(q.T, g.len) * p.H * p.dv * p.dk;
    } else {
        g.len = (int)std::min<long long>(((long long)q.T + 127) / 128 * 128, 0x7fffff80LL);
    }
    // The tensor cores take bfloat16 prompts, but not calls of few tokens a sequence:
    // a block there costs 16 us whatever its length up to 128 tokens, the scan
    // below 7 us for 16 tokens, 12 for 32 (one sequence, 32 heads of 128 x 128; 64
    // sequences: 244 us against 154 for 4 tokens each, 162 for 16, 243 for 24, 250
    // for 32). One sequence may hold nearly all of the tokens (0.37 us each here), so
    // the longest there can be must not take more than about twice those blocks' time.
    const long long waves = ((long long)q.n_seq * p.H * p.dv / 128 + SMS - 1) / SMS;
    const bool few = q.T <= 24LL * q.n_seq && q.T - q.n_seq <= 85 * waves;
    if (!few && ssm_tc_supported(p)) return launch_ssm_tc(p, q, g, split, st);
    return dispatch_ssm(p, [&](auto s, auto t, auto dk) -> cudaError_t {
        using ST = decltype(s);
        using IT = decltype(t);
        constexpr int DK = decltype(dk)::value;
        const long long tiles = (long long)q.T / g.len + q.n_seq;
        auto go = [&](auto rows) -> cudaError_t {
            constexpr int ROWS = decltype(rows)::value;
            const long long blocks = (long long)p.H * (p.dv / ROWS);  // of a segment
            if (split) {
                ssm_scan_kernel<ST, IT, DK, ROWS, true><<<(unsigned)(q.T / g.len * blocks), 4 * ROWS, 0, st>>>(p, q, g);
                cudaError_t e = cudaGetLastError();
                if (e == cudaSuccess) e = launch_ssm_join(p, q, g, st);
                if (e != cudaSuccess) return e;
            }
            ssm_scan_kernel<ST, IT, DK, ROWS, false><<<(unsigned)(tiles * blocks), 4 * ROWS, 0, st>>>(p, q, g);
            return cudaGetLastError();
        };
        if (tiles * p.H * (p.dv / 64) < 2 * SMS) return go(std::integral_constant<int, 16>{});
        return go(std::integral_constant<int, 64>{});
    });
}

}  // namespace dl
