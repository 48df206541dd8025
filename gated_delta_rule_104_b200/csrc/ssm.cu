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
// out as that is: a state row over a group of lanes, 16 bytes each, R = 4 rows'
// loads in flight per lane before any arithmetic, a shuffle sum per row, no
// shared memory.
template <class ST, class IT, int DK>
__global__ void __launch_bounds__(256) ssm_step_kernel(const SsmParams p, const SeqIdx q, long long num_units) {
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
    float bb[VEC], cc[VEC], xr[R], dt, da;
    load_vec<VEC>(static_cast<const IT *>(in.b) + b * in.b_stride + g * DK + col, bb);
    load_vec<VEC>(static_cast<const IT *>(in.c) + b * in.c_stride + g * DK + col, cc);
    const IT *x = static_cast<const IT *>(in.x) + b * in.x_stride + (long long)h * p.dv + r0 + sub;
#pragma unroll
    for (int r = 0; r < R; ++r) xr[r] = to_f(x[r * RPW]);
    step_size<IT>(in, b, h, dt, da);
    const float D = in.D ? in.D[h] : 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float s[VEC], y = 0.f;
        StateVec<ST>::unpack(raw[r], s);
        const float dx = dt * xr[r];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            s[e] = fmaf(s[e], da, dx * bb[e]);
            y = fmaf(s[e], cc[e], y);
        }
        y = group_sum<G>(y);
        st_stream(srow + (long long)r * RPW * DK, StateVec<ST>::pack(s));
        if (lane % G == 0) {
            const int row = r0 + r * RPW + sub;
            y = fmaf(D, xr[r], y);
            if (in.z) y *= silu_f<IT>(to_f(static_cast<const IT *>(in.z)[b * in.z_stride + (long long)h * p.dv + row]));
            store_f(static_cast<IT *>(p.y) + (b * p.H + h) * p.dv + row, y);
        }
    }
}

// Prompts, token by token: a block of 256 threads keeps 64 rows of one head's
// state in registers (8 columns of 2 or 4 rows a thread) for the whole
// sequence, so the state moves once; the operands of 16 tokens are staged as
// floats, the next 16 tokens' loads in flight meanwhile.
constexpr int SCAN_TOK = 16, SCAN_ROWS = 64;

template <class ST>
__device__ __forceinline__ void load_state8(const ST *p, float (&s)[8]) { load_vec<8>(p, s); }
__device__ __forceinline__ void store_state8(float *p, const float (&s)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(s[0], s[1], s[2], s[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(s[4], s[5], s[6], s[7]);
}
__device__ __forceinline__ void store_state8(bf16 *p, const float (&s)[8]) {
    *reinterpret_cast<uint4 *>(p) = StateVec<bf16>::pack(s);
}
__device__ __forceinline__ void store4(float *p, const float (&y)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(y[0], y[1], y[2], y[3]);
}
__device__ __forceinline__ void store4(bf16 *p, const float (&y)[4]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3]));
}

template <class ST, class IT, int DK>
__global__ void __launch_bounds__(256) ssm_scan_kernel(const SsmParams p, const SeqIdx q) {
    constexpr int LPR = DK / 8, RG = 256 / LPR, RPT = SCAN_ROWS / RG;  // lanes a row, row groups, rows a thread
    constexpr int BE = SCAN_TOK * DK / 256;                            // b (and c) elements a thread stages
    __shared__ float xs[SCAN_TOK][SCAN_ROWS], ys[SCAN_TOK][SCAN_ROWS], bs[SCAN_TOK][DK], cs[SCAN_TOK][DK];
    __shared__ float dts[SCAN_TOK], das[SCAN_TOK];
    const int tid = threadIdx.x;
    const long long gid = (long long)blockIdx.x * 256 + tid;
    if (gid < q.n_seq) seq_check(q, (int)gid);
    const int tiles = p.dv / SCAN_ROWS;
    const int i = (int)(blockIdx.x / (unsigned)(p.H * tiles)), rest = (int)(blockIdx.x - (unsigned)i * (p.H * tiles));
    const int h = rest / tiles, r0 = (rest - h * tiles) * SCAN_ROWS;
    int s0, n;
    const int slot = seq_slot(q, i);
    if (!seq_range(q, i, s0, n) || slot < 0 || n == 0) return;
    const dl_ssm &in = p.in;
    const int g = h / (p.H / p.G);
    const IT *x = static_cast<const IT *>(in.x) + (long long)s0 * in.x_stride + (long long)h * p.dv + r0;
    const IT *z = in.z ? static_cast<const IT *>(in.z) + (long long)s0 * in.z_stride + (long long)h * p.dv + r0 : nullptr;
    const IT *b = static_cast<const IT *>(in.b) + (long long)s0 * in.b_stride + g * DK;
    const IT *c = static_cast<const IT *>(in.c) + (long long)s0 * in.c_stride + g * DK;
    IT *y = static_cast<IT *>(p.y) + ((long long)s0 * p.H + h) * p.dv + r0;
    const float D = in.D ? in.D[h] : 0.f;

    // staging: thread t takes 4 x of token t / 16 and BE elements of b and c
    const int xt = tid >> 4, xc = (tid & 15) * 4, bt = tid * BE / DK, bc = tid * BE % DK;
    float rx[4], rb[BE], rc[BE], rdt = 0.f, rda = 1.f;
    auto fetch = [&](int t0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) rx[e] = 0.f;
#pragma unroll
        for (int e = 0; e < BE; ++e) rb[e] = rc[e] = 0.f;
        rdt = 0.f;
        rda = 1.f;
        if (t0 + xt < n) load_vec<4>(x + (long long)(t0 + xt) * in.x_stride + xc, rx);
        if (t0 + bt < n) {
            load_vec<BE>(b + (long long)(t0 + bt) * in.b_stride + bc, rb);
            load_vec<BE>(c + (long long)(t0 + bt) * in.c_stride + bc, rc);
        }
        if (tid < SCAN_TOK && t0 + tid < n) step_size<IT>(in, (long long)s0 + t0 + tid, h, rdt, rda);
    };
    fetch(0);

    const int rg = tid / LPR, lr = tid % LPR, col = lr * 8;
    ST *S = static_cast<ST *>(p.S) + (((long long)slot * p.H + h) * p.dv + r0) * DK + col;
    float s[RPT][8];
#pragma unroll
    for (int r = 0; r < RPT; ++r) load_state8(S + (long long)(rg + RG * r) * DK, s[r]);

    for (int t0 = 0; t0 < n; t0 += SCAN_TOK) {
        const int m = min(SCAN_TOK, n - t0);
        __syncthreads();  // the previous tokens' operands and outputs have been read
#pragma unroll
        for (int e = 0; e < 4; ++e) xs[xt][xc + e] = rx[e];
#pragma unroll
        for (int e = 0; e < BE; ++e) {
            bs[bt][bc + e] = rb[e];
            cs[bt][bc + e] = rc[e];
        }
        if (tid < SCAN_TOK) {
            dts[tid] = rdt;
            das[tid] = rda;
        }
        __syncthreads();
        fetch(t0 + SCAN_TOK);
        for (int t = 0; t < m; ++t) {
            const float dt = dts[t], da = das[t];
            float bb[8], cc[8], dot[RPT];
            load_vec<8>(&bs[t][col], bb);
            load_vec<8>(&cs[t][col], cc);
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                const float dx = dt * xs[t][rg + RG * r];
                float acc = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s[r][e] = fmaf(s[r][e], da, dx * bb[e]);
                    acc = fmaf(s[r][e], cc[e], acc);
                }
                dot[r] = group_sum<LPR>(acc);
            }
#pragma unroll
            for (int r = 0; r < RPT; ++r)
                if (lr == r) ys[t][rg + RG * r] = dot[r];
        }
        __syncthreads();
        if (xt < m) {
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
#pragma unroll
    for (int r = 0; r < RPT; ++r) store_state8(S + (long long)(rg + RG * r) * DK, s[r]);
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
    if (ssm_tc_supported(p)) return launch_ssm_tc(p, q, work, st);
    return dispatch_ssm(p, [&](auto s, auto t, auto dk) -> cudaError_t {
        using ST = decltype(s);
        using IT = decltype(t);
        constexpr int DK = decltype(dk)::value;
        const long long blocks = (long long)q.n_seq * p.H * (p.dv / SCAN_ROWS);
        ssm_scan_kernel<ST, IT, DK><<<(unsigned)blocks, 256, 0, st>>>(p, q);
        return cudaGetLastError();
    });
}

}  // namespace dl
