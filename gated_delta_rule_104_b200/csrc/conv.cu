// Short causal convolution along the tokens, for ragged prompts and for single
// tokens, with each slot's last taps - 1 inputs as its state.
//
//   y_t[c] = act(bias[c] + sum_{j < K} w[c, j] x_{t-K+1+j}[c])
//
// HBM-bound (2 K + 5 operations per element moved twice; the activation's two
// special-function operations take three quarters of the copy's time): every
// input and output moves once. A thread owns 16 bytes of channels and walks TT
// tokens with the K - 1 inputs before them in registers, so an input is loaded
// once and used K times. Its next 12 tokens are on the way to its own places in
// shared memory (asynchronous copies that no other thread reads, so no
// barriers): enough in flight without holding registers. With 8 tokens' loads
// in registers instead, one block fitted an SM and 16263 tokens of 4352
// channels took 106 us of a floor of 43; it takes 57 this way.
// A prompt's first tile reads its slot's history and also writes the new one
// (the last K - 1 inputs, from x): no other thread reads that history, so the
// update needs no second launch.
#include "launch.h"

namespace dl {

namespace {

// VEC elements as loaded (VEC = 1: any alignment; else 16 bytes).
template <class T, int VEC>
struct Raw {
    T v[VEC];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (VEC == 1)
            v[0] = *p;
        else
            *reinterpret_cast<uint4 *>(v) = *reinterpret_cast<const uint4 *>(p);
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (VEC == 1)
            *p = v[0];
        else
            *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(v);
    }
};
template <class T, int VEC>
struct alignas(16) RawV : Raw<T, VEC> {};

template <class T, int K, int VEC>
struct Filter {
    float w[VEC][K], bias[VEC];
    __device__ __forceinline__ void load(const ConvParams &p, int ch) {
        const T *wp = static_cast<const T *>(p.w) + (long long)ch * K;
        if constexpr (VEC == 1) {
#pragma unroll
            for (int j = 0; j < K; ++j) w[0][j] = to_f(wp[j]);
        } else {  // VEC K elements: K times 16 bytes
            float f[VEC * K];
            load_vec<VEC * K>(wp, f);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
#pragma unroll
                for (int j = 0; j < K; ++j) w[e][j] = f[e * K + j];
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) bias[e] = 0.f;
        if (p.bias) {
            const T *bp = static_cast<const T *>(p.bias) + ch;
            if constexpr (VEC > 1) {
                if (p.bias16)
                    load_vec<VEC>(bp, bias);
                else
#pragma unroll
                    for (int e = 0; e < VEC; ++e) bias[e] = to_f(bp[e]);
            } else {
                bias[0] = to_f(bp[0]);
            }
        }
    }
};

// act of a pair of sums, to the output's type.
template <class T, bool SILU>
__device__ __forceinline__ void finish_pair(T *out, uint64_t acc) {
    if constexpr (SILU) acc = silu2<T>(acc);
    if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint32_t *>(out) = pack_bf2(acc);
    } else {
        unpair(acc, out[0], out[1]);
    }
}
template <class T>
__device__ __forceinline__ uint64_t load_pair(const T *v) {
    if constexpr (sizeof(T) == 2)
        return pair_bf(*reinterpret_cast<const uint32_t *>(v));
    else
        return pair(v[0], v[1]);
}

// The wide path's walk over tokens t0 .. t1 - 1 of one thread's VEC channels:
// x and y at the sequence's first row, `ring` the thread's places in shared
// memory (RING of them, 256 apart), hist the K - 1 inputs before t0.
constexpr int GROUP = 4, GROUPS = 3, RING = GROUP * GROUPS;  // tokens of one wait, waits in flight
template <class T, int K, int VEC, bool SILU>
__device__ __forceinline__ void walk_wide(const ConvParams &p, const T *x, T *y, int t0, int t1, uint4 *ring, int ch,
                                          const RawV<T, VEC> (&hist)[K - 1]) {
    constexpr int PAIRS = VEC / 2;
    const int C = p.channels;
    auto fetch = [&](int g) {  // the g-th GROUP of tokens
#pragma unroll
        for (int u = 0; u < GROUP; ++u) {
            const int t = t0 + g * GROUP + u;
            if (t < t1) cp_async16(ring + ((g % GROUPS) * GROUP + u) * 256, x + (long long)t * p.x_stride);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int g = 0; g < GROUPS - 1; ++g) fetch(g);
    uint64_t w[PAIRS][K], bias[PAIRS], win[K - 1 + GROUP][PAIRS];
    {
        Filter<T, K, VEC> f;
        f.load(p, ch);
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) {
            bias[e] = pair(f.bias[2 * e], f.bias[2 * e + 1]);
#pragma unroll
            for (int j = 0; j < K; ++j) w[e][j] = pair(f.w[2 * e][j], f.w[2 * e + 1][j]);
        }
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) win[j][e] = load_pair(&hist[j].v[2 * e]);
    int g = 0;
    for (int t = t0; t < t1; t += GROUP, ++g) {
        fetch(g + GROUPS - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(GROUPS - 1) : "memory");
#pragma unroll
        for (int u = 0; u < GROUP; ++u) {
            if (t + u < t1) {
                RawV<T, VEC> in, out;
                *reinterpret_cast<uint4 *>(in.v) = ring[((g % GROUPS) * GROUP + u) * 256];
#pragma unroll
                for (int e = 0; e < PAIRS; ++e) {
                    win[K - 1 + u][e] = load_pair(&in.v[2 * e]);
                    uint64_t acc = bias[e];
#pragma unroll
                    for (int j = 0; j < K; ++j) acc = fma2(w[e][j], win[u + j][e], acc);
                    finish_pair<T, SILU>(&out.v[2 * e], acc);
                }
                out.store(y + (long long)(t + u) * C);
            }
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
#pragma unroll
            for (int e = 0; e < PAIRS; ++e) win[j][e] = win[GROUP + j][e];
    }
}

template <class T, int K, int VEC, int TT>
__global__ void __launch_bounds__(256, VEC > 1 ? 2 : 1) conv_prompt_kernel(const ConvParams p, const SeqIdx q, int nv) {
    using R = RawV<T, VEC>;
    constexpr int U = 8;  // tokens whose loads are in flight (VEC = 1)
    static_assert(TT % U == 0 && TT >= K, "tile");
    extern __shared__ uint4 ring[];
    const long long gid = (long long)blockIdx.x * 256 + threadIdx.x;
    if (gid < q.n_seq) seq_check(q, (int)gid);
    const long long tile = gid / nv;
    if (tile >= (long long)q.T / TT + q.n_seq) return;
    const int ch = (int)(gid - tile * nv) * VEC;
    int in_seq = 0, s0, n;
    const int i = seq_of_tile(q, (int)tile, TT, in_seq);
    if (i < 0 || !seq_range(q, i, s0, n)) return;
    const int slot = seq_slot(q, i);
    if (slot < 0 || in_seq >= (n + TT - 1) / TT) return;
    const int t0 = in_seq * TT, t1 = min(t0 + TT, n), C = p.channels;
    const T *x = static_cast<const T *>(p.x) + (long long)s0 * p.x_stride + ch;
    T *y = static_cast<T *>(p.y) + (long long)s0 * C + ch;
    R hist[K - 1];
    if (t0 == 0) {
        T *st = static_cast<T *>(p.state) + (long long)slot * (K - 1) * C + ch;
#pragma unroll
        for (int j = 0; j < K - 1; ++j) hist[j].load(st + (long long)j * C);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {  // the slot's new history
            const int pos = n - (K - 1) + j;
            R r;
            if (pos >= 0) {
                r.load(x + (long long)pos * p.x_stride);
            } else {  // hist[pos + K - 1], by constant indices
#pragma unroll
                for (int m = 0; m < K - 1; ++m)
                    if (m == pos + K - 1) r = hist[m];
            }
            r.store(st + (long long)j * C);
        }
    } else {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) hist[j].load(x + (long long)(t0 - (K - 1) + j) * p.x_stride);
    }
    if constexpr (VEC > 1) {
        if (p.silu)
            walk_wide<T, K, VEC, true>(p, x, y, t0, t1, ring + threadIdx.x, ch, hist);
        else
            walk_wide<T, K, VEC, false>(p, x, y, t0, t1, ring + threadIdx.x, ch, hist);
    } else {
        Filter<T, K, 1> f;
        f.load(p, ch);
        float win[K - 1 + U];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) win[j] = to_f(hist[j].v[0]);
        for (int t = t0; t < t1; t += U) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (t + u < t1) win[K - 1 + u] = to_f(x[(long long)(t + u) * p.x_stride]);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t + u < t1) {
                    float acc = f.bias[0];
#pragma unroll
                    for (int j = 0; j < K; ++j) acc = fmaf(f.w[0][j], win[u + j], acc);
                    store_f(y + (long long)(t + u) * C, p.silu ? silu_f<T>(acc) : acc);
                }
            }
#pragma unroll
            for (int j = 0; j < K - 1; ++j) win[j] = win[U + j];
        }
    }
}

template <class T, int K, int VEC>
__global__ void __launch_bounds__(256) conv_step_kernel(const ConvParams p, const SeqIdx q, int nv) {
    using R = RawV<T, VEC>;
    const long long gid = (long long)blockIdx.x * 256 + threadIdx.x;
    if (gid < q.n_seq) seq_check(q, (int)gid);
    const long long row = gid / nv;
    if (row >= q.n_seq) return;
    const int ch = (int)(gid - row * nv) * VEC, C = p.channels;
    const int slot = seq_slot(q, (int)row);
    if (slot < 0) return;
    T *st = static_cast<T *>(p.state) + (long long)slot * (K - 1) * C + ch;
    R in[K];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) in[j].load(st + (long long)j * C);
    in[K - 1].load(static_cast<const T *>(p.x) + row * p.x_stride + ch);
    Filter<T, K, VEC> f;
    f.load(p, ch);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) in[j + 1].store(st + (long long)j * C);
    R out;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        float acc = f.bias[e];
#pragma unroll
        for (int j = 0; j < K; ++j) acc = fmaf(f.w[e][j], to_f(in[j].v[e]), acc);
        store_f(&out.v[e], p.silu ? silu_f<T>(acc) : acc);
    }
    out.store(static_cast<T *>(p.y) + row * C + ch);
}

// Tokens a thread walks: 32 where that leaves every SM full (each tile reads its
// K - 1 rows of history again), 8 in smaller calls, whose time is a chain of
// loads (776 tokens of 1541 channels: 11.6 us by 32, 7.0 by 8).
constexpr int TT_LONG = 32, TT_SHORT = 8;
constexpr long long FILL = 148 * 2 * 256;

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// f(T{}, K constant, VEC constant): VEC fills 16 bytes where every row, the
// filter and the histories allow it, else 1.
template <class F>
cudaError_t dispatch_conv(const ConvParams &p, F &&f) {
    auto with_k = [&](auto t, auto vec) -> cudaError_t {
        switch (p.taps) {
            case 2: return f(t, std::integral_constant<int, 2>{}, vec);
            case 3: return f(t, std::integral_constant<int, 3>{}, vec);
            case 4: return f(t, std::integral_constant<int, 4>{}, vec);
        }
        return cudaErrorInvalidValue;
    };
    auto with_t = [&](auto t) -> cudaError_t {
        constexpr int V = 16 / (int)sizeof(t);
        const bool wide = p.channels % V == 0 && p.x_stride % V == 0 && aligned16(p.x) && aligned16(p.y) &&
                          aligned16(p.state) && aligned16(p.w);
        return wide ? with_k(t, std::integral_constant<int, V>{}) : with_k(t, std::integral_constant<int, 1>{});
    };
    return p.dt == DL_BF16 ? with_t(bf16{}) : with_t(float{});
}

}  // namespace

cudaError_t launch_conv_prompt(const ConvParams &conv, const SeqIdx &q, cudaStream_t st) {
    ConvParams p = conv;
    p.bias16 = aligned16(p.bias);
    return dispatch_conv(p, [&](auto t, auto k, auto vec) -> cudaError_t {
        using T = decltype(t);
        constexpr int K = decltype(k)::value, V = decltype(vec)::value;
        const int nv = p.channels / V;
        auto go = [&](auto tt) -> cudaError_t {
            constexpr int TT = decltype(tt)::value;
            const long long threads = ((long long)q.T / TT + q.n_seq) * nv;
            const size_t smem = V > 1 ? RING * 256 * sizeof(uint4) : 0;
            auto kern = conv_prompt_kernel<T, K, V, TT>;
            const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kern), smem);
            if (e != cudaSuccess) return e;
            kern<<<(unsigned)((threads + 255) / 256), 256, smem, st>>>(p, q, nv);
            return cudaGetLastError();
        };
        if ((long long)q.T / TT_LONG * nv >= FILL) return go(std::integral_constant<int, TT_LONG>{});
        return go(std::integral_constant<int, TT_SHORT>{});
    });
}

cudaError_t launch_conv_step(const ConvParams &conv, const SeqIdx &q, cudaStream_t st) {
    ConvParams p = conv;
    p.bias16 = aligned16(p.bias);
    return dispatch_conv(p, [&](auto t, auto k, auto vec) -> cudaError_t {
        using T = decltype(t);
        constexpr int K = decltype(k)::value, V = decltype(vec)::value;
        const int nv = p.channels / V;
        const long long threads = (long long)q.n_seq * nv;
        conv_step_kernel<T, K, V><<<(unsigned)((threads + 255) / 256), 256, 0, st>>>(p, q, nv);
        return cudaGetLastError();
    });
}

}  // namespace dl
