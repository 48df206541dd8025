// Root-mean-square norm of rows with the residual's addition and an output in
// 8 bits with scales, and the values of such rows.
//
//   h = x + residual,  y = h / sqrt(mean(h^2) + eps) * weight
//
// HBM-bound: every operand moves once. A row stays in the registers of its
// threads from its one load to its store, so the mean, the 8-bit scales (the
// largest |y| of a row or of 128 columns) and the codes need no second pass.
// The weight is fetched before the row's sum is reduced. All of it is fp32;
// each output is rounded once.
#include <cuda_fp8.h>

#include "launch.h"

namespace dl {

namespace {

template <int N>
__device__ __forceinline__ void load_n(const float *p, float (&x)[N]) {
    if constexpr (N == 1)
        x[0] = *p;
    else
        load_vec<N>(p, x);
}
template <int N>
__device__ __forceinline__ void load_n(const bf16 *p, float (&x)[N]) {
    if constexpr (N == 1)
        x[0] = to_f(*p);
    else
        load_vec<N>(p, x);
}
template <int N>
__device__ __forceinline__ void store_n(float *p, const float (&x)[N]) {
    if constexpr (N == 1) {
        *p = x[0];
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            *reinterpret_cast<float4 *>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    }
}
template <int N>
__device__ __forceinline__ void store_n(bf16 *p, const float (&x)[N]) {
    if constexpr (N == 1) {
        *p = __float2bfloat16_rn(x[0]);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 8)
            *reinterpret_cast<uint4 *>(p + i) = make_uint4(pack_bf2(x[i], x[i + 1]), pack_bf2(x[i + 2], x[i + 3]),
                                                           pack_bf2(x[i + 4], x[i + 5]), pack_bf2(x[i + 6], x[i + 7]));
    }
}

// The scale of a group whose largest |y| is m: NaN where m is no finite number.
__device__ __forceinline__ float scale_of(float m, float top) { return m <= 3.402823466e38f ? m / top : __int_as_float(0x7fffffff); }

// x / scale correctly rounded: by the row's reciprocal where i8_fast(scale)
// (see i8_code), else by division; 0 for scale 0.
template <bool FAST>
__device__ __forceinline__ float over_scale(float x, float scale, float inv) {
    if constexpr (FAST) {
        const float q0 = __fmul_rn(x, inv);
        return fmaf(fmaf(-q0, scale, x), inv, q0);
    }
    return scale == 0.f ? 0.f : x / scale;
}
template <bool FAST>
__device__ __forceinline__ uint32_t e4m3_pack2(float a, float b, float scale, float inv) {
    const float2 v = make_float2(over_scale<FAST>(a, scale, inv), over_scale<FAST>(b, scale, inv));
    return (uint32_t)__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
}

// N codes of a group with the given scale at p (N-byte aligned for N = 8).
template <bool FAST, int N>
__device__ __forceinline__ void store_codes(uint8_t *p, const float (&y)[N], float scale, float inv, bool i8) {
    if constexpr (N == 1) {
        if (i8)
            *p = (uint8_t)(FAST ? i8_code(y[0], scale, inv) : i8_code_div(y[0], scale));
        else
            *p = (uint8_t)e4m3_pack2<FAST>(y[0], 0.f, scale, inv);
    } else {
        uint32_t w[N / 4];
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            w[i] = i8 ? i8_pack4<FAST>(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3], scale, inv)
                      : e4m3_pack2<FAST>(y[4 * i], y[4 * i + 1], scale, inv) |
                            (e4m3_pack2<FAST>(y[4 * i + 2], y[4 * i + 3], scale, inv) << 16);
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
}
template <int N>
__device__ __forceinline__ void store_codes(uint8_t *p, const float (&y)[N], float scale, bool i8) {
    if (i8_fast(scale))
        store_codes<true, N>(p, y, scale, i8_inv(scale), i8);
    else
        store_codes<false, N>(p, y, scale, 0.f, i8);
}

// One value over the blockDim.x threads of a row: blockDim.x == 32 (any
// number of rows a block) or blockDim.y == 1.
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, float *red) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, off);
        v = MAX ? max_nan(v, o) : v + o;
    }
    if (blockDim.x == 32) return v;
    const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < nw ? red[lane] : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, off);
        v = MAX ? max_nan(v, o) : v + o;
    }
    return v;
}

// CH chunks of VEC columns per thread. VEC = 8 (16-byte accesses): chunk c of
// thread t starts at column (c blockDim.x + t) 8, so 16 lanes hold a group of
// 128. VEC = 1 (any alignment): a warp holds whole groups, 4 chunks each.
template <class XT, class RT, bool RES, class WT, int VEC, int CH>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const NormParams p) {
    __shared__ float red[2][32];
    const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = row < p.rows;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5, width = p.width;
    auto column = [&](int c) {
        return VEC == 1 ? ((c >> 2) * nw + warp) * 128 + (c & 3) * 32 + lane : (c * (int)blockDim.x + (int)threadIdx.x) * VEC;
    };
    const XT *x = static_cast<const XT *>(p.x) + row * p.x_stride;
    float h[CH][VEC], w[CH][VEC];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int col = column(c);
        const bool in = live && col < width;
        if (in) {
            load_n<VEC>(x + col, h[c]);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) h[c][e] = 0.f;
        }
        if constexpr (RES) {
            float r[VEC];
            if (in) {
                load_n<VEC>(static_cast<const RT *>(p.res) + row * width + col, r);
#pragma unroll
                for (int e = 0; e < VEC; ++e) h[c][e] += r[e];
            }
        }
    }
    auto load_w = [&](int c) {
        const int col = column(c);
        if (col < width) load_n<VEC>(static_cast<const WT *>(p.w) + col, w[c]);
    };
    if constexpr (VEC * CH <= 16) {  // (more would spill at 1024 threads)
#pragma unroll
        for (int c = 0; c < CH; ++c) load_w(c);
    }
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss = fmaf(h[c][e], h[c][e], ss);
        if constexpr (RES) {
            const int col = column(c);
            if (live && col < width) store_n<VEC>(static_cast<RT *>(p.res_out) + row * width + col, h[c]);
        }
    }
    const float r = rsqrtf(row_reduce<false>(ss, red[0]) / (float)width + p.eps);
    float m = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        if constexpr (VEC * CH > 16) load_w(c);
        const bool in = live && column(c) < width;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            h[c][e] = in ? h[c][e] * r * w[c][e] : 0.f;
            m = max_nan(m, fabsf(h[c][e]));
        }
    }
    const bool i8 = p.y_dt == DL_I8;
    if (p.y_dt == DL_F32 || p.y_dt == DL_BF16) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = column(c);
            if (!live || col >= width) continue;
            if (p.y_dt == DL_F32)
                store_n<VEC>(static_cast<float *>(p.y) + row * width + col, h[c]);
            else
                store_n<VEC>(static_cast<bf16 *>(p.y) + row * width + col, h[c]);
        }
        return;
    }
    const float top = i8 ? 127.f : 448.f;
    uint8_t *y = static_cast<uint8_t *>(p.y) + row * width;
    if (p.group == 0) {
        const float scale = scale_of(row_reduce<true>(m, red[1]), top);
        if (live && threadIdx.x == 0) p.scale[row] = scale;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int col = column(c);
            if (live && col < width) store_codes<VEC>(y + col, h[c], scale, i8);
        }
        return;
    }
    const int groups = (width + 127) / 128;
    if constexpr (VEC == 1) {
#pragma unroll
        for (int g = 0; g < CH / 4; ++g) {
            float gm = 0.f;
#pragma unroll
            for (int c = 4 * g; c < 4 * g + 4; ++c) gm = max_nan(gm, fabsf(h[c][0]));
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) gm = max_nan(gm, __shfl_xor_sync(0xffffffffu, gm, off));
            const float scale = scale_of(gm, top);
            const int gi = g * nw + warp;
            if (live && lane == 0 && gi < groups) p.scale[row * groups + gi] = scale;
#pragma unroll
            for (int c = 4 * g; c < 4 * g + 4; ++c) {
                const int col = column(c);
                if (live && col < width) store_codes<VEC>(y + col, h[c], scale, i8);
            }
        }
    } else {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float gm = 0.f;
#pragma unroll
            for (int e = 0; e < VEC; ++e) gm = max_nan(gm, fabsf(h[c][e]));
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) gm = max_nan(gm, __shfl_xor_sync(0xffffffffu, gm, off));
            const float scale = scale_of(gm, top);
            const int col = column(c);
            if (live && col < width) {
                if (col % 128 == 0) p.scale[row * groups + col / 128] = scale;
                store_codes<VEC>(y + col, h[c], scale, i8);
            }
        }
    }
}

template <class OT, int VEC>
__global__ void __launch_bounds__(256)
rows_from_8bit_kernel(const uint8_t *__restrict__ codes, const float *__restrict__ scale, OT *__restrict__ out,
                      long long chunks, int per_row, int groups, int group, bool i8) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= chunks) return;
    long long row;  // 32-bit division where it holds
    if (chunks <= 0xffffffffLL)
        row = (unsigned)i / (unsigned)per_row;
    else
        row = i / per_row;
    const int col = (int)(i - row * per_row) * VEC;
    const float s = scale[row * groups + (group ? col / group : 0)];
    alignas(16) uint8_t raw[VEC];
    if constexpr (VEC == 16)
        *reinterpret_cast<uint4 *>(raw) = __ldcs(reinterpret_cast<const uint4 *>(codes + i * VEC));
    else
        raw[0] = codes[i];
    float x[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        if (i8)
            x[e] = (float)(int8_t)raw[e] * s;
        else
            x[e] = __half2float(__half(__nv_cvt_fp8_to_halfraw(raw[e], __NV_E4M3))) * s;
    }
    store_n<VEC>(out + i * VEC, x);
}

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t size_of(dl_dtype t) { return t == DL_F32 ? 4 : t == DL_BF16 ? 2 : 1; }

template <class XT, class RT, bool RES, class WT>
cudaError_t launch_typed(const NormParams &p, cudaStream_t st) {
    const bool wide = p.width % 8 == 0 && aligned(p.x, 16) && (size_t)p.x_stride * sizeof(XT) % 16 == 0 &&
                      aligned(p.w, 16) && aligned(p.y, size_of(p.y_dt) == 1 ? 8 : 16) &&
                      (!RES || (aligned(p.res, 16) && aligned(p.res_out, 16)));
    auto go = [&](auto kern, int threads) {
        const int nt = (threads + 31) / 32 * 32, rpb = nt == 32 ? 8 : 1;
        kern<<<(unsigned)((p.rows + rpb - 1) / rpb), dim3(nt, rpb), 0, st>>>(p);
        return cudaGetLastError();
    };
    if (wide) {
        if (p.width <= 4096) return go(rms_norm_kernel<XT, RT, RES, WT, 8, 1>, p.width / 8);
        if (p.width <= 16384) return go(rms_norm_kernel<XT, RT, RES, WT, 8, 2>, (p.width / 8 + 1) / 2);
        return go(rms_norm_kernel<XT, RT, RES, WT, 8, 4>, (p.width / 8 + 3) / 4);
    }
    // Single columns: a warp on one group as long as that gives a block, then on as
    // few as fit (1021 rows of 2501 bfloat16 columns to 8 bits: 9.8 us with one, 11.0
    // with two, 16.0 with four; 500 of 5001: 8.7 us with two, 11.0 with four; 300 of
    // 15999: 19.7 us with four, 46 with eight, which no longer fit the registers).
    const int groups = (p.width + 127) / 128;
    if (groups <= 32) return go(rms_norm_kernel<XT, RT, RES, WT, 1, 4>, groups * 32);
    if (groups <= 64) return go(rms_norm_kernel<XT, RT, RES, WT, 1, 8>, (groups + 1) / 2 * 32);
    if (groups <= 128) return go(rms_norm_kernel<XT, RT, RES, WT, 1, 16>, (groups + 3) / 4 * 32);
    return go(rms_norm_kernel<XT, RT, RES, WT, 1, 32>, (groups + 7) / 8 * 32);
}

}  // namespace

cudaError_t launch_rms_norm(const NormParams &p, cudaStream_t st) {
    auto with_w = [&](auto x, auto r, auto res) -> cudaError_t {
        using XT = decltype(x);
        using RT = decltype(r);
        constexpr bool RES = decltype(res)::value;
        return p.w_dt == DL_BF16 ? launch_typed<XT, RT, RES, bf16>(p, st) : launch_typed<XT, RT, RES, float>(p, st);
    };
    auto with_r = [&](auto x) -> cudaError_t {
        if (!p.res) return with_w(x, float{}, std::false_type{});
        return p.r_dt == DL_BF16 ? with_w(x, bf16{}, std::true_type{}) : with_w(x, float{}, std::true_type{});
    };
    return p.x_dt == DL_BF16 ? with_r(bf16{}) : with_r(float{});
}

cudaError_t launch_rows_from_8bit(const void *codes, dl_dtype c_dt, const float *scale, int group, void *out,
                                  dl_dtype out_dt, long long rows, int width, cudaStream_t st) {
    const bool i8 = c_dt == DL_I8, wide = width % 16 == 0 && aligned(codes, 16) && aligned(out, 16);
    const int per_row = wide ? width / 16 : width, groups = group ? (width + group - 1) / group : 1;
    const long long chunks = rows * per_row;
    const unsigned blocks = (unsigned)((chunks + 255) / 256);
    const uint8_t *c = static_cast<const uint8_t *>(codes);
    auto go = [&](auto o) {
        using OT = decltype(o);
        OT *dst = static_cast<OT *>(out);
        if (wide)
            rows_from_8bit_kernel<OT, 16><<<blocks, 256, 0, st>>>(c, scale, dst, chunks, per_row, groups, group, i8);
        else
            rows_from_8bit_kernel<OT, 1><<<blocks, 256, 0, st>>>(c, scale, dst, chunks, per_row, groups, group, i8);
        return cudaGetLastError();
    };
    return out_dt == DL_BF16 ? go(bf16{}) : go(float{});
}

}  // namespace dl
