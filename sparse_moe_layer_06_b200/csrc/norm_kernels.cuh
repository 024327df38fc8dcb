// norm_kernels.cuh -- residual addition + root-mean-square norm (with E4M3
// codes of the normed rows) and its backward pass.
//
//   s = x + res                      residual_out = s rounded to the row type
//   y = (s * w) * r,  r = (mean(s^2) + eps)^-1/2
//   codes: scale = pow2_scale(max |y|) of the rounded y, q = e4m3(y / scale)
//
// backward, with h = residual_out as it is stored, n = h * r, g = dy * w:
//   dx = r * (g - n * mean(g * n)) + dres,    dw = sum over rows of dy * n
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "device_common.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kNormMaxH = 16384;
constexpr int kNormVec = 4;  // 16-byte vectors of a row per thread

// The 16-byte vector of values f rounded to the row type.
template <typename T>
__device__ __forceinline__ uint4 pack_vec(const float (&f)[16 / sizeof(T)]) {
    uint4 q;
    if constexpr (sizeof(T) == 2) {
        __nv_bfloat162* h2 = reinterpret_cast<__nv_bfloat162*>(&q);
#pragma unroll
        for (int e = 0; e < 4; ++e) h2[e] = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
    } else {
        q = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                       __float_as_uint(f[3]));
    }
    return q;
}

// Sum of a and of b over the threads of one row: a warp, or the whole CTA of
// blockDim.x threads (kWarp false; s_red holds 2 * 32 floats, and the caller
// leaves a barrier between two uses of it).  With kMaxB b takes the maximum.
// Every thread gets both results, added in one fixed order.
template <bool kWarp, bool kMaxB>
__device__ __forceinline__ void row_reduce(float& a, float& b, float* s_red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        const float ob = __shfl_xor_sync(0xffffffffu, b, o);
        b = kMaxB ? fmaxf(b, ob) : b + ob;
    }
    if constexpr (!kWarp) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
        if (lane == 0) {
            s_red[warp] = a;
            s_red[32 + warp] = b;
        }
        __syncthreads();
        a = lane < nw ? s_red[lane] : 0.0f;
        b = lane < nw ? s_red[32 + lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            const float ob = __shfl_xor_sync(0xffffffffu, b, o);
            b = kMaxB ? fmaxf(b, ob) : b + ob;
        }
    }
}

// One row per warp (kWarp: blockDim.x / 32 rows per CTA) or per CTA.  A row
// stays in registers between its only read and its only write, so outputs may
// overlay the inputs of the same rows.  Both statistics come from one
// reduction: y = (s * w) * r is monotone in s * w for the row's r >= 0, so the
// largest |y| is the rounded product of the largest |s * w| with r.
template <typename T, bool kWarp>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(
    const T* x, const T* res, const T* __restrict__ weight, float eps, int64_t n_rows, int H,
    T* res_out, T* y, uint8_t* y_q, float* __restrict__ y_scale) {
    constexpr int kVE = 16 / static_cast<int>(sizeof(T));
    __shared__ float s_red[64];
    const int tx = kWarp ? (threadIdx.x & 31) : threadIdx.x;
    const int nt = kWarp ? 32 : blockDim.x;
    const int64_t row = kWarp ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) +
                                    (threadIdx.x >> 5)
                              : static_cast<int64_t>(blockIdx.x);
    if (kWarp && row >= n_rows) return;
    const int nv = H / kVE;
    ptx::grid_dep_wait();
    const uint4* xr = reinterpret_cast<const uint4*>(x + row * H);
    const uint4* rr = reinterpret_cast<const uint4*>(res ? res + row * H : nullptr);
    const uint4* wr = reinterpret_cast<const uint4*>(weight);
    uint4 xv[kNormVec], rv[kNormVec], wv[kNormVec];
#pragma unroll
    for (int u = 0; u < kNormVec; ++u) {
        const int v = tx + u * nt;
        xv[u] = rv[u] = wv[u] = make_uint4(0, 0, 0, 0);
        if (v < nv) {
            xv[u] = xr[v];
            if (res) rv[u] = rr[v];
            wv[u] = wr[v];
        }
    }
    float s[kNormVec][kVE];
    float sq = 0.0f, big = 0.0f;
#pragma unroll
    for (int u = 0; u < kNormVec; ++u) {
        unpack_vec<T>(xv[u], s[u]);
        float w[kVE];
        unpack_vec<T>(wv[u], w);
        if (res) {
            float b[kVE];
            unpack_vec<T>(rv[u], b);
#pragma unroll
            for (int e = 0; e < kVE; ++e) s[u][e] += b[e];
            if (res_out && tx + u * nt < nv)
                reinterpret_cast<uint4*>(res_out + row * H)[tx + u * nt] = pack_vec<T>(s[u]);
        } else if (res_out && tx + u * nt < nv) {
            reinterpret_cast<uint4*>(res_out + row * H)[tx + u * nt] = xv[u];
        }
#pragma unroll
        for (int e = 0; e < kVE; ++e) {
            sq = fmaf(s[u][e], s[u][e], sq);
            s[u][e] *= w[e];
            big = fmaxf(big, fabsf(s[u][e]));
        }
    }
    row_reduce<kWarp, true>(sq, big, s_red);
    const float r = 1.0f / sqrtf(sq / static_cast<float>(H) + eps);
    float inv = 0.0f;
    if (y_q) {
        float amax = big * r;
        if constexpr (sizeof(T) == 2) amax = __bfloat162float(__float2bfloat16_rn(amax));
        const float sc = pow2_scale_f(amax);
        inv = 1.0f / sc;  // exact: power of two
        if (tx == 0) y_scale[row] = sc;
    }
#pragma unroll
    for (int u = 0; u < kNormVec; ++u) {
        const int v = tx + u * nt;
        if (v >= nv) continue;
#pragma unroll
        for (int e = 0; e < kVE; ++e) s[u][e] *= r;
        const uint4 q = pack_vec<T>(s[u]);
        if (y) reinterpret_cast<uint4*>(y + row * H)[v] = q;
        if (y_q) {
            // the codes are those of the stored (rounded) row, so they equal
            // the ones the FP8 forward makes itself of y
            float f[kVE];
            unpack_vec<T>(q, f);
            uint32_t c[kVE / 4];
#pragma unroll
            for (int k = 0; k < kVE / 4; ++k)
                c[k] = static_cast<uint32_t>(ptx::e4m3x2(f[4 * k] * inv, f[4 * k + 1] * inv)) |
                       (static_cast<uint32_t>(
                            ptx::e4m3x2(f[4 * k + 2] * inv, f[4 * k + 3] * inv))
                        << 16);
            if constexpr (kVE == 8)
                reinterpret_cast<uint2*>(y_q + row * H)[v] = make_uint2(c[0], c[1]);
            else
                reinterpret_cast<uint32_t*>(y_q + row * H)[v] = c[0];
        }
    }
}

// Backward over rows blockIdx.x, blockIdx.x + gridDim.x, ...: dx of each row,
// and the CTA's share of dw, kept in registers and written once to
// partial[blockIdx.x].  Thread tx owns the same columns of every row.
template <typename T>
__global__ void __launch_bounds__(1024) add_rmsnorm_backward_kernel(
    const T* dy, const T* dres, const T* h, const T* __restrict__ weight, float eps,
    int64_t n_rows, int H, T* dx, float* __restrict__ partial) {
    constexpr int kVE = 16 / static_cast<int>(sizeof(T));
    __shared__ float s_red[2][64];
    const int tx = threadIdx.x, nt = blockDim.x;
    const int nv = H / kVE;
    ptx::grid_dep_wait();
    uint4 wv[kNormVec];
    float dw[kNormVec][kVE];
#pragma unroll
    for (int u = 0; u < kNormVec; ++u) {
        const int v = tx + u * nt;
        wv[u] = v < nv ? reinterpret_cast<const uint4*>(weight)[v] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < kVE; ++e) dw[u][e] = 0.0f;
    }
    int flip = 0;
    for (int64_t row = blockIdx.x; row < n_rows; row += gridDim.x, flip ^= 1) {
        uint4 hv[kNormVec], gv[kNormVec], rv[kNormVec];
#pragma unroll
        for (int u = 0; u < kNormVec; ++u) {
            const int v = tx + u * nt;
            hv[u] = gv[u] = rv[u] = make_uint4(0, 0, 0, 0);
            if (v < nv) {
                hv[u] = reinterpret_cast<const uint4*>(h + row * H)[v];
                gv[u] = reinterpret_cast<const uint4*>(dy + row * H)[v];
                if (dres) rv[u] = reinterpret_cast<const uint4*>(dres + row * H)[v];
            }
        }
        float sq = 0.0f, dot = 0.0f;
#pragma unroll
        for (int u = 0; u < kNormVec; ++u) {
            float hf[kVE], gf[kVE], wf[kVE];
            unpack_vec<T>(hv[u], hf);
            unpack_vec<T>(gv[u], gf);
            unpack_vec<T>(wv[u], wf);
#pragma unroll
            for (int e = 0; e < kVE; ++e) {
                sq = fmaf(hf[e], hf[e], sq);
                dot = fmaf(gf[e] * wf[e], hf[e], dot);
            }
        }
        // two scratch rows in turn: the barrier inside the next row's reduction
        // separates this row's reads from the writes two rows later
        row_reduce<false, false>(sq, dot, s_red[flip]);
        const float r = 1.0f / sqrtf(sq / static_cast<float>(H) + eps);
        const float c = r * r * (dot / static_cast<float>(H));  // mean(g * n) * r
#pragma unroll
        for (int u = 0; u < kNormVec; ++u) {
            const int v = tx + u * nt;
            float hf[kVE], gf[kVE], wf[kVE], rf[kVE];
            unpack_vec<T>(hv[u], hf);
            unpack_vec<T>(gv[u], gf);
            unpack_vec<T>(wv[u], wf);
            unpack_vec<T>(rv[u], rf);
#pragma unroll
            for (int e = 0; e < kVE; ++e) {
                dw[u][e] = fmaf(gf[e], hf[e] * r, dw[u][e]);
                rf[e] = fmaf(r, gf[e] * wf[e] - hf[e] * c, rf[e]);
            }
            if (v < nv) reinterpret_cast<uint4*>(dx + row * H)[v] = pack_vec<T>(rf);
        }
    }
#pragma unroll
    for (int u = 0; u < kNormVec; ++u) {
        const int v = tx + u * nt;
        if (v < nv) {
            float4* p = reinterpret_cast<float4*>(partial + static_cast<int64_t>(blockIdx.x) * H) +
                        v * (kVE / 4);
#pragma unroll
            for (int e = 0; e < kVE; e += 4)
                p[e / 4] = make_float4(dw[u][e], dw[u][e + 1], dw[u][e + 2], dw[u][e + 3]);
        }
    }
}

// dw[c] = sum of partial[0..n)[c] in a fixed order: 8 warps take every 8th row
// of 32 columns, then their sums are added in warp order.
__global__ void __launch_bounds__(256) reduce_columns_kernel(const float* __restrict__ partial,
                                                             int n, int H,
                                                             float* __restrict__ dw) {
    __shared__ float s_sum[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;  // H is a multiple of 64
    ptx::grid_dep_wait();
    float a = 0.0f;
#pragma unroll 8
    for (int i = warp; i < n; i += 8) a += partial[static_cast<int64_t>(i) * H + c];
    s_sum[warp][lane] = a;
    __syncthreads();
    if (warp == 0) {
        a = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) a += s_sum[w][lane];
        dw[c] = a;
    }
}

}  // namespace moe
