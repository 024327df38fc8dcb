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
// blockDim.x threads (kWarp false; s_red holds 2 * 32 floats, and a barrier lies
// between two uses of it).  With kMaxB b takes the maximum.
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

// Asynchronous copy of one 16-byte vector of a row into the thread's own bytes
// of the ring, and the wait for all but the newest N rows of copies.
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void ring_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A row in registers -> residual_out, y, codes.  Both statistics come from one
// reduction: y = (s * w) * r is monotone in s * w for the row's r >= 0, so the
// largest |y| is the rounded product of the largest |s * w| with r.
template <typename T, bool kWarp, int VPT>
__device__ __forceinline__ void norm_row(const uint4 (&xv)[VPT], const uint4 (&rv)[VPT],
                                         const uint4 (&wv)[VPT], bool has_res, float eps, int H,
                                         int tx, int nt, T* res_out, T* y, uint8_t* y_q,
                                         float* y_scale, float* s_red) {
    constexpr int kVE = 16 / static_cast<int>(sizeof(T));
    const int nv = H / kVE;
    float s[VPT][kVE];
    float sq = 0.0f, big = 0.0f;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        unpack_vec<T>(xv[u], s[u]);
        float w[kVE];
        unpack_vec<T>(wv[u], w);
        if (has_res) {
            float b[kVE];
            unpack_vec<T>(rv[u], b);
#pragma unroll
            for (int e = 0; e < kVE; ++e) s[u][e] += b[e];
        }
        if (res_out && tx + u * nt < nv)
            reinterpret_cast<uint4*>(res_out)[tx + u * nt] = pack_vec<T>(s[u]);
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
        if (tx == 0) *y_scale = sc;
    }
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const int v = tx + u * nt;
        if (v >= nv) continue;
#pragma unroll
        for (int e = 0; e < kVE; ++e) s[u][e] *= r;
        const uint4 q = pack_vec<T>(s[u]);
        if (y) reinterpret_cast<uint4*>(y)[v] = q;
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
            if constexpr (kVE == 8) reinterpret_cast<uint2*>(y_q)[v] = make_uint2(c[0], c[1]);
            else reinterpret_cast<uint32_t*>(y_q)[v] = c[0];
        }
    }
}

// Short rows: one per warp, four per CTA, VPT vectors per lane.
template <typename T, int VPT>
__global__ void __launch_bounds__(128) add_rmsnorm_short_kernel(
    const T* x, const T* res, const T* __restrict__ weight, float eps, int64_t n_rows, int H,
    T* res_out, T* y, uint8_t* y_q, float* __restrict__ y_scale) {
    constexpr int kVE = 16 / static_cast<int>(sizeof(T));
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= n_rows) return;
    const int nv = H / kVE;
    ptx::grid_dep_wait();
    uint4 xv[VPT], rv[VPT], wv[VPT];
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const int v = lane + u * 32;
        xv[u] = rv[u] = wv[u] = make_uint4(0, 0, 0, 0);
        if (v < nv) {
            xv[u] = reinterpret_cast<const uint4*>(x + row * H)[v];
            if (res) rv[u] = reinterpret_cast<const uint4*>(res + row * H)[v];
            wv[u] = reinterpret_cast<const uint4*>(weight)[v];
        }
    }
    norm_row<T, true, VPT>(xv, rv, wv, res != nullptr, eps, H, lane, 32,
                           res_out ? res_out + row * H : nullptr, y ? y + row * H : nullptr,
                           y_q ? y_q + row * H : nullptr, y_q ? y_scale + row : nullptr, nullptr);
}

// Rows blockIdx.x, blockIdx.x + gridDim.x, ..., one at a time per CTA, VPT
// vectors per thread.  The inputs of the next D - 1 rows are on their way into a
// ring in shared memory; each thread copies and reads its own columns only, so
// the ring needs no barrier, and an output may overlay the inputs of the same
// row.  (One row per CTA without the ring left the loads' latency in the open:
// 65 us against 39 for 4096 rows of 6144 bf16 with residual and codes.)
template <typename T, int VPT, int D, int MaxThreads>
__global__ void __launch_bounds__(MaxThreads) add_rmsnorm_kernel(
    const T* x, const T* res, const T* __restrict__ weight, float eps, int64_t n_rows, int H,
    T* res_out, T* y, uint8_t* y_q, float* __restrict__ y_scale) {
    constexpr int kVE = 16 / static_cast<int>(sizeof(T));
    extern __shared__ __align__(16) uint8_t s_ring[];
    __shared__ float s_red[2][64];
    const int tx = threadIdx.x, nt = blockDim.x;
    const int nv = H / kVE;
    uint4* ring = reinterpret_cast<uint4*>(s_ring);  // [D][x, res][nv]
    const int per_stage = (res ? 2 : 1) * nv;
    ptx::grid_dep_wait();
    auto fill = [&](int64_t row, int stage) {
        if (row < n_rows) {
#pragma unroll
            for (int u = 0; u < VPT; ++u) {
                const int v = tx + u * nt;
                if (v < nv) {
                    uint4* dst = ring + stage * per_stage + v;
                    ptx::cp_async_16(dst, reinterpret_cast<const uint4*>(x + row * H) + v, 16);
                    if (res)
                        ptx::cp_async_16(dst + nv,
                                         reinterpret_cast<const uint4*>(res + row * H) + v, 16);
                }
            }
        }
        ring_commit();
    };
#pragma unroll
    for (int d = 0; d < D; ++d) fill(blockIdx.x + static_cast<int64_t>(d) * gridDim.x, d);
    uint4 wv[VPT];
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const int v = tx + u * nt;
        wv[u] = v < nv ? reinterpret_cast<const uint4*>(weight)[v] : make_uint4(0, 0, 0, 0);
    }
    int stage = 0, flip = 0;
    for (int64_t row = blockIdx.x; row < n_rows; row += gridDim.x, flip ^= 1) {
        ring_wait<D - 1>();
        uint4 xv[VPT], rv[VPT];
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int v = tx + u * nt;
            xv[u] = rv[u] = make_uint4(0, 0, 0, 0);
            if (v < nv) {
                xv[u] = ring[stage * per_stage + v];
                if (res) rv[u] = ring[stage * per_stage + nv + v];
            }
        }
        fill(row + static_cast<int64_t>(D) * gridDim.x, stage);
        if (++stage == D) stage = 0;
        // two scratch rows in turn: the barrier inside the next row's reduction
        // separates this row's reads from the writes two rows later
        norm_row<T, false, VPT>(xv, rv, wv, res != nullptr, eps, H, tx, nt,
                                res_out ? res_out + row * H : nullptr, y ? y + row * H : nullptr,
                                y_q ? y_q + row * H : nullptr, y_q ? y_scale + row : nullptr,
                                s_red[flip]);
    }
}

// Backward over rows blockIdx.x, blockIdx.x + gridDim.x, ..., with the same ring:
// dx of each row, and the CTA's share of dw, kept in registers (a thread owns the
// same columns of every row) and written once to partial[blockIdx.x].  Rows of
// more than 1024 vectors take up to 1024 threads, so 64 registers each: a thread
// with 16 columns reads its part of the ring once more instead of keeping it (45 us
// for 2048 rows of 12288 bf16; spilled, it took 87; the fp32 forms still spill 16 and
// 36 bytes).  4096 rows of 6144 bf16 take
// 37 us, 5.4 TB/s, and the sum over the CTAs 2 us more.
template <typename T, int VPT, int D, int MaxThreads>
__global__ void __launch_bounds__(MaxThreads) add_rmsnorm_backward_kernel(
    const T* dy, const T* dres, const T* h, const T* __restrict__ weight, float eps,
    int64_t n_rows, int H, T* dx, float* __restrict__ partial) {
    constexpr int kVE = 16 / static_cast<int>(sizeof(T));
    extern __shared__ __align__(16) uint8_t s_ring[];
    __shared__ float s_red[2][64];
    const int tx = threadIdx.x, nt = blockDim.x;
    const int nv = H / kVE;
    constexpr bool kReread = VPT * kVE == 16 && MaxThreads == 1024;
    uint4* ring = reinterpret_cast<uint4*>(s_ring);  // [D][h, dy, dres][nv]
    const int per_stage = (dres ? 3 : 2) * nv;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    auto fill = [&](int64_t row, int stage) {
        if (row < n_rows) {
#pragma unroll
            for (int u = 0; u < VPT; ++u) {
                const int v = tx + u * nt;
                if (v < nv) {
                    uint4* dst = ring + stage * per_stage + v;
                    ptx::cp_async_16(dst, reinterpret_cast<const uint4*>(h + row * H) + v, 16);
                    ptx::cp_async_16(dst + nv, reinterpret_cast<const uint4*>(dy + row * H) + v,
                                     16);
                    if (dres)
                        ptx::cp_async_16(dst + 2 * nv,
                                         reinterpret_cast<const uint4*>(dres + row * H) + v, 16);
                }
            }
        }
        ring_commit();
    };
#pragma unroll
    for (int d = 0; d < D; ++d) fill(blockIdx.x + static_cast<int64_t>(d) * gridDim.x, d);
    uint4 wv[VPT];
    float dw[VPT][kVE];
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const int v = tx + u * nt;
        wv[u] = v < nv ? reinterpret_cast<const uint4*>(weight)[v] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < kVE; ++e) dw[u][e] = 0.0f;
    }
    int stage = 0, flip = 0;
    for (int64_t row = blockIdx.x; row < n_rows; row += gridDim.x, flip ^= 1) {
        ring_wait<D - 1>();
        const uint4* in = ring + stage * per_stage;
        const int from = stage;
        uint4 kept[kReread ? 1 : VPT][3];
        if constexpr (!kReread) {
#pragma unroll
            for (int u = 0; u < VPT; ++u) {
                const int v = tx + u * nt;
                kept[u][0] = kept[u][1] = kept[u][2] = make_uint4(0, 0, 0, 0);
                if (v < nv) {
                    kept[u][0] = in[v];
                    kept[u][1] = in[nv + v];
                    if (dres) kept[u][2] = in[2 * nv + v];
                }
            }
            fill(row + static_cast<int64_t>(D) * gridDim.x, from);
        }
        // vector u of h (0), dy (1) or dres (2)
        auto get = [&](int which, int u) {
            if constexpr (!kReread) return kept[u][which];
            const int v = tx + u * nt;
            return v < nv ? in[which * nv + v] : make_uint4(0, 0, 0, 0);
        };
        if (++stage == D) stage = 0;
        float sq = 0.0f, dot = 0.0f;
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            float hf[kVE], gf[kVE], wf[kVE];
            unpack_vec<T>(get(0, u), hf);
            unpack_vec<T>(get(1, u), gf);
            unpack_vec<T>(wv[u], wf);
#pragma unroll
            for (int e = 0; e < kVE; ++e) {
                sq = fmaf(hf[e], hf[e], sq);
                dot = fmaf(gf[e] * wf[e], hf[e], dot);
            }
        }
        row_reduce<false, false>(sq, dot, s_red[flip]);
        const float r = 1.0f / sqrtf(sq / static_cast<float>(H) + eps);
        const float c = r * r * (dot / static_cast<float>(H));  // mean(g * n) * r
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int v = tx + u * nt;
            float hf[kVE], gf[kVE], wf[kVE], rf[kVE];
            unpack_vec<T>(get(0, u), hf);
            unpack_vec<T>(get(1, u), gf);
            unpack_vec<T>(wv[u], wf);
            unpack_vec<T>(dres ? get(2, u) : make_uint4(0, 0, 0, 0), rf);
#pragma unroll
            for (int e = 0; e < kVE; ++e) {
                dw[u][e] = fmaf(gf[e], hf[e] * r, dw[u][e]);
                rf[e] = fmaf(r, gf[e] * wf[e] - hf[e] * c, rf[e]);
            }
            if (v < nv) reinterpret_cast<uint4*>(dx + row * H)[v] = pack_vec<T>(rf);
        }
        if constexpr (kReread) fill(row + static_cast<int64_t>(D) * gridDim.x, from);
    }
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
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

// dw[c] = sum of partial[0..n)[c] in a fixed order: 32 warps take every 32nd row
// of 32 columns, then their sums are added in warp order.
__global__ void __launch_bounds__(1024) reduce_columns_kernel(const float* __restrict__ partial,
                                                              int n, int H,
                                                              float* __restrict__ dw) {
    __shared__ float s_sum[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;  // H is a multiple of 64
    ptx::grid_dep_wait();
    float a = 0.0f;
#pragma unroll 4
    for (int i = warp; i < n; i += 32) a += partial[static_cast<int64_t>(i) * H + c];
    s_sum[warp][lane] = a;
    __syncthreads();
    if (warp == 0) {
        a = 0.0f;
#pragma unroll
        for (int w = 0; w < 32; ++w) a += s_sum[w][lane];
        dw[c] = a;
    }
}

}  // namespace moe
