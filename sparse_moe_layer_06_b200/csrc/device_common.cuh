// device_common.cuh -- device pieces that more than one translation unit of the
// library uses: the device error word, the tile-schedule layout, the dispatch's
// lane masks and block scan, 16-byte vector unpacking and the power-of-two
// E4M3 scale.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "route_topk.cuh"

namespace moe {

enum DeviceError : int { DEV_OK = 0, DEV_ERR_TIMEOUT = 5, DEV_ERR_BAD_INDEX = 6 };

__device__ __forceinline__ void set_device_error(int32_t* status, int code) {
    if (status) atomicCAS(status, 0, code);
}

// Device-built tile schedule for nseg segments (a segment = the rows that
// share one weight matrix).  int32 array of 5*(nseg+1) entries:
//   prefix[nseg+1]  exclusive prefix sum of per-segment chunk counts
//   b_row0[nseg]    first row of the segment in its B tensor map
//   out_row0[nseg]  first row of the segment in the output row space
//   rows[nseg]      rows in the segment
//   chunk_len[nseg] rows per chunk (multiple of 16, <= NMAX)
// Tiles are ordered (segment, chunk, weight block) with the weight block
// fastest, so the CTAs working at the same time share one chunk of token rows
// and, across neighbouring chunks, the same weight blocks through L2.
struct SchedPtrs {
    const int32_t* prefix;
    const int32_t* b_row0;
    const int32_t* out_row0;
    const int32_t* rows;
    const int32_t* chunk_len;
};

__host__ __device__ inline SchedPtrs sched_ptrs(const int32_t* base, int nseg) {
    SchedPtrs p;
    p.prefix = base;
    p.b_row0 = base + (nseg + 1);
    p.out_row0 = base + 2 * (nseg + 1);
    p.rows = base + 3 * (nseg + 1);
    p.chunk_len = base + 4 * (nseg + 1);
    return p;
}

constexpr int kMaxSegments = 257;  // 256 routed experts + 1 shared expert

// ------------------------------------------------------------------ dispatch

constexpr int kPermTokens = 256;  // tokens per dispatch chunk (one CTA, 8 warps)
constexpr int kPermWarps = kPermTokens / 32;

// Build, for the warp's 32 tokens, one bit mask per expert of the lanes whose
// token routes to it.  A token's k experts must be distinct; a repeat, or an
// index outside [0,E), is reported through `status` and skipped.
__device__ __forceinline__ void build_lane_masks(const int32_t* __restrict__ idx, int64_t T, int E,
                                                 int k, int64_t t, uint32_t* warp_masks,
                                                 int32_t* status) {
    const int lane = threadIdx.x & 31;
    if (t < T) {
        for (int j = 0; j < k; ++j) {
            const int e = idx[t * k + j];
            if (e < 0 || e >= E) {
                set_device_error(status, DEV_ERR_BAD_INDEX);
                continue;
            }
            const uint32_t old = atomicOr(&warp_masks[e], 1u << lane);
            if (old & (1u << lane)) set_device_error(status, DEV_ERR_BAD_INDEX);
        }
    }
}

// Exclusive prefix sum over the CTA (blockDim.x a multiple of 32, <= 1024).
// `s_warp` is 32 ints of shared scratch; every thread must call it.
__device__ __forceinline__ int block_exclusive_scan(int v, int* s_warp, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nwarps = blockDim.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = lane < nwarps ? s_warp[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    const int result = (warp > 0 ? s_warp[warp - 1] : 0) + x - v;
    if (total) *total = s_warp[nwarps - 1];
    __syncthreads();
    return result;
}

// ------------------------------------------------------------------ vectors and scales

// The 16 / sizeof(T) values of a 16-byte vector as fp32.
template <typename T>
__device__ __forceinline__ void unpack_vec(const uint4& q, float (&f)[16 / sizeof(T)]) {
    if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162* h2 = reinterpret_cast<const __nv_bfloat162*>(&q);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 v = __bfloat1622float2(h2[e]);
            f[2 * e] = v.x;
            f[2 * e + 1] = v.y;
        }
    } else {
        f[0] = __uint_as_float(q.x);
        f[1] = __uint_as_float(q.y);
        f[2] = __uint_as_float(q.z);
        f[3] = __uint_as_float(q.w);
    }
}

// Scale of an E4M3 channel whose largest magnitude is amax: 2^n with n the
// smallest integer such that 448 * 2^n >= amax, and 1 for amax = 0.  n is held
// to [-126, 120], where 2^n and 2^-n are both normal: the upper end is what the
// largest finite float needs (an infinite amax takes it too, its codes then
// saturate), and below the lower end the codes only lose subnormal magnitudes.
// amax = m * 2^e with 1 <= m < 2, and 448 = 1.75 * 2^8: n = e - 8 where
// m <= 1.75, else e - 7.
__device__ __forceinline__ float pow2_scale_f(float amax) {
    if (!(amax > 0.0f)) return 1.0f;
    const uint32_t bits = __float_as_uint(amax);
    const int e = static_cast<int>(bits >> 23) - 127;  // (-127 for subnormal amax: clamped below)
    int n = (bits & 0x7fffffu) <= 0x600000u ? e - 8 : e - 7;
    n = min(max(n, -126), 120);
    return __uint_as_float(static_cast<uint32_t>(n + 127) << 23);
}

}  // namespace moe
