// w4_kernels.cuh -- the experts' products with 4-bit weights and group scales.
//
// A weight is w = (u - 8) * s: u its 4-bit code, s the bf16 scale of its group
// of G (32, 64 or 128) consecutive weights along the contraction.  Products
// run on m16n8k16 bf16 MMAs with the weights as the 16-row operand, unpacked
// in registers, and the token rows as the 8 columns: u - 8 is exact in bf16,
// so a group's sum of (u - 8) * x carries fp32 rounding only; it is scaled and
// added to the fp32 total once per group.
//
// Layout.  Each matrix (gate/up: rows i of both, contraction H; down: rows h,
// contraction I) is cut into pair tiles of 2 x 16 rows (gate/up: 16 gate rows
// and the 16 up rows of the same i; down: 32 rows) and blocks of 128 along the
// contraction; the codes of a pair tile and block are 2 KB, those of a tile
// lie one block behind the other, so a warp reads one contiguous stream.  The
// 16 x 128 half of a block is 1 KB, 32 bytes (one load) for each of 32 lanes:
// lane 4r + c holds rows r (low nibble of each byte) and r + 8 (high nibble),
// word 2a + b of its 8 the k = 32 a + 8 c + 4 b + {0, 2, 1, 3} (one per byte):
// the A fragment of one MMA, a nibble of each half word per register.
// The matching B fragments of two MMAs are 8 consecutive values of a token row
// (one 16-byte load).  Scales: [tile][block][r 8][128/G][half][r, r + 8] bf16.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "device_common.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kW4Block = 128;       // contraction length of a block
constexpr int kW4BlockBytes = 2048; // codes of a pair tile's block
constexpr int kW4Threads = 256;

struct W4Args {
    const uint8_t* q;          // codes of expert 0's matrix
    const __nv_bfloat16* sc;   // its scales
    const uint8_t* q_shared;   // the same of the shared expert (segment `special`)
    const __nv_bfloat16* sc_shared;
    int64_t q_stride, sc_stride;  // bytes / scales from one expert to the next
    const int32_t* sched;      // tile schedule of nseg segments (chunk j: rows from j * 8 NT)
    int32_t nseg, special;
    const __nv_bfloat16* rows; // token rows [*, K] (down: [*, K/8, {hi, lo}, 8])
    const int32_t* row_src;    // gate/up: token of each routed row (special: the row itself)
    int32_t K, tiles;          // contraction length, pair tiles
    void* out;                 // gate/up: h rows as above; down: fp32 [*, ld]
    int32_t ld;
    const float* row_w;        // down: routing weight of each routed row
    int32_t routed_rows;       // rows from here on have weight 1
    float clip;
};

// 32 bytes that are read once: past L1, first to leave L2.
__device__ __forceinline__ void ldg_stream(const void* p, uint32_t (&v)[8]) {
    asm volatile(
        "ld.global.nc.L1::no_allocate.L2::evict_first.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7])
        : "l"(p));
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The 8 codes of a word as the A fragment of one MMA: 0x4300 | u is the bf16
// value 128 + u, and subtracting 136 leaves u - 8 exactly.
__device__ __forceinline__ void w4_fragment(uint32_t w, uint32_t (&a)[4]) {
    const __nv_bfloat162 off = __float2bfloat162_rn(136.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), off);
        a[i] = *reinterpret_cast<const uint32_t*>(&d);
    }
}

// The codes and scales of one block of a pair tile, as one lane holds them.
template <int SUB>
struct W4Stage {
    uint32_t a[2][8];          // [half]: word 2 * k32 + MMA
    __nv_bfloat162 s[SUB][2];  // [group][half]: scales of rows r and r + 8
};

template <int SUB>
__device__ __forceinline__ void w4_load(W4Stage<SUB>& st, const uint8_t* q,
                                        const __nv_bfloat16* sc) {
#pragma unroll
    for (int h = 0; h < 2; ++h) ldg_stream(q + h * 1024, st.a[h]);
    if constexpr (SUB == 1) {
        *reinterpret_cast<uint2*>(&st.s[0][0]) = __ldg(reinterpret_cast<const uint2*>(sc));
    } else {
#pragma unroll
        for (int u = 0; u < SUB; u += 2)
            *reinterpret_cast<uint4*>(&st.s[u][0]) =
                __ldg(reinterpret_cast<const uint4*>(sc + u * 4));
    }
}

// One warp per task: a pair tile against up to 8 NT token rows of one segment,
// over the whole contraction.  Tasks are numbered (segment, tile, chunk).
template <int NT, bool DOWN, int SUB>
__global__ void __launch_bounds__(kW4Threads) w4_product_kernel(const W4Args args) {
    const int lane = threadIdx.x & 31;
    const int r = lane >> 2, c = lane & 3;
    const int nkb = args.K / kW4Block;
    const SchedPtrs sp = sched_ptrs(args.sched, args.nseg);
    if constexpr (!DOWN) ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int64_t total = static_cast<int64_t>(sp.prefix[args.nseg]) * args.tiles;
    bool waited = !DOWN;
    for (int64_t task = static_cast<int64_t>(blockIdx.x) * (kW4Threads / 32) + (threadIdx.x >> 5);
         task < total; task += static_cast<int64_t>(gridDim.x) * (kW4Threads / 32)) {
        // segment: the last one whose first task is not behind this one
        int lo = 0, hi = args.nseg - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (static_cast<int64_t>(sp.prefix[mid]) * args.tiles <= task) lo = mid;
            else hi = mid - 1;
        }
        const int seg = lo;
        const int chunks = sp.prefix[seg + 1] - sp.prefix[seg];
        const int in_seg = static_cast<int>(task - static_cast<int64_t>(sp.prefix[seg]) * args.tiles);
        const int tile = in_seg / chunks;
        const int row0 = (in_seg - tile * chunks) * (8 * NT);
        const int nrows = min(8 * NT, sp.rows[seg] - row0);
        const bool special = seg == args.special;
        const uint8_t* q = (special ? args.q_shared : args.q + seg * args.q_stride) +
                           static_cast<int64_t>(tile) * nkb * kW4BlockBytes + lane * 32;
        const __nv_bfloat16* sc = (special ? args.sc_shared : args.sc + seg * args.sc_stride) +
                                  (static_cast<int64_t>(tile) * nkb * 8 + r) * SUB * 4;
        W4Stage<SUB> st[2];
        w4_load<SUB>(st[0], q, sc);
        if (nkb > 1) w4_load<SUB>(st[1], q + kW4BlockBytes, sc + 32 * SUB);
        if (!waited) {
            ptx::grid_dep_wait();
            waited = true;
        }
        // token rows: columns past the chunk's last row repeat it (not stored)
        const __nv_bfloat16* b[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int row = sp.b_row0[seg] + row0 + min(8 * n + r, nrows - 1);
            const int64_t at = (!DOWN && !special) ? args.row_src[row] : row;
            b[n] = args.rows + at * args.K * (DOWN ? 2 : 1) + c * (DOWN ? 16 : 8);
        }
        float tot[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) tot[h][n][i] = 0.0f;

        auto block = [&](const W4Stage<SUB>& s, int kb) {
            float acc[2][NT][4];
#pragma unroll
            for (int k32 = 0; k32 < 4; ++k32) {
                if (k32 % (4 / SUB) == 0) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[h][n][i] = 0.0f;
                }
                uint4 bv[NT], bl[DOWN ? NT : 1];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int64_t at = (static_cast<int64_t>(kb) * 128 + k32 * 32) * (DOWN ? 2 : 1);
                    bv[n] = *reinterpret_cast<const uint4*>(b[n] + at);
                    if constexpr (DOWN) bl[n] = *reinterpret_cast<const uint4*>(b[n] + at + 8);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t f[4];
                    w4_fragment(s.a[h][2 * k32], f);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma_bf16(acc[h][n], f, bv[n].x, bv[n].y);
                        if constexpr (DOWN) mma_bf16(acc[h][n], f, bl[n].x, bl[n].y);
                    }
                    w4_fragment(s.a[h][2 * k32 + 1], f);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma_bf16(acc[h][n], f, bv[n].z, bv[n].w);
                        if constexpr (DOWN) mma_bf16(acc[h][n], f, bl[n].z, bl[n].w);
                    }
                }
                if ((k32 + 1) % (4 / SUB) == 0) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float2 sv = __bfloat1622float2(s.s[k32 / (4 / SUB)][h]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            tot[h][n][0] = fmaf(sv.x, acc[h][n][0], tot[h][n][0]);
                            tot[h][n][1] = fmaf(sv.x, acc[h][n][1], tot[h][n][1]);
                            tot[h][n][2] = fmaf(sv.y, acc[h][n][2], tot[h][n][2]);
                            tot[h][n][3] = fmaf(sv.y, acc[h][n][3], tot[h][n][3]);
                        }
                    }
                }
            }
        };
        for (int kb = 0; kb < nkb; kb += 2) {
            block(st[0], kb);
            if (kb + 2 < nkb) w4_load<SUB>(st[0], q + static_cast<int64_t>(kb + 2) * kW4BlockBytes, sc + static_cast<int64_t>(kb + 2) * 32 * SUB);
            if (kb + 1 < nkb) {
                block(st[1], kb + 1);
                if (kb + 3 < nkb) w4_load<SUB>(st[1], q + static_cast<int64_t>(kb + 3) * kW4BlockBytes, sc + static_cast<int64_t>(kb + 3) * 32 * SUB);
            }
        }
        // lane 4r + c holds rows r and r + 8 of both halves, columns 2c, 2c + 1
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = 8 * n + 2 * c + j;
                if (col >= nrows) continue;
                const int64_t m = sp.out_row0[seg] + row0 + col;
                if constexpr (!DOWN) {
                    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(args.out) + m * args.ld * 2 +
                                       tile * 32 + r;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        float g = tot[0][n][2 * t + j], u = tot[1][n][2 * t + j];
                        // compare-select clamp: NaN passes through
                        g = g > args.clip ? args.clip : (g < -args.clip ? -args.clip : g);
                        u = u > args.clip ? args.clip : (u < -args.clip ? -args.clip : u);
                        const float v = g / (1.0f + __expf(-g)) * u;
                        const __nv_bfloat16 hi = __float2bfloat16_rn(v);
                        // the remainder of a non-finite value would be NaN
                        const float rem = v - __bfloat162float(hi);
                        o[t * 16] = hi;
                        o[t * 16 + 8] = __float2bfloat16_rn(isfinite(rem) ? rem : 0.0f);
                    }
                } else {
                    const float wt = m < args.routed_rows ? args.row_w[m] : 1.0f;
                    float* o = static_cast<float*>(args.out) + m * args.ld + tile * 32 + r;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int t = 0; t < 2; ++t)
                            o[h * 16 + t * 8] = wt * tot[h][n][2 * t + j];
                }
            }
        }
    }
    if (!waited) ptx::grid_dep_wait();
}

// Dispatch of up to kPermTokens tokens in one CTA of 512 threads: histogram,
// offsets, tile schedules and stable positions (row order: expert, token), as
// the three dispatch launches compute them for any number of tokens.  pos of
// an assignment with an expert out of range is -1.
__global__ void __launch_bounds__(512) w4_dispatch_kernel(
    const int32_t* __restrict__ idx, const float* __restrict__ topk_w, int T, int E, int k,
    int num_shared, int nmax, int32_t* sched_gu, int32_t* sched_dn, int32_t* __restrict__ pos,
    int32_t* __restrict__ src, float* __restrict__ row_w, int32_t* status) {
    __shared__ uint32_t masks[kPermWarps][kMaxExperts];
    __shared__ int32_t wbase[kPermWarps][kMaxExperts];
    __shared__ int s_warp[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < kPermWarps * kMaxExperts; i += blockDim.x) (&masks[0][0])[i] = 0u;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    __syncthreads();
    if (warp < kPermWarps) build_lane_masks(idx, T, E, k, tid, masks[warp], status);
    __syncthreads();
    int cnt = 0;
    if (tid < E) {
#pragma unroll
        for (int w = 0; w < kPermWarps; ++w) cnt += __popc(masks[w][tid]);
    }
    const int off = block_exclusive_scan(cnt, s_warp, nullptr);
    if (tid < E) {
        int running = off;
#pragma unroll
        for (int w = 0; w < kPermWarps; ++w) {
            wbase[w][tid] = running;
            running += __popc(masks[w][tid]);
        }
    }
    const int nseg = E + num_shared;
    const bool shared = num_shared && tid == E;
    const int rows = tid < E ? cnt : (shared ? T : 0);
    int total = 0;
    const int pre = block_exclusive_scan((rows + nmax - 1) / nmax, s_warp, &total);
    if (tid < nseg) {
        const int o0 = shared ? T * k : off;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const SchedPtrs sp = sched_ptrs(which == 0 ? sched_gu : sched_dn, nseg);
            const_cast<int32_t*>(sp.prefix)[tid] = pre;
            const_cast<int32_t*>(sp.b_row0)[tid] = shared && which == 0 ? 0 : o0;
            const_cast<int32_t*>(sp.out_row0)[tid] = o0;
            const_cast<int32_t*>(sp.rows)[tid] = rows;
            if (tid == 0) const_cast<int32_t*>(sp.prefix)[nseg] = total;
        }
    }
    __syncthreads();
    if (tid < T) {
        const uint32_t lt = (1u << lane) - 1u;
        for (int j = 0; j < k; ++j) {
            const int e = idx[tid * k + j];
            int p = -1;
            if (e >= 0 && e < E) {
                p = wbase[warp][e] + __popc(masks[warp][e] & lt);
                src[p] = tid;
                row_w[p] = topk_w[tid * k + j];
            }
            pos[tid * k + j] = p;
        }
    }
}

// Encoder: one CTA of 128 threads per 16-row half of a pair tile and block.
// Row i of the half and k of the block come from in[...] with the strides of
// the matrix (gate/up: k contiguous; down: rows contiguous).
// scale = bf16(max |w| / 7) (1 where that is 0, NaN where the group holds a
// value that is not finite), code = nearest integer to w / scale, ties to
// even, held to [-7, 7], plus 8.
template <typename T, int SUB>
__global__ void __launch_bounds__(128) w4_encode_kernel(const T* __restrict__ w, int I, int H,
                                                        uint8_t* __restrict__ q,
                                                        __nv_bfloat16* __restrict__ scales) {
    __shared__ float tile[16][kW4Block + 1];
    __shared__ float s_sc[16][4];
    const int tid = threadIdx.x;
    const int64_t n = blockIdx.y;  // expert
    // halves of the gate/up tiles' blocks, then of the down tiles'
    const int gu = (I / 16) * (H / kW4Block) * 2;
    int id = blockIdx.x;
    const bool down = id >= gu;
    if (down) id -= gu;
    const int half = id & 1;
    const int nkb = (down ? I : H) / kW4Block;
    const int kb = (id >> 1) % nkb, t = (id >> 1) / nkb;
    const T* in = w + n * 3 * I * H;
    if (!down) {
        in += static_cast<int64_t>(half) * I * H + static_cast<int64_t>(t) * 16 * H + kb * kW4Block;
        for (int i = tid; i < 16 * kW4Block; i += 128)
            tile[i / kW4Block][i % kW4Block] =
                static_cast<float>(in[static_cast<int64_t>(i / kW4Block) * H + i % kW4Block]);
    } else {
        in += 2 * static_cast<int64_t>(I) * H + static_cast<int64_t>(kb) * kW4Block * H + t * 32 +
              half * 16;
        for (int i = tid; i < 16 * kW4Block; i += 128)
            tile[i % 16][i / 16] = static_cast<float>(in[static_cast<int64_t>(i / 16) * H + i % 16]);
    }
    __syncthreads();
    {
        // thread (row, eighth) scans 16 values; a group is 8 / SUB eighths
        const int row = tid >> 3, part = tid & 7;
        float amax = 0.0f;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float v = tile[row][part * 16 + i];
            amax = fmaxf(amax, fabsf(v));
            bad |= !isfinite(v);
        }
#pragma unroll
        for (int o = 1; o < 8 / SUB; o <<= 1) {
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            bad |= __shfl_xor_sync(0xffffffffu, bad ? 1 : 0, o) != 0;
        }
        float s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(amax, 7.0f)));
        if (s == 0.0f) s = 1.0f;
        if (bad) s = __int_as_float(0x7fc00000);
        if (part % (8 / SUB) == 0) s_sc[row][part / (8 / SUB)] = s;
    }
    __syncthreads();
    const int64_t unit = static_cast<int64_t>(t) * nkb + kb;  // block of a pair tile
    {
        uint8_t* qo = q + n * (3ll * I * H / 2) + (down ? static_cast<int64_t>(I) * H : 0) +
                      unit * kW4BlockBytes + half * 1024;
        for (int word = tid; word < 256; word += 128) {
            const int ln = word >> 3, wd = word & 7;
            const int r = ln >> 2, c = ln & 3;
            const int k0 = 32 * (wd >> 1) + 8 * c + 4 * (wd & 1);
            uint32_t out = 0;
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const int row = r + 8 * (p & 1);
                const int k = k0 + 2 * ((p >> 1) & 1) + (p >> 2);
                const float v = tile[row][k], s = s_sc[row][k / (kW4Block / SUB)];
                int code = 0;
                if (s == s) {
                    // nearest of the two neighbours by the sign of the exact
                    // remainder at their midpoint (s has 8 significant bits
                    // and the midpoint 4, so the product is exact)
                    const float lo = floorf(__fdiv_rn(v, s));
                    const float rem = fmaf(-s, lo + 0.5f, v);
                    const int l = static_cast<int>(lo);
                    code = rem > 0.0f ? l + 1 : (rem < 0.0f ? l : l + (l & 1));
                    code = min(7, max(-7, code));
                }
                out |= static_cast<uint32_t>(code + 8) << (4 * p);
            }
            reinterpret_cast<uint32_t*>(qo)[word] = out;
        }
    }
    if (tid < 16 * SUB) {
        const int row = tid / SUB, g = tid % SUB;
        __nv_bfloat16* so = scales + n * (3ll * I * H / (kW4Block / SUB)) +
                            (down ? 2ll * I * H / (kW4Block / SUB) : 0) + unit * 32 * SUB;
        so[((row % 8) * SUB + g) * 4 + half * 2 + row / 8] = __float2bfloat16_rn(s_sc[row][g]);
    }
}

}  // namespace moe
