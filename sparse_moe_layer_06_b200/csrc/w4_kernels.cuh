// w4_kernels.cuh -- the experts' products with 4-bit weights and group scales.
//
// A weight is w = (u - 8) * s: u its 4-bit code, s the bf16 scale of its group
// of G (32, 64 or 128) consecutive weights along the contraction.
//
// The products run on m16n8k32 integer MMAs (u8 codes x s8 limbs, exact s32
// sums).  A mask of a packed word is an A register as it stands, the low nibbles
// u of one row or the high ones, 16 u, of another: two ALU steps for 8 codes (a
// bf16 fragment takes 7, and ran the first form of these kernels into the ALU
// pipe, which has half rate).  A token row is split, per block of 128 values,
// into a power-of-two scale a and 16-bit integers v = 256 hi + lo with two s8
// limbs: bf16 values down to 2^-6 of the block's largest are exact, smaller ones
// off by at most a / 2, 2^-14.9 of the largest.  On rows without outliers that is
// far inside the bf16 output's rounding (4e-6 of an output against 1.7e-3).  Beside
// an outlier it is not: 1000 times the others, which hidden states have, and an
// output whose weight there is 0 was off by 1%.  So where the values below 1024 a are
// three quarters of a block or more and lose more than 2^-9 of their norm (about what
// bf16 takes of fp32 values), the block is marked: the remainders x - a v, exact in
// fp32, are split in the same way into a second integer with a scale of its own, and
// a chunk's blocks with such a row are taken a second time; a value is then off by at
// most 2^-29.8 of the block's largest.  (Of 10^6 blocks of normally, uniformly or
// exponentially distributed values, or of products of such, none is marked.  64
// tokens, 256 experts: 673 us a call for ordinary rows, 797 with three such channels
// in every row, 1056 with eight; the code for it costs ordinary rows 0 to 3%.)
// With the sums of the limbs of each group,
//   sum_k (u_k - 8) s x_k = s a (256 (sum u hi - 8 sum hi) + (sum u lo - 8 sum lo)):
// the accumulators start from -8 times the limb sums, and the joined integer,
// below 2^29, is converted, scaled and added to the fp32 total once per group.
//
// Layout.  Each matrix (gate/up: rows i of both, contraction H; down: rows h,
// contraction I) is cut into pair tiles of 2 x 16 rows (gate/up: 16 gate rows
// and the 16 up rows of the same i; down: 32 rows) and blocks of 128 along the
// contraction; the codes of a pair tile and block are 2 KB, those of a tile
// lie one block behind the other, so a warp reads one contiguous stream.  The
// 16 x 128 half of a block is 1 KB, 32 bytes (one load) for each of 32 lanes:
// lane 4r + c holds rows r (low nibble of each byte) and r + 8 (high nibble),
// word 2a + b of its 8 the k = 32 a + 8 c + 4 b + {0, 2, 1, 3} (one per byte):
// with both words of a, the A fragments of one MMA.
// Scales: [tile][block][r 8][128/G][half][r, r + 8] bf16.
// Limbs of a row and block, 256 bytes: [a / 2][limb][c 4][a % 2][8 bytes], the 8
// bytes in the order of the two words; in an array of their own the multiples of
// the limb sums, the scale and whether there is a second integer (whose limbs and
// sums lie in two more such arrays), w4_meta_words words per row and block.
//
// Measured, with 256 experts of 6144 x 2048, eight per token, and a shared one: 64
// tokens take 435 and 233 us for the two products (2.9 and 1.45 GB of codes and
// scales: 6.7 and 6.2 TB/s), 256 tokens 784 and 402 us, where the issue slots bound
// (53% of the cycles with 3 warps a scheduler, each waiting mostly on its own
// previous instruction; DRAM at 51%).  One token: 28 and 19 us for 9 experts, of
// which 17 and 9 are the weights' share and the rest the start of each launch.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>
#include <type_traits>

#include "device_common.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kW4Block = 128;       // contraction length of a block
constexpr int kW4BlockBytes = 2048; // codes of a pair tile's block
constexpr int kW4RowBytes = 256;    // limbs of a row's block
constexpr int kW4MaxK = 65536;      // longest contraction (a row's limbs: 147 KB)

// Shape of a launch whose tasks have up to 8 NT rows, in groups of 128 / SUB: one
// CTA per SM.  One column tile leaves 128 registers a thread and so 16 warps; two,
// or the scales of groups of 32, take up to 168 (for 37 tokens of 32 experts of
// 7168 x 2048 and groups of 32 the two products took a tenth longer with 16 warps;
// for 256 tokens and two column tiles 14 warps take a fifth longer than 12).  The
// forms with two column tiles spill 20 to 106 bytes, that with one and groups of 64
// spills 16.
template <int NT, int SUB>
struct W4Shape {
    static constexpr int kWarps = NT == 1 && SUB < 4 ? 16 : 12;
    static constexpr int kMostLog = kWarps == 16 ? 4 : 3;  // log2 of the warps that share a tile
    static constexpr int kAhead = NT;  // blocks behind its next one that L2 has on the way
    static constexpr int kVals = 2 * NT * 4 * 32;         // fp32 sums of a tile
    static constexpr int kSumBytes = 2 * kWarps * kVals * 4;  // two buffers of them
    static constexpr int kSlack = 8 * NT * kW4RowBytes;   // rows read past the last block
};

// Beside a row's block stand -8 times the sums of its two limbs over each group
// of at most 64 values (w4_sums of them: a pair of int32 each), then the scale and
// the mark of a second integer (0 or 1); words of that per row and block, whole
// 16-byte vectors.
__host__ __device__ constexpr int w4_sums(int sub) { return sub == 4 ? 4 : 2; }
__host__ __device__ constexpr int w4_meta_words(int sub) { return sub == 4 ? 12 : 8; }
__host__ __device__ constexpr int w4_mark(int sub) { return 2 * w4_sums(sub) + 1; }
constexpr int kW4MaxMeta = 12;

// The integers of rows: limbs, and group sums with scales.
struct W4Rows {
    uint8_t* limbs;
    uint32_t* meta;
};

// Rows of K values that fit beside the sums and the schedule (5 KB) in a CTA's
// shared memory, at most 8 NT.
template <int NT, int SUB>
int w4_rows_cap(int64_t K) {
    using S = W4Shape<NT, SUB>;
    const int64_t row = K / kW4Block * (kW4RowBytes + 4 * w4_meta_words(SUB));
    const int64_t cap = (220 * 1024 - S::kSumBytes - S::kSlack) / row;
    return static_cast<int>(cap < 8 * NT ? cap : 8 * NT);
}

struct W4Args {
    const uint8_t* q;          // codes of expert 0's matrix
    const __nv_bfloat16* sc;   // its scales
    const uint8_t* q_shared;   // the same of the shared expert (segment `special`)
    const __nv_bfloat16* sc_shared;
    int64_t q_stride, sc_stride;  // bytes / scales from one expert to the next
    const int32_t* sched;      // tile schedule of nseg segments (chunk j: rows from j * cap)
    int32_t nseg, special;
    W4Rows rows, rest;         // the token rows' integers, and the second ones
    const int32_t* row_src;    // gate/up: token of each routed row (special: the row itself)
    int32_t K, tiles, cap;     // contraction length, pair tiles, rows of a chunk
    float* out;                // gate/up: h rows, down: weighted rows; fp32 [*, ld]
    int32_t ld;
    const float* row_w;        // down: routing weight of each routed row
    int32_t routed_rows;       // rows from here on have weight 1
    float clip;
};

// d = c + a b
__device__ __forceinline__ void mma_u8s8(int32_t (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, const int32_t (&c)[4]) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(c[0]), "r"(c[1]),
          "r"(c[2]), "r"(c[3]));
}

// 32 bytes that are read once: past L1, first to leave L2.
__device__ __forceinline__ void ldg_stream(const void* p, uint32_t (&v)[8]) {
    asm volatile(
        "ld.global.nc.L1::no_allocate.L2::evict_first.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7])
        : "l"(p));
}

// Brings bytes (a multiple of 16, 16-byte aligned) on their way into L2.
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// The codes and scales of one block of a pair tile, as one lane holds them.
template <int SUB>
struct W4Stage {
    uint32_t a[2][8];  // [half]: word 2 * k32 + j
    uint2 s[SUB];      // [group]: half 0's and half 1's scales of rows r and r + 8
};

// The four values v of each lane (128 of a block) as the integers rint(v / a) of one
// scale, by one warp, and what is left of them in v.  The scale is the power of two a
// with 16191 <= amax / a <= 32384, which leaves both limbs in range (32640 would need
// 128).  A block with a value that is not finite gets a NaN scale, so its row's results
// are NaN.  Returns whether the block is marked: at most 32 values from 1024 a on, and
// the others lose more than 2^-9 of their 2-norm.  (An output's weights are hardly 0 at
// more than 32 larger values; a block of 128 normally distributed ones has 111 to 119 of
// them, and without that condition 2.5e-5 of such blocks would be marked, a few in each
// call for 256 tokens, each of which held its CTA up by 100 us.)
__device__ __forceinline__ bool w4_split_values(float (&v)[4], int sub, uint8_t* __restrict__ out,
                                                uint32_t* __restrict__ meta) {
    const int lane = threadIdx.x & 31;
    float amax = 0.0f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        amax = fmaxf(amax, fabsf(v[i]));
        bad |= !isfinite(v[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    bad = __any_sync(0xffffffffu, bad);
    // amax = m * 2^e, 1 <= m < 2; a = 2^(e-14), twice that for m > 253/128.  a and
    // 1 / a stay normal: blocks below 2^-112 keep an absolute step of 2^-127
    const uint32_t bits = __float_as_uint(amax);
    int n = static_cast<int>(bits >> 23) - 127 - 14 + ((bits & 0x7fffffu) > 0x7d0000u ? 1 : 0);
    n = min(max(n, -126), 126);
    const float scale = __uint_as_float(static_cast<uint32_t>(n + 127) << 23);
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - n) << 23);
    out += (lane >> 4) * 128 + ((lane & 7) >> 1) * 16 + ((lane >> 3) & 1) * 8 + (lane & 1) * 4;
    uint32_t hi = 0, lo = 0;
    int sum_hi = 0, sum_lo = 0;
    float off = 0.0f;  // sum of (u - t)^2 - 2^-18 u^2 over the small u = v / a
    int large = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float u = v[i] * inv;
        const int t = bad ? 0 : __float2int_rn(u);
        const int l = static_cast<int8_t>(t & 0xff), h = (t - l) >> 8;
        const int at = ((i & 1) << 1) | (i >> 1);  // bytes k, k + 2, k + 1, k + 3
        hi |= static_cast<uint32_t>(h & 0xff) << (8 * at);
        lo |= static_cast<uint32_t>(l & 0xff) << (8 * at);
        sum_hi += h;
        sum_lo += l;
        const float rest = u - static_cast<float>(t);  // exact: |t| < 2^15, |rest| <= 1/2
        const bool small = fabsf(u) < 1024.0f;
        if (small) off += rest * rest - 0x1p-18f * (u * u);
        large += __popc(__ballot_sync(0xffffffffu, !small));
        v[i] = rest * scale;
    }
    *reinterpret_cast<uint32_t*>(out) = hi;
    *reinterpret_cast<uint32_t*>(out + 64) = lo;
    const int sums = w4_sums(sub), per = 32 / sums;  // lanes of a group
    for (int o = 1; o < per; o <<= 1) {
        sum_hi += __shfl_xor_sync(0xffffffffu, sum_hi, o);
        sum_lo += __shfl_xor_sync(0xffffffffu, sum_lo, o);
    }
    if (lane % per == 0)
        *reinterpret_cast<int2*>(meta + lane / per * 2) = make_int2(-8 * sum_hi, -8 * sum_lo);
    if (lane == 0) meta[2 * sums] = bad ? 0x7fc00000u : __float_as_uint(scale);
    // (at the smallest scale the remainders would have no smaller one)
    if (bad || n <= -126 || large > 32) return false;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) off += __shfl_xor_sync(0xffffffffu, off, o);
    return off > 0.0f;
}

// Row block `unit` of rows in [*, K] order, by one warp: lane l has the values
// 4 l .. 4 l + 3.
template <typename T>
__device__ __forceinline__ void w4_split_block(const T* __restrict__ rows, int sub, int64_t unit,
                                               const W4Rows& out, const W4Rows& rest) {
    const int lane = threadIdx.x & 31;
    float v[4];
    const T* in = rows + unit * kW4Block + lane * 4;
    if constexpr (sizeof(T) == 2) {
        const uint2 q = *reinterpret_cast<const uint2*>(in);
        const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&q.x));
        const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&q.y));
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    } else {
        const float4 q = *reinterpret_cast<const float4*>(in);
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    }
    const int64_t m = unit * w4_meta_words(sub);
    const bool more = w4_split_values(v, sub, out.limbs + unit * kW4RowBytes, out.meta + m);
    if (lane == 0) out.meta[m + w4_mark(sub)] = more ? 1 : 0;
    if (more) {
        w4_split_values(v, sub, rest.limbs + unit * kW4RowBytes, rest.meta + m);
        if (lane == 0) rest.meta[m + w4_mark(sub)] = 1;
    }
}

template <typename T>
__global__ void __launch_bounds__(256) w4_split_kernel(const T* __restrict__ rows, int64_t units,
                                                       int sub, W4Rows out, W4Rows rest) {
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (unit < units) w4_split_block<T>(rows, sub, unit, out, rest);
}

// The tile schedule in shared memory.
struct W4Sched {
    int32_t prefix[kMaxSegments + 1], b_row0[kMaxSegments], out_row0[kMaxSegments],
        rows[kMaxSegments];
};

// What a chunk of so many rows counts for when the CTAs share out the tasks.  With
// equal shares the CTAs that met the larger chunks set the time: their loads come
// later than the others', which take the memory's bandwidth meanwhile.
constexpr int kW4CostFew = 3, kW4CostOne = 5, kW4CostTwo = 8;
template <int NT>
__device__ __forceinline__ int w4_cost(int rows) {
    if (NT == 1) return rows <= 4 ? kW4CostFew : kW4CostOne;
    return rows <= 8 ? kW4CostOne : kW4CostTwo;
}

// First task that starts at place x or behind it; a segment s with its tiles takes
// the places from cost[s] * tiles on.
template <int NT>
__device__ __forceinline__ int64_t w4_task_at(const W4Sched& sp, const int32_t* cost, int nseg,
                                              int cap, int tiles, int64_t x) {
    const int at = static_cast<int>(x / tiles);
    if (at >= cost[nseg]) return static_cast<int64_t>(sp.prefix[nseg]) * tiles;
    int lo = 0, hi = nseg - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cost[mid] <= at) lo = mid;
        else hi = mid - 1;
    }
    const int chunks = sp.prefix[lo + 1] - sp.prefix[lo], full = w4_cost<NT>(cap);
    const int j = min((at - cost[lo]) / full, chunks - 1);
    const int rest = static_cast<int>(x - static_cast<int64_t>(cost[lo] + j * full) * tiles);
    const int own = w4_cost<NT>(min(cap, sp.rows[lo] - j * cap));
    return static_cast<int64_t>(sp.prefix[lo] + j) * tiles + (rest + own - 1) / own;
}

// A round of a CTA: `tiles` tiles from `tile` on of one chunk of rows (chunk
// number `group` of the launch), each shared by 2^log_ks warps.
struct W4Round {
    int group, seg, row0, nrows;  // the chunk's segment and rows of it
    int tile, tiles;
    int log_ks;
    int left;  // tasks of the CTA behind this round
};

// Segment and rows of chunk p.group: the segment is the last whose first chunk
// is not behind it.
__device__ __forceinline__ void w4_find_chunk(W4Round& p, const W4Sched& sp, int nseg, int cap) {
    int lo = 0, hi = nseg - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sp.prefix[mid] <= p.group) lo = mid;
        else hi = mid - 1;
    }
    p.seg = lo;
    p.row0 = (p.group - sp.prefix[lo]) * cap;
    p.nrows = min(cap, sp.rows[lo] - p.row0);
}

// The round behind `p` (p.tiles = 0: the first one, p.tile its tile): as many
// tiles as the warps hold at 2^base warps each, or, for fewer tiles than that,
// as many as keep all warps busy.
template <int kWarps>
__device__ __forceinline__ void w4_next_round(W4Round& p, const W4Sched& sp, int all_tiles,
                                              int nseg, int cap, int base, int most) {
    p.tile += p.tiles;
    if (p.tile == all_tiles) {
        p.tile = 0;
        ++p.group;
        w4_find_chunk(p, sp, nseg, cap);
    }
    const int rem = min(all_tiles - p.tile, p.left);
    int l = base;
    while (l < most && (kWarps >> l) > rem) ++l;
    p.log_ks = l;
    p.tiles = min(kWarps >> l, rem);
    p.left -= p.tiles;
}

// One CTA per SM takes a run of consecutive tasks, numbered (segment, chunk,
// tile), each a pair tile against the chunk's rows.  The chunk's limbs lie in
// shared memory (16-byte piece p of a row and block at p ^ 4 (row % 2), so that
// the 8 lanes of a read meet different banks): taken through L1 instead, they
// cost more than the weights (700 us for the gate/up of 64 tokens).  2^log_ks
// warps share a tile, each with a part of its blocks; their fp32 sums are added in
// shared memory in warp order.  The weights stream through registers past L1, one
// block at a time and across rounds, with a prefetch of the next kAhead blocks into
// L2.  (Two or three blocks in registers were slower, 1.39 and 1.54 against 1.33 ms
// a call for 256 tokens: they cost spills, and the warps cover the way from L2.
// Further ahead costs more than it hides: 434 us with 1, 440 with 2, 462 with 4 for
// the gate/up of 64 tokens; with two column tiles 1.38 ms a call with 1, 1.33 with
// 2, 1.34 with 4 for 256 tokens.)
template <int NT, bool DOWN, int SUB>
__global__ void __launch_bounds__(W4Shape<NT, SUB>::kWarps * 32, 1)
    w4_product_kernel(const W4Args args) {
    using S = W4Shape<NT, SUB>;
    constexpr int kWarps = S::kWarps, kVals = S::kVals;
    constexpr int kMeta = w4_meta_words(SUB);
    extern __shared__ __align__(128) uint8_t s_dyn[];
    float(*s_sum)[kWarps][kVals] = reinterpret_cast<float(*)[kWarps][kVals]>(s_dyn);
    uint8_t* s_rows = s_dyn + S::kSumBytes;  // [block][cap rows][256]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane >> 2, c = lane & 3;
    const int nkb = args.K / kW4Block, cap = args.cap;
    uint32_t* s_meta = reinterpret_cast<uint32_t*>(s_rows + nkb * cap * kW4RowBytes);
    __shared__ W4Sched sp;
    __shared__ uint32_t s_marks[kW4MaxK / kW4Block / 32];
    if constexpr (!DOWN) ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    {
        const SchedPtrs from = sched_ptrs(args.sched, args.nseg);
        for (int i = threadIdx.x; i <= args.nseg; i += kWarps * 32) {
            sp.prefix[i] = from.prefix[i];
            if (i < args.nseg) {
                sp.b_row0[i] = from.b_row0[i];
                sp.out_row0[i] = from.out_row0[i];
                sp.rows[i] = from.rows[i];
            }
        }
    }
    __syncthreads();
    // this CTA's run of tasks
    int64_t begin, end;
    {
        __shared__ int32_t cost[kMaxSegments + 1];
        __shared__ int s_warp[32];
        int v = 0;
        if (threadIdx.x < args.nseg && sp.rows[threadIdx.x] > 0) {
            // chunks before the segment's last
            const int full = sp.prefix[threadIdx.x + 1] - sp.prefix[threadIdx.x] - 1;
            v = full * w4_cost<NT>(cap) + w4_cost<NT>(sp.rows[threadIdx.x] - full * cap);
        }
        int all = 0;
        const int before = block_exclusive_scan(v, s_warp, &all);
        if (threadIdx.x < args.nseg) cost[threadIdx.x] = before;
        if (threadIdx.x == args.nseg) cost[args.nseg] = all;
        __syncthreads();
        // (odd lanes find the end)
        const int64_t x =
            static_cast<int64_t>(all) * args.tiles * (blockIdx.x + (lane & 1)) / gridDim.x;
        const int64_t task = w4_task_at<NT>(sp, cost, args.nseg, cap, args.tiles, x);
        begin = __shfl_sync(0xffffffffu, task, 0);
        end = __shfl_sync(0xffffffffu, task, 1);
    }
    const int run = static_cast<int>(end - begin);
    if (run == 0) {
        if constexpr (DOWN) ptx::grid_dep_wait();
        return;
    }
    // warps per tile: the fewest blocks on any warp's way, a round counting as
    // two more for its barrier and sums
    int most = 0, base = 0;
    while (most < S::kMostLog && (2 << most) <= nkb) ++most;
    for (int l = 0, best = 0x7fffffff; l <= most; ++l) {
        const int cost = ((run + (kWarps >> l) - 1) / (kWarps >> l)) * (((nkb - 1) >> l) + 3);
        if (cost < best) {
            best = cost;
            base = l;
        }
    }

    W4Round cur{}, next{};
    {
        cur.group = static_cast<int>(begin / args.tiles);
        cur.tile = static_cast<int>(begin - static_cast<int64_t>(cur.group) * args.tiles);
        cur.left = run;
        w4_find_chunk(cur, sp, args.nseg, cap);
        w4_next_round<kWarps>(cur, sp, args.tiles, args.nseg, cap, base, most);
    }
    // the warp's part of a round: n blocks, its tile's codes and scales from the
    // first of them on
    struct Part {
        const uint8_t* q;
        const uint8_t* sc;
        int n;
    };
    auto part_of = [&](const W4Round& p) {
        const int slot = warp >> p.log_ks, part = warp & ((1 << p.log_ks) - 1);
        const int kb0 = part * nkb >> p.log_ks;
        const bool special = p.seg == args.special;
        const int64_t unit = static_cast<int64_t>(p.tile + slot) * nkb + kb0;
        Part w;
        w.q = (special ? args.q_shared : args.q + p.seg * args.q_stride) + unit * kW4BlockBytes;
        w.sc = reinterpret_cast<const uint8_t*>(
                   special ? args.sc_shared : args.sc + p.seg * args.sc_stride) +
               unit * 64 * SUB;
        w.n = slot < p.tiles ? ((part + 1) * nkb >> p.log_ks) - kb0 : 0;
        return w;
    };
    W4Stage<SUB> s;
    auto load = [&](const Part& w, int i) {
        if (i < w.n) {
            const uint8_t* p = w.q + static_cast<int64_t>(i) * kW4BlockBytes + lane * 32;
            ldg_stream(p, s.a[0]);
            ldg_stream(p + 1024, s.a[1]);
            p = w.sc + static_cast<int64_t>(i) * 64 * SUB + r * 8 * SUB;
            if constexpr (SUB == 1) {
                s.s[0] = __ldg(reinterpret_cast<const uint2*>(p));
            } else {
#pragma unroll
                for (int u = 0; u < SUB; u += 2) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p + u * 8));
                    s.s[u] = make_uint2(v.x, v.y);
                    s.s[u + 1] = make_uint2(v.z, v.w);
                }
            }
        }
    };
    auto prefetch = [&](const Part& w, int i) {
        if (i < w.n && lane == 0) {
            prefetch_l2(w.q + static_cast<int64_t>(i) * kW4BlockBytes, kW4BlockBytes);
            prefetch_l2(w.sc + static_cast<int64_t>(i) * 64 * SUB, 64 * SUB);
        }
    };
    Part mine = part_of(cur), then{};
    // the chunk's rows into shared memory (asynchronous copies of this thread); whether
    // the thread met the mark of a second integer
    auto fetch_rows = [&](const W4Round& p) {
        const int first = sp.b_row0[p.seg] + p.row0;
        const bool direct = DOWN || p.seg == args.special;
        bool marked = false;
        for (int row = warp; row < p.nrows; row += kWarps) {
            const int64_t m = (direct ? first + row : args.row_src[first + row]);
            const uint8_t* src = args.rows.limbs + m * nkb * kW4RowBytes;
            for (int i = lane; i < nkb * 16; i += 32)
                ptx::cp_async_16(s_rows + ((i >> 4) * cap + row) * kW4RowBytes +
                                     ((i & 15) ^ ((row & 1) * 4)) * 16,
                                 src + i * 16, 16);
            const uint32_t* meta = args.rows.meta + m * nkb * kMeta;
            for (int i = lane; i < nkb * kMeta; i += 32) {
                const uint32_t v = meta[i];
                s_meta[((i / kMeta) * cap + row) * kMeta + i % kMeta] = v;
                marked |= i % kMeta == w4_mark(SUB) && v != 0;
            }
        }
        return marked;
    };
    // bits of the blocks in which a row of the chunk in shared memory has a mark, by one warp
    auto find_marks = [&](int nrows) {
        for (int kb = 0; kb < nkb; kb += 32) {
            uint32_t any = 0;
            if (kb + lane < nkb)
                for (int row = 0; row < nrows; ++row)
                    any |= s_meta[((kb + lane) * cap + row) * kMeta + w4_mark(SUB)];
            any = __ballot_sync(0xffffffffu, any != 0);
            if (lane == 0) s_marks[kb / 32] = any;
        }
    };
    // the marked blocks of the chunk's rows (asynchronous copies, a warp to a block and
    // row): the second integers, 0 for rows without a mark, in the first ones' place, or
    // the first ones again
    auto fetch_marked = [&](const W4Round& p, const W4Rows& from, bool all) {
        const int first = sp.b_row0[p.seg] + p.row0;
        const bool direct = DOWN || p.seg == args.special;
        int turn = 0;
#pragma unroll 1
        for (int word = 0; word * 32 < nkb; ++word)
#pragma unroll 1
            for (uint32_t w = s_marks[word]; w; w &= w - 1)
#pragma unroll 1
                for (int row = 0; row < p.nrows; ++row) {
                    if (turn++ % kWarps != warp) continue;
                    const int kb = word * 32 + __ffs(w) - 1, at = kb * cap + row;
                    const int64_t m = direct ? first + row : args.row_src[first + row];
                    const uint32_t has = all || s_meta[at * kMeta + w4_mark(SUB)] ? 16 : 0;
                    if (lane < 16)
                        ptx::cp_async_16(s_rows + at * kW4RowBytes + (lane ^ ((row & 1) * 4)) * 16,
                                         from.limbs + (m * nkb + kb) * kW4RowBytes + lane * 16, has);
                    else if (lane - 16 < kMeta / 4)
                        ptx::cp_async_16(s_meta + at * kMeta + (lane - 16) * 4,
                                         from.meta + (m * nkb + kb) * kMeta + (lane - 16) * 4, has);
                }
    };
    load(mine, 0);
    for (int i = 1; i <= S::kAhead; ++i) prefetch(mine, i);
    if constexpr (DOWN) ptx::grid_dep_wait();  // (the weights and the schedule are older)
    bool marked = fetch_rows(cur);
    ptx::cp_async_wait_all();
    marked = __syncthreads_or(marked);

    // (a round over a chunk with marks goes round once more for each run of the warp's
    // marked blocks; `at`: the block behind the run at hand, -1 before the first)
    for (int buffer = 0, at = -1;;) {
        const bool more = cur.left > 0;
        if (more) {
            next = cur;
            w4_next_round<kWarps>(next, sp, args.tiles, args.nseg, cap, base, most);
            then = part_of(next);
        }
        float tot[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) tot[h][n][i] = 0.0f;
        // offsets of the lane's row r and of its columns' sums and scales (rows
        // past the chunk's last hold anything: their columns are not stored)
        const int kb0 = (warp & ((1 << cur.log_ks) - 1)) * nkb >> cur.log_ks;
        const bool few = NT == 1 && cur.nrows <= 4;
        uint32_t b, m;
        auto start_at = [&](int kb) {
            b = few ? (kb * cap + (r & 3)) * kW4RowBytes + ((((r >> 2) ^ (r & 1)) << 2) | c) * 16
                    : (kb * cap + r) * kW4RowBytes + (c ^ ((r & 1) * 4)) * 16;
            m = (kb * cap + 2 * (few ? c & 1 : c)) * kMeta;
        };
        start_at(at < 0 ? kb0 : at - mine.n);
        // Limbs of the lane's columns.  With 12 warps those past the chunk's rows
        // are zeros and not read, which saves power more than time (3% of a call for
        // 256 tokens, calls in a row under the power limit); with 16 the loads would
        // come late (3% more for 64 tokens).
        constexpr bool kLive = kWarps == 12;
        uint4 bv[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int l = 0; l < 2; ++l)
                if (kLive) bv[n][l] = make_uint4(0, 0, 0, 0);
        // one weight block against N column tiles (those that the chunk has rows for)
        auto block = [&](auto tiles) {
            constexpr int N = decltype(tiles)::value;
            constexpr int kSums = w4_sums(SUB);
            // with one column tile the accumulators of both halves fit, a whole
            // block long where that is a group; with two, the halves of a group of
            // at most 64 run one after the other
            constexpr bool kBoth = N == 1, kWhole = kBoth && SUB == 1;
            int32_t acc[kBoth ? 2 : 1][2][N][4];  // [half][limb hi, lo]
            int32_t from[2][N][4];  // the limb sums' multiples (row r + 8: 16 u)
            auto start = [&](int g) {
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t* p = s_meta + m + (8 * n + j) * kMeta;
                        int2 v;
                        if constexpr (kWhole) {
                            const int4 q = *reinterpret_cast<const int4*>(p);
                            v = make_int2(q.x + q.z, q.y + q.w);
                        } else {
                            v = *reinterpret_cast<const int2*>(p + 2 * g);
                        }
                        from[0][n][j] = v.x;
                        from[0][n][2 + j] = 16 * v.x;
                        from[1][n][j] = v.y;
                        from[1][n][2 + j] = 16 * v.y;
                    }
            };
            // the block's sum of s (256 hi + lo), before the rows' scales
            float part[2][N][4];
            auto finish = [&](const int32_t (&a)[2][N][4], int h, int g, bool first) {
                const uint2 s2 = s.s[g];
                const uint32_t sw = h ? s2.y : s2.x;
                const float2 sv = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&sw));
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float v = static_cast<float>(a[0][n][i] * 256 + a[1][n][i]);
                        const float w = i < 2 ? sv.x : sv.y;
                        part[h][n][i] = first ? w * v : fmaf(w, v, part[h][n][i]);
                    }
            };
            auto step = [&](int32_t (&a)[2][N][4], int h, int k32, bool first) {
                const uint32_t w0 = s.a[h][2 * k32], w1 = s.a[h][2 * k32 + 1];
                const uint32_t f[4] = {w0 & 0x0f0f0f0fu, w0 & 0xf0f0f0f0u, w1 & 0x0f0f0f0fu,
                                       w1 & 0xf0f0f0f0u};
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int l = 0; l < 2; ++l)
                        mma_u8s8(a[l][n], f, (k32 & 1) ? bv[n][l].z : bv[n][l].x,
                                 (k32 & 1) ? bv[n][l].w : bv[n][l].y,
                                 first ? from[l][n] : a[l][n]);
            };
            if constexpr (kWhole) start(0);
#pragma unroll
            for (int k64 = 0; k64 < 2; ++k64) {
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int l = 0; l < 2; ++l)
                        // (piece 8 k64 + 4 l + c, its bit 2 flipped in odd rows)
                        if (!kLive || n * 8 + r < cur.nrows)
                            bv[n][l] = *reinterpret_cast<const uint4*>(
                                s_rows + (b ^ (l * 64)) + k64 * 128 + n * 8 * kW4RowBytes);
                if constexpr (kWhole) {
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            step(acc[h], h, 2 * k64 + kk, 2 * k64 + kk == 0);
                } else {
#pragma unroll
                    for (int g = 0; g < (SUB == 4 ? 2 : 1); ++g) {
                        const int sum = SUB == 4 ? 2 * k64 + g : k64;
                        const int scale_of = SUB == 1 ? 0 : sum;
                        constexpr int kSteps = SUB == 4 ? 1 : 2;
                        start(sum);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if constexpr (kBoth) {
                                if (h) continue;
#pragma unroll
                                for (int kk = 0; kk < kSteps; ++kk)
#pragma unroll
                                    for (int x = 0; x < 2; ++x)
                                        step(acc[x], x, 2 * k64 + g + kk, kk == 0);
#pragma unroll
                                for (int x = 0; x < 2; ++x)
                                    finish(acc[x], x, scale_of, k64 + g == 0);
                            } else {
#pragma unroll
                                for (int kk = 0; kk < kSteps; ++kk)
                                    step(acc[0], h, 2 * k64 + g + kk, kk == 0);
                                finish(acc[0], h, scale_of, k64 + g == 0);
                            }
                        }
                    }
                }
            }
            if constexpr (kWhole) {
#pragma unroll
                for (int h = 0; h < 2; ++h) finish(acc[h], h, 0, true);
            }
            float scale[N][2];
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    scale[n][j] =
                        __uint_as_float(s_meta[m + (8 * n + j) * kMeta + 2 * kSums]);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        tot[h][n][i] = fmaf(scale[n][i & 1], part[h][n][i], tot[h][n][i]);
            b += cap * kW4RowBytes;
            m += cap * kMeta;
        };
        // One weight block against up to four rows: column r of the one tile is limb
        // r / 4 of row r % 4, which halves the MMAs, conversions and reads.  The two
        // limbs' sums stay apart until the end of the round.
        auto block4 = [&]() {
            constexpr int kSums = w4_sums(SUB);
            constexpr int kSteps = SUB == 4 ? 1 : (SUB == 2 ? 2 : 4);  // MMAs of a group
            const uint32_t* p[2] = {s_meta + m, s_meta + m + kMeta};
            int32_t acc[2][4];
            float part[2][4];
            uint4 v;
#pragma unroll
            for (int k32 = 0; k32 < 4; ++k32) {
                if (k32 % 2 == 0)
                    v = *reinterpret_cast<const uint4*>(s_rows + b + k32 * 64);
                const int g = k32 / kSteps;
                int32_t from[4];
                if (k32 % kSteps == 0) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        from[j] = static_cast<int32_t>(p[j][2 * g + (c >> 1)]);
                        if (SUB == 1) from[j] += static_cast<int32_t>(p[j][2 + (c >> 1)]);
                        from[2 + j] = 16 * from[j];
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t w0 = s.a[h][2 * k32], w1 = s.a[h][2 * k32 + 1];
                    const uint32_t f[4] = {w0 & 0x0f0f0f0fu, w0 & 0xf0f0f0f0u, w1 & 0x0f0f0f0fu,
                                           w1 & 0xf0f0f0f0u};
                    if (k32 % kSteps == 0)
                        mma_u8s8(acc[h], f, (k32 & 1) ? v.z : v.x, (k32 & 1) ? v.w : v.y, from);
                    else
                        mma_u8s8(acc[h], f, (k32 & 1) ? v.z : v.x, (k32 & 1) ? v.w : v.y, acc[h]);
                }
                if (k32 % kSteps == kSteps - 1) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t sw = h ? s.s[g].y : s.s[g].x;
                        const float2 sv =
                            __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&sw));
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float x = static_cast<float>(acc[h][i]), w = i < 2 ? sv.x : sv.y;
                            part[h][i] = g == 0 ? w * x : fmaf(w, x, part[h][i]);
                        }
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = __uint_as_float(p[i & 1][2 * kSums]) * (c < 2 ? 256.0f : 1.0f);
#pragma unroll
                for (int h = 0; h < 2; ++h) tot[h][0][i] = fmaf(a, part[h][i], tot[h][0][i]);
            }
            b += cap * kW4RowBytes;
            m += cap * kMeta;
        };
        auto blocks = [&](auto tiles) {
#pragma unroll 1
            for (int kb = 0; kb < mine.n; ++kb) {
                const int ahead = kb + 1 + S::kAhead;
                if (ahead < mine.n) prefetch(mine, ahead);
                else if (more) prefetch(then, ahead - mine.n);
                if constexpr (decltype(tiles)::value == 0) block4();
                else block(tiles);
                load(mine, kb + 1);
            }
        };
        if (few) blocks(std::integral_constant<int, 0>{});
        else if (NT == 1 || cur.nrows <= 8) blocks(std::integral_constant<int, 1>{});
        else blocks(std::integral_constant<int, NT>{});
        if (few) {
            // lane 4r + c (c < 2) adds the low limbs of its columns, those of lane + 2
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tot[h][0][i] += __shfl_xor_sync(0xffffffffu, tot[h][0][i], 2);
        }
        // (the value of lane 4r + c, index i: row r + 8 (i / 2) of half h, column
        // 8n + 2c + i % 2; row r + 8 carries 16 u)
        auto store = [&](float g, float u, int tile, int h, int n, int i) {
            const int col = 8 * n + 2 * c + (i & 1);
            if (col >= cur.nrows) return;
            const int64_t row = sp.out_row0[cur.seg] + cur.row0 + col;
            if (i >= 2) {
                g *= 0.0625f;
                u *= 0.0625f;
            }
            if constexpr (!DOWN) {
                // compare-select clamp: NaN passes through
                g = g > args.clip ? args.clip : (g < -args.clip ? -args.clip : g);
                u = u > args.clip ? args.clip : (u < -args.clip ? -args.clip : u);
                args.out[row * args.ld + tile * 16 + (i >> 1) * 8 + r] =
                    g / (1.0f + __expf(-g)) * u;
            } else {
                const float wt = row < args.routed_rows ? args.row_w[row] : 1.0f;
                args.out[row * args.ld + tile * 32 + h * 16 + (i >> 1) * 8 + r] = wt * g;
            }
        };
        // a tile of one warp's own needs neither the sums nor the barrier
        const int ks = 1 << cur.log_ks, slot = warp >> cur.log_ks, part = warp & (ks - 1);
        if (ks == 1 && !marked) {
            if (slot < cur.tiles) {
#pragma unroll
                for (int h = 0; h < (DOWN ? 2 : 1); ++h)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            store(tot[h][n][i], tot[1][n][i], cur.tile + slot, h, n, i);
            }
        } else {
            float* sums = s_sum[buffer][warp];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float& to = sums[((h * NT + n) * 4 + i) * 32 + lane];
                        to = at < 0 ? tot[h][n][i] : to + tot[h][n][i];
                    }
        }
        if (marked) {
            const Part whole = part_of(cur);
            if (at < 0) {
                if (warp == 0) find_marks(cur.nrows);
                __syncthreads();  // (and every warp is done with the rows)
                fetch_marked(cur, args.rest, false);
                at = kb0;
                for (int kb = lane; kb < whole.n; kb += 32)
                    if (s_marks[(kb0 + kb) >> 5] >> ((kb0 + kb) & 31) & 1)
                        prefetch_l2(whole.q + static_cast<int64_t>(kb) * kW4BlockBytes,
                                    kW4BlockBytes);
                ptx::cp_async_wait_all();
                __syncthreads();
            }
            uint32_t w = 0;
            for (; at < kb0 + whole.n; at = (at | 31) + 1) {
                w = s_marks[at >> 5] >> (at & 31);
                if (w) break;
            }
            if (w) at += __ffs(w) - 1;
            const int left = kb0 + whole.n - at;
            if (left > 0) {
                w >>= __ffs(w) - 1;
                mine.n = min(left, w == 0xffffffffu ? 32 : __ffs(~w) - 1);
                mine.q = whole.q + static_cast<int64_t>(at - kb0) * kW4BlockBytes;
                mine.sc = whole.sc + static_cast<int64_t>(at - kb0) * 64 * SUB;
                at += mine.n;
                load(mine, 0);
                continue;
            }
            at = -1;
        }
        // the next round's first weights are on their way before this one is
        // added up, and its rows while it is
        // (the second integers of a chunk took its marked blocks' place)
        const bool other_rows = more && (next.group != cur.group || marked);
        if (more) {
            mine = then;
            load(mine, 0);
        }
        // (two buffers of sums in turn: the barrier of the next round that uses one
        // lies between this round's reads and the writes of the one after)
        if (ks > 1 || other_rows) __syncthreads();
        bool next_marked = marked;
        if (other_rows) {
            if (next.group != cur.group) next_marked = fetch_rows(next);
            else fetch_marked(cur, args.rows, true);
        }
        if (ks > 1 || marked) {
            const float(*from)[kVals] = &s_sum[buffer][slot << cur.log_ks];
            if (ks > 1) buffer ^= 1;
            constexpr int kOut = DOWN ? kVals : kVals / 2;
            for (int v = slot < cur.tiles ? part * 32 + lane : kOut; v < kOut; v += ks * 32) {
                float g = 0.0f, u = 0.0f;
                for (int w = 0; w < ks; ++w) {
                    g += from[w][v];
                    if constexpr (!DOWN) u += from[w][v + kVals / 2];
                }
                store(g, u, cur.tile + slot, v / (kVals / 2), (v >> 7) % NT, (v >> 5) & 3);
            }
        }
        if (!more) break;
        if (other_rows) {
            ptx::cp_async_wait_all();
            marked = __syncthreads_or(next_marked);
        }
        cur = next;
    }
}

// Dispatch of up to kPermTokens tokens in one CTA (the first) of 512 threads:
// histogram, offsets, tile schedules and stable positions (row order: expert,
// token), as the three dispatch launches compute them for any number of tokens.
// pos of an assignment with an expert out of range is -1.  The other CTAs split
// the token rows into limbs meanwhile.
__global__ void __launch_bounds__(512) w4_dispatch_kernel(
    const int32_t* __restrict__ idx, const float* __restrict__ topk_w, int T, int E, int k,
    int num_shared, int32_t* sched_gu, int nmax_gu, int32_t* sched_dn, int nmax_dn,
    int32_t* __restrict__ pos,
    int32_t* __restrict__ src, float* __restrict__ row_w, int32_t* status,
    const __nv_bfloat16* __restrict__ x, int64_t units, int sub, W4Rows x_rows,
    W4Rows x_rest) {
    if (blockIdx.x > 0) {
        ptx::grid_dep_wait();
        ptx::grid_dep_launch();
        const int64_t unit = (static_cast<int64_t>(blockIdx.x) - 1) * 16 + (threadIdx.x >> 5);
        if (unit < units) w4_split_block<__nv_bfloat16>(x, sub, unit, x_rows, x_rest);
        return;
    }
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
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const int nmax = which == 0 ? nmax_gu : nmax_dn;
        int total = 0;
        const int pre = block_exclusive_scan((rows + nmax - 1) / nmax, s_warp, &total);
        if (tid < nseg) {
            const int o0 = shared ? T * k : off;
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

// Encoder, for weights as they are loaded: one CTA of 128 threads per 16-row half of
// a pair tile and block.  16 experts of 6144 x 2048 take 1.41 to 1.46 ms from bf16
// and 1.47 to 1.54 from fp32, 1.1 and 1.8 TB/s (the down part reads 32 or 64 bytes
// of a row at a time).
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
