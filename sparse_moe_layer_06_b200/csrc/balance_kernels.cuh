// balance_kernels.cuh -- the router's balance loss over packed sequences and
// its gradient with respect to the logits.
//
// Sequence s holds the tokens [offsets[s], offsets[s+1]) whose mask is set,
// n_s of them; S of the sequences have n_s > 0.  With p_t = softmax(logits_t +
// bias) over the experts and count[s,e] the selections of expert e:
//   P[s,e] = (1/n_s) sum_t p_t[e]      f[s,e] = count[s,e] / (n_s k)
//   loss   = (1/S) sum_s E sum_e P[s,e] f[s,e]
//   dlogits[t,e] = grad E/(S n_s) p_t[e] (f[s,e] - sum_j p_t[j] f[s,j])
// (f is piecewise constant, so it has no gradient).  The sums over tokens are
// taken in a fixed order: per window of consecutive tokens and sequence in
// fp32, then over a sequence's windows in fp64.
#pragma once

#include <cstdint>

#include "device_common.cuh"
#include "ptx.cuh"

namespace moe {

// A token's E logits lie in one warp, NP per lane: expert lane + 32 i in slot i,
// or, with VEC, expert 128 (i / 4) + 4 lane + i % 4 (E a multiple of 4, rows 16
// byte aligned), so that a lane loads four at a time.
template <bool VEC>
__device__ __forceinline__ int slot_expert(int i) {
    const int lane = threadIdx.x & 31;
    return VEC ? 128 * (i >> 2) + 4 * lane + (i & 3) : lane + 32 * i;
}

// v[i] = row[expert of slot i], `fill` beyond the E experts.
template <int NP, bool VEC>
__device__ __forceinline__ void load_slots(const float* __restrict__ row, int E, float fill,
                                           float (&v)[NP]) {
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < NP; i += 4) {
            const int e = slot_expert<VEC>(i);
            float4 q = make_float4(fill, fill, fill, fill);
            if (e < E) q = *reinterpret_cast<const float4*>(row + e);
            v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int e = slot_expert<VEC>(i);
            v[i] = e < E ? row[e] : fill;
        }
    }
}

__device__ __forceinline__ float warp_max(float v) {
    float m;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

// First sequence that ends behind token t (n_seq if none), by one warp: 64 places
// of the range are looked at in each round, so up to 64 sequences take one load,
// up to 4096 two, one behind the other.  Offsets that are not in order give some sequence
// number, never one out of range.
__device__ __forceinline__ int first_sequence(const int32_t* __restrict__ offsets, int n_seq,
                                              int64_t t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, len = n_seq;
    while (len > 0) {
        const int step = (len + 63) / 64;
        // sequence lo + (lane + 1) step - 1 and all before it end at t or earlier?
        const int at = (lane + 1) * step - 1, at2 = at + 32 * step;
        const bool before = at < len && offsets[lo + at + 1] <= t;
        const bool before2 = at2 < len && offsets[lo + at2 + 1] <= t;
        const int n = __popc(__ballot_sync(0xffffffffu, before)) +
                      __popc(__ballot_sync(0xffffffffu, before2));
        lo += n * step;
        len = step == 1 ? 0 : min(step - 1, len - n * step);
    }
    return min(lo, n_seq);
}

// Bits of the tokens t, t + kStep, ... (32 of them) that lie before `end` and have
// their mask set.
template <int kStep>
__device__ __forceinline__ uint32_t live_tokens(const uint8_t* __restrict__ mask, int64_t t,
                                                int64_t end) {
    const int lane = threadIdx.x & 31;
    t += lane * kStep;
    return __ballot_sync(0xffffffffu, t < end && (!mask || mask[t]));
}

// Tokens whose logits a warp has on the way at once: 4 KB of 256 experts, which
// at 24 warps per SM covers the memory's latency (one token ahead did not: 34 us
// against 27 for the gradient of 65536 x 256 logits).
constexpr int kBalBatch = 4;

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Numerators of the softmax of one token's logits l plus the bias (read again
// for each token: registers hold the logits on the way instead).  A token whose
// logits are all -inf (every expert masked off) has no distribution: its
// probabilities are 0.
template <int NP, bool VEC>
__device__ __forceinline__ void numerators(const float* __restrict__ bias, int E, float (&l)[NP]) {
    if (bias) {
        float b[NP];
        load_slots<NP, VEC>(bias, E, 0.0f, b);
#pragma unroll
        for (int i = 0; i < NP; ++i) l[i] += b[i];
    }
    float mx = l[0];
#pragma unroll
    for (int i = 1; i < NP; ++i) mx = fmaxf(mx, l[i]);
    mx = warp_max(mx);
    if (mx == -INFINITY) mx = 0.0f;  // (a NaN logit still gives NaN below)
    // (the difference first: the products of the lowest floats are infinite)
    constexpr float kLog2e = 1.44269504f;
#pragma unroll
    for (int i = 0; i < NP; ++i) l[i] = exp2_approx((l[i] - mx) * kLog2e);
}

// Adds a token, its logits l and the lane's selection e, to the lane's sums of
// probabilities and the CTA's counts.
template <int NP, bool VEC>
__device__ __forceinline__ void add_token(const float* __restrict__ bias, int E, int k, int e,
                                          float (&l)[NP], float (&acc)[NP], int32_t* s_cnt,
                                          int32_t* status) {
    if ((threadIdx.x & 31) < k) {
        if (e >= 0 && e < E) atomicAdd(&s_cnt[e], 1);
        else set_device_error(status, DEV_ERR_BAD_INDEX);
    }
    numerators<NP, VEC>(bias, E, l);
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < NP; ++i) z += l[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    const float inv = z == 0.0f ? 0.0f : 1.0f / z;
#pragma unroll
    for (int i = 0; i < NP; ++i) acc[i] = fmaf(l[i], inv, acc[i]);
}

// Floats from one slot of partial sums to the next: whole 16-byte vectors.
__host__ __device__ constexpr int balance_pad(int E) { return (E + 3) & ~3; }

// Pass 1: CTA b sums the probabilities and counts of the tokens of window b
// ([b * win, (b+1) * win)) for each sequence s that the window touches, into
// slot b + s: along the windows and sequences in order either b or s grows by
// one, so no two pairs share a slot.
template <int NP, bool VEC>
__global__ void __launch_bounds__(256, 3) balance_partial_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias,
    const int32_t* __restrict__ idx, const uint8_t* __restrict__ mask,
    const int32_t* __restrict__ offsets, int n_seq, int64_t T, int E, int k, int win,
    float* __restrict__ part_p, int32_t* __restrict__ part_c, int32_t* __restrict__ part_n,
    uint32_t* __restrict__ ticket, int32_t* status) {
    __shared__ float s_sum[8][kMaxExperts];
    __shared__ int32_t s_cnt[kMaxExperts];
    __shared__ int32_t s_tok;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    if (blockIdx.x == 0 && tid == 0) *ticket = 0;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * win;
    const int64_t t1 = min(T, t0 + win);
    int s = offsets ? first_sequence(offsets, n_seq, t0) : 0;
    for (; s < n_seq; ++s) {
        const int64_t o0 = offsets ? offsets[s] : 0, o1 = offsets ? offsets[s + 1] : T;
        if (o0 >= t1) break;
        const int64_t lo = max(t0, o0), hi = min(t1, o1);
        if (lo >= hi) continue;
        s_cnt[tid] = 0;
        if (tid == 0) s_tok = 0;
        __syncthreads();
        float acc[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) acc[i] = 0.0f;
        int ntok = 0;
        // each warp takes every eighth token (an eighth of the window each left warps
        // waiting where a sequence ends inside it: 38 us against 28 for 65536 tokens of
        // 256 experts in 37 sequences)
        uint32_t bits = 0;
        const int len = static_cast<int>(hi - lo);
        const float* rows = logits + lo * E;
        const int32_t* sel = idx + lo * k;
        for (int t = warp; t < len; t += 8 * kBalBatch) {
            if ((t >> 3 & 31) == 0) bits = live_tokens<8>(mask ? mask + lo : nullptr, t, len);
            const uint32_t live = bits >> (t >> 3 & 31);
            float l[kBalBatch][NP];
            int e[kBalBatch];
#pragma unroll
            for (int u = 0; u < kBalBatch; ++u) {
                if (live >> u & 1) {
                    e[u] = lane < k ? sel[(t + 8 * u) * k + lane] : 0;
                    load_slots<NP, VEC>(rows + (t + 8 * u) * E, E, -INFINITY, l[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < kBalBatch; ++u) {
                if (!(live >> u & 1)) continue;
                ++ntok;
                add_token<NP, VEC>(bias, E, k, e[u], l[u], acc, s_cnt, status);
            }
        }
        if (lane == 0 && ntok) atomicAdd(&s_tok, ntok);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int x = slot_expert<VEC>(i);
            if (x < E) s_sum[warp][x] = acc[i];
        }
        __syncthreads();
        const int64_t slot = static_cast<int64_t>(blockIdx.x) + s;
        const int pad = balance_pad(E);
        if (tid < E) {
            float a = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; ++w) a += s_sum[w][tid];
            part_p[slot * pad + tid] = a;
            part_c[slot * pad + tid] = s_cnt[tid];
        }
        if (tid == 0) part_n[slot] = s_tok;
        __syncthreads();
    }
}

// Pass 2: CTA (s, c) adds the windows of sequence s for the experts from 4 g c on
// (fp64, window order within each of kBalFinal / g interleaved groups of g threads,
// four experts to a thread, then group order) and writes their P and counts, with
// c = 0 the token count too; the CTA that finishes last adds all losses in order.
// Few long sequences take narrow groups, so many of them: 2048 tokens of 32 experts
// leave 256 windows to add.
constexpr int kBalFinal = 512;  // threads

__global__ void __launch_bounds__(kBalFinal) balance_final_kernel(
    const float* __restrict__ part_p, const int32_t* __restrict__ part_c,
    const int32_t* __restrict__ part_n, const int32_t* __restrict__ offsets, int n_seq, int64_t T,
    int E, int k, int win, int log_g, float* __restrict__ P_out, int32_t* __restrict__ counts,
    int32_t* __restrict__ tokens, double* seq_loss, uint32_t* ticket, float* __restrict__ loss,
    int32_t* status) {
    constexpr int kWarps = kBalFinal / 32;
    __shared__ __align__(16) double s_p[kBalFinal * 4];   // [group][expert of the CTA]
    __shared__ __align__(16) int32_t s_c[kBalFinal * 4];
    __shared__ double s_red[kWarps];
    __shared__ int32_t s_n[kWarps];
    __shared__ bool s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    ptx::grid_dep_wait();
    const int s = blockIdx.x;
    int64_t o0 = 0, o1 = T;
    if (offsets) {
        o0 = offsets[s];
        o1 = offsets[s + 1];
        if (o0 < 0 || o1 < o0 || o1 > T) {
            if (tid == 0) set_device_error(status, DEV_ERR_BAD_INDEX);
            o1 = o0 = 0;  // counts as empty
        }
    }
    const int per = 4 << log_g, e0 = blockIdx.y * per;  // the CTA's experts
    const int64_t b0 = o0 / win, b1 = o1 > o0 ? (o1 - 1) / win : b0 - 1;
    {
        const int groups = kBalFinal >> log_g, e = e0 + (tid & ((1 << log_g) - 1)) * 4;
        const int pad = balance_pad(E);
        double p[4] = {0.0, 0.0, 0.0, 0.0};
        int4 c = make_int4(0, 0, 0, 0);
        if (e < pad) {
#pragma unroll 8
            for (int64_t b = b0 + (tid >> log_g); b <= b1; b += groups) {
                const float4 v = *reinterpret_cast<const float4*>(part_p + (b + s) * pad + e);
                const int4 d = *reinterpret_cast<const int4*>(part_c + (b + s) * pad + e);
                p[0] += v.x, p[1] += v.y, p[2] += v.z, p[3] += v.w;
                c.x += d.x, c.y += d.y, c.z += d.z, c.w += d.w;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s_p[tid * 4 + i] = p[i];
        *reinterpret_cast<int4*>(&s_c[tid * 4]) = c;
    }
    int32_t n = 0;
    for (int64_t b = b0 + tid; b <= b1; b += kBalFinal) n += part_n[b + s];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0) s_n[warp] = n;
    __syncthreads();
    n = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) n += s_n[w];
    double prod = 0.0;
    const int e = e0 + tid;
    if (tid < per && e < E) {
        double p = 0.0;
        int32_t c = 0;
#pragma unroll 8
        for (int i = tid; i < kBalFinal * 4; i += per) {
            p += s_p[i];
            c += s_c[i];
        }
        p = n > 0 ? p / n : 0.0;
        P_out[static_cast<int64_t>(s) * E + e] = static_cast<float>(p);
        counts[static_cast<int64_t>(s) * E + e] = c;
        if (n > 0) prod = p * (static_cast<double>(c) / (static_cast<double>(n) * k));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) prod += __shfl_xor_sync(0xffffffffu, prod, o);
    if (lane == 0) s_red[warp] = prod;
    __syncthreads();
    if (tid == 0) {
        double a = 0.0;
#pragma unroll
        for (int w = 0; w < kMaxExperts / 32; ++w) a += s_red[w];
        if (blockIdx.y == 0) tokens[s] = n;
        seq_loss[static_cast<int64_t>(s) * gridDim.y + blockIdx.y] = a * E;
        __threadfence();
        s_last = atomicAdd(ticket, 1u) == gridDim.x * gridDim.y - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    double a = 0.0;
    int used = 0;
    for (int64_t i = tid; i < static_cast<int64_t>(n_seq) * gridDim.y; i += kBalFinal) {
        a += __ldcg(seq_loss + i);
        if (i < n_seq) used += __ldcg(tokens + i) > 0 ? 1 : 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        used += __shfl_xor_sync(0xffffffffu, used, o);
    }
    if (lane == 0) {
        s_red[warp] = a;
        s_n[warp] = used;
    }
    __syncthreads();
    if (tid == 0) {
        a = 0.0;
        used = 0;
        for (int w = 0; w < kWarps; ++w) {
            a += s_red[w];
            used += s_n[w];
        }
        tokens[n_seq] = used;
        *loss = used > 0 ? static_cast<float>(a / used) : 0.0f;
    }
}

// Both passes for one sequence of a small batch, in one CTA of 16 warps: warp w
// takes every 16th token from w on, and the warps' sums are added in fp64 in warp
// order.
constexpr int kBalOneWarps = 16;

template <int NP, bool VEC>
__global__ void __launch_bounds__(kBalOneWarps * 32) balance_one_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias,
    const int32_t* __restrict__ idx, const uint8_t* __restrict__ mask,
    const int32_t* __restrict__ offsets, int64_t T, int E, int k, float* __restrict__ P_out,
    int32_t* __restrict__ counts, int32_t* __restrict__ tokens, float* __restrict__ loss,
    int32_t* status) {
    __shared__ float s_sum[kBalOneWarps][kMaxExperts];
    __shared__ int32_t s_cnt[kMaxExperts];
    __shared__ double s_red[kBalOneWarps];
    __shared__ int32_t s_n[kBalOneWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid < kMaxExperts) s_cnt[tid] = 0;
    __syncthreads();
    ptx::grid_dep_wait();
    int64_t o0 = 0, o1 = T;
    if (offsets) {
        o0 = offsets[0];
        o1 = offsets[1];
        if (o0 < 0 || o1 < o0 || o1 > T) {
            if (tid == 0) set_device_error(status, DEV_ERR_BAD_INDEX);
            o1 = o0 = 0;  // counts as empty
        }
    }
    float acc[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) acc[i] = 0.0f;
    int ntok = 0;
    for (int64_t t = o0 + warp; t < o1; t += kBalOneWarps * kBalBatch) {
        float l[kBalBatch][NP];
        int e[kBalBatch];
        bool live[kBalBatch];
#pragma unroll
        for (int u = 0; u < kBalBatch; ++u) {
            const int64_t at = t + u * kBalOneWarps;
            live[u] = at < o1 && (!mask || mask[at]);
            if (live[u]) {
                e[u] = lane < k ? idx[at * k + lane] : 0;
                load_slots<NP, VEC>(logits + at * E, E, -INFINITY, l[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < kBalBatch; ++u) {
            if (!live[u]) continue;
            ++ntok;
            add_token<NP, VEC>(bias, E, k, e[u], l[u], acc, s_cnt, status);
        }
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int x = slot_expert<VEC>(i);
        if (x < E) s_sum[warp][x] = acc[i];
    }
    if (lane == 0) s_n[warp] = ntok;
    __syncthreads();
    int n = 0;
#pragma unroll
    for (int w = 0; w < kBalOneWarps; ++w) n += s_n[w];
    double prod = 0.0;
    if (tid < E) {
        double p = 0.0;
#pragma unroll
        for (int w = 0; w < kBalOneWarps; ++w) p += s_sum[w][tid];
        p = n > 0 ? p / n : 0.0;
        const int32_t c = s_cnt[tid];
        P_out[tid] = static_cast<float>(p);
        counts[tid] = c;
        if (n > 0) prod = p * (static_cast<double>(c) / (static_cast<double>(n) * k));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) prod += __shfl_xor_sync(0xffffffffu, prod, o);
    if (lane == 0) s_red[warp] = prod;
    __syncthreads();
    if (tid == 0) {
        double a = 0.0;
#pragma unroll
        for (int w = 0; w < kMaxExperts / 32; ++w) a += s_red[w];
        tokens[0] = n;
        tokens[1] = n > 0 ? 1 : 0;
        *loss = static_cast<float>(a * E);
    }
}

// Gradient of the loss.  Each warp takes `run` consecutive tokens, kBalBatch at
// a time, and keeps the selection shares f of its current sequence in registers.
// With c = 1/E, sum_j p_j (f_j - c) + c = sum_j p_j f_j: the shares are taken
// relative to the uniform one, so that of a small difference f - p.f only the
// rounding of f itself is lost, 2^-24 of f, and none of the sums'.
template <int NP, bool VEC>
__global__ void __launch_bounds__(256, 2) balance_backward_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias,
    const uint8_t* __restrict__ mask, const int32_t* __restrict__ offsets, int n_seq, int64_t T,
    int E, int k, int run, const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens,
    const float* __restrict__ grad, float* __restrict__ dlogits) {
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t t0 = w * run, t1 = min(T, t0 + run);
    if (t0 >= T) return;
    ptx::grid_dep_wait();
    int s = -1;                    // sequence of the token at hand
    int64_t seq0 = 0, seq1 = -1;   // its tokens; none yet
    float f[NP];
    float scale = 0.0f;
    uint32_t bits = 0;
    for (int64_t t = t0; t < t1; t += kBalBatch) {
        if (((t - t0) & 31) == 0) bits = live_tokens<1>(mask, t, t1);
        const uint32_t live = bits >> ((t - t0) & 31);
        float l[kBalBatch][NP];
#pragma unroll
        for (int u = 0; u < kBalBatch; ++u)
            if (live >> u & 1) load_slots<NP, VEC>(logits + (t + u) * E, E, -INFINITY, l[u]);
#pragma unroll
        for (int u = 0; u < kBalBatch; ++u) {
            if (t + u >= t1) break;
            if (seq1 <= t + u) {
                // the next sequence that ends behind this token
                if (!offsets) {
                    s = 0;
                    seq1 = T;
                } else {
                    s = first_sequence(offsets, n_seq, t + u);
                    seq0 = s < n_seq ? offsets[s] : T;
                    seq1 = s < n_seq ? offsets[s + 1] : T;
                }
                const int n = s < n_seq ? tokens[s] : 0, used = tokens[n_seq];
                const float inv = n > 0 ? 1.0f / (static_cast<float>(n) * k) : 0.0f;
                scale = n > 0 ? *grad * static_cast<float>(E) /
                                    (static_cast<float>(used) * static_cast<float>(n))
                              : 0.0f;
                const float c = 1.0f / static_cast<float>(E);
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const int e = slot_expert<VEC>(i);
                    f[i] = e < E && n > 0 ? counts[static_cast<int64_t>(s) * E + e] * inv - c
                                          : 0.0f;
                }
            }
            if ((live >> u & 1) && seq0 <= t + u && scale != 0.0f) {
                numerators<NP, VEC>(bias, E, l[u]);
                float z = 0.0f, dot = 0.0f;
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    z += l[u][i];
                    dot = fmaf(l[u][i], f[i], dot);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    z += __shfl_xor_sync(0xffffffffu, z, o);
                    dot += __shfl_xor_sync(0xffffffffu, dot, o);
                }
                const float inv = z == 0.0f ? 0.0f : 1.0f / z;
                const float a = scale * inv, ad = a * (dot * inv);
#pragma unroll
                for (int i = 0; i < NP; ++i) l[u][i] *= fmaf(a, f[i], -ad);
            } else {
#pragma unroll
                for (int i = 0; i < NP; ++i) l[u][i] = 0.0f;
            }
            float* out = dlogits + (t + u) * E;
            if constexpr (VEC) {
#pragma unroll
                for (int i = 0; i < NP; i += 4) {
                    const int e = slot_expert<VEC>(i);
                    if (e < E)
                        *reinterpret_cast<float4*>(out + e) =
                            make_float4(l[u][i], l[u][i + 1], l[u][i + 2], l[u][i + 3]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const int e = slot_expert<VEC>(i);
                    if (e < E) out[e] = l[u][i];
                }
            }
        }
    }
}

}  // namespace moe
