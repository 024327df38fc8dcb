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

constexpr int kBalPer = kMaxExperts / 32;  // experts per lane

// First sequence that ends behind token t (n_seq if none).  Offsets that are
// not in order give some sequence number, never one out of range.
__device__ __forceinline__ int first_sequence(const int32_t* __restrict__ offsets, int n_seq,
                                              int64_t t) {
    int lo = 0, hi = n_seq;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (offsets[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// Softmax of one token's E logits by one warp, lane + 32 i holding expert
// lane + 32 i.  A token whose logits are all -inf (every expert masked off)
// has no distribution: its probabilities are 0.
__device__ __forceinline__ void token_probs(const float* __restrict__ row,
                                            const float* __restrict__ bias, int E,
                                            float (&p)[kBalPer]) {
    const int lane = threadIdx.x & 31;
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < kBalPer; ++i) {
        const int e = lane + 32 * i;
        p[i] = e < E ? row[e] : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < kBalPer; ++i) {
        const int e = lane + 32 * i;
        if (bias && e < E) p[i] += bias[e];
        mx = fmaxf(mx, p[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (mx == -INFINITY) mx = 0.0f;  // (a NaN logit still gives NaN below)
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < kBalPer; ++i) {
        p[i] = expf(p[i] - mx);
        z += p[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    const float inv = z == 0.0f ? 0.0f : 1.0f / z;
#pragma unroll
    for (int i = 0; i < kBalPer; ++i) p[i] *= inv;
}

// Pass 1: CTA b sums the probabilities and counts of the tokens of window b
// ([b * win, (b+1) * win)) for each sequence s that the window touches, into
// slot b + s: along the windows and sequences in order either b or s grows by
// one, so no two pairs share a slot.
__global__ void __launch_bounds__(256) balance_partial_kernel(
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
        float acc[kBalPer];
#pragma unroll
        for (int i = 0; i < kBalPer; ++i) acc[i] = 0.0f;
        int ntok = 0;
        for (int64_t t = lo + warp; t < hi; t += 8) {
            if (mask && !mask[t]) continue;
            ++ntok;
            if (lane < k) {
                const int e = idx[t * k + lane];
                if (e >= 0 && e < E) atomicAdd(&s_cnt[e], 1);
                else set_device_error(status, DEV_ERR_BAD_INDEX);
            }
            float p[kBalPer];
            token_probs(logits + t * E, bias, E, p);
#pragma unroll
            for (int i = 0; i < kBalPer; ++i) acc[i] += p[i];
        }
        if (lane == 0 && ntok) atomicAdd(&s_tok, ntok);
#pragma unroll
        for (int i = 0; i < kBalPer; ++i) s_sum[warp][lane + 32 * i] = acc[i];
        __syncthreads();
        const int64_t slot = static_cast<int64_t>(blockIdx.x) + s;
        if (tid < E) {
            float a = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; ++w) a += s_sum[w][tid];
            part_p[slot * E + tid] = a;
            part_c[slot * E + tid] = s_cnt[tid];
        }
        if (tid == 0) part_n[slot] = s_tok;
        __syncthreads();
    }
}

// Pass 2: CTA s adds the windows of sequence s (fp64, window order within each
// of kBalGroups interleaved groups, then group order) and writes its P, counts
// and token count; the CTA that finishes last adds the sequences' losses in
// sequence order.
constexpr int kBalGroups = 4;

__global__ void __launch_bounds__(kBalGroups* kMaxExperts) balance_final_kernel(
    const float* __restrict__ part_p, const int32_t* __restrict__ part_c,
    const int32_t* __restrict__ part_n, const int32_t* __restrict__ offsets, int n_seq, int64_t T,
    int E, int k, int win, float* __restrict__ P_out, int32_t* __restrict__ counts,
    int32_t* __restrict__ tokens, double* seq_loss, uint32_t* ticket, float* __restrict__ loss,
    int32_t* status) {
    __shared__ double s_p[kBalGroups][kMaxExperts];
    __shared__ int32_t s_c[kBalGroups][kMaxExperts];
    __shared__ double s_red[32];
    __shared__ int32_t s_n[32];
    __shared__ bool s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int e = tid % kMaxExperts, g = tid / kMaxExperts;
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
    const int64_t b0 = o0 / win, b1 = o1 > o0 ? (o1 - 1) / win : b0 - 1;
    double p = 0.0;
    int32_t c = 0, n = 0;
    if (e < E) {
#pragma unroll 4
        for (int64_t b = b0 + g; b <= b1; b += kBalGroups) {
            p += part_p[(b + s) * E + e];
            c += part_c[(b + s) * E + e];
        }
    }
    s_p[g][e] = p;
    s_c[g][e] = c;
    for (int64_t b = b0 + tid; b <= b1; b += blockDim.x) n += part_n[b + s];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0) s_n[warp] = n;
    __syncthreads();
    n = s_n[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    double prod = 0.0;
    if (g == 0 && e < E) {
#pragma unroll
        for (int i = 1; i < kBalGroups; ++i) {
            p += s_p[i][e];
            c += s_c[i][e];
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
        seq_loss[s] = a * E;
        tokens[s] = n;
        __threadfence();
        s_last = atomicAdd(ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    double a = 0.0;
    int used = 0;
    for (int i = tid; i < n_seq; i += blockDim.x) {
        a += __ldcg(seq_loss + i);
        used += __ldcg(tokens + i) > 0 ? 1 : 0;
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
        for (int w = 0; w < 32; ++w) {
            a += s_red[w];
            used += s_n[w];
        }
        tokens[n_seq] = used;
        *loss = used > 0 ? static_cast<float>(a / used) : 0.0f;
    }
}

// Gradient of the loss.  Each warp takes `run` consecutive tokens and keeps the
// selection shares f of its current sequence in registers.  With
// c = 1/E, sum_j p_j (f_j - c) + c = sum_j p_j f_j: taking the shares relative
// to the uniform one loses nothing of a small difference f - p.f to rounding.
__global__ void __launch_bounds__(256) balance_backward_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias,
    const uint8_t* __restrict__ mask, const int32_t* __restrict__ offsets, int n_seq, int64_t T,
    int E, int k, int run, const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens,
    const float* __restrict__ grad, float* __restrict__ dlogits) {
    const int lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t t0 = w * run, t1 = min(T, t0 + run);
    if (t0 >= T) return;
    ptx::grid_dep_wait();
    const int used = tokens[n_seq];
    const float g = used > 0 ? *grad * static_cast<float>(E) / static_cast<float>(used) : 0.0f;
    int s = offsets ? first_sequence(offsets, n_seq, t0) : 0;
    int loaded = -1;
    float f[kBalPer];
    float scale = 0.0f;
    for (int64_t t = t0; t < t1; ++t) {
        if (offsets)
            while (s < n_seq && offsets[s + 1] <= t) ++s;
        const bool live = s < n_seq && (!offsets || offsets[s] <= t) && (!mask || mask[t]);
        float p[kBalPer];
        if (live) {
            if (loaded != s) {
                loaded = s;
                const int n = tokens[s];
                const float inv = n > 0 ? 1.0f / (static_cast<float>(n) * k) : 0.0f;
                scale = n > 0 ? g / static_cast<float>(n) : 0.0f;
                const float c = 1.0f / static_cast<float>(E);
#pragma unroll
                for (int i = 0; i < kBalPer; ++i) {
                    const int e = lane + 32 * i;
                    f[i] = e < E ? counts[static_cast<int64_t>(s) * E + e] * inv - c : 0.0f;
                }
            }
            token_probs(logits + t * E, bias, E, p);
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < kBalPer; ++i) dot = fmaf(p[i], f[i], dot);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
#pragma unroll
            for (int i = 0; i < kBalPer; ++i) p[i] = scale * (p[i] * (f[i] - dot));
        } else {
#pragma unroll
            for (int i = 0; i < kBalPer; ++i) p[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kBalPer; ++i) {
            const int e = lane + 32 * i;
            if (e < E) dlogits[t * E + e] = p[i];
        }
    }
}

}  // namespace moe
