// ops_api.cu -- host side of the operators around the layer: the pre-norm and
// its backward pass, the balance loss and its gradient, and the experts'
// products with 4-bit weights.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "host_common.cuh"
#include "internal.hpp"
#include "balance_kernels.cuh"
#include "norm_kernels.cuh"
#include "w4_kernels.cuh"

namespace moe {
namespace {

// ------------------------------------------------------------------ norm

int32_t check_norm(const moe_problem* p, float eps) {
    MOE_TRY(check_problem(p));
    if (p->H > kNormMaxH) return MOE_ERR_UNSUPPORTED;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// How a launch over rows of H values covers them: VPT 16-byte vectors per
// thread (2 up to `two` vectors, 4 above), CTAs per SM (about `per_sm` threads),
// and the depth of their rings.
struct RowShape {
    int nv, vpt, threads, ctas, depth, smem;
};

constexpr int kNormThreadsPerSM = 768, kNormBackThreadsPerSM = 512;
// Longest rows that take two vectors per thread (longer ones four).  Forward: 100
// us with two and 96 with four for 8192 rows of 4352 fp32.  Backward, which keeps
// its share of dw too: 89 and 213 us.
constexpr int kNormTwo = 1024, kNormBackTwo = 2048;
constexpr int kRingBytesPerSM = 200 * 1024;

RowShape row_shape(const moe_problem* p, int inputs, int per_sm, int two) {
    RowShape r;
    const int row_bytes = p->H * (p->dtype == MOE_BF16 ? 2 : 4);
    r.nv = row_bytes / 16;
    r.vpt = r.nv <= two ? 2 : 4;
    r.threads = std::max(32, ((r.nv + r.vpt - 1) / r.vpt + 31) / 32 * 32);
    r.ctas = std::max(1, std::min(8, per_sm / r.threads));
    const int rows = kRingBytesPerSM / r.ctas / (inputs * row_bytes);
    r.depth = rows >= 4 ? 4 : (rows >= 2 ? 2 : 1);
    r.smem = r.depth * inputs * row_bytes;
    return r;
}

// Lets `kern` take the ring's shared memory, once per device.
template <typename K>
bool allow_ring(K kern, std::atomic<uint64_t>& configured) {
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (bit && (configured.load() & bit)) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kRingBytesPerSM) != cudaSuccess)
        return false;
    configured.fetch_or(bit);
    return true;
}

template <typename T, int VPT, int D, int MaxThreads>
int32_t launch_norm(const moe_problem* p, const RowShape& r, const void* x, const void* res,
                    const void* weight, float eps, void* res_out, void* y, uint8_t* y_q,
                    float* y_scale, cudaStream_t s) {
    auto kern = add_rmsnorm_kernel<T, VPT, D, MaxThreads>;
    static std::atomic<uint64_t> configured{0};
    if (!allow_ring(kern, configured)) return MOE_ERR_CUDA;
    const int64_t most = static_cast<int64_t>(sm_count()) * r.ctas;
    MOE_LAUNCH("add_rmsnorm", s,
               if (launch_ex(kern, static_cast<int>(std::min<int64_t>(p->T, most)), r.threads,
                             r.smem, s, pdl_enabled(), static_cast<const T*>(x),
                             static_cast<const T*>(res), static_cast<const T*>(weight), eps, p->T,
                             p->H, static_cast<T*>(res_out), static_cast<T*>(y), y_q, y_scale) !=
                   cudaSuccess) return MOE_ERR_CUDA);
    return MOE_OK;
}

template <typename T, int VPT>
int32_t launch_norm_short(const moe_problem* p, const void* x, const void* res,
                          const void* weight, float eps, void* res_out, void* y, uint8_t* y_q,
                          float* y_scale, cudaStream_t s) {
    MOE_LAUNCH("add_rmsnorm_short", s,
               if (launch_ex(add_rmsnorm_short_kernel<T, VPT>, static_cast<int>((p->T + 3) / 4),
                             128, 0, s, pdl_enabled(), static_cast<const T*>(x),
                             static_cast<const T*>(res), static_cast<const T*>(weight), eps, p->T,
                             p->H, static_cast<T*>(res_out), static_cast<T*>(y), y_q, y_scale) !=
                   cudaSuccess) return MOE_ERR_CUDA);
    return MOE_OK;
}

template <typename T>
int32_t run_norm(const moe_problem* p, const void* x, const void* res, const void* weight,
                 float eps, void* res_out, void* y, uint8_t* y_q, float* y_scale,
                 cudaStream_t s) {
    const RowShape r = row_shape(p, res ? 2 : 1, kNormThreadsPerSM, kNormTwo);
    if (r.nv <= 64)
        return launch_norm_short<T, 2>(p, x, res, weight, eps, res_out, y, y_q, y_scale, s);
    if (r.nv <= 128)
        return launch_norm_short<T, 4>(p, x, res, weight, eps, res_out, y, y_q, y_scale, s);
#define MOE_NORM(V, D, N) \
    return launch_norm<T, V, D, N>(p, r, x, res, weight, eps, res_out, y, y_q, y_scale, s)
    // (the other shapes belong to no width up to kNormMaxH)
    constexpr int kMost = sizeof(T) == 2 ? 512 : 1024;  // threads of the widest row
    if (r.vpt == 2 && r.depth == 4) MOE_NORM(2, 4, 512);
    if (r.vpt == 4 && r.depth == 4) MOE_NORM(4, 4, kMost);
    if (r.vpt == 4 && r.depth == 2) MOE_NORM(4, 2, kMost);
    if constexpr (sizeof(T) == 4) {
        if (r.vpt == 4) MOE_NORM(4, 1, 1024);
    }
    return MOE_ERR_UNSUPPORTED;
#undef MOE_NORM
}

// CTAs of the backward pass, as many rows for each (the workspace holds a
// partial dw of each CTA; the count goes by 148 SMs on any device, so that it
// depends on the problem only).
constexpr int64_t kNormBackSMs = 148;
int64_t norm_backward_ctas(const moe_problem* p) {
    if (p->T <= 0) return 1;
    const int64_t most = kNormBackSMs * row_shape(p, 3, kNormBackThreadsPerSM, kNormBackTwo).ctas;
    const int64_t per = (p->T + most - 1) / most;
    return (p->T + per - 1) / per;
}

template <typename T, int VPT, int D, int MaxThreads>
int32_t launch_norm_backward(const moe_problem* p, const RowShape& r, const void* dy,
                             const void* dres, const void* h, const void* weight, float eps,
                             void* dx, float* dweight, float* partial, cudaStream_t s) {
    auto kern = add_rmsnorm_backward_kernel<T, VPT, D, MaxThreads>;
    static std::atomic<uint64_t> configured{0};
    if (!allow_ring(kern, configured)) return MOE_ERR_CUDA;
    const int ctas = static_cast<int>(norm_backward_ctas(p));
    MOE_LAUNCH("add_rmsnorm_backward", s,
               if (launch_ex(kern, ctas, r.threads, r.smem, s, pdl_enabled(),
                             static_cast<const T*>(dy), static_cast<const T*>(dres),
                             static_cast<const T*>(h), static_cast<const T*>(weight), eps, p->T,
                             p->H, static_cast<T*>(dx), partial) != cudaSuccess)
                   return MOE_ERR_CUDA);
    MOE_LAUNCH("add_rmsnorm_dweight", s,
               if (launch_ex(reduce_columns_kernel, p->H / 32, 1024, 0, s, pdl_enabled(),
                             static_cast<const float*>(partial), ctas, p->H, dweight) !=
                   cudaSuccess) return MOE_ERR_CUDA);
    return MOE_OK;
}

template <typename T>
int32_t run_norm_backward(const moe_problem* p, const void* dy, const void* dres, const void* h,
                          const void* weight, float eps, void* dx, float* dweight,
                          float* partial, cudaStream_t s) {
    const RowShape r = row_shape(p, dres ? 3 : 2, kNormBackThreadsPerSM, kNormBackTwo);
#define MOE_NORM(V, D, N) \
    return launch_norm_backward<T, V, D, N>(p, r, dy, dres, h, weight, eps, dx, dweight, partial, s)
    // (the other shapes belong to no width up to kNormMaxH)
    if (r.vpt == 2 && r.depth == 4 && r.threads <= 512) MOE_NORM(2, 4, 512);
    if (r.vpt == 2 && r.depth == 4) MOE_NORM(2, 4, 1024);
    if (r.vpt == 2 && r.depth == 2 && r.threads > 512) MOE_NORM(2, 2, 1024);
    if constexpr (sizeof(T) == 4) {
        if (r.vpt == 4 && r.depth == 2) MOE_NORM(4, 2, 1024);
        if (r.vpt == 4 && r.depth == 1) MOE_NORM(4, 1, 1024);
    }
    return MOE_ERR_UNSUPPORTED;
#undef MOE_NORM
}

// ------------------------------------------------------------------ balance loss

constexpr int32_t kMaxSequences = 1 << 20;

// Tokens per window, a multiple of the CTA's 8 warps: at most 3 windows per SM,
// which is what its registers hold at once.
int balance_window(int64_t T) {
    return static_cast<int>(8 * std::max<int64_t>(1, (T + 8 * 444 - 1) / (8 * 444)));
}

// Up to this many tokens one sequence takes one CTA and one launch: 4.2 us a call
// for 64 x 256 logits in a captured graph, 5.5 in two launches; 6.2 and 5.5 for 128
// (called one by one, where the host bounds, 8.5 and 11.5 us for both).
constexpr int64_t kBalOneTokens = 96;

// log2 of the threads of pass 2 that share a window's experts, four each: eight or
// sixteen, and so up to four CTAs a sequence, while these are no more than the SMs.
int balance_log_group(int64_t E, int64_t n_seq) {
    int g = E <= 32 ? 3 : 4;
    while ((4 << g) < E && (E + (4 << g) - 1) / (4 << g) * n_seq > 148) ++g;
    return g;
}
int64_t balance_chunks(int64_t E, int64_t n_seq) {
    const int per = 4 << balance_log_group(E, n_seq);
    return (E + per - 1) / per;
}

struct BalanceLayout {
    size_t status, ticket, part_p, part_c, part_n, seq_loss, total;
};

BalanceLayout balance_layout(const moe_problem* p, int64_t n_seq) {
    BalanceLayout L{};
    Carve c;
    const int64_t win = balance_window(p->T);
    const int64_t slots = std::max<int64_t>(1, (p->T + win - 1) / win) + n_seq;
    L.status = c.take(256);
    L.ticket = c.take(4);
    L.part_p = c.take(slots * balance_pad(p->E) * 4);
    L.part_c = c.take(slots * balance_pad(p->E) * 4);
    L.part_n = c.take(slots * 4);
    L.seq_loss = c.take(n_seq * balance_chunks(p->E, n_seq) * 8);
    L.total = c.off;
    return L;
}

// Calls f with the kernels' experts per lane and whether they load them four at
// a time: more than 64 experts, rows of a multiple of 4, aligned arrays.
template <typename F>
int32_t with_slots(int E, bool aligned, F f) {
    if (E > 64 && E % 4 == 0 && aligned) {
        if (E > 128) return f(std::integral_constant<int, 8>{}, std::true_type{});
        return f(std::integral_constant<int, 4>{}, std::true_type{});
    }
    if (E > 128) return f(std::integral_constant<int, 8>{}, std::false_type{});
    if (E > 64) return f(std::integral_constant<int, 4>{}, std::false_type{});
    if (E > 32) return f(std::integral_constant<int, 2>{}, std::false_type{});
    return f(std::integral_constant<int, 1>{}, std::false_type{});
}

int32_t check_sequences(const int32_t* offsets, int32_t n_seq) {
    if (n_seq < 1 || (!offsets && n_seq != 1)) return MOE_ERR_INVALID_ARG;
    if (n_seq > kMaxSequences) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// ------------------------------------------------------------------ 4-bit experts

int32_t check_w4(const moe_problem* p, int32_t group) {
    MOE_TRY(check_problem(p));
    if (p->H % kW4Block != 0 || p->I % kW4Block != 0) return MOE_ERR_UNSUPPORTED;
    if (group != 32 && group != 64 && group != 128) return MOE_ERR_UNSUPPORTED;
    // a chunk of one row has to fit in a CTA's shared memory
    if (p->H > kW4MaxK || p->I > kW4MaxK) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

struct W4Layout {
    size_t status, route, idx, w, hist, base, counts, offsets, sched_gu, sched_dn, pos, src,
        row_w, h, y, total;
    // integers of the rows of x and of h: limbs and sums, and the second ones
    size_t x_limbs[2], x_meta[2], h_limbs[2], h_meta[2];
};

W4Layout w4_layout(const moe_problem* p, bool with_route) {
    W4Layout L{};
    Carve c;
    const int64_t T = p->T, H = p->H, E = p->E, I = p->I, k = p->top_k, S = p->num_shared;
    // the router's workspace (error word first), or the error word alone
    L.status = c.take(with_route ? moe_workspace_size(p, MOE_CALL_ROUTE) : 256);
    if (with_route) {
        L.idx = c.take(T * k * 4);
        L.w = c.take(T * k * 4);
    }
    L.hist = c.take(dispatch_chunks(T) * E * 4);
    L.base = c.take(dispatch_chunks(T) * E * 4);
    L.counts = c.take(E * 4);
    L.offsets = c.take((E + 1) * 4);
    L.sched_gu = c.take(schedule_bytes());
    L.sched_dn = c.take(schedule_bytes());
    L.pos = c.take(T * k * 4);
    L.src = c.take(T * k * 4);
    L.row_w = c.take(T * k * 4);
    for (int i = 0; i < 2; ++i) {
        L.x_limbs[i] = c.take(T * H * 2);
        L.x_meta[i] = c.take(T * (H / kW4Block) * kW4MaxMeta * 4);
        L.h_limbs[i] = c.take(T * (k + S) * I * 2);
        L.h_meta[i] = c.take(T * (k + S) * (I / kW4Block) * kW4MaxMeta * 4);
    }
    L.h = c.take(T * (k + S) * I * 4);
    L.y = c.take(T * (k + S) * H * 4);
    L.total = c.off;
    return L;
}

// 8-row column tiles per task, from the mean rows per expert (the host does not know
// which experts are the fuller ones): one leaves registers for 16 warps, two read a
// weight once for 16 rows.  Measured with uniform routing (256 experts of
// 6144 x 2048, groups of 64, calls in a row), one against two tiles: 0.93 and 1.04
// ms at 96 tokens (3 rows), 1.04 and 1.09 at 128 (4), 1.18 and 1.14 at 160 (5),
// 1.56 and 1.39 at 256, 2.75 and 2.50 at 512.
int w4_column_tiles(double mean_rows) { return mean_rows <= 4.5 ? 1 : 2; }

int w4_cap(int nt, int64_t K, int sub) {
    if (sub == 1) return nt == 1 ? w4_rows_cap<1, 1>(K) : w4_rows_cap<2, 1>(K);
    if (sub == 2) return nt == 1 ? w4_rows_cap<1, 2>(K) : w4_rows_cap<2, 2>(K);
    return nt == 1 ? w4_rows_cap<1, 4>(K) : w4_rows_cap<2, 4>(K);
}

template <int NT, bool DOWN, int SUB>
int32_t launch_w4_n(const W4Args& a, int64_t max_tasks, cudaStream_t s) {
    auto kern = w4_product_kernel<NT, DOWN, SUB>;
    constexpr int threads = W4Shape<NT, SUB>::kWarps * 32;
    int dev = 0;
    cudaGetDevice(&dev);
    static std::atomic<uint64_t> configured{0};
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!bit || !(configured.load() & bit)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024) !=
            cudaSuccess)
            return MOE_ERR_CUDA;
        configured.fetch_or(bit);
    }
    const int smem = W4Shape<NT, SUB>::kSumBytes + W4Shape<NT, SUB>::kSlack +
                     a.K / kW4Block * a.cap * (kW4RowBytes + 4 * w4_meta_words(SUB));
    const int grid =
        static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(sm_count(), max_tasks)));
    MOE_LAUNCH(DOWN ? "expert_down_w4" : "expert_gate_up_w4", s,
               if (launch_ex(kern, grid, threads, smem, s, pdl_enabled(), a) != cudaSuccess)
                   return MOE_ERR_CUDA);
    return MOE_OK;
}

template <bool DOWN>
int32_t launch_w4(int nt, int group, const W4Args& a, int64_t max_tasks, cudaStream_t s) {
    const int key = nt * 1000 + group;
    switch (key) {
        case 1032: return launch_w4_n<1, DOWN, 4>(a, max_tasks, s);
        case 1064: return launch_w4_n<1, DOWN, 2>(a, max_tasks, s);
        case 1128: return launch_w4_n<1, DOWN, 1>(a, max_tasks, s);
        case 2032: return launch_w4_n<2, DOWN, 4>(a, max_tasks, s);
        case 2064: return launch_w4_n<2, DOWN, 2>(a, max_tasks, s);
        case 2128: return launch_w4_n<2, DOWN, 1>(a, max_tasks, s);
        default: return MOE_ERR_UNSUPPORTED;
    }
}

int32_t run_experts_w4(const moe_problem* p, int32_t group, const void* x, const int32_t* idx,
                       const float* w, const uint8_t* eq, const void* es, const uint8_t* sq,
                       const void* ss, void* out, void* ws, const W4Layout& L, cudaStream_t s) {
    const int64_t T = p->T, H = p->H, E = p->E, I = p->I, k = p->top_k, S = p->num_shared;
    int32_t* status = at<int32_t>(ws, L.status);
    int32_t* sg = at<int32_t>(ws, L.sched_gu);
    int32_t* sd = at<int32_t>(ws, L.sched_dn);
    int32_t* pos = at<int32_t>(ws, L.pos);
    int32_t* src = at<int32_t>(ws, L.src);
    float* row_w = at<float>(ws, L.row_w);
    const int sub = kW4Block / group;
    const int nt = w4_column_tiles(static_cast<double>(T * k) / E);
    const int cap_gu = w4_cap(nt, H, sub), cap_dn = w4_cap(nt, I, sub);
    const bool pdl = pdl_enabled();
    const __nv_bfloat16* xb = static_cast<const __nv_bfloat16*>(x);
    W4Rows x_rows[2], h_rows[2];
    for (int i = 0; i < 2; ++i) {
        x_rows[i] = {at<uint8_t>(ws, L.x_limbs[i]), at<uint32_t>(ws, L.x_meta[i])};
        h_rows[i] = {at<uint8_t>(ws, L.h_limbs[i]), at<uint32_t>(ws, L.h_meta[i])};
    }
    const int64_t x_units = T * (H / kW4Block);
    if (T <= kPermTokens) {
        MOE_LAUNCH("dispatch_w4", s,
                   if (launch_ex(w4_dispatch_kernel, 1 + static_cast<int>((x_units + 15) / 16),
                                 512, 0, s, pdl, idx, w, static_cast<int>(T), p->E, p->top_k,
                                 p->num_shared, sg, cap_gu, sd, cap_dn, pos, src, row_w, status,
                                 xb, x_units, sub, x_rows[0], x_rows[1]) != cudaSuccess)
                       return MOE_ERR_CUDA);
    } else {
        // (an assignment with an expert out of range keeps position -1)
        if (cudaMemsetAsync(pos, 0xff, static_cast<size_t>(T * k) * 4, s) != cudaSuccess)
            return MOE_ERR_CUDA;
        MOE_TRY(dispatch_rows(p, idx, w, at<int32_t>(ws, L.hist), at<int32_t>(ws, L.base),
                              at<int32_t>(ws, L.counts), at<int32_t>(ws, L.offsets), sg, cap_gu,
                              sd, cap_dn, pos, src, row_w, status, s));
        MOE_LAUNCH("split_rows_w4", s,
                   if (launch_ex(w4_split_kernel<__nv_bfloat16>,
                                 static_cast<int>((x_units + 7) / 8), 256, 0, s, pdl, xb, x_units,
                                 sub, x_rows[0], x_rows[1]) != cudaSuccess)
                       return MOE_ERR_CUDA);
    }
    const int nseg = static_cast<int>(E + S);
    // at most this many chunks of `cap` rows over all segments
    const auto max_chunks = [&](int64_t cap) {
        return std::min<int64_t>(T * k, T * k / cap + E) + (S ? (T + cap - 1) / cap : 0);
    };
    W4Args a{};
    a.nseg = nseg;
    a.special = S ? static_cast<int32_t>(E) : -1;
    a.q_stride = 3 * I * H / 2;
    a.sc_stride = 3 * I * H / group;
    a.routed_rows = static_cast<int32_t>(T * k);
    a.row_w = row_w;
    a.row_src = src;
    a.clip = (p->clip_limit > 0.0f && std::isfinite(p->clip_limit)) ? p->clip_limit : INFINITY;
    a.q = eq;
    a.sc = static_cast<const __nv_bfloat16*>(es);
    a.q_shared = sq;
    a.sc_shared = static_cast<const __nv_bfloat16*>(ss);
    a.sched = sg;
    a.rows = x_rows[0];
    a.rest = x_rows[1];
    a.cap = cap_gu;
    a.K = static_cast<int32_t>(H);
    a.tiles = static_cast<int32_t>(I / 16);
    a.out = at<float>(ws, L.h);
    a.ld = static_cast<int32_t>(I);
    MOE_TRY(launch_w4<false>(nt, group, a, max_chunks(cap_gu) * a.tiles, s));
    const int64_t h_units = T * (k + S) * (I / kW4Block);
    MOE_LAUNCH("split_h_w4", s,
               if (launch_ex(w4_split_kernel<float>, static_cast<int>((h_units + 7) / 8), 256, 0,
                             s, pdl, static_cast<const float*>(a.out), h_units, sub, h_rows[0],
                             h_rows[1]) != cudaSuccess) return MOE_ERR_CUDA);
    a.q = eq + I * H;
    a.sc = static_cast<const __nv_bfloat16*>(es) + 2 * I * H / group;
    a.q_shared = sq ? sq + I * H : nullptr;
    a.sc_shared = ss ? static_cast<const __nv_bfloat16*>(ss) + 2 * I * H / group : nullptr;
    a.sched = sd;
    a.rows = h_rows[0];
    a.rest = h_rows[1];
    a.cap = cap_dn;
    a.K = static_cast<int32_t>(I);
    a.tiles = static_cast<int32_t>(H / 32);
    a.out = at<float>(ws, L.y);
    a.ld = static_cast<int32_t>(H);
    MOE_TRY(launch_w4<true>(nt, group, a, max_chunks(cap_dn) * a.tiles, s));
    return combine_rows_f32(p, at<float>(ws, L.y), pos, static_cast<__nv_bfloat16*>(out), status,
                            s);
}

bool aligned32(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 31u) == 0; }

// Checks of the two 4-bit entry points.
int32_t check_w4_call(const moe_problem* p, int32_t group, const void* x, const uint8_t* eq,
                      const void* es, const uint8_t* sq, const void* ss, const void* out,
                      const void* ws) {
    MOE_TRY(check_w4(p, group));
    if (p->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
    if (!eq || !es || !ws || (p->T > 0 && (!x || !out))) return MOE_ERR_INVALID_ARG;
    if (p->num_shared && (!sq || !ss)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(eq) || !aligned16(es) || !aligned16(out) || !aligned16(ws) ||
        (sq && !aligned16(sq)) || (ss && !aligned16(ss)))
        return MOE_ERR_INVALID_ARG;
    // the codes are read in 32-byte vectors
    if (!aligned32(eq) || (sq && !aligned32(sq))) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

}  // namespace

size_t operator_workspace(const moe_problem* p, int32_t call) {
    switch (call) {
        case MOE_CALL_ADD_RMSNORM_BACKWARD:
            if (p->H > kNormMaxH) return 0;
            return 256 + static_cast<size_t>(norm_backward_ctas(p)) * p->H * 4;
        case MOE_CALL_BALANCE_LOSS: return balance_layout(p, 1).total;
        case MOE_CALL_EXPERTS_W4:
        case MOE_CALL_FORWARD_W4:
            if (check_w4(p, kW4Block) != MOE_OK || p->dtype != MOE_BF16) return 0;
            return w4_layout(p, call == MOE_CALL_FORWARD_W4).total;
        default: return 0;
    }
}

}  // namespace moe

using namespace moe;

extern "C" {

int32_t moe_add_rmsnorm(const moe_problem* p, const void* x, const void* residual,
                        const void* weight, float eps, void* residual_out, void* y, uint8_t* y_q,
                        float* y_scale, void* stream) {
    MOE_TRY(check_norm(p, eps));
    if (!weight) return MOE_ERR_INVALID_ARG;
    // (an empty batch's row pointers may be null)
    if (p->T > 0 && (!x || (!y && !y_q) || (!y_q) != (!y_scale))) return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(residual_out) ||
        !aligned16(y) || !aligned16(y_q))
        return MOE_ERR_INVALID_ARG;
    if (p->T == 0) return MOE_OK;
    if (residual_out && residual_out == y) return MOE_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p->dtype == MOE_BF16)
        return run_norm<__nv_bfloat16>(p, x, residual, weight, eps, residual_out, y, y_q, y_scale,
                                       s);
    return run_norm<float>(p, x, residual, weight, eps, residual_out, y, y_q, y_scale, s);
}

int32_t moe_add_rmsnorm_backward(const moe_problem* p, const void* dy, const void* dresidual,
                                 const void* h, const void* weight, float eps, void* dx,
                                 float* dweight, void* ws, size_t ws_bytes, void* stream) {
    MOE_TRY(check_norm(p, eps));
    if (!weight || !dweight || !ws || (p->T > 0 && (!dy || !h || !dx))) return MOE_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(dresidual) || !aligned16(h) || !aligned16(weight) ||
        !aligned16(dx) || !aligned16(ws))
        return MOE_ERR_INVALID_ARG;
    if (ws_bytes < operator_workspace(p, MOE_CALL_ADD_RMSNORM_BACKWARD)) return MOE_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p->T == 0) {
        // the sum over no rows
        if (cudaMemsetAsync(dweight, 0, static_cast<size_t>(p->H) * 4, s) != cudaSuccess)
            return MOE_ERR_CUDA;
        return MOE_OK;
    }
    float* partial = at<float>(ws, 256);
    if (p->dtype == MOE_BF16)
        return run_norm_backward<__nv_bfloat16>(p, dy, dresidual, h, weight, eps, dx, dweight,
                                                partial, s);
    return run_norm_backward<float>(p, dy, dresidual, h, weight, eps, dx, dweight, partial, s);
}

size_t moe_balance_loss_workspace_size(const moe_problem* p, int32_t n_seq) {
    if (check_problem(p) != MOE_OK || n_seq < 1 || n_seq > kMaxSequences) return 0;
    return balance_layout(p, n_seq).total;
}

int32_t moe_balance_loss(const moe_problem* p, const float* logits, const float* bias,
                         const int32_t* topk_idx, const uint8_t* token_mask,
                         const int32_t* seq_offsets, int32_t n_seq, float* loss, int32_t* counts,
                         int32_t* tokens, float* mean_prob, void* ws, size_t ws_bytes,
                         void* stream) {
    MOE_TRY(check_problem(p));
    MOE_TRY(check_sequences(seq_offsets, n_seq));
    if ((p->T > 0 && (!logits || !topk_idx)) || !loss || !counts || !tokens || !mean_prob || !ws)
        return MOE_ERR_INVALID_ARG;
    if (!aligned16(ws)) return MOE_ERR_INVALID_ARG;
    const BalanceLayout L = balance_layout(p, n_seq);
    if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int win = balance_window(p->T);
    const int nwin = static_cast<int>(std::max<int64_t>(1, (p->T + win - 1) / win));
    int32_t* status = at<int32_t>(ws, L.status);
    float* part_p = at<float>(ws, L.part_p);
    int32_t* part_c = at<int32_t>(ws, L.part_c);
    int32_t* part_n = at<int32_t>(ws, L.part_n);
    uint32_t* ticket = at<uint32_t>(ws, L.ticket);
    if (n_seq == 1 && p->T <= kBalOneTokens)
        return with_slots(p->E, aligned16(logits) && aligned16(bias),
                          [&](auto np, auto vec) -> int32_t {
            MOE_LAUNCH("balance_one", s,
                       if (launch_ex(balance_one_kernel<decltype(np)::value, decltype(vec)::value>,
                                     1, kBalOneWarps * 32, 0, s, pdl_enabled(), logits, bias,
                                     topk_idx, token_mask, seq_offsets, p->T, p->E, p->top_k,
                                     mean_prob, counts, tokens, loss, status) != cudaSuccess)
                           return MOE_ERR_CUDA);
            return MOE_OK;
        });
    MOE_TRY(with_slots(p->E, aligned16(logits) && aligned16(bias),
                       [&](auto np, auto vec) -> int32_t {
        MOE_LAUNCH("balance_partial", s,
                   if (launch_ex(balance_partial_kernel<decltype(np)::value, decltype(vec)::value>,
                                 nwin, 256, 0, s, pdl_enabled(), logits, bias, topk_idx,
                                 token_mask, seq_offsets, static_cast<int>(n_seq), p->T, p->E,
                                 p->top_k, win, part_p, part_c, part_n, ticket, status) !=
                       cudaSuccess) return MOE_ERR_CUDA);
        return MOE_OK;
    }));
    MOE_LAUNCH("balance_final", s,
               if (launch_ex(balance_final_kernel,
                             dim3(static_cast<unsigned>(n_seq),
                                  static_cast<unsigned>(balance_chunks(p->E, n_seq))),
                             kBalFinal, 0, s,
                             pdl_enabled(), static_cast<const float*>(part_p),
                             static_cast<const int32_t*>(part_c),
                             static_cast<const int32_t*>(part_n), seq_offsets,
                             static_cast<int>(n_seq), p->T, p->E, p->top_k, win,
                             balance_log_group(p->E, n_seq), mean_prob, counts, tokens,
                             at<double>(ws, L.seq_loss), ticket, loss, status) != cudaSuccess)
                   return MOE_ERR_CUDA);
    return MOE_OK;
}

int32_t moe_balance_loss_backward(const moe_problem* p, const float* logits, const float* bias,
                                  const uint8_t* token_mask, const int32_t* seq_offsets,
                                  int32_t n_seq, const int32_t* counts, const int32_t* tokens,
                                  const float* grad_loss, float* dlogits, void* stream) {
    MOE_TRY(check_problem(p));
    MOE_TRY(check_sequences(seq_offsets, n_seq));
    if (p->T == 0) return MOE_OK;
    if (!logits || !counts || !tokens || !grad_loss || !dlogits || dlogits == logits)
        return MOE_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // consecutive tokens per warp: 16 warps per SM, which are resident at once
    const int64_t warps = 148 * 16;
    const int run = static_cast<int>((p->T + warps - 1) / warps);
    const int grid = static_cast<int>((p->T + 8 * run - 1) / (8 * run));
    return with_slots(
        p->E, aligned16(logits) && aligned16(bias) && aligned16(dlogits),
        [&](auto np, auto vec) -> int32_t {
            MOE_LAUNCH(
                "balance_backward", s,
                if (launch_ex(balance_backward_kernel<decltype(np)::value, decltype(vec)::value>,
                              grid, 256, 0, s, pdl_enabled(), logits, bias, token_mask,
                              seq_offsets, static_cast<int>(n_seq), p->T, p->E, p->top_k, run,
                              counts, tokens, grad_loss, dlogits) != cudaSuccess)
                    return MOE_ERR_CUDA);
            return MOE_OK;
        });
}

int32_t moe_quantize_weights_w4(const moe_problem* p, int32_t group_size, int32_t n_experts,
                                const void* w, uint8_t* q, void* scales, void* stream) {
    MOE_TRY(check_w4(p, group_size));
    if (!w || !q || !scales) return MOE_ERR_INVALID_ARG;
    if (!aligned16(w) || !aligned16(q) || !aligned16(scales)) return MOE_ERR_INVALID_ARG;
    if (n_experts < 1 || n_experts > 65535) return MOE_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 grid(static_cast<unsigned>(3ll * p->I * p->H / (16 * kW4Block)),
                    static_cast<unsigned>(n_experts));
    __nv_bfloat16* sc = static_cast<__nv_bfloat16*>(scales);
    auto go = [&](auto* in) -> int32_t {
        using T = std::remove_const_t<std::remove_pointer_t<decltype(in)>>;
        auto kern = group_size == 128 ? w4_encode_kernel<T, 1>
                                      : (group_size == 64 ? w4_encode_kernel<T, 2>
                                                          : w4_encode_kernel<T, 4>);
        MOE_LAUNCH("quantize_weights_w4", s, kern<<<grid, 128, 0, s>>>(in, p->I, p->H, q, sc));
        return MOE_OK;
    };
    if (p->dtype == MOE_BF16) return go(static_cast<const __nv_bfloat16*>(w));
    return go(static_cast<const float*>(w));
}

int32_t moe_experts_w4(const moe_problem* p, int32_t group_size, const void* x,
                       const int32_t* topk_idx, const float* topk_w, const uint8_t* expert_q,
                       const void* expert_scale, const uint8_t* shared_q,
                       const void* shared_scale, void* out, void* ws, size_t ws_bytes,
                       void* stream) {
    MOE_TRY(check_w4_call(p, group_size, x, expert_q, expert_scale, shared_q, shared_scale, out,
                          ws));
    if (p->T > 0 && (!topk_idx || !topk_w)) return MOE_ERR_INVALID_ARG;
    const W4Layout L = w4_layout(p, false);
    if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
    if (p->T == 0) return MOE_OK;
    return run_experts_w4(p, group_size, x, topk_idx, topk_w, expert_q, expert_scale, shared_q,
                          shared_scale, out, ws, L, static_cast<cudaStream_t>(stream));
}

int32_t moe_forward_w4(const moe_problem* p, int32_t group_size, const void* x,
                       const void* gate_w, const float* bias, const uint8_t* expert_q,
                       const void* expert_scale, const uint8_t* shared_q,
                       const void* shared_scale, void* out, int32_t* idx_out, float* w_out,
                       void* ws, size_t ws_bytes, void* stream) {
    MOE_TRY(check_w4_call(p, group_size, x, expert_q, expert_scale, shared_q, shared_scale, out,
                          ws));
    if (!gate_w || !aligned16(gate_w)) return MOE_ERR_INVALID_ARG;
    const W4Layout L = w4_layout(p, true);
    if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
    if (p->T == 0) return MOE_OK;
    int32_t* idx = idx_out ? idx_out : at<int32_t>(ws, L.idx);
    float* w = w_out ? w_out : at<float>(ws, L.w);
    MOE_TRY(moe_route(p, x, gate_w, bias, idx, w, ws, ws_bytes, stream));
    return run_experts_w4(p, group_size, x, idx, w, expert_q, expert_scale, shared_q, shared_scale,
                          out, ws, L, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
