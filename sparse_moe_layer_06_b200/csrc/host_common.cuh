// host_common.cuh -- host-side pieces that every entry point shares: the
// launch counter and the per-kernel event profiler, problem checks, workspace
// carving and the launch helper.  Included by each translation unit of the
// library.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <mutex>
#include <utility>
#include <vector>

#include "../../include/moe.h"
#include "route_topk.cuh"

namespace moe {

// ------------------------------------------------------------------ launch bookkeeping

inline std::atomic<int64_t> g_launches{0};

struct ProfRecord {
    const char* name;
    cudaEvent_t start, stop;
};

struct Profiler {
    std::mutex mu;
    bool on = false;
    std::vector<cudaEvent_t> pool;  // 2 per record
    std::vector<ProfRecord> recs;
    size_t cap = 0;
};
inline Profiler g_prof;

struct LaunchScope {
    cudaEvent_t stop = nullptr;
    cudaStream_t stream;
    LaunchScope(const char* name, cudaStream_t s) : stream(s) {
        if (!g_prof.on) return;
        std::lock_guard<std::mutex> lk(g_prof.mu);
        if (!g_prof.on || g_prof.recs.size() >= g_prof.cap) return;
        ProfRecord r{name, g_prof.pool[2 * g_prof.recs.size()],
                     g_prof.pool[2 * g_prof.recs.size() + 1]};
        cudaEventRecord(r.start, s);
        stop = r.stop;
        g_prof.recs.push_back(r);
    }
    ~LaunchScope() {
        g_launches.fetch_add(1, std::memory_order_relaxed);
        if (stop) cudaEventRecord(stop, stream);
    }
};

#define MOE_LAUNCH(name, stream, ...)              \
    do {                                           \
        LaunchScope scope_(name, stream);          \
        __VA_ARGS__;                               \
        cudaError_t e_ = cudaGetLastError();       \
        if (e_ != cudaSuccess) return MOE_ERR_CUDA; \
    } while (0)

// ------------------------------------------------------------------ device info

inline int sm_count() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    static int cache[64] = {0};
    if (dev < 64 && cache[dev]) return cache[dev];
    int n = 0;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (n <= 0) n = 148;
    if (dev < 64) cache[dev] = n;
    return n;
}

// ------------------------------------------------------------------ problem checks

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int32_t check_problem(const moe_problem* p) {
    if (!p) return MOE_ERR_INVALID_ARG;
    if (p->T < 0) return MOE_ERR_INVALID_ARG;
    if (p->dtype != MOE_F32 && p->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
    if (p->H < 64 || p->H % 64 != 0 || p->I < 64 || p->I % 64 != 0) return MOE_ERR_UNSUPPORTED;
    // top_k <= 32: the router and the row gather keep one selection per lane
    if (p->E < 1 || p->E > kMaxExperts || p->top_k < 1 || p->top_k > p->E || p->top_k > 32)
        return MOE_ERR_UNSUPPORTED;
    if (p->num_shared != 0 && p->num_shared != 1) return MOE_ERR_UNSUPPORTED;
    if (p->T * static_cast<int64_t>(p->top_k + p->num_shared) >= (int64_t(1) << 31))
        return MOE_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(p->E) * 3 * p->I >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
    if (!std::isfinite(p->routed_scale)) return MOE_ERR_INVALID_ARG;
    if (std::isnan(p->clip_limit)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

inline int env_int(const char* name, int dflt) {
    const char* e = std::getenv(name);
    return e ? std::atoi(e) : dflt;
}

// ------------------------------------------------------------------ workspace carving

struct Carve {
    size_t off = 0;
    size_t take(size_t bytes) {
        size_t o = off;
        off += (bytes + 255) & ~size_t(255);
        return o;
    }
};

template <typename T>
T* at(void* ws, size_t off) {
    return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

// ------------------------------------------------------------------ launches

// Kernel launch on stream s; with pdl the launch may begin before the
// previous launch on the stream has finished (programmatic stream
// serialization): the kernel must then wait (griddepcontrol.wait) before it
// reads anything the previous launch writes.
template <typename... KArgs, typename... Args>
cudaError_t launch_ex(void (*kern)(KArgs...), dim3 grid, int threads, int smem, cudaStream_t s,
                      bool pdl, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// Programmatic dependent launch along the forward's kernel chain (MOE_PDL=0
// turns it off): each kernel may start while its predecessor finishes, does
// its independent set-up (in the expert GEMMs: streams its first weight
// tiles), then waits for the predecessor before reading its outputs.
inline bool pdl_enabled() {
    const bool v = env_int("MOE_PDL", 1) != 0;
    return v;
}

#define MOE_TRY(expr)                      \
    do {                                   \
        int32_t r_ = (expr);               \
        if (r_ != MOE_OK) return r_;       \
    } while (0)

}  // namespace moe
