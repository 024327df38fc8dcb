// internal.hpp -- host functions of moe_api.cu that the operators in
// ops_api.cu share, and the other way round (no part of the C ABI).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/moe.h"

namespace moe {

// moe_api.cu: histogram, offsets, tile schedules and stable positions of the
// (token, slot) rows, in three launches.
int32_t dispatch_rows(const moe_problem* p, const int32_t* idx, const float* topk_w,
                      int32_t* hist, int32_t* base, int32_t* counts, int32_t* offsets,
                      int32_t* sched_gu, int nmax_gu, int32_t* sched_dn, int nmax_dn,
                      int32_t* pos, int32_t* src, float* row_w, int32_t* status, cudaStream_t s);
int64_t dispatch_chunks(int64_t T);
size_t schedule_bytes();

// moe_api.cu: fixed-order sum of each token's weighted fp32 rows into bf16.
int32_t combine_rows_f32(const moe_problem* p, const float* y, const int32_t* pos,
                         __nv_bfloat16* out, int32_t* status, cudaStream_t s);

// ops_api.cu: workspace bytes of its entry points (0: unsupported problem).
size_t operator_workspace(const moe_problem* p, int32_t call);

}  // namespace moe
