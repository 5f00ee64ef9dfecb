// Internal launcher interface of the attention operators (step tables, cache
// append, attention).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "nvfp4.h"

namespace nvfp4 {

constexpr int64_t kStepMaxRequests = 8192;

// Device status values of the attention operators (NVFP4_ERR_INVALID_ARG *
// 100 + site).
constexpr int kStatusPlan = NVFP4_ERR_INVALID_ARG * 100 + 31;
constexpr int kStatusSlot = NVFP4_ERR_INVALID_ARG * 100 + 32;

cudaError_t launch_attn_plan(const nvfp4_step_t& step, int* status, int num_sms, cudaStream_t stream);

cudaError_t launch_kv_append(const __nv_bfloat16* k, int64_t ldk, int64_t hk, const __nv_bfloat16* v, int64_t ldv,
                             int64_t hv, const int32_t* slot, int64_t tokens, const nvfp4_kv_cache_t& cache,
                             int* status, int num_sms, cudaStream_t stream);

// Keys and values of an attention call: packed rows (block_table NULL), or
// the paged cache.
struct AttnKV {
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    int64_t ldk, hk, ldv, hv;          // packed: row and head pitches (elements)
    const int32_t* block_table;        // paged
    int64_t table_cols, table_ld, page_size, pages, page_stride;
};

cudaError_t launch_attn(const nvfp4_step_t& step, const nvfp4_attn_io_t& io, const AttnKV& kv, int num_sms,
                        cudaStream_t stream);

}  // namespace nvfp4
