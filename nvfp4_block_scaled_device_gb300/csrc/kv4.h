// Internal launcher interface of the operators around a layer's cache: norms
// and rotation of heads, the 4-bit cache and its attention, pages.
#pragma once

#include "attn.h"

namespace nvfp4 {

// Device status of the page operators (NVFP4_ERR_INVALID_ARG * 100 + site).
constexpr int kStatusPages = NVFP4_ERR_INVALID_ARG * 100 + 34;

// Rows of a request, on average, from which a step's keys are expanded once (us that way
// and straight from the codes, 40 rows: 32 requests of 200 to 4000 keys 91 and 113, 8 of
// 2000 43 and 42, 1 of 8000 47 and 41; 60 rows: 64 of 100 to 2000 93 and 160; 20 rows: 8 of
// 2000 45 and 24, 1 of 8000 55 and 24).
constexpr int64_t kExpandRows = 40;

constexpr int64_t kMaxPages = 1 << 20;      // of the page operators (a bit each in shared memory)
constexpr int kMaxPlanes = 64;              // of one copying launch
constexpr int64_t kPageCopyChunk = 16384;   // bytes of a page that a block copies

struct PageCopyPlanes {
    nvfp4_plane_t p[kMaxPlanes];
};

// The heads of nvfp4_qk_norm_rope, or (heads 0, no norms, no rotation) the rows
// of nvfp4_kv4_append.
cudaError_t launch_heads(const nvfp4_heads_t& heads, int* status, int num_sms, cudaStream_t stream);

// The rows of a 4-bit cache that a step sees, into a bf16 cache's pages; scaled:
// times the cache's global scales (else code times E4M3 scale, exact: K in bf16, V as
// halves in the bf16 cache's place, what nvfp4_attn_paged4's own variant reads);
// unless_few: only where the step's schedule does not have few_passes.
cudaError_t launch_kv4_expand(const nvfp4_kv4_cache_t& cache, const nvfp4_step_t& step, const nvfp4_kv_cache_t& out,
                              bool scaled, bool unless_few, int num_sms, cudaStream_t stream);

// Attention over a 4-bit cache (args.k_g, v_g and the paged fields set).
cudaError_t launch_attn4(const AttnArgs& args, const nvfp4_kv4_cache_t& cache, const __nv_bfloat16* q, int64_t ldq,
                         int64_t hq, int64_t requests, int num_sms, cudaStream_t stream);

cudaError_t launch_pages_fork(const nvfp4_pages_t& t, const int32_t* src, const int32_t* dst, int64_t n,
                              const int32_t* free_pages, int64_t free_count, const int32_t* cursor,
                              int32_t* cursor_out, int32_t* copy_src, int32_t* copy_dst, int* status, int num_sms,
                              cudaStream_t stream);

cudaError_t launch_pages_free(const nvfp4_pages_t& t, int32_t* free_pages, int32_t* free_count, int32_t* table_out,
                              int64_t table_out_ld, int32_t* move_src, int32_t* move_dst, int* status,
                              cudaStream_t stream);

cudaError_t launch_pages_copy(const PageCopyPlanes& planes, int n_planes, int64_t max_bytes, int64_t pages,
                              const int32_t* src, const int32_t* dst, int64_t n, int* status, int num_sms,
                              cudaStream_t stream);

}  // namespace nvfp4
