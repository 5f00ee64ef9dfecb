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

// ---- attention schedule (built by the plan kernel, walked by the attention)
//
// A row tile is 128 rows of the attention's MMAs: the `group` query heads of
// one kv head for kAttnRows / group consecutive tokens (row = token * group +
// head).  A work item is a QTile for one kv head: up to two row tiles of one
// request, over the 128-key tiles that any of its rows sees.  The items, all
// kv heads of a QTile one after the other, form one axis of `units`: for each
// item kItemUnits for its start and end, then one per key tile.  CTA c takes
// the key tiles among units [c * per_cta, (c + 1) * per_cta), so that every
// CTA has about the same work whatever the lengths.  A boundary that would
// leave fewer than kMinPart tiles of an item on one side moves to that edge of
// the item (snap_unit).
constexpr int kAttnRows = 128;
constexpr int kAttnKeys = 128;
constexpr int kAttnMaxCtas = 256;
constexpr int kItemUnits = 2;
constexpr int kItemUnits4 = 2, kChunksOfTile = 4;
constexpr int kPassRows = 32;

struct QTile {
    int32_t tok0, n_tok;     // packed rows (tokens) tok0 .. tok0 + n_tok - 1
    int32_t req, pos0;       // the request, the position of token tok0
    int32_t kv_end;          // no row sees keys from kv_end on
    int32_t tile0, tiles;    // key tiles tile0 .. tile0 + tiles - 1
    int32_t unit0;           // units before this QTile; it has (kItemUnits + tiles) * kv_heads
};
static_assert(sizeof(QTile) == 32, "QTile");

struct ScheduleHead {
    int32_t units, per_cta, qtiles;
    // The second axis, for the attention that gives each warp its own share
    // (attn4.cu): an item is kItemUnits4 units, then one per 32 keys of its tiles,
    // kChunksOfTile for each; QTile i begins at 4 unit0 - (4 kItemUnits -
    // kItemUnits4) kv_heads i.  CTA c takes units c * per_cta4 .. as above.
    int32_t units4, per_cta4;      // 0: too long for it
    int32_t most_tokens;           // of a QTile
    // few passes of kPassRows rows over the keys suffice, on average and for each CTA
    int32_t few_passes;
    int32_t pad[9];
    int32_t first[kAttnMaxCtas];   // QTile of the first unit of CTA c ...
    QTile start[kAttnMaxCtas];     // ... and a copy of it, next to what a CTA reads first
    int32_t first4[kAttnMaxCtas];  // the same of the second axis
    QTile start4[kAttnMaxCtas];
};
static_assert(sizeof(ScheduleHead) % 16 == 0, "QTiles follow the head, 16-byte aligned");

inline __host__ __device__ const QTile* schedule_tiles(const ScheduleHead* h)
{
    return reinterpret_cast<const QTile*>(h + 1);
}

// Units of the second axis before QTile i.
inline __host__ __device__ int units4_before(int unit0, int kv_heads, int i)
{
    return kChunksOfTile * unit0 - (kChunksOfTile * kItemUnits - kItemUnits4) * kv_heads * i;
}

// Boundary r (units from the item's start) of an item of `item` units.  A part
// costs its CTA 3 to 5 us beside its tiles (1.1 to 1.7 us each), so short items
// are not shared.  At least 3 tiles a part: prompts of 1 to 499 tokens 18.6 us,
// one of 8192 523; 5: 21.8, 534; 2: 21.7, 529.
constexpr int kMinPart = 3;
inline __host__ __device__ int snap_unit(int r, int item)
{
    const bool head = r < kItemUnits + kMinPart, tail = item - r < kMinPart;
    return r >= item ? item : head && tail ? (2 * r < item ? 0 : item) : head ? 0 : tail ? item : r;
}

// The same on the second axis, in chunks of 32 keys.
constexpr int kMinPart4 = 8;
inline __host__ __device__ int snap_unit4(int r, int item)
{
    const bool head = r < kItemUnits4 + kMinPart4, tail = item - r < kMinPart4;
    return r >= item ? item : head && tail ? (2 * r < item ? 0 : item) : head ? 0 : tail ? item : r;
}

// Tokens of a row tile.
inline __host__ __device__ int row_tile_tokens(int group) { return kAttnRows / group; }

// QTiles of any step of that many requests and tokens, at most.
inline int64_t max_qtiles(int64_t requests, int64_t tokens, int64_t group)
{
    const int64_t per = 2 * row_tile_tokens((int)group);
    const int64_t n = tokens / per + requests;
    return n < tokens ? n : tokens;
}

cudaError_t launch_attn_plan(const nvfp4_step_t& step, int* status, int num_sms, cudaStream_t stream);

cudaError_t launch_kv_append(const __nv_bfloat16* k, int64_t ldk, int64_t hk, const __nv_bfloat16* v, int64_t ldv,
                             int64_t hv, const int32_t* slot, int64_t tokens, const nvfp4_kv_cache_t& cache,
                             int* status, int num_sms, cudaStream_t stream);

// Workspace of the attention kernel: tickets (zero between calls), then two
// partial slots per CTA: the unnormalised outputs [head_dim / 4][256 rows][4]
// of an item that other CTAs share, its rows' maxima and sums.
constexpr size_t kAttnTicketBytes = (size_t)kAttnMaxCtas * 8 * 4;
constexpr int64_t kAttnSlotRows = 2 * kAttnRows;
constexpr int64_t kAttnSlotFloats = kAttnSlotRows * (128 + 2);
inline size_t attn_workspace_bytes(int ctas) { return kAttnTicketBytes + (size_t)ctas * 2 * kAttnSlotFloats * 4; }

// Arguments of the attention kernel (tensor maps apart).
struct AttnArgs {
    const ScheduleHead* sched;
    __nv_bfloat16* out;
    int64_t ldo, ho;
    float* lse;
    const int32_t* cu_end;   // rows *cu_end .. tokens - 1 of out are zeroed, of lse -inf; NULL: not written
    int64_t tokens;
    int heads, kv_heads, group, head_dim;
    int row_tokens;      // tokens of a row tile
    int window;
    float scale;
    // attention over a 4-bit cache, or over rows taken out of one (k_g NULL: neither)
    const float* k_g;    // device scalars that multiply every score and every output
    const float* v_g;
    int skip_few;        // over bf16 rows it returns at once where the schedule has few_passes, over 4 bits where not
    // paged cache (block_table NULL: packed keys)
    const int32_t* block_table;
    int64_t table_ld;
    int page_size;
    int fold;            // pages of 16 rows of 128 columns: copied whole
    int* tickets;
    float* partials;
    int* status;
};

// map_q: [head_dim, heads, tokens], boxes {64, group, tokens of a row tile};
// map_k, map_v: packed [head_dim, kv_heads, tokens], boxes {64, 1, 128}, or
// the cache [head_dim, page_size, kv_heads, pages], boxes {64, page_size, 1, 1}, or
// (args.fold) [64, 16, 2 halves, kv_heads, pages], boxes {64, 16, 2, 1, 1}; all with
// 128-byte swizzle.
cudaError_t launch_attn(const CUtensorMap& map_q, const CUtensorMap& map_k, const CUtensorMap& map_v,
                        const AttnArgs& args, int num_sms, cudaStream_t stream);

}  // namespace nvfp4
