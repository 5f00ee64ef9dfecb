// The tables of one serving step (nvfp4_attn_plan) and the write of its new
// K and V rows into the paged cache (nvfp4_kv_append).
//
// Plan.  Everything follows from two prefix sums over the requests, of the
// new tokens and of the pages they open.  Every block computes both sums for
// all requests in shared memory (a few KB of lengths out of L2) instead of
// waiting for a first kernel to do it, then fills its own slice of the
// tables; so the whole plan is one launch without a grid-wide wait.  The
// tables are small (a few hundred KB at most): the launch and the dependent
// reads set the time, not bandwidth (64 decoding requests 5.6 us; 4096 requests
// of 1 to 13 new tokens 15.9 us).  Only a cursor that is advanced in place is
// stored by a second launch (cursor_kernel).
#include "attn.h"
#include "common.cuh"
#include "internal.h"

namespace nvfp4 {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kMaxPosition = 1 << 30;
constexpr int64_t kMaxUnits = (int64_t)1 << 30;   // of a schedule (a call of seconds): the rest is not worked on

struct PlanParams {
    nvfp4_step_t s;
    int* status;
    int page_shift;
    int ctas;                // the attention kernel's grid
    int schedulers;          // blocks that build the schedule
};

__device__ __forceinline__ void report(int* status, int code)
{
    if (status) atomicCAS(status, 0, code);
}

// Pages that q new tokens behind c cached ones open (pages of 2^shift tokens).
__device__ __forceinline__ int64_t pages_opened(int64_t c, int64_t q, int shift)
{
    const int64_t round = ((int64_t)1 << shift) - 1;
    return ((c + q + round) >> shift) - ((c + round) >> shift);
}

__device__ __forceinline__ int64_t warp_incl_sum(int64_t v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

// Block-wide exclusive prefix sums over the threads of two values at once;
// the totals in *ta, *tb.  Every thread of the block calls it.
__device__ __forceinline__ void block_prefix(int64_t& a, int64_t& b, int64_t (*warp_sums)[2], int64_t* ta, int64_t* tb)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t ia = warp_incl_sum(a, lane), ib = warp_incl_sum(b, lane);
    __syncthreads();                // the sums of an earlier call have been read
    if (lane == 31) {
        warp_sums[warp][0] = ia;
        warp_sums[warp][1] = ib;
    }
    __syncthreads();
    int64_t all_a = 0, all_b = 0;
    a = ia - a;
    b = ib - b;
#pragma unroll
    for (int w = 0; w < kPlanWarps; w++) {
        if (w < warp) {
            a += warp_sums[w][0];
            b += warp_sums[w][1];
        }
        all_a += warp_sums[w][0];
        all_b += warp_sums[w][1];
    }
    *ta = all_a;
    *tb = all_b;
}

// The last of n ascending entries that is at or below v (entry 0 is).
__device__ __forceinline__ int last_at_or_below(const int32_t* x, int n, int64_t v)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (x[mid] <= v) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// The attention's schedule, by the last blocks of the grid, each of which works
// out all of it and writes its share (one SM would take 6 ns for each QTile's
// store): the QTiles of all requests in
// order, the prefix sum of their units, and the QTile of each CTA's first
// unit.  A thread takes consecutive QTiles, walking from request to request:
// once for their units, once (the sums known) to write them.  cu: new tokens
// before each request, ctx: cached tokens, tile0: room for R + 1 int32 (all
// shared memory).
__device__ void build_schedule(const PlanParams& p, const int32_t* cu, const int32_t* ctx, int32_t* tile0,
                               int64_t (*warp_sums)[2], int* longest, int block, int blocks)
{
    const nvfp4_step_t& s = p.s;
    const int R = (int)s.requests, t = threadIdx.x;
    const int per_tile = 2 * row_tile_tokens((int)(s.heads / s.kv_heads));
    const int Hkv = (int)s.kv_heads;
    ScheduleHead* head = static_cast<ScheduleHead*>(s.schedule);
    QTile* tiles = const_cast<QTile*>(schedule_tiles(head));
    // QTiles before each request
    const int per = ((R + kPlanThreads - 1) / kPlanThreads) | 1;     // (odd: no bank conflicts)
    int64_t before = 0, unused = 0, total = 0, unused_total;
    for (int r = t * per; r < min(R, (t + 1) * per); r++) before += (cu[r + 1] - cu[r] + per_tile - 1) / per_tile;
    block_prefix(before, unused, warp_sums, &total, &unused_total);
    for (int r = t * per; r < min(R, (t + 1) * per); r++) {
        tile0[r] = (int32_t)before;
        before += (cu[r + 1] - cu[r] + per_tile - 1) / per_tile;
    }
    if (t == 0) {
        tile0[R] = (int32_t)total;
        *longest = 1;
    }
    __syncthreads();
    const int n = (int)total, each = ((n + kPlanThreads - 1) / kPlanThreads) | 1;
    const int i0 = min(n, t * each), i1 = min(n, i0 + each);
    // (32-bit from here: positions up to 2^30)
    const int cap = (int)min(s.page_size ? s.table_cols * s.page_size : (int64_t)kMaxPosition, (int64_t)kMaxPosition);
    const int window = (int)s.window;
    const int r0 = i0 < i1 ? last_at_or_below(tile0, R, i0) : 0;
    auto tile_of = [&](int i, int& r) {
        while (tile0[r + 1] <= i) r++;           // (requests without new tokens have no QTile)
        const int off = (i - tile0[r]) * per_tile, q_len = cu[r + 1] - cu[r];
        QTile q = {};
        q.tok0 = cu[r] + off;
        q.n_tok = min(per_tile, q_len - off);
        q.req = r;
        q.pos0 = min(min(ctx[r], kMaxPosition) + off, kMaxPosition);
        const int begin = window ? max(q.pos0 + 1 - window, 0) : 0;
        q.kv_end = min(q.pos0 + q.n_tok, cap);
        q.tile0 = begin / kAttnKeys;
        // at least one tile, so that rows that see no key are written too
        q.tiles = max((q.kv_end + kAttnKeys - 1) / kAttnKeys - q.tile0, 1);
        return q;
    };
    int64_t unit = 0, units = 0;
    int most = 1;
    for (int i = i0, r = r0; i < i1; i++) {
        const int item = kItemUnits + tile_of(i, r).tiles;
        unit += (int64_t)item * Hkv;
        most = max(most, item);
    }
    atomicMax(longest, __reduce_max_sync(0xffffffffu, most));
    block_prefix(unit, unused, warp_sums, &units, &unused_total);   // (its barriers order *longest too)
    if (units > kMaxUnits) {
        // ends with a whole item (one cut off would never collect its tickets)
        int64_t at = unit;
        for (int i = i0, r = r0; i < i1 && at <= kMaxUnits; i++) {
            const int64_t item = kItemUnits + tile_of(i, r).tiles, next = at + item * Hkv;
            if (next > kMaxUnits) *longest = (int)(at + (kMaxUnits - at) / item * item);
            at = next;
        }
        __syncthreads();
        units = *longest;
        if (t == 0) report(p.status, kStatusPlan);
    }
    const int share = (int)((units + p.ctas - 1) / p.ctas);
    const int per_cta = max(share, min(kItemUnits + kMinPart, *longest));
    if (t == 0 && block == 0) {
        head->units = (int32_t)units;
        head->per_cta = per_cta;
        head->qtiles = n;
    }
    if (t * blocks / kPlanThreads != block) return;
    int c = (int)((min(unit, units) + per_cta - 1) / per_cta);       // the next CTA to start
    for (int i = i0, r = r0; i < i1; i++) {
        QTile q = tile_of(i, r);
        q.unit0 = (int)min(unit, units);
        unit += (int64_t)(kItemUnits + q.tiles) * Hkv;
        tiles[i] = q;
        for (const int next = (int)min(unit, units); c * per_cta < next; c++) {
            head->first[c] = i;
            head->start[c] = q;
        }
    }
}

// shared memory, int32: cu [R+1] (new tokens before each request, at most
// `tokens`), first [R+1] (pages taken before each request), ctx [R] (cached
// tokens)
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p)
{
    extern __shared__ int32_t sh[];
    __shared__ int64_t s_sums[kPlanWarps][2];
    __shared__ int s_longest;
    griddep_launch_dependents();
    // (The lengths may come from the previous kernel, and what it writes while
    // this one is already there is no constant: plain loads, not __ldg, here
    // and in the other kernels of a step.)
    griddep_wait();
    const nvfp4_step_t& s = p.s;
    const int R = (int)s.requests;
    const bool paged = s.page_size != 0;
    int32_t* cu = sh;
    int32_t* first = sh + R + 1;
    int32_t* ctx = first + R + 1;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int64_t P = paged ? s.page_size : 1, round = P - 1;
    const int sft = p.page_shift;
    const int64_t kIntMax = 0x7fffffff;
    const int64_t cursor = paged && s.cursor ? *s.cursor : 0;

    // the lengths, negative ones as zero
    bool bad = false;
    for (int r = t; r < R; r += kPlanThreads) {
        const int q = s.q_len[r], c = s.ctx_len ? s.ctx_len[r] : 0;
        bad |= q < 0 || c < 0;
        cu[r] = max(q, 0);
        ctx[r] = max(c, 0);
    }
    __syncthreads();
    // prefix sums over the requests: thread t takes the requests per*t ..
    const int per = ((R + kPlanThreads - 1) / kPlanThreads) | 1;     // (odd: no bank conflicts)
    int64_t bq = 0, bn = 0, total_q = 0, total_n = 0;
    for (int r = t * per; r < min(R, (t + 1) * per); r++) {
        bq += cu[r];
        if (paged) bn += pages_opened(ctx[r], cu[r], sft);
    }
    block_prefix(bq, bn, s_sums, &total_q, &total_n);
    const int64_t cap = s.tokens;
    for (int r = t * per; r < min(R, (t + 1) * per); r++) {
        const int q = cu[r];
        cu[r] = (int32_t)min(bq, cap);
        first[r] = (int32_t)min(bn, kIntMax);
        bq += q;
        if (paged) bn += pages_opened(ctx[r], q, sft);
    }
    if (t == 0) {
        cu[R] = (int32_t)min(total_q, cap);
        first[R] = (int32_t)min(total_n, kIntMax);
        if (total_q > cap) bad = true;
    }
    if (bad && blockIdx.x == 0) report(p.status, kStatusPlan);
    __syncthreads();
    const int blocks = gridDim.x - p.schedulers;
    if ((int)blockIdx.x >= blocks) {
        build_schedule(p, cu, ctx, first, s_sums, &s_longest, blockIdx.x - blocks, p.schedulers);
        return;
    }
    const int32_t T = cu[R];

    // per-request tables
    for (int r = blockIdx.x * kPlanThreads + t; r < R; r += blocks * kPlanThreads) {
        s.cu_q[r] = cu[r];
        s.kv_len[r] = (int32_t)min((int64_t)ctx[r] + (cu[r + 1] - cu[r]), kIntMax);
    }
    if (blockIdx.x == 0 && t == 0) s.cu_q[R] = T;
    if (paged && s.free_pages) {
        // the pages opened, a warp per request
        for (int r = blockIdx.x * kPlanWarps + warp; r < R; r += blocks * kPlanWarps) {
            const int64_t have = (ctx[r] + round) >> sft;
            // (first: exact below its limit)
            const int64_t taken = first[r + 1] < kIntMax ? first[r + 1] - first[r]
                                                         : pages_opened(ctx[r], max(s.q_len[r], 0), sft);
            // (no further than the table's last column, whatever the lengths ask for)
            const int64_t room = max(s.table_cols - have, (int64_t)0), n = min(taken, room);
            bool missing = taken > room;
            for (int64_t x = lane; x < n; x += 32) {
                const int64_t at = cursor + first[r] + x;
                const bool ok = at >= 0 && at < s.free_count;
                s.block_table[r * s.table_ld + have + x] = ok ? s.free_pages[at] : -1;
                missing |= !ok;
            }
            if (missing) report(p.status, kStatusPlan);
        }
        if (blockIdx.x == 0 && t == 0 && s.cursor_out && s.cursor_out != s.cursor)
            *s.cursor_out = (int32_t)min(cursor + total_n, kIntMax);
    }

    // per-token tables
    for (int64_t i = (int64_t)blockIdx.x * kPlanThreads + t; i < cap; i += (int64_t)blocks * kPlanThreads) {
        int pos = 0, slot = -1;
        if (i < T) {
            const int r = last_at_or_below(cu, R, i);     // the request that row i is of
            const int64_t at = (int64_t)ctx[r] + (i - cu[r]);
            pos = (int)min(at, kIntMax);
            if (s.heads && at >= kMaxPosition) report(p.status, kStatusPlan);   // beyond the schedule's positions
            if (paged) {
                const int64_t j = at >> sft, have = (ctx[r] + round) >> sft;
                int64_t page = -1;
                if (j < s.table_cols) {
                    if (!s.free_pages || j < have) {
                        page = s.block_table[r * s.table_ld + j];
                    } else {
                        const int64_t f = cursor + first[r] + (j - have);
                        if (f >= 0 && f < s.free_count) page = s.free_pages[f];
                    }
                }
                const int64_t sl = page * P + (at & round);
                if (page >= 0 && sl <= kIntMax)
                    slot = (int)sl;
                else
                    report(p.status, kStatusPlan);
            }
        }
        if (s.pos) s.pos[i] = pos;
        if (paged) s.slot[i] = slot;
    }
}

// *cursor_out where it is cursor itself.  The plan's blocks read the cursor
// when they start, and nothing orders a block's start before another's end: a
// store from within the plan could reach a block that has yet to read, and give
// its requests pages that are others'.  So the word changes once the plan has
// completed, by a block that counts the pages again (64 requests 5.6 us with
// the cursor apart, 7.0 with it in place; 4096 requests 15.7 and 17.6).
constexpr int kCursorThreads = 512;

__global__ void __launch_bounds__(kCursorThreads) cursor_kernel(const PlanParams p)
{
    __shared__ int64_t s_sums[kCursorThreads / 32];
    griddep_launch_dependents();
    griddep_wait();
    const nvfp4_step_t& s = p.s;
    int64_t n = 0;
    for (int r = threadIdx.x; r < (int)s.requests; r += kCursorThreads)
        n += pages_opened(max(s.ctx_len ? s.ctx_len[r] : 0, 0), max(s.q_len[r], 0), p.page_shift);
    n = warp_incl_sum(n, threadIdx.x & 31);
    if ((threadIdx.x & 31) == 31) s_sums[threadIdx.x >> 5] = n;
    __syncthreads();
    if (threadIdx.x == 0) {
        n = *s.cursor;
        for (int w = 0; w < kCursorThreads / 32; w++) n += s_sums[w];
        *s.cursor_out = (int32_t)min(n, (int64_t)0x7fffffff);
    }
}

// ---------------------------------------------------------------- append
// One 16-byte vector of a head's row per thread: a block copies whole packed
// rows (both K and V, every kv head), kAppendRows of them at a time, all
// their loads in flight before the first store.  Bound by HBM: 16272 tokens of
// 8 heads of 128 columns (133 MB read and written) 22.9 us, 5.8 TB/s; a decode
// step's 17 tokens 2.0 us.
constexpr int kAppendThreads = 256;
constexpr int kAppendRows = 4;

struct AppendParams {
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    int64_t ldk, hk, ldv, hv;
    const int32_t* slot;
    int64_t tokens;
    nvfp4_kv_cache_t c;
    int page_shift;
    int* status;
};

__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p)
{
    griddep_launch_dependents();
    griddep_wait();
    const int dv = (int)(p.c.head_dim / 8);             // vectors of a head's row
    const int per = (int)p.c.kv_heads * dv;             // vectors of a packed row of K (or V)
    const int64_t slots = p.c.pages << p.page_shift;
    const int64_t mask = p.c.page_size - 1;
    const int64_t hstride = p.c.page_size * p.c.head_dim;
    for (int64_t t0 = (int64_t)blockIdx.x * kAppendRows; t0 < p.tokens; t0 += (int64_t)gridDim.x * kAppendRows) {
        int64_t dst[kAppendRows];
        bool ok[kAppendRows];
#pragma unroll
        for (int u = 0; u < kAppendRows; u++) {
            const int64_t sl = t0 + u < p.tokens ? p.slot[t0 + u] : -1;
            ok[u] = sl >= 0 && sl < slots;
            if (!ok[u] && sl != -1 && threadIdx.x == 0) report(p.status, kStatusSlot);
            dst[u] = (sl >> p.page_shift) * p.c.page_stride + (sl & mask) * p.c.head_dim;
        }
        for (int x = threadIdx.x; x < 2 * per; x += kAppendThreads) {
            const bool is_v = x >= per;
            const int y = is_v ? x - per : x;
            const int h = y / dv, d = 8 * (y - h * dv);
            const __nv_bfloat16* src = is_v ? p.v + h * p.hv + d : p.k + h * p.hk + d;
            const int64_t ld = is_v ? p.ldv : p.ldk;
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(is_v ? p.c.v : p.c.k) + h * hstride + d;
            uint4 val[kAppendRows];
#pragma unroll
            for (int u = 0; u < kAppendRows; u++)
                if (ok[u]) val[u] = *reinterpret_cast<const uint4*>(src + (t0 + u) * ld);
#pragma unroll
            for (int u = 0; u < kAppendRows; u++)
                if (ok[u]) *reinterpret_cast<uint4*>(out + dst[u]) = val[u];
        }
    }
}

int log2_of(int64_t v)
{
    int s = 0;
    while (((int64_t)1 << s) < v) s++;
    return s;
}

}  // namespace

cudaError_t launch_attn_plan(const nvfp4_step_t& step, int* status, int num_sms, cudaStream_t stream)
{
    const size_t smem = (size_t)(step.requests + 1) * 12;
    static int attr_set_for_device[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && !attr_set_for_device[dev]) {
        e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)((kStepMaxRequests + 1) * 12));
        if (e != cudaSuccess) return e;
        attr_set_for_device[dev] = 1;
    }
    PlanParams p;
    p.s = step;
    p.status = status;
    p.page_shift = step.page_size ? log2_of(step.page_size) : 0;
    const int64_t by_tokens = (step.tokens + kPlanThreads - 1) / kPlanThreads;
    const int64_t by_requests = (step.requests + kPlanWarps - 1) / kPlanWarps;
    int64_t grid = by_tokens > by_requests ? by_tokens : by_requests;
    if (grid > num_sms) grid = num_sms;
    p.schedulers = 0;
    if (step.heads) {
        const int64_t n = max_qtiles(step.requests, step.tokens, step.heads / step.kv_heads) / kPlanThreads;
        p.schedulers = (int)(n < 1 ? 1 : n > 16 ? 16 : n);
        grid += p.schedulers;
    }
    p.ctas = num_sms < kAttnMaxCtas ? num_sms : kAttnMaxCtas;
    e = launch_programmatic(plan_kernel, dim3((unsigned)grid), dim3(kPlanThreads), smem, stream, p);
    if (e != cudaSuccess || !step.page_size || !step.free_pages || !step.cursor || step.cursor_out != step.cursor)
        return e;
    return launch_programmatic(cursor_kernel, dim3(1), dim3(kCursorThreads), 0, stream, p);
}

cudaError_t launch_kv_append(const __nv_bfloat16* k, int64_t ldk, int64_t hk, const __nv_bfloat16* v, int64_t ldv,
                             int64_t hv, const int32_t* slot, int64_t tokens, const nvfp4_kv_cache_t& cache,
                             int* status, int num_sms, cudaStream_t stream)
{
    AppendParams p = {k, v, ldk, hk, ldv, hv, slot, tokens, cache, log2_of(cache.page_size), status};
    int64_t grid = (tokens + kAppendRows - 1) / kAppendRows;
    if (grid > (int64_t)num_sms * 8) grid = (int64_t)num_sms * 8;
    return launch_programmatic(append_kernel, dim3((unsigned)grid), dim3(kAppendThreads), 0, stream, p);
}

}  // namespace nvfp4
