// The tables of one serving step (nvfp4_attn_plan) and the write of its new
// K and V rows into the paged cache (nvfp4_kv_append).
//
// Plan.  Everything follows from two prefix sums over the requests, of the
// new tokens and of the pages they open.  Every block computes both sums for
// all requests in shared memory (a few KB of lengths out of L2) instead of
// waiting for a first kernel to do it, then fills its own slice of the
// tables; so the whole plan is one launch without a grid-wide wait.  The
// tables are small (a few hundred KB at most): the launch and the dependent
// reads set the time, not bandwidth.
#include "attn.h"
#include "common.cuh"
#include "internal.h"

namespace nvfp4 {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int64_t kMaxUnits = (int64_t)1 << 30;   // of a schedule (a call of seconds): the rest is not worked on

struct PlanParams {
    nvfp4_step_t s;
    int* status;
    int page_shift;
    int ctas;                // the attention kernel's grid
};

__device__ __forceinline__ void report(int* status, int code)
{
    if (status) atomicCAS(status, 0, code);
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

// A request's lengths, with negative ones taken as zero.
struct Lens {
    int64_t ctx, q;
    bool bad;
};

__device__ __forceinline__ Lens lens_of(const nvfp4_step_t& s, int r)
{
    const int q = __ldg(s.q_len + r), c = s.ctx_len ? __ldg(s.ctx_len + r) : 0;
    return {c < 0 ? 0 : c, q < 0 ? 0 : q, q < 0 || c < 0};
}

// Block-wide inclusive prefix sum over the threads (kPlanThreads of them);
// total: the sum of all.  Every thread of the block calls it.
__device__ __forceinline__ int64_t block_incl_sum(int64_t v, int64_t* warp_sums, int64_t* total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = warp_incl_sum(v, lane);
    __syncthreads();                // the sums of an earlier call have been read
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlanWarps; w++) {
        if (w < warp) before += warp_sums[w];
        all += warp_sums[w];
    }
    *total = all;
    return v + before;
}

// The attention's schedule, by one block: the QTiles of all requests in
// order, the prefix sum of their units, and the QTile of each CTA's first
// unit.  cu: new tokens before each request (shared memory); tile0: room for
// R + 1 int32 in shared memory.
__device__ void build_schedule(const PlanParams& p, const int32_t* cu, int32_t* tile0, int64_t* warp_sums)
{
    const nvfp4_step_t& s = p.s;
    const int R = (int)s.requests, t = threadIdx.x;
    const int per_tile = 2 * row_tile_tokens((int)(s.heads / s.kv_heads));
    ScheduleHead* head = static_cast<ScheduleHead*>(s.schedule);
    QTile* tiles = const_cast<QTile*>(schedule_tiles(head));
    // QTiles before each request
    const int per = (R + kPlanThreads - 1) / kPlanThreads;
    int64_t mine = 0, total = 0;
    for (int r = t * per; r < min(R, (t + 1) * per); r++) mine += (cu[r + 1] - cu[r] + per_tile - 1) / per_tile;
    int64_t before = block_incl_sum(mine, warp_sums, &total) - mine;
    for (int r = t * per; r < min(R, (t + 1) * per); r++) {
        tile0[r] = (int32_t)before;
        before += (cu[r + 1] - cu[r] + per_tile - 1) / per_tile;
    }
    if (t == 0) {
        tile0[R] = (int32_t)total;
        warp_sums[kPlanWarps] = 1;                  // units of the longest item
    }
    __syncthreads();
    const int n = (int)total;
    const int64_t cap = s.page_size ? s.table_cols * s.page_size : 0x7fffffff;
    int64_t units = 0;
    for (int base = 0; base < n; base += kPlanThreads) {
        const int i = base + t;
        QTile q = {};
        int64_t u = 0;
        if (i < n) {
            int lo = 0, hi = R - 1;      // the last request whose first QTile is at or before i
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (tile0[mid] <= i) lo = mid; else hi = mid - 1;
            }
            const int off = (i - tile0[lo]) * per_tile, q_len = cu[lo + 1] - cu[lo];
            const int64_t ctx = lens_of(s, lo).ctx;
            q.tok0 = cu[lo] + off;
            q.n_tok = min(per_tile, q_len - off);
            q.req = lo;
            q.kv_row = cu[lo];
            const int64_t pos0 = min(ctx + off, (int64_t)0x7fffffff - q.n_tok);
            q.pos0 = (int32_t)pos0;
            const int64_t end = min(min(pos0 + q.n_tok, ctx + q_len), cap);
            const int64_t begin = s.window ? max(pos0 + 1 - s.window, (int64_t)0) : 0;
            q.kv_end = (int32_t)end;
            q.tile0 = (int32_t)(begin / kAttnKeys);
            // at least one tile, so that rows that see no key are written too
            q.tiles = (int32_t)max((end + kAttnKeys - 1) / kAttnKeys - q.tile0, (int64_t)1);
            u = (int64_t)(kItemUnits + q.tiles) * s.kv_heads;
            atomicMax(reinterpret_cast<unsigned long long*>(warp_sums + kPlanWarps), (unsigned long long)(kItemUnits + q.tiles));
        }
        int64_t sum = 0;
        const int64_t incl = block_incl_sum(u, warp_sums, &sum);
        if (i < n) {
            q.unit0 = (int32_t)min(units + incl - u, kMaxUnits);
            tiles[i] = q;
        }
        units += sum;
    }
    if (units > kMaxUnits) {
        units = kMaxUnits;
        if (t == 0) report(p.status, kStatusPlan);
    }
    __syncthreads();
    const int64_t share = (units + p.ctas - 1) / p.ctas;
    const int64_t least = min((int64_t)(kItemUnits + kMinPart), warp_sums[kPlanWarps]);
    const int64_t per_cta = share > least ? share : least;
    if (t == 0) {
        head->units = (int32_t)units;
        head->per_cta = (int32_t)per_cta;
        head->qtiles = n;
    }
    for (int i = t; i < n; i += kPlanThreads) {     // each thread reads the entries it wrote
        const QTile q = tiles[i];
        const int64_t u1 = min(q.unit0 + (int64_t)(kItemUnits + q.tiles) * s.kv_heads, units);
        for (int64_t c = (q.unit0 + per_cta - 1) / per_cta; c * per_cta < u1; c++) {
            head->first[c] = i;
            head->start[c] = q;
        }
    }
}

// shared memory: cu [R+1] int32 (new tokens before each request, at most
// `tokens`), first [R+1] int32 (pages taken before each request)
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p)
{
    extern __shared__ int32_t sh[];
    __shared__ int64_t s_sums[kPlanWarps + 1];
    griddep_launch_dependents();
    griddep_wait();                 // the lengths may come from the previous kernel
    const nvfp4_step_t& s = p.s;
    const int R = (int)s.requests;
    const bool paged = s.page_size != 0;
    int32_t* cu = sh;
    int32_t* first = sh + R + 1;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int64_t P = paged ? s.page_size : 1, round = P - 1;
    const int sft = p.page_shift;

    // prefix sums over the requests: thread t takes the requests
    // per*t .. per*t + per - 1
    const int per = (R + kPlanThreads - 1) / kPlanThreads;
    int64_t sq = 0, sn = 0;
    bool bad = false;
    for (int j = 0; j < per; j++) {
        const int r = t * per + j;
        if (r >= R) break;
        const Lens l = lens_of(s, r);
        bad |= l.bad;
        sq += l.q;
        if (paged) sn += ((l.ctx + l.q + round) >> sft) - ((l.ctx + round) >> sft);
    }
    int64_t total_q = 0, total_n = 0;
    int64_t bq = block_incl_sum(sq, s_sums, &total_q) - sq;
    int64_t bn = paged ? block_incl_sum(sn, s_sums, &total_n) - sn : 0;
    const int64_t cap = s.tokens;
    const int64_t cursor = paged && s.cursor ? __ldg(s.cursor) : 0;
    const int64_t kIntMax = 0x7fffffff;
    for (int j = 0; j < per; j++) {
        const int r = t * per + j;
        if (r >= R) break;
        const Lens l = lens_of(s, r);
        cu[r] = (int32_t)min(bq, cap);
        first[r] = (int32_t)min(bn, kIntMax);
        bq += l.q;
        if (paged) bn += ((l.ctx + l.q + round) >> sft) - ((l.ctx + round) >> sft);
    }
    if (t == 0) {
        cu[R] = (int32_t)min(total_q, cap);
        if (total_q > cap) bad = true;
    }
    const bool scheduler = s.heads != 0 && blockIdx.x == gridDim.x - 1;   // the last block builds the schedule
    if (bad && blockIdx.x == 0) report(p.status, kStatusPlan);
    __syncthreads();
    if (scheduler) {
        build_schedule(p, cu, first, s_sums);
        return;
    }
    const int blocks = s.heads ? gridDim.x - 1 : gridDim.x;
    const int32_t T = cu[R];

    // per-request tables: a warp per request
    for (int r = blockIdx.x * kPlanWarps + warp; r < R; r += blocks * kPlanWarps) {
        const Lens l = lens_of(s, r);
        const int q = cu[r + 1] - cu[r];
        if (lane == 0) {
            s.cu_q[r] = cu[r];
            if (r == R - 1) s.cu_q[R] = T;
            s.kv_len[r] = (int32_t)min(l.ctx + q, kIntMax);
        }
        if (paged && s.free_pages) {
            const int64_t have = (l.ctx + round) >> sft, need = (l.ctx + l.q + round) >> sft;
            for (int64_t j = have + lane; j < need; j += 32) {
                const int64_t at = cursor + first[r] + (j - have);
                const bool ok = at >= 0 && at < s.free_count && j < s.table_cols;
                if (j < s.table_cols) s.block_table[r * s.table_ld + j] = ok ? __ldg(s.free_pages + at) : -1;
                if (!ok) report(p.status, kStatusPlan);
            }
        }
    }
    if (paged && blockIdx.x == 0 && t == 0 && s.cursor_out && s.free_pages)
        *s.cursor_out = (int32_t)min(cursor + total_n, kIntMax);

    // per-token tables
    for (int64_t i = (int64_t)blockIdx.x * kPlanThreads + t; i < cap; i += (int64_t)blocks * kPlanThreads) {
        int pos = 0, slot = -1;
        if (i < T) {
            // the last request that starts at or before row i and has rows
            int lo = 0, hi = R - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (cu[mid] <= i) lo = mid; else hi = mid - 1;
            }
            const int64_t ctx = lens_of(s, lo).ctx;
            const int64_t at = ctx + (i - cu[lo]);
            pos = (int)min(at, kIntMax);
            if (paged) {
                const int64_t j = at >> sft, have = (ctx + round) >> sft;
                int64_t page = -1;
                if (j < s.table_cols) {
                    if (!s.free_pages || j < have) {
                        page = s.block_table[lo * s.table_ld + j];
                    } else {
                        const int64_t f = cursor + first[lo] + (j - have);
                        if (f >= 0 && f < s.free_count) page = __ldg(s.free_pages + f);
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

// ---------------------------------------------------------------- append
// One 16-byte vector of a head's row per thread: a block copies whole packed
// rows (both K and V, every kv head), kAppendRows of them at a time, all
// their loads in flight before the first store.
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
            const int64_t sl = t0 + u < p.tokens ? __ldg(p.slot + t0 + u) : -1;
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
                if (ok[u]) val[u] = __ldg(reinterpret_cast<const uint4*>(src + (t0 + u) * ld));
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
    const size_t smem = (size_t)(step.requests + 1) * 8;
    static int attr_set_for_device[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && !attr_set_for_device[dev]) {
        e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)((kStepMaxRequests + 1) * 8));
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
    if (step.heads) grid++;
    p.ctas = num_sms < kAttnMaxCtas ? num_sms : kAttnMaxCtas;
    return launch_programmatic(plan_kernel, dim3((unsigned)grid), dim3(kPlanThreads), smem, stream, p);
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
