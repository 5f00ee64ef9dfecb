// Pages of a paged cache: requests that fork, pages that come free, pages moved
// together, and the copies that go with them.
//
// No count of users is kept for a page: a page is in use while a request's row
// of the block table has it among its first ceil(ctx_len / page_size) entries.
// Forked requests share pages by having them in both rows, and a request ends
// when its length becomes zero.  The free list is made anew from the tables by
// a sweep, whose result does not depend on what was freed when, or twice.
//
// The tables are small next to the cache (4096 requests of 512 pages: 8 MB):
// the launch and the dependent reads set the time.  The sweep is one launch of one
// cluster of 16 CTAs, so that the steps between which everyone has to wait (all
// pages marked, all moves known) are cluster barriers instead of launches, and
// the marks are bits in the CTAs' shared memory instead of a workspace to be kept
// at zero.  (64 requests of up to 246 pages 5.0 us; 400 of up to 255, 19569 pages
// moved together, 17.9; 23.0 with 8 CTAs and longer segments.)
#include "common.cuh"
#include "internal.h"
#include "kv4.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 16;
constexpr int kSegment = 64;           // entries of a table's row that a warp takes at a time (256: 20.2 us below)
constexpr int kGroup = 8;              // words of the bit map per entry of its prefix sum

__device__ __forceinline__ void report(int* status, int code)
{
    if (status) atomicCAS(status, 0, code);
}

// Exclusive prefix sum over the block's threads; the total in *all.
__device__ __forceinline__ int block_prefix(int v, int* warp_sums, int* all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();                   // the sums of an earlier call have been read
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
        if (w < warp) before += warp_sums[w];
        total += warp_sums[w];
    }
    *all = total;
    return before + x - v;
}

// Entries of request r's row that hold its pages (of 2^shift rows); more than
// the table has are reported and cut.
__device__ __forceinline__ int held_entries(int ctx, int shift, int64_t cols, bool* bad)
{
    const int64_t need = ((int64_t)max(ctx, 0) + ((int64_t)1 << shift) - 1) >> shift;
    *bad |= ctx < 0 || need > cols;
    return (int)min(need, cols);
}

// ------------------------------------------------------------------- fork
struct ForkParams {
    nvfp4_pages_t t;
    const int32_t* src;
    const int32_t* dst;
    int n;
    const int32_t* free_pages;
    int64_t free_count;
    const int32_t* cursor;
    int32_t* cursor_out;
    int32_t* copy_src;
    int32_t* copy_dst;
    int* status;
    int shift;
    int cursor_only;
};

// Every CTA looks at all pairs (which of them count, and how many free pages
// the earlier ones take) in its shared memory: first [R] the first pair with
// this destination, at [n] the pair's free page (-1: none, -2: the pair does
// not count), src_bits [R / 32] the requests that are sources.  Then the warps
// write the rows, a segment at a time.  No row or length that is read is
// written.  A cursor that is advanced in place is stored by a launch of its own
// (cursor_only), as in the plan: the CTAs read it when they start.
__global__ void __launch_bounds__(kThreads) fork_kernel(const ForkParams p)
{
    extern __shared__ int32_t sh[];
    __shared__ int s_sums[kWarps];
    griddep_launch_dependents();
    griddep_wait();
    const int R = (int)p.t.requests, n = p.n, t = threadIdx.x, lane = t & 31;
    int32_t* first = sh;
    int32_t* at = first + R;
    uint32_t* src_bits = reinterpret_cast<uint32_t*>(at + n);
    const int64_t cols = p.t.table_cols, ld = p.t.table_ld;
    const int mask = (1 << p.shift) - 1;
    const int64_t cursor = p.cursor ? *p.cursor : 0;

    for (int r = t; r < R; r += kThreads) first[r] = 0x7fffffff;
    for (int w = t; w < (R + 31) / 32; w += kThreads) src_bits[w] = 0;
    __syncthreads();
    for (int i = t; i < n; i += kThreads) {
        const int s = p.src[i], d = p.dst[i];
        if (s >= 0 && s < R) atomicOr(&src_bits[s >> 5], 1u << (s & 31));
        if (d >= 0 && d < R) atomicMin(&first[d], i);
    }
    __syncthreads();
    const int per = (n + kThreads - 1) / kThreads;
    bool bad = false;
    int fresh = 0, all = 0;
    for (int i = t * per; i < min(n, (t + 1) * per); i++) {
        const int s = p.src[i], d = p.dst[i];
        bool ok = s >= 0 && s < R && d >= 0 && d < R && first[d] == i && !(src_bits[d >> 5] >> (d & 31) & 1);
        int a = -2;
        if (ok) {
            const int ctx = p.t.ctx_len[s];
            bool cut = false;
            held_entries(ctx, p.shift, cols, &cut);
            ok = !cut;
            if (ok) a = ctx & mask ? fresh++ : -1;
        }
        bad |= !ok;
        at[i] = a;                     // (free pages counted from this thread's first)
    }
    const int before = block_prefix(fresh, s_sums, &all);
    for (int i = t * per; i < min(n, (t + 1) * per); i++) {
        if (at[i] < 0) continue;
        const int64_t f = cursor + before + at[i];
        int32_t page = f >= 0 && f < p.free_count ? p.free_pages[f] : -1;
        if (page >= p.t.pages) page = -1;
        bad |= page < 0;
        at[i] = page < 0 ? -3 : page;  // -3: a page that the list did not have
    }
    __syncthreads();

    if (p.cursor_only || (blockIdx.x == 0 && p.cursor_out && p.cursor_out != p.cursor)) {
        if (t == 0) *p.cursor_out = (int32_t)min(cursor + all, (int64_t)0x7fffffff);
        if (p.cursor_only) return;
    }
    if (bad && blockIdx.x == 0) report(p.status, kStatusPages);
    const int segments = (int)((cols + kSegment - 1) / kSegment);
    const int64_t units = (int64_t)n * segments;
    for (int64_t u = (int64_t)blockIdx.x * kWarps + (t >> 5); u < units; u += (int64_t)gridDim.x * kWarps) {
        const int i = (int)(u / segments), seg = (int)(u - (int64_t)i * segments);
        const int page = at[i];
        if (page == -2) {
            if (seg == 0 && lane == 0) p.copy_src[i] = p.copy_dst[i] = -1;
            continue;
        }
        const int s = p.src[i], d = p.dst[i], ctx = p.t.ctx_len[s];
        const int need = (int)(((int64_t)ctx + mask) >> p.shift);
        const int last = page == -1 ? -1 : need - 1;         // the entry that is not shared
        const int32_t* from = p.t.block_table + s * ld;
        int32_t* to = p.t.block_table + d * ld;
        const int j1 = (int)min(cols, (int64_t)(seg + 1) * kSegment);
#pragma unroll 8
        for (int j = seg * kSegment + lane; j < j1; j += 32) {
            const int32_t e = j < need ? from[j] : -1;
            to[j] = j == last ? max(page, -1) : e;
        }
        if (seg == 0 && lane == 0) {
            p.copy_src[i] = page >= 0 ? from[last] : -1;
            p.copy_dst[i] = max(page, -1);
            p.t.ctx_len[d] = ctx;
        }
    }
}

// ------------------------------------------------------------------- free
struct FreeParams {
    nvfp4_pages_t t;
    int32_t* free_pages;
    int32_t* free_count;
    int32_t* table_out;                // NULL: the pages stay where they are
    int64_t table_out_ld;
    int32_t* move_src;
    int32_t* move_dst;
    int* status;
    int shift;
    int words, groups;                 // of the bit map, of its prefix sum
};

__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Shared memory: bits [words] (a page in use), pre [groups] (pages in use
// before each group of kGroup words).
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) free_kernel(const FreeParams p)
{
    extern __shared__ uint32_t bits[];
    __shared__ int s_sums[kWarps];
    griddep_launch_dependents();
    griddep_wait();
    const int R = (int)p.t.requests, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int rank = (int)cluster_ctarank(), W = p.words, G = p.groups, pages = (int)p.t.pages;
    int* pre = reinterpret_cast<int*>(bits + W);
    const int64_t cols = p.t.table_cols, ld = p.t.table_ld;
    const int segments = (int)((cols + kSegment - 1) / kSegment);
    const int64_t units = (int64_t)R * segments;
    const int unit0 = rank * kWarps + warp;

    // the pages in use, each CTA those of its share of the table
    for (int w = t; w < W; w += kThreads) bits[w] = 0;
    __syncthreads();
    bool bad = false;
    // (a warp's next units' lengths are read 32 at a time)
    constexpr int kStep = kCluster * kWarps;
    int held = 0;
    auto held_of = [&](int64_t u, int i) {
        if ((i & 31) == 0) {
            const int64_t mine = u + (int64_t)lane * kStep;
            held = mine < units ? held_entries(p.t.ctx_len[mine / segments], p.shift, cols, &bad) : 0;
        }
        return __shfl_sync(0xffffffffu, held, i & 31);
    };
    for (int64_t u = unit0, i = 0; u < units; u += kStep, i++) {
        const int r = (int)(u / segments), seg = (int)(u - (int64_t)r * segments);
        const int j1 = min(held_of(u, (int)i), (seg + 1) * kSegment);
        const int32_t* row = p.t.block_table + r * ld;
#pragma unroll 8
        for (int j = seg * kSegment + lane; j < j1; j += 32) {
            const int32_t e = row[j];
            if (e >= 0 && e < pages) atomicOr(&bits[e >> 5], 1u << (e & 31));
            else bad = true;
        }
    }
    if (bad) report(p.status, kStatusPages);
    cluster_sync_all();
    // CTA c joins a slice of the words and gives it to everyone (no other CTA
    // reads or writes that slice meanwhile)
    const int slice = (W + kCluster - 1) / kCluster, w0 = min(W, rank * slice), w1 = min(W, w0 + slice);
    for (int w = w0 + t; w < w1; w += kThreads) {
        uint32_t at[kCluster], v = 0;
#pragma unroll
        for (int c = 0; c < kCluster; c++) at[c] = map_to_cta(smem_u32(bits + w), c);
#pragma unroll
        for (int c = 0; c < kCluster; c++) v |= ld_cluster(at[c]);
#pragma unroll
        for (int c = 0; c < kCluster; c++) st_cluster(at[c], v);
    }
    cluster_sync_all();

    const int per = (G + kThreads - 1) / kThreads;
    int n = 0, used = 0;
    for (int g = t * per; g < min(G, (t + 1) * per); g++)
        for (int w = g * kGroup; w < min(W, (g + 1) * kGroup); w++) n += __popc(bits[w]);
    n = block_prefix(n, s_sums, &used);
    for (int g = t * per; g < min(G, (t + 1) * per); g++) {
        pre[g] = n;
        for (int w = g * kGroup; w < min(W, (g + 1) * kGroup); w++) n += __popc(bits[w]);
    }
    __syncthreads();
    // pages in use below page e (e < 32 W)
    auto used_below = [&](int e) {
        const int w = e >> 5;
        int x = pre[w / kGroup] + __popc(bits[w] & ((1u << (e & 31)) - 1));
        for (int y = w & ~(kGroup - 1); y < w; y++) x += __popc(bits[y]);
        return x;
    };
    const bool compact = p.table_out != nullptr;
    // `used` itself may be one past the last word's bits
    const int low = !compact ? 0 : used < 32 * W ? used_below(used) : used;      // pages in use that stay
    const int free_n = pages - used, moves = compact ? used - low : 0;
    if (rank == 0 && t == 0) *p.free_count = free_n;
    for (int w = w0 + warp; w < w1; w += kWarps) {
        const int e = 32 * w + lane, below = used_below(e);
        const bool in_use = bits[w] >> lane & 1;
        if (e >= pages) continue;
        if (!compact) {
            if (!in_use) p.free_pages[e - below] = e;
        } else if (e >= used) {
            p.free_pages[e - used] = e;
            if (in_use) p.move_src[below - low] = e;
        } else if (!in_use) {
            p.move_dst[e - below] = e;
        }
    }
    for (int i = free_n + rank * kThreads + t; i < pages; i += kCluster * kThreads) p.free_pages[i] = -1;
    if (!compact) return;              // (no CTA reads another's shared memory from here on)
    for (int i = moves + rank * kThreads + t; i < pages / 2; i += kCluster * kThreads) p.move_src[i] = p.move_dst[i] = -1;
    __threadfence();
    cluster_sync_all();                // the moves are known (and every entry has been read)
    for (int64_t u = unit0, i = 0; u < units; u += kStep, i++) {
        const int r = (int)(u / segments), seg = (int)(u - (int64_t)r * segments);
        const int need = held_of(u, (int)i);
        const int32_t* row = p.t.block_table + r * ld;
        int32_t* out = p.table_out + r * p.table_out_ld;
        const int j1 = (int)min(cols, (int64_t)(seg + 1) * kSegment);
#pragma unroll 8
        for (int j = seg * kSegment + lane; j < j1; j += 32) {
            int32_t e = -1;
            if (j < need) {
                e = row[j];
                if (e >= used && e < pages) e = __ldcg(p.move_dst + used_below(e) - low);
            }
            out[j] = e;
        }
    }
}

// ------------------------------------------------------------------- copy
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;           // 16-byte vectors of a thread, all loaded before the first is stored
constexpr int kCopyChunk = (int)kPageCopyChunk;
static_assert(kCopyChunk == kCopyThreads * kCopyVecs * 16, "a vector of each thread");

struct CopyParams {
    PageCopyPlanes planes;
    const int32_t* src;
    const int32_t* dst;
    int64_t n, pages;
    int chunks;
    int* status;
};

// blockIdx.y: a chunk of 16 KB of the pages of one plane; along x the pairs.  A
// warp reads the ids of its block's next 32 pairs at once.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams p)
{
    griddep_launch_dependents();
    griddep_wait();
    const int y = blockIdx.y / p.chunks, chunk = blockIdx.y - y * p.chunks, lane = threadIdx.x & 31;
    const nvfp4_plane_t& plane = p.planes.p[y];
    const int64_t off = (int64_t)chunk * kCopyChunk + threadIdx.x * 16;
    if ((int64_t)chunk * kCopyChunk >= plane.page_bytes) return;
    char* base = static_cast<char*>(plane.base) + off;
    for (int64_t i0 = blockIdx.x; i0 < p.n; i0 += 32 * (int64_t)gridDim.x) {
        const int64_t mine = i0 + lane * (int64_t)gridDim.x;
        int32_t a = mine < p.n ? p.src[mine] : -1, b = mine < p.n ? p.dst[mine] : -1;
        const bool none = a < 0 || b < 0 || a >= p.pages || b >= p.pages;
        if (none && (a != -1 || b != -1) && blockIdx.y == 0 && threadIdx.x < 32) report(p.status, kStatusPages);
        for (unsigned left = __ballot_sync(0xffffffffu, !none); left; left &= left - 1) {
            const int l = __ffs(left) - 1;
            const int64_t from = __shfl_sync(0xffffffffu, a, l) * plane.page_stride;
            const int64_t to = __shfl_sync(0xffffffffu, b, l) * plane.page_stride;
            uint4 v[kCopyVecs];
#pragma unroll
            for (int x = 0; x < kCopyVecs; x++)
                if (off + x * kCopyThreads * 16 < plane.page_bytes)
                    v[x] = *reinterpret_cast<const uint4*>(base + from + x * kCopyThreads * 16);
#pragma unroll
            for (int x = 0; x < kCopyVecs; x++)
                if (off + x * kCopyThreads * 16 < plane.page_bytes)
                    *reinterpret_cast<uint4*>(base + to + x * kCopyThreads * 16) = v[x];
        }
    }
}

int log2_of(int64_t v)
{
    int s = 0;
    while (((int64_t)1 << s) < v) s++;
    return s;
}

// More dynamic shared memory than 48 KB, once per device.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, int (&done)[64])
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && done[dev])) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done[dev] = 1;
    return e;
}

}  // namespace

cudaError_t launch_pages_fork(const nvfp4_pages_t& t, const int32_t* src, const int32_t* dst, int64_t n,
                              const int32_t* free_pages, int64_t free_count, const int32_t* cursor,
                              int32_t* cursor_out, int32_t* copy_src, int32_t* copy_dst, int* status, int num_sms,
                              cudaStream_t stream)
{
    static int done[64] = {0};
    constexpr int kMost = (int)(2 * kStepMaxRequests + kStepMaxRequests / 32) * 4;
    cudaError_t e = allow_smem(fork_kernel, kMost, done);
    if (e != cudaSuccess) return e;
    ForkParams p = {t, src, dst, (int)n, free_pages, free_pages ? free_count : 0, cursor, cursor_out,
                    copy_src, copy_dst, status, log2_of(t.page_size), 0};
    const size_t smem = (size_t)(t.requests + n + (t.requests + 31) / 32) * 4;
    const int64_t units = n * ((t.table_cols + kSegment - 1) / kSegment), want = (units + kWarps - 1) / kWarps;
    const unsigned grid = (unsigned)(want < 1 ? 1 : want < num_sms ? want : num_sms);
    e = launch_programmatic(fork_kernel, dim3(grid), dim3(kThreads), smem, stream, p);
    if (e != cudaSuccess || !cursor_out || cursor_out != cursor) return e;
    p.cursor_only = 1;
    return launch_programmatic(fork_kernel, dim3(1), dim3(kThreads), smem, stream, p);
}

cudaError_t launch_pages_free(const nvfp4_pages_t& t, int32_t* free_pages, int32_t* free_count, int32_t* table_out,
                              int64_t table_out_ld, int32_t* move_src, int32_t* move_dst, int* status,
                              cudaStream_t stream)
{
    static int done[64] = {0}, wide[64] = {0};
    constexpr int kMost = (int)(kMaxPages / 32 + kMaxPages / 32 / kGroup) * 4;
    cudaError_t e = allow_smem(free_kernel, kMost, done);
    int dev = 0;
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !wide[dev])) {
        e = cudaFuncSetAttribute(free_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);    // more than 8 CTAs
        if (e == cudaSuccess && dev < 64) wide[dev] = 1;
    }
    if (e != cudaSuccess) return e;
    FreeParams p = {t, free_pages, free_count, table_out, table_out_ld, move_src, move_dst, status,
                    log2_of(t.page_size), 0, 0};
    p.words = (int)((t.pages + 31) / 32);
    p.groups = (p.words + kGroup - 1) / kGroup;
    return launch_programmatic(free_kernel, dim3(kCluster), dim3(kThreads), (size_t)(p.words + p.groups) * 4, stream, p);
}

cudaError_t launch_pages_copy(const PageCopyPlanes& planes, int n_planes, int64_t max_bytes, int64_t pages,
                              const int32_t* src, const int32_t* dst, int64_t n, int* status, int num_sms,
                              cudaStream_t stream)
{
    CopyParams p = {planes, src, dst, n, pages, (int)((max_bytes + kCopyChunk - 1) / kCopyChunk), status};
    const int64_t ny = (int64_t)n_planes * p.chunks, want = ((int64_t)num_sms * 8 + ny - 1) / ny;
    return launch_programmatic(copy_kernel, dim3((unsigned)(n < want ? n : want), (unsigned)ny), dim3(kCopyThreads), 0,
                               stream, p);
}

}  // namespace nvfp4
