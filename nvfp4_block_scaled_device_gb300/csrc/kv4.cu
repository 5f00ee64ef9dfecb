// Rows on their way into and out of a layer's cache: norms and rotation of the
// query and key heads (nvfp4_qk_norm_rope), the write of rows into a cache in 4
// bits (nvfp4_kv4_append), and the rows of a step out of it (nvfp4_kv4_expand).
#include "common.cuh"
#include "internal.h"
#include "kv4.h"

namespace nvfp4 {
namespace {

__device__ __forceinline__ void report(int* status, int code)
{
    if (status) atomicCAS(status, 0, code);
}

int log2_of(int64_t v)
{
    int s = 0;
    while (((int64_t)1 << s) < v) s++;
    return s;
}

// ------------------------------------------------------------------ heads
// y = x / sqrt(mean(x^2) + eps) * w, then the rotation, in binary32, rounded
// once.  A head's row is D / 8 lanes of one 16-byte vector each, so that the
// mean is a few shuffles, interleaved pairs lie in one lane and those of halves
// in two; a warp takes 32 / (D / 8) rows of one token at a time and keeps the
// token's cosines and sines over its rows.  K rows go to k_out or, with those
// of V, into the cache, in 4 bits from the bf16 value (so that the pass gives
// what the two calls give); a block of 16 columns is two lanes.
//
// Bound by HBM with many tokens (2 B in, 2 B out a column); with few by the
// launch and one dependent chain of loads, so the rows of a token are spread
// over as many warps as there is room for.
constexpr int kHeadThreads = 256;
constexpr int kHeadWarps = kHeadThreads / 32;
constexpr int kHeadBatch = 4;          // rows of a lane loaded before the first is worked on

enum { kToRows = 0, kToCache = 1, kToCache4 = 2 };

struct HeadsParams {
    nvfp4_heads_t h;
    nvfp4_kv_cache_t c;                // kToCache
    nvfp4_kv4_cache_t c4;              // kToCache4
    int lanes;                         // of a row: a power of two >= head_dim / 8
    int rows;                          // of a token: q, k and (into a cache) v heads
    int per;                           // batches of kHeadBatch rows a lane of a warp's unit
    int units;                         // of a token
    int page_shift;
    int wide_tables;                   // the tables can be read in 16-byte vectors
    int* status;
};

__device__ __forceinline__ uint4 pack8(const float* v)
{
    return make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]), cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void unpack8(uint4 x, float* v)
{
    v[0] = bf16_lo(x.x), v[1] = bf16_hi(x.x), v[2] = bf16_lo(x.y), v[3] = bf16_hi(x.y);
    v[4] = bf16_lo(x.z), v[5] = bf16_hi(x.z), v[6] = bf16_lo(x.w), v[7] = bf16_hi(x.w);
}

// Largest magnitude of two bf16x2, NaN if one is.
__device__ __forceinline__ uint32_t amax_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7fff7fffu), "r"(b & 0x7fff7fffu));
    return r;
}

// n table entries from `at` on (n 4 or 8).
template <int kN>
__device__ __forceinline__ void load_table(const float* t, int64_t at, bool wide, float* out)
{
    if (wide) {
#pragma unroll
        for (int i = 0; i < kN; i += 4) {
            const float4 x = *reinterpret_cast<const float4*>(t + at + i);
            out[i] = x.x, out[i + 1] = x.y, out[i + 2] = x.z, out[i + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kN; i++) out[i] = t[at + i];
    }
}

template <int kTo>
__global__ void __launch_bounds__(kHeadThreads) heads_kernel(const __grid_constant__ HeadsParams p)
{
    griddep_launch_dependents();
    griddep_wait();
    const nvfp4_heads_t& h = p.h;
    const int lane = threadIdx.x & 31, L = p.lanes, D = (int)h.head_dim;
    const int sub = lane / L, col = 8 * (lane & (L - 1)), at_once = 32 / L;
    const bool in_row = col < D;
    const int64_t unit = (int64_t)blockIdx.x * kHeadWarps + (threadIdx.x >> 5);
    const int64_t t = unit / p.units;
    if (t >= h.tokens) return;
    const int row0 = (int)(unit - t * p.units) * p.per * kHeadBatch * at_once;
    const int Hq = (int)h.heads, Hk = Hq + (int)h.kv_heads;

    // the angles of this lane's columns: of 4 pairs, or of 8 columns and their other halves
    const int rd = (int)h.rope_dim, rot0 = D - rd, half = rd / 2;
    float c[8], s[8];
    bool rotate = false;
    if (h.pos && in_row && col + 8 > rot0) {
        int64_t at = h.pos[t];
        if (at < 0 || at >= h.positions) {
            if (col + 8 >= D && sub == 0) report(p.status, kStatusRope);
            at = at < 0 ? 0 : h.positions - 1;
        }
        at *= h.table_ld;
        rotate = true;
        if (h.halves) {
            const int i = col - rot0 < half ? col - rot0 : col - rot0 - half;
            load_table<8>(h.cos_t, at + i, p.wide_tables, c);
            load_table<8>(h.sin_t, at + i, p.wide_tables, s);
        } else if (col >= rot0 && (col - rot0) % 8 == 0) {
            load_table<4>(h.cos_t, at + (col - rot0) / 2, p.wide_tables, c);
            load_table<4>(h.sin_t, at + (col - rot0) / 2, p.wide_tables, s);
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int x = col + 2 * i - rot0;
                c[i] = x >= 0 ? h.cos_t[at + x / 2] : 1.0f;
                s[i] = x >= 0 ? h.sin_t[at + x / 2] : 0.0f;
            }
        }
    }
    const int partner = lane + (col - rot0 < half ? rd / 16 : -rd / 16);
    float wq[8], wk[8];
    if (h.q_norm && in_row) unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(h.q_norm) + col), wq);
    if (h.k_norm && in_row) unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(h.k_norm) + col), wk);
    int64_t slot = -1;
    float g_k = 0.0f, g_v = 0.0f;
    if (kTo != kToRows) {
        const int64_t slots = (kTo == kToCache ? p.c.pages : p.c4.pages) << p.page_shift;
        slot = h.slot[t];
        if (slot != -1 && (slot < 0 || slot >= slots)) {
            if (lane == 0 && row0 == 0) report(p.status, kStatusSlot);
            slot = -1;
        }
        if (kTo == kToCache4) g_k = *p.c4.k_g, g_v = *p.c4.v_g;
    }
    const int64_t page = slot >> p.page_shift, in_page = slot & (((int64_t)1 << p.page_shift) - 1);

    for (int b = 0; b < p.per; b++) {
        uint4 x[kHeadBatch];
        const int r0 = row0 + b * kHeadBatch * at_once + sub;
        if (r0 - sub >= p.rows) return;
#pragma unroll
        for (int u = 0; u < kHeadBatch; u++) {
            const int r = r0 + u * at_once;
            const void* base = r < Hq ? h.q : r < Hk ? h.k : h.v;
            const int64_t ld = r < Hq ? h.ldq : r < Hk ? h.ldk : h.ldv, hd = r < Hq ? h.hq : r < Hk ? h.hk : h.hv;
            const int i = r < Hq ? r : r < Hk ? r - Hq : r - Hk;
            x[u] = make_uint4(0, 0, 0, 0);
            if (in_row && r < p.rows)
                x[u] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + t * ld + i * hd + col);
        }
#pragma unroll
        for (int u = 0; u < kHeadBatch; u++) {
            const int r = r0 + u * at_once;
            const bool is_q = r < Hq, is_v = r >= Hk;
            const int i = is_q ? r : is_v ? r - Hk : r - Hq;
            const bool norm = !is_v && (is_q ? h.q_norm : h.k_norm) != nullptr;
            float v[8];
            unpack8(x[u], v);
            if (h.q_norm || h.k_norm) {                    // (all lanes: the sum goes over lanes of other rows' kinds)
                float sum = 0.0f;
#pragma unroll
                for (int y = 0; y < 8; y++) sum += v[y] * v[y];
                for (int o = L / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (norm) {
                    const float inv = rsqrtf(sum / (float)D + h.eps);
#pragma unroll
                    for (int y = 0; y < 8; y++) v[y] = v[y] * inv * (is_q ? wq[y] : wk[y]);
                }
            }
            if (h.pos) {
                if (h.halves) {
#pragma unroll
                    for (int y = 0; y < 8; y++) {
                        const float other = __shfl_sync(0xffffffffu, v[y], rotate ? partner : lane);
                        if (rotate && !is_v)
                            v[y] = col - rot0 < half ? __fsub_rn(__fmul_rn(v[y], c[y]), __fmul_rn(other, s[y]))
                                                     : __fadd_rn(__fmul_rn(other, s[y]), __fmul_rn(v[y], c[y]));
                    }
                } else if (rotate && !is_v) {
#pragma unroll
                    for (int y = 0; y < 4; y++) {
                        // (columns before the rotated ones are not touched: 1 and 0 would lose a -0 or a NaN's partner)
                        if (col + 2 * y < rot0) continue;
                        const float a = v[2 * y], d = v[2 * y + 1];
                        v[2 * y] = __fsub_rn(__fmul_rn(a, c[y]), __fmul_rn(d, s[y]));
                        v[2 * y + 1] = __fadd_rn(__fmul_rn(a, s[y]), __fmul_rn(d, c[y]));
                    }
                }
            }
            const uint4 y = norm || (h.pos && !is_v) ? pack8(v) : x[u];
            const bool here = in_row && r < p.rows;
            if (is_q || (!is_v && h.k_out)) {
                if (here)
                    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_q ? h.q_out : h.k_out) +
                                              t * (is_q ? h.ldqo : h.ldko) + i * (is_q ? h.hqo : h.hko) + col) = y;
            }
            if (kTo == kToCache && !is_q && here && slot >= 0) {
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(is_v ? p.c.v : p.c.k);
                *reinterpret_cast<uint4*>(out + page * p.c.page_stride + (((int64_t)i << p.page_shift) + in_page) * D + col) = y;
            }
            if (kTo == kToCache4) {
                unpack8(y, v);
                uint32_t m = amax_bf16x2(amax_bf16x2(y.x, y.y), amax_bf16x2(y.z, y.w));
                m = amax_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = amax_bf16x2(m, m >> 16 | m << 16);
                if (!is_q && here && slot >= 0) {
                    float amax = bf16_lo(m);
                    const bool nan = amax != amax;
                    constexpr float kMost = 3.3895313892515355e38f;      // of bf16
                    if (!(amax <= kMost)) {
                        amax = kMost;
#pragma unroll
                        for (int z = 0; z < 8; z++) v[z] = fminf(fmaxf(v[z], -kMost), kMost);
                    }
                    uint32_t sc, codes = quant_half_block(v, is_v ? g_v : g_k, amax, &sc);
                    if (nan) sc = 0x7f, codes = 0;
                    const int64_t at = ((int64_t)i << p.page_shift) + in_page;
                    *reinterpret_cast<uint32_t*>((is_v ? p.c4.v : p.c4.k) + page * p.c4.page_stride + at * (D / 2) + col / 2) =
                        codes;
                    if ((col & 8) == 0)
                        (is_v ? p.c4.v_sf : p.c4.k_sf)[page * p.c4.sf_stride + at * (D / 16) + col / 16] = (uint8_t)sc;
                }
            }
        }
    }
}

template <int kTo>
cudaError_t run_heads(HeadsParams& p, int num_sms, cudaStream_t stream)
{
    const int batch = kHeadBatch * (32 / p.lanes), most = (p.rows + batch - 1) / batch;
    // as many warps as fill the GPU, each with as many rows of its token as that leaves
    const int64_t per = p.h.tokens * most / ((int64_t)num_sms * 64);
    p.per = (int)(per < 1 ? 1 : per > most ? most : per);
    p.units = (most + p.per - 1) / p.per;
    const int64_t blocks = (p.h.tokens * p.units + kHeadWarps - 1) / kHeadWarps;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return launch_programmatic(heads_kernel<kTo>, dim3((unsigned)blocks), dim3(kHeadThreads), 0, stream, p);
}

// ----------------------------------------------------------------- expand
// A page's rows of all heads are one run of half blocks (8 columns: 4 bytes of
// codes, a scale that two share, 16 bytes out), so nothing but the pages at a
// request's ends has to know which row it is at.  Every block sums up the
// pages of all requests in shared memory and takes its share of them.
// Bound by HBM: 0.56 B in, 2 B out a column.
constexpr int kExpandThreads = 256;
constexpr int kExpandVecs = 8;                      // half blocks of a thread
constexpr int kExpandChunk = kExpandThreads * kExpandVecs;

struct ExpandParams {
    nvfp4_kv4_cache_t c;
    nvfp4_kv_cache_t out;
    const int32_t* cu_q;
    const int32_t* kv_len;
    const int32_t* block_table;
    int64_t table_ld;
    int requests, table_cols, window, page_shift, scaled;
    int halves;                                     // half blocks of a page of K
    int chunks;                                     // of kExpandChunk
};

// First position that a new token of request r sees, and the end.
__device__ __forceinline__ int2 seen_rows(const ExpandParams& p, int r)
{
    const int q = p.cu_q[r + 1] - p.cu_q[r], kv = p.kv_len[r];
    if (q <= 0) return make_int2(0, 0);
    const int64_t cap = (int64_t)p.table_cols << p.page_shift;
    return make_int2(p.window ? max(kv - q + 1 - p.window, 0) : 0, (int)min((int64_t)kv, cap));
}

__global__ void __launch_bounds__(kExpandThreads) expand_kernel(const __grid_constant__ ExpandParams p)
{
    extern __shared__ int32_t pre[];                // [requests + 1] pages before each request
    __shared__ int s_sums[kExpandThreads / 32];
    griddep_launch_dependents();
    griddep_wait();
    const int R = p.requests, t = threadIdx.x, lane = t & 31, warp = t >> 5, P = 1 << p.page_shift;
    const int per = (R + kExpandThreads - 1) / kExpandThreads;
    auto pages_of = [&](int r) {
        const int2 x = seen_rows(p, r);
        return x.x < x.y ? ((x.y - 1) >> p.page_shift) - (x.x >> p.page_shift) + 1 : 0;
    };
    int n = 0;
    for (int r = t * per; r < min(R, (t + 1) * per); r++) n += pages_of(r);
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s_sums[warp] = incl;
    __syncthreads();
    int at = incl - n;
    for (int w = 0; w < warp; w++) at += s_sums[w];
    for (int r = t * per; r < min(R, (t + 1) * per); r++) {
        pre[r] = at;
        at += pages_of(r);
    }
    if (t == kExpandThreads - 1) pre[R] = at;
    __syncthreads();
    const int64_t units = (int64_t)pre[R] * 2 * p.chunks;
    const int per_row = (int)p.c.head_dim / 8;
    const float g[2] = {p.scaled ? *p.c.k_g : 1.0f, p.scaled ? *p.c.v_g : 1.0f};
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int i = (int)(u / (2 * p.chunks)), part = (int)(u - (int64_t)i * 2 * p.chunks);
        const bool is_v = part >= p.chunks;
        const int h0 = (is_v ? part - p.chunks : part) * kExpandChunk + t;
        int lo = 0, hi = R - 1;                     // the request that page i is of
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pre[mid] <= i) lo = mid; else hi = mid - 1;
        }
        const int2 seen = seen_rows(p, lo);
        const int j = (seen.x >> p.page_shift) + i - pre[lo];
        const int64_t page = p.block_table[lo * p.table_ld + j];
        if (page < 0 || page >= p.c.pages) continue;
        const int r0 = seen.x - (j << p.page_shift), r1 = seen.y - (j << p.page_shift);   // rows r0 .. r1 - 1 of the page
        const bool whole = r0 <= 0 && r1 >= P;
        const uint8_t* codes = (is_v ? p.c.v : p.c.k) + page * p.c.page_stride;
        const uint8_t* sf = (is_v ? p.c.v_sf : p.c.k_sf) + page * p.c.sf_stride;
        uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_v ? p.out.v : p.out.k) + page * p.out.page_stride);
        uint32_t w[kExpandVecs];
        uint32_t sc[kExpandVecs];
#pragma unroll
        for (int x = 0; x < kExpandVecs; x++) {
            const int hb = h0 + x * kExpandThreads;
            if (hb < p.halves) {
                w[x] = *reinterpret_cast<const uint32_t*>(codes + (int64_t)hb * 4);
                sc[x] = sf[hb >> 1];
            }
        }
#pragma unroll
        for (int x = 0; x < kExpandVecs; x++) {
            const int hb = h0 + x * kExpandThreads;
            if (hb >= p.halves) continue;
            if (!whole) {
                const int row = (hb / per_row) & (P - 1);
                if (row < r0 || row >= r1) continue;
            }
            const float f = e4m3_to_f32(sc[x]);
            const float gg = g[is_v ? 1 : 0];
            uint32_t o[4];
#pragma unroll
            for (int y = 0; y < 4; y++) {
                const float2 v = e2m1x2_to_f32(w[x] >> (8 * y));
                // (code times scale is exact)
                o[y] = cvt_bf16x2(v.x * f * gg, v.y * f * gg);
            }
            out[hb] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

}  // namespace

cudaError_t launch_heads(const nvfp4_heads_t& heads, int* status, int num_sms, cudaStream_t stream)
{
    HeadsParams p = {};
    p.h = heads;
    p.status = status;
    p.lanes = 1 << log2_of((heads.head_dim + 7) / 8);
    const bool to_cache = heads.slot != nullptr;
    p.rows = (int)(heads.heads + heads.kv_heads * (to_cache ? 2 : 1));
    p.wide_tables = heads.pos && heads.table_ld % 4 == 0 && ((uintptr_t)heads.cos_t | (uintptr_t)heads.sin_t) % 16 == 0;
    if (!to_cache) return run_heads<kToRows>(p, num_sms, stream);
    if (heads.cache) {
        p.c = *heads.cache;
        p.page_shift = log2_of(p.c.page_size);
        return run_heads<kToCache>(p, num_sms, stream);
    }
    p.c4 = *heads.cache4;
    p.page_shift = log2_of(p.c4.page_size);
    return run_heads<kToCache4>(p, num_sms, stream);
}

cudaError_t launch_kv4_expand(const nvfp4_kv4_cache_t& cache, const nvfp4_step_t& step, const nvfp4_kv_cache_t& out,
                              bool scaled, int num_sms, cudaStream_t stream)
{
    ExpandParams p = {};
    p.c = cache;
    p.out = out;
    p.cu_q = step.cu_q;
    p.kv_len = step.kv_len;
    p.block_table = step.block_table;
    p.table_ld = step.table_ld;
    p.requests = (int)step.requests;
    p.table_cols = (int)step.table_cols;
    p.window = step.heads ? (int)step.window : 0;
    p.page_shift = log2_of(cache.page_size);
    p.scaled = scaled;
    p.halves = (int)(cache.kv_heads * cache.page_size * cache.head_dim / 8);
    p.chunks = (p.halves + kExpandChunk - 1) / kExpandChunk;
    return launch_programmatic(expand_kernel, dim3((unsigned)num_sms * 8), dim3(kExpandThreads),
                               (size_t)(step.requests + 1) * 4, stream, p);
}

}  // namespace nvfp4
