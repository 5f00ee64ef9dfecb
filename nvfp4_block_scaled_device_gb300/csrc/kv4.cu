// Rows on their way into and out of a layer's cache: norms and rotation of the
// query and key heads (nvfp4_qk_norm_rope), the write of rows into a cache in 4
// bits (nvfp4_kv4_append), and the rows of a step out of it (nvfp4_kv4_expand).
#include <cuda_fp16.h>

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
// in two; a warp takes 32 / (D / 8) rows of one token and kind (q, k, v) at a
// time and keeps the token's cosines and sines over its rows.  Arithmetic on
// pairs of columns (two binary32 operations an instruction: without it, and with
// the kinds mixed in a warp, the pass was bound by its instructions, 195 us where
// it now takes 87).  K rows go to k_out or, with those of V, into the cache,
// in 4 bits from the bf16 value (so that the pass gives what the two calls give);
// a block of 16 columns is two lanes.
//
// Bound by HBM's latency with many tokens (2 B in, 2 B out a column): 16272 tokens of 40
// query and 8 key heads, with the values into the bf16 cache, 87 us for 475 MB (5.5 TB/s; blocks
// of 64 registers, 8 to an SM, 91 then: 9 blocks 92, 6 blocks 115, 10 and fewer rows at
// once 104).  Into the 4-bit cache 102 us for 427 MB (4.2 TB/s; 94 with interleaved
// pairs): 78 M instructions of a warp instead of 59 M, as a lane quantizes half a block
// of K.  Part of a head rotated 91 to 117, heads of 96 columns 94 and (4 bits) 116,
// of 64 columns 65 and 81.  With few tokens by the launch and one dependent chain of
// loads, so the rows of a token
// are spread over as many warps as there is room for (8 tokens 2.6 us).
constexpr int kHeadThreads = 128;
constexpr int kHeadWarps = kHeadThreads / 32;
constexpr int kHeadBatch = 4;          // rows of a lane loaded before the first is worked on
constexpr int kHeadBlocks = 8;             // of an SM

enum { kToRows = 0, kToCache = 1, kToCache4 = 2 };
enum { kNoRope = 0, kPairs = 1, kHalves = 2 };

struct HeadsParams {
    nvfp4_heads_t h;
    nvfp4_kv_cache_t c;                // kToCache
    nvfp4_kv4_cache_t c4;              // kToCache4
    int lanes;                         // of a row: a power of two >= head_dim / 8
    int per;                           // batches of a warp's unit
    int units_q, units_k, units;       // units of a token: of q, of k, of all kinds
    int page_shift;
    int wide_tables;                   // the tables can be read in 16-byte vectors
    int* status;
};

// Two binary32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
        " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ void unpack4(uint4 x, float2* v)
{
    v[0] = make_float2(bf16_lo(x.x), bf16_hi(x.x));
    v[1] = make_float2(bf16_lo(x.y), bf16_hi(x.y));
    v[2] = make_float2(bf16_lo(x.z), bf16_hi(x.z));
    v[3] = make_float2(bf16_lo(x.w), bf16_hi(x.w));
}

// Largest magnitude of two bf16x2, NaN if one is.
__device__ __forceinline__ uint32_t amax_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7fff7fffu), "r"(b & 0x7fff7fffu));
    return r;
}

// Two bf16, no more than `far` from 0.
__device__ __forceinline__ uint32_t clamp_bf16x2(uint32_t x, uint32_t far)
{
    asm("min.bf16x2 %0, %0, %1;\n max.bf16x2 %0, %0, %2;" : "+r"(x) : "r"(far), "r"(far | 0x80008000u));
    return x;
}

constexpr float kMostBf16 = 3.3895313892515355e38f;

// Scales of a cache's blocks: 6 g and its correctly rounded reciprocal.
struct BlockScale {
    float g, d, rd;
};
__device__ __forceinline__ BlockScale block_scale(float g)
{
    const float d = __fmul_rn(6.0f, g);
    return BlockScale{g, d, __frcp_rn(d)};
}

// One block's scale and codes, nvfp4_quantize's bit for bit: each lane has kVecs
// vectors of it (8 columns), amax is the block's, *sc its scale.  The quotients v /
// den are those of div_by_recip in pairs of columns, negated (q = -v y, q + (v + q
// den) (-y): the remainder's sign needs no operation, and a zero keeps the sign
// that the codes' XOR then turns around).  They are right for dividends whose quotients
// are far from overflow: amax no more than 448 d (the scale is 448 from there on; an
// infinity is the largest bf16 number), then v no more than 8 den (the code is 6).
template <int kVecs>
__device__ __forceinline__ void quant_block(const uint4* x, uint32_t amax_bits, const BlockScale& b, uint32_t* codes, uint32_t* sc)
{
    float amax = bf16_lo(amax_bits);
    const float most = __fmul_rn(448.0f, b.d);
    const bool odd = !(amax < most), nan = amax != amax;             // too large, an infinity or NaN in it
    if (odd) amax = fminf(most, kMostBf16);
    const uint32_t s = cvt_e4m3(div_by_recip(amax, b.d, b.rd));
    const float den = __fmul_rn(e4m3_to_f32(s), b.g);
    const float ny = -__frcp_rn(s ? den : 1.0f);
    const float2 ny2 = make_float2(ny, ny), den2 = make_float2(den, den);
#pragma unroll
    for (int i = 0; i < kVecs; i++) {
        uint4 z = x[i];
        if (odd) {
            const float far = fminf(__fmul_rn(8.0f, den), kMostBf16);
            const uint32_t far2 = cvt_bf16x2(far, far);
            z = make_uint4(clamp_bf16x2(z.x, far2), clamp_bf16x2(z.y, far2), clamp_bf16x2(z.z, far2), clamp_bf16x2(z.w, far2));
        }
        float2 v[4];
        unpack4(z, v);
        float q[8];
#pragma unroll
        for (int y = 0; y < 4; y++) {
            const float2 q0 = mul2(v[y], ny2), r = fma2(fma2(q0, den2, v[y]), ny2, q0);
            q[2 * y] = r.x, q[2 * y + 1] = r.y;
        }
        codes[i] = s == 0 || nan ? 0u : cvt_e2m1x8(q) ^ 0x88888888u;
    }
    *sc = nan ? 0x7fu : s;
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

// A lane's place in a warp's rows, and where these come from and go.
struct HeadRows {
    const __nv_bfloat16* src;          // this lane's columns of row 0, and of a row kHeadBatch * at_once on ...
    int64_t step;                      // ... elements from one of its rows to the next
    __nv_bfloat16* out;                // NULL: none
    int64_t step_out;
    uint8_t* codes;                    // kToCache4: of the slot's row 0 (NULL: none), its scale, bytes from one to the next
    uint8_t* sf;
    uint32_t step_codes, step_sf;
    float g;
    __nv_bfloat16* also;               // k_out beside a cache
    int64_t step_also;
    int left;                          // rows from this lane's first on (in steps)
};

// The weights count a power of two less and 1 / rms as much more, which no result
// of ordinary size notices: a row whose squares are beyond binary32 is 0 (1 / rms
// is), not 0 times an infinite product (of weights up to 2^15).
constexpr float kLess = 1.0f / 65536.0f;

// What a lane does to its 8 columns of a row.
struct HeadMath {
    int L;                             // lanes of a row
    float inv_d, eps;
    // with a norm: column pair y becomes (v[y] * p[y] + other * q[y]) / (kLess rms), where
    // `other` is the partner lane's pair (halves) or the pair's columns exchanged:
    // kLess times weight times cosine, the other one's weight times sine with its sign
    float2 p[4], q[4];
    // without: the rotation in single operations
    float c[8], s[8];
    bool rotate;
    int skip;                          // pairs of the lane before the rotated ones
    float sign;
    int partner;
    bool scale_lane;
};

// The rows of a warp's unit.  kNorm: times w / rms; kRope: rotated; kTo: bf16 to
// out, or codes and scales; kWhole: a row is 16 whole lanes, all of them rotated.
template <int kTo, int kRope, bool kNorm, bool kWhole>
__device__ __forceinline__ void work_rows(HeadRows& q, int batches, const HeadMath& h)
{
    const BlockScale scale = block_scale(kTo == kToCache4 ? q.g : 1.0f);
#pragma unroll 1
    for (;;) {
        uint4 x[kHeadBatch];
#pragma unroll
        for (int i = 0; i < kHeadBatch; i++)
            x[i] = i < q.left ? *reinterpret_cast<const uint4*>(q.src + i * q.step) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kHeadBatch; i++) {
            uint4 y = x[i];
            if (kNorm) {
                float2 v[4], r[4];
                unpack4(x[i], v);
                float2 sq = mul2(v[0], v[0]);
#pragma unroll
                for (int z = 1; z < 4; z++) sq = fma2(v[z], v[z], sq);
                float sum = sq.x + sq.y;
#pragma unroll
                for (int o = 8; o; o >>= 1) {
                    const float other = __shfl_xor_sync(0xffffffffu, sum, o);
                    if (kWhole || o < h.L) sum += other;
                }
                const float inv = rsqrtf(sum * h.inv_d + h.eps) * (1.0f / kLess);
#pragma unroll
                for (int z = 0; z < 4; z++) r[z] = mul2(v[z], h.p[z]);
                if (kRope == kHalves) {
                    // (the bf16 row itself goes between the lanes)
                    const uint4 ox = make_uint4(__shfl_sync(0xffffffffu, x[i].x, h.partner), __shfl_sync(0xffffffffu, x[i].y, h.partner),
                                                __shfl_sync(0xffffffffu, x[i].z, h.partner), __shfl_sync(0xffffffffu, x[i].w, h.partner));
                    unpack4(ox, v);
                }
#pragma unroll
                for (int z = 0; z < 4; z++) {
                    if (kRope != kNoRope) {
                        const float2 turned = fma2(kRope == kPairs ? make_float2(v[z].y, v[z].x) : v[z], h.q[z], r[z]);
                        // (a column that is not rotated takes nothing of its neighbour, which may be infinite)
                        if (kWhole || (kRope == kPairs ? z >= h.skip : h.rotate)) r[z] = turned;
                    }
                    r[z] = mul2(r[z], make_float2(inv, inv));
                }
                y = make_uint4(cvt_bf16x2(r[0].x, r[0].y), cvt_bf16x2(r[1].x, r[1].y), cvt_bf16x2(r[2].x, r[2].y), cvt_bf16x2(r[3].x, r[3].y));
            } else if (kRope != kNoRope) {
                // (products rounded first: the sum with a factor of 1 or -1 is one operation)
                float2 v[4];
                unpack4(x[i], v);
#pragma unroll
                for (int z = 0; z < 4; z++) {
                    if (kRope == kHalves) {
                        const float2 other = make_float2(__shfl_sync(0xffffffffu, v[z].x, h.partner), __shfl_sync(0xffffffffu, v[z].y, h.partner));
                        const float2 r = fma2(mul2(other, make_float2(h.s[2 * z], h.s[2 * z + 1])), make_float2(h.sign, h.sign),
                                              mul2(v[z], make_float2(h.c[2 * z], h.c[2 * z + 1])));
                        if (h.rotate) v[z] = r;
                    } else {
                        const float2 r = fma2(mul2(make_float2(v[z].y, v[z].x), make_float2(h.s[z], h.s[z])), make_float2(-1.0f, 1.0f),
                                              mul2(v[z], make_float2(h.c[z], h.c[z])));
                        // (columns before the rotated ones are not touched: 1 and 0 would lose a -0 or a NaN's partner)
                        if (z >= h.skip) v[z] = r;
                    }
                }
                y = make_uint4(cvt_bf16x2(v[0].x, v[0].y), cvt_bf16x2(v[1].x, v[1].y), cvt_bf16x2(v[2].x, v[2].y), cvt_bf16x2(v[3].x, v[3].y));
            }
            const bool here = i < q.left;
            // (leaves L2 first: rows to come are read through it; 16272 tokens 87 us, 91 without)
            if (q.out && here) __stcs(reinterpret_cast<uint4*>(q.out + i * q.step_out), y);
            if (kTo != kToRows && q.also && here) *reinterpret_cast<uint4*>(q.also + i * q.step_also) = y;
            if (kTo == kToCache4 && q.codes) {
                uint32_t m = amax_bf16x2(amax_bf16x2(y.x, y.y), amax_bf16x2(y.z, y.w));
                m = amax_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = amax_bf16x2(m, m >> 16 | m << 16);
                uint32_t sc, codes;
                quant_block<1>(&y, m, scale, &codes, &sc);
                if (here) {
                    *reinterpret_cast<uint32_t*>(q.codes + (uint64_t)i * q.step_codes) = codes;
                    if (h.scale_lane) q.sf[(uint64_t)i * q.step_sf] = (uint8_t)sc;
                }
            }
        }
        q.left -= kHeadBatch;
        if (--batches == 0 || !__any_sync(0xffffffffu, q.left > 0)) break;
        q.src += kHeadBatch * q.step;
        if (q.out) q.out += kHeadBatch * q.step_out;
        if (kTo != kToRows && q.also) q.also += kHeadBatch * q.step_also;
        if (kTo == kToCache4 && q.codes) {
            q.codes += (uint64_t)kHeadBatch * q.step_codes;
            q.sf += (uint64_t)kHeadBatch * q.step_sf;
        }
    }
}

// Rows as they are into the 4-bit cache: unit u of token t's rows of k or v, `per`
// times kHeadBatch rows for each that L lanes of 8 columns would have.  A lane has a
// whole block of 16 columns (so that what is done once per block is done once) of
// two rows at a time.  16272 tokens of 8 heads: 18.0 us for 85 MB (4.7 TB/s; with half
// a block to a lane 25, bound by its instructions; then, without the loads' hint, 19.7, and
// with warps that loop over tokens, the next one's rows on their way, 19.8).
__device__ __forceinline__ void append_rows(const HeadsParams& p, uint32_t t, bool is_v, int u, int lane, int L, int D)
{
    const nvfp4_heads_t& h = p.h;
    const int lanes = L / 2, at_once = 32 / lanes, col = 16 * (lane & (lanes - 1));
    const int first = u * p.per * (kHeadBatch / 2) * at_once, end = min((int)h.kv_heads, first + p.per * (kHeadBatch / 2) * at_once);
    const int64_t slots = p.c4.pages << p.page_shift, slot = h.slot[t];
    if (slot < 0 || slot >= slots) {
        if (slot != -1 && lane == 0 && u == 0) report(p.status, kStatusSlot);
        return;
    }
    if (col >= D) return;
    const int64_t page = slot >> p.page_shift, pitch = is_v ? h.hv : h.hk;
    const uint32_t in_page = (uint32_t)slot & ((1u << p.page_shift) - 1);
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_v ? h.v : h.k) + t * (is_v ? h.ldv : h.ldk) + col;
    uint8_t* codes = (is_v ? p.c4.v : p.c4.k) + page * p.c4.page_stride + col / 2;
    uint8_t* sf = (is_v ? p.c4.v_sf : p.c4.k_sf) + page * p.c4.sf_stride + col / 16;
    const BlockScale scale = block_scale(*(is_v ? p.c4.v_g : p.c4.k_g));
#pragma unroll 1
    for (int r = first + lane / lanes; r < end; r += 2 * at_once) {
        uint4 x[2][2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const uint4* from = reinterpret_cast<const uint4*>(src + (r + i * at_once) * pitch);
            // (nothing reads the bf16 rows of a cached token again: they leave L2 first)
#pragma unroll
            for (int y = 0; y < 2; y++) x[i][y] = i == 0 || r + at_once < end ? __ldcs(from + y) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if (i && r + at_once >= end) break;
            uint32_t m = amax_bf16x2(amax_bf16x2(amax_bf16x2(x[i][0].x, x[i][0].y), amax_bf16x2(x[i][0].z, x[i][0].w)),
                                     amax_bf16x2(amax_bf16x2(x[i][1].x, x[i][1].y), amax_bf16x2(x[i][1].z, x[i][1].w)));
            m = amax_bf16x2(m, m >> 16 | m << 16);
            uint32_t w[2], sc;
            quant_block<2>(x[i], m, scale, w, &sc);
            const uint32_t at = ((uint32_t)(r + i * at_once) << p.page_shift) + in_page;
            *reinterpret_cast<uint2*>(codes + (uint64_t)at * (D / 2)) = make_uint2(w[0], w[1]);
            sf[(uint64_t)at * (D / 16)] = (uint8_t)sc;
        }
    }
}

// nvfp4_kv4_append.
template <bool kWhole>
__global__ void __launch_bounds__(kHeadThreads, kHeadBlocks) append_kernel(const __grid_constant__ HeadsParams p)
{
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t unit = blockIdx.x * kHeadWarps + (threadIdx.x >> 5), t = unit / (uint32_t)p.units;
    if (t >= p.h.tokens) return;
    const int u = (int)(unit - t * p.units);
    const bool is_v = u >= p.units_k;
    append_rows(p, t, is_v, is_v ? u - p.units_k : u, threadIdx.x & 31, kWhole ? 16 : p.lanes, kWhole ? 128 : (int)p.h.head_dim);
}

template <int kTo, int kRope, bool kWhole>
__global__ void __launch_bounds__(kHeadThreads, kHeadBlocks) heads_kernel(const __grid_constant__ HeadsParams p)
{
    griddep_launch_dependents();
    griddep_wait();
    const nvfp4_heads_t& h = p.h;
    const int lane = threadIdx.x & 31, L = kWhole ? 16 : p.lanes, D = kWhole ? 128 : (int)h.head_dim;
    const int sub = lane / L, col = 8 * (lane & (L - 1)), at_once = 32 / L;
    const bool in_row = kWhole || col < D;
    const uint32_t unit = blockIdx.x * kHeadWarps + (threadIdx.x >> 5), t = unit / (uint32_t)p.units;
    if (t >= h.tokens) return;
    // the warp's rows: of one kind
    int u = (int)(unit - t * p.units);
    const bool is_q = u < p.units_q, is_v = kTo != kToRows && u >= p.units_q + p.units_k;
    u -= is_q ? 0 : is_v ? p.units_q + p.units_k : p.units_q;
    if (kTo == kToCache4 && is_v) {
        append_rows(p, t, true, u, lane, L, D);
        return;
    }
    const int rows = (int)(is_q ? h.heads : h.kv_heads), r0 = u * p.per * kHeadBatch * at_once + sub;
    const int64_t pitch = is_q ? h.hq : is_v ? h.hv : h.hk, ld = is_q ? h.ldq : is_v ? h.ldv : h.ldk;
    HeadRows q = {};
    q.src = static_cast<const __nv_bfloat16*>(is_q ? h.q : is_v ? h.v : h.k) + t * ld + r0 * pitch + col;
    q.step = at_once * pitch;
    q.left = in_row && r0 < rows ? (rows - r0 + at_once - 1) / at_once : 0;
    const int64_t pitch_out = is_q ? h.hqo : h.hko;
    __nv_bfloat16* rows_out = static_cast<__nv_bfloat16*>(is_q ? h.q_out : is_v ? nullptr : h.k_out);
    if (rows_out) rows_out += t * (is_q ? h.ldqo : h.ldko) + r0 * pitch_out + col;
    q.out = rows_out;
    q.step_out = at_once * pitch_out;
    if (kTo != kToRows && !is_q) {
        const int64_t slots = (kTo == kToCache ? p.c.pages : p.c4.pages) << p.page_shift;
        const int64_t slot = h.slot[t];
        const bool ok = slot >= 0 && slot < slots;
        if (!ok && slot != -1 && lane == 0 && u == 0) report(p.status, kStatusSlot);
        const int64_t page = slot >> p.page_shift, at = ((int64_t)r0 << p.page_shift) + (slot & (((int64_t)1 << p.page_shift) - 1));
        if (kTo == kToCache) {
            q.also = rows_out;
            q.step_also = q.step_out;
            q.out = ok ? static_cast<__nv_bfloat16*>(is_v ? p.c.v : p.c.k) + page * p.c.page_stride + at * D + col : nullptr;
            q.step_out = (int64_t)(at_once << p.page_shift) * D;
        } else {
            q.also = rows_out;
            q.step_also = q.step_out;
            q.out = nullptr;
            q.codes = ok ? p.c4.k + page * p.c4.page_stride + at * (D / 2) + col / 2 : nullptr;
            q.sf = p.c4.k_sf + page * p.c4.sf_stride + at * (D / 16) + col / 16;
            q.step_codes = (at_once << p.page_shift) * (D / 2);
            q.step_sf = (at_once << p.page_shift) * (D / 16);
            q.g = *p.c4.k_g;
        }
    }
    HeadMath m;
    m.L = L;
    m.inv_d = 1.0f / (float)D;
    m.eps = h.eps;
    m.scale_lane = (col & 8) == 0;
    const __nv_bfloat16* weight = static_cast<const __nv_bfloat16*>(is_q ? h.q_norm : is_v ? nullptr : h.k_norm);
    if (kTo == kToCache && is_v) {
        work_rows<kTo, kNoRope, false, kWhole>(q, p.per, m);
        return;
    }

    // the angles of this lane's columns: of 4 pairs, or of 8 columns and their other halves
    const int rd = kWhole ? D : (int)h.rope_dim, rot0 = D - rd, half = rd / 2;
    constexpr int kAngles = kRope == kHalves ? 8 : 4;
    m.rotate = kRope != kNoRope && in_row && (kWhole || col + 8 > rot0);
    const bool low = col - rot0 < half;
    m.partner = !m.rotate ? lane : low ? lane + rd / 16 : lane - rd / 16;
    m.skip = m.rotate ? max(rot0 - col, 0) / 2 : 4;
    m.sign = low ? -1.0f : 1.0f;
#pragma unroll
    for (int i = 0; i < kAngles; i++) m.c[i] = 1.0f, m.s[i] = 0.0f;
    if (kRope != kNoRope && m.rotate) {
        int64_t at = h.pos[t];
        if (at < 0 || at >= h.positions) {
            if (col + 8 >= D && sub == 0) report(p.status, kStatusRope);
            at = at < 0 ? 0 : h.positions - 1;
        }
        at *= h.table_ld;
        if (kRope == kHalves) {
            const int i = low ? col - rot0 : col - rot0 - half;
            load_table<kAngles>(h.cos_t, at + i, p.wide_tables, m.c);
            load_table<kAngles>(h.sin_t, at + i, p.wide_tables, m.s);
        } else if (kWhole || (col >= rot0 && (col - rot0) % 8 == 0)) {
            load_table<kAngles>(h.cos_t, at + (col - rot0) / 2, p.wide_tables, m.c);
            load_table<kAngles>(h.sin_t, at + (col - rot0) / 2, p.wide_tables, m.s);
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int y = col + 2 * i - rot0;
                if (y < 0) continue;
                m.c[i] = h.cos_t[at + y / 2];
                m.s[i] = h.sin_t[at + y / 2];
            }
        }
    }
    if (!weight) {
        work_rows<kTo, kRope, false, kWhole>(q, p.per, m);
        return;
    }
    float2 w[4] = {}, o[4] = {};
    if (in_row) {
        unpack4(*reinterpret_cast<const uint4*>(weight + col), w);
        if (kRope == kHalves && m.rotate) unpack4(*reinterpret_cast<const uint4*>(weight + (low ? col + half : col - half)), o);
    }
#pragma unroll
    for (int y = 0; y < 4; y++) w[y] = mul2(w[y], make_float2(kLess, kLess)), o[y] = mul2(o[y], make_float2(kLess, kLess));
#pragma unroll
    for (int y = 0; y < 4; y++) {
        if (kRope == kHalves) {
            m.p[y] = mul2(w[y], make_float2(m.c[2 * y], m.c[2 * y + 1]));
            m.q[y] = mul2(o[y], make_float2(m.sign * m.s[2 * y], m.sign * m.s[2 * y + 1]));
        } else if (kRope == kPairs) {
            m.p[y] = mul2(w[y], make_float2(m.c[y], m.c[y]));
            m.q[y] = mul2(make_float2(w[y].y, w[y].x), make_float2(-m.s[y], m.s[y]));
        } else {
            m.p[y] = w[y];
        }
    }
    work_rows<kTo, kRope, true, kWhole>(q, p.per, m);
}

template <int kTo>
cudaError_t run_heads(HeadsParams& p, int num_sms, cudaStream_t stream)
{
    const int batch = kHeadBatch * (32 / p.lanes);
    const int64_t q = (p.h.heads + batch - 1) / batch, kv = (p.h.kv_heads + batch - 1) / batch;
    // as many warps as fill the GPU, each with as many rows of its token as that leaves
    // (no more than the smaller kind has, so that a block's warps end together)
    const int64_t most = q && (!kv || q < kv) ? q : kv, per = p.h.tokens * (q + (kTo != kToRows ? 2 : 1) * kv) / ((int64_t)num_sms * 64);
    p.per = (int)(per < 1 ? 1 : per > most ? most : per);
    p.units_q = (int)((q + p.per - 1) / p.per);
    p.units_k = (int)((kv + p.per - 1) / p.per);
    p.units = p.units_q + p.units_k * (kTo != kToRows ? 2 : 1);
    const int64_t blocks = (p.h.tokens * p.units + kHeadWarps - 1) / kHeadWarps;
    if (blocks * kHeadWarps > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks), block(kHeadThreads);
    const bool rope = p.h.pos, whole = p.h.head_dim == 128 && (!rope || p.h.rope_dim == 128);
    auto go = [&](void (*kernel)(HeadsParams)) { return launch_programmatic(kernel, grid, block, 0, stream, p); };
    if (kTo == kToCache4 && !p.h.heads && !rope && !p.h.k_norm && !p.h.k_out)
        return p.h.head_dim == 128 ? go(append_kernel<true>) : go(append_kernel<false>);
    if (!rope) return whole ? go(heads_kernel<kTo, kNoRope, true>) : go(heads_kernel<kTo, kNoRope, false>);
    if (p.h.halves) return whole ? go(heads_kernel<kTo, kHalves, true>) : go(heads_kernel<kTo, kHalves, false>);
    return whole ? go(heads_kernel<kTo, kPairs, true>) : go(heads_kernel<kTo, kPairs, false>);
}

// ----------------------------------------------------------------- expand
// Two E2M1 codes (a byte, the first in the low nibble) -> two halves (exact).
__device__ __forceinline__ __half2 e2m1x2_to_f16x2(uint32_t b)
{
    uint32_t h;
    asm("{\n .reg .b8 x, a, b, c;\n mov.b32 {x, a, b, c}, %1;\n cvt.rn.f16x2.e2m1x2 %0, x;\n}" : "=r"(h) : "r"(b));
    return *reinterpret_cast<const __half2*>(&h);
}

// A page's rows of all heads are one run of half blocks (8 columns: 4 bytes of
// codes, a scale that two share, 16 bytes out), so nothing but the pages at a
// request's ends has to know which row it is at.  Every block sums up the
// pages of all requests in shared memory and takes its share of them.
// 0.56 B in, 2 B out a column; 16272 rows of 8 heads 17.9 us (4.8 TB/s; the
// bytes alone would take 12.7).  Bound by its instructions, 12.2 M of a warp (issue active 71 %,
// beside 29 MB of HBM traffic: the rest stays in L2), after some 3 us until the first
// codes are there: lengths, table, codes one after the other; 4 half blocks to a
// thread 18.1, 2 23.3.  Pages of less than a chunk (one head of 16 rows of 128
// columns: 256 half blocks) leave threads idle.
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
    int requests, table_cols, window, page_shift;
    int halves;                                     // half blocks of a page of K
    int chunks;                                     // of kExpandChunk
    const ScheduleHead* unless_few;                 // nothing to do where its few_passes is set; NULL: there is
};

// First position that a new token of request r sees, and the end.
__device__ __forceinline__ int2 seen_rows(const ExpandParams& p, int r)
{
    const int q = p.cu_q[r + 1] - p.cu_q[r], kv = p.kv_len[r];
    if (q <= 0) return make_int2(0, 0);
    const int64_t cap = (int64_t)p.table_cols << p.page_shift;
    return make_int2(p.window ? max(kv - q + 1 - p.window, 0) : 0, (int)min((int64_t)kv, cap));
}

// kScaled: times the global scales, bf16; else without them, K as bf16 and V as halves.
template <bool kScaled>
__global__ void __launch_bounds__(kExpandThreads) expand_kernel(const __grid_constant__ ExpandParams p)
{
    extern __shared__ int32_t pre[];                // [requests + 1] pages before each request
    __shared__ int s_sums[kExpandThreads / 32];
    griddep_launch_dependents();
    griddep_wait();
    if (p.unless_few && p.unless_few->few_passes) return;
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
    const float g[2] = {kScaled ? *p.c.k_g : 1.0f, kScaled ? *p.c.v_g : 1.0f};
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int i = (int)(u / (2 * p.chunks)), part = (int)(u - (int64_t)i * 2 * p.chunks);
        const bool is_v = part >= p.chunks, halves = is_v && !kScaled;
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
                const __half2 h = e2m1x2_to_f16x2(w[x] >> (8 * y));
                // (code times scale is exact, in bf16 and as halves)
                if (halves) {
                    const __half2 z = __hmul2(h, __float2half2_rn(f));
                    o[y] = *reinterpret_cast<const uint32_t*>(&z);
                } else {
                    const float2 v = __half22float2(h);
                    o[y] = kScaled ? cvt_bf16x2(v.x * f * gg, v.y * f * gg) : cvt_bf16x2(v.x * f, v.y * f);
                }
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
                              bool scaled, bool unless_few, int num_sms, cudaStream_t stream)
{
    ExpandParams p = {};
    p.unless_few = unless_few ? static_cast<const ScheduleHead*>(step.schedule) : nullptr;
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
    p.halves = (int)(cache.kv_heads * cache.page_size * cache.head_dim / 8);
    p.chunks = (p.halves + kExpandChunk - 1) / kExpandChunk;
    return launch_programmatic(scaled ? expand_kernel<true> : expand_kernel<false>, dim3((unsigned)num_sms * 8), dim3(kExpandThreads),
                               (size_t)(step.requests + 1) * 4, stream, p);
}

}  // namespace nvfp4
