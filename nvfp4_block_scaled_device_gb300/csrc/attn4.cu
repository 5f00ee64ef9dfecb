// Attention over the 4-bit cache, on warp-level MMAs:
//   s_j = scale * q.k_j over the keys j a row sees, out = sum_j softmax_j(s) v_j,
// with k_j = E2M1 code * E4M3 scale * *k_g, v_j likewise.
//
// A decode step is few rows against many keys: 72 bytes of keys and as many of
// values a key of 128 columns, each read once, and what has to be done for them
// is to turn codes into numbers.  So nothing is written back to shared memory:
// every warp has its own ring of groups of 16 keys (cp.async), turns a group's
// codes into the fragments of mma.m16n8k16 in registers (cvt of two codes to two
// halves, times the scale: six bits of significand, exact in half precision)
// and multiplies
//   S^T = K Q^T      16 keys x 8 rows at a time, over 16 columns
//   O^T += V^T P^T   16 columns x 8 rows at a time, over the 16 keys
// so that 8 rows, not 16, fill an instruction.  The order of a product's inner
// index is free as long as both operands have it: a lane takes 32 columns of a
// key in a row (one 16-byte read), and of the values 16 columns of four keys;
// P^T comes out of S^T by transposing its 8 x 8 blocks (movmatrix).
//   Softmax: 2^(c s - m), c = scale * log2(e) * *k_g, statistics and sums in
// binary32; m only moves when a score has outgrown it by 2^8, which one vote per
// group finds out.  P is rounded to half precision, 2^-11 relative, and carried
// 2^6 above 1 so that what is below 2^-20 of the largest loses bits only.  Q is
// scaled by a power of two to the top of half precision's range (its bf16 bits
// fit down to 2^-28 of the row's largest).
//
// Work is cut as in attn.cu (the plan's schedule: equal key tiles per CTA).  The
// warps of a CTA take the groups of its piece of an item in turn, with rows,
// maxima and sums of their own, and are joined in shared memory at its end; the
// pieces of an item that several CTAs share are joined by the last of them, in
// CTA order.  No CTA waits for another.
//
// More than 8 kNT rows of an item take several passes over its keys.
#include <cuda_fp16.h>

#include "attn.h"
#include "attn_walk.cuh"
#include "common.cuh"
#include "internal.h"
#include "kv4.h"

namespace nvfp4 {
namespace {

constexpr int kHalf = 16;              // keys of a page's smallest run, and of an MMA
constexpr int kChunk = 2 * kHalf;      // keys of a ring's stage
constexpr float kLazy = 8.0f;          // log2 of the growth that P may carry
constexpr float kLift = 6.0f;          // log2 of P at m
constexpr float kLog2e = 1.4426950408889634f;

template <int kDP, int kNT>
struct Cfg4 {
    static constexpr int kWarps = kNT == 1 ? 16 : 8;
    static constexpr int kStages = kNT == 1 ? 2 : 3;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kRows = 8 * kNT;
    static constexpr int kAtOnce = kNT == 1 ? 2 : 1;             // halves of a chunk worked on together
    static constexpr int kRowBytes = kDP / 2;
    static constexpr int kCodes = kHalf * kRowBytes;             // of K or V of half a chunk
    static constexpr int kScales = kHalf * kDP / 16;
    static constexpr int kHalfBytes = 2 * (kCodes + kScales);    // K, V, scales of K, scales of V
    static constexpr int kStageBytes = 2 * kHalfBytes;
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    // O of all warps for kJoin tiles of 8 rows: two rows and 4 words of padding a line
    static constexpr int kJoin = 16 / kWarps;
    static constexpr int kLine = 2 * kDP + 4;
    static constexpr int kWarpO = kJoin * 4 * kLine;             // floats
    static constexpr int kOffO = kRing;
    static constexpr int kOffQ = kOffO + kWarps * kWarpO * 4;    // Q's rows (bf16), then (kNT > 1) its fragments
    static constexpr int kOffFrag = kOffQ + kRows * kDP * 2;
    static constexpr int kOffM = kOffFrag + (kNT > 1 ? kNT * (kDP / 16) * 32 * 8 : 0);
    static constexpr int kSmem = kOffM + kWarps * kRows * 2 * 4;
    static constexpr int kQVecs = kRows * kDP / 8 / kThreads > 0 ? kRows * kDP / 8 / kThreads : 1;
    static_assert(kSmem <= 232448 - 1024, "shared memory per block");
};

// One pass of a CTA over the keys of a piece, for up to kRows of its rows.  The
// first warp writes them down two ahead, in shared memory, for all to read.
struct Pass {
    int valid;
    int rows, r0;            // rows of the piece's item; the pass is for rows r0 ..
    int tok0, pos0, hk;
    int kv_end, key_end;     // no row sees keys from kv_end on; the piece ends at key_end
    int lo, lo_all, hi_all;  // some row sees key lo; all see lo_all .. hi_all - 1
    int kb, ke;              // keys of the pass (kb a multiple of kChunk)
    int cta0, parts;
    int last;                // of the piece
    const int32_t* table;    // the request's pages
};

struct Params4 {
    AttnArgs a;
    const uint8_t* k;
    const uint8_t* v;
    const uint8_t* k_sf;
    const uint8_t* v_sf;
    uint32_t page_stride, sf_stride;           // bytes
    const __nv_bfloat16* q;
    int64_t ldq, hq;
    int pages, page_shift;
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }
// Eight E2M1 codes -> four f16x2 (exact).  The bytes are taken apart in the asm
// block, where they cost nothing: from shifts the conversions take 2.5
// instructions each instead of one.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t* out)
{
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
        : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
        : "r"(w));
}
__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi)
{
    uint32_t y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t b)
{
    uint32_t y;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"((uint16_t)b));
    return y;
}
// 16 (8) bytes of global memory into shared memory, kAt bytes on from both
// addresses; `real` 0: zeros instead.
template <int kAt>
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t real)
{
    asm volatile("cp.async.cg.shared.global [%0 + %3], [%1 + %3], 16, %2;" ::"r"(dst), "l"(src), "r"(real), "n"(kAt) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src, uint32_t real)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(real) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// The passes of CTA `cta` in order.
template <int kRows>
struct Passes {
    Pieces pieces;
    Piece p;
    int r0, rows;

    __device__ __forceinline__ Passes(const AttnArgs& a, int cta) : pieces(a, cta), r0(0), rows(0) {}
    __device__ __forceinline__ void next(const AttnArgs& a, Pass* out, int lane)
    {
        r0 += kRows;
        bool valid = true;
        if (r0 >= rows) {
            valid = pieces.next(p);
            r0 = 0;
            rows = valid ? p.n_tok * a.group : 0;
        }
        if (lane) return;
        out->valid = valid;
        if (!valid) return;
        const int t0 = r0 / a.group, t1 = (min(rows, r0 + kRows) - 1) / a.group;
        const int hi = min(p.pos0 + t1 + 1, p.kv_end), key_end = min((p.tile0 + p.n) * kAttnKeys, p.kv_end);
        out->rows = rows;
        out->r0 = r0;
        out->tok0 = p.tok0;
        out->pos0 = p.pos0;
        out->hk = p.hk;
        out->kv_end = p.kv_end;
        out->key_end = key_end;
        out->lo = a.window ? max(p.pos0 + t0 + 1 - a.window, 0) : 0;
        out->lo_all = a.window ? max(p.pos0 + t1 + 1 - a.window, 0) : 0;
        out->hi_all = min(p.pos0 + t0 + 1, key_end);
        out->kb = max(p.tile0 * kAttnKeys, out->lo) & ~(kChunk - 1);
        out->ke = min(key_end, hi);
        out->cta0 = p.cta0;
        out->parts = p.parts;
        out->last = r0 + kRows >= rows;
        out->table = a.block_table + p.req * a.table_ld;
    }
};

template <int kDP, int kNT, bool kFull>
__global__ void __launch_bounds__(Cfg4<kDP, kNT>::kThreads, 1) attn4_kernel(const __grid_constant__ Params4 prm)
{
    using C = Cfg4<kDP, kNT>;
    constexpr int kSteps = kDP / 16;           // MMAs over a key's columns; of 16 columns of O
    constexpr int kH = C::kAtOnce;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_last;
    __shared__ Pass s_pass[3];
    const AttnArgs& a = prm.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
    const int cta = blockIdx.x, D = kFull ? kDP : a.head_dim, nb = D / 16;
    uint8_t* ring = smem + warp * (C::kStages * C::kStageBytes);
    const uint32_t ring_addr = smem_u32(ring);
    float* o_all = reinterpret_cast<float*>(smem + C::kOffO);
    float2* m_all = reinterpret_cast<float2*>(smem + C::kOffM);            // [warp][row] m, l
    uint4* q_rows = reinterpret_cast<uint4*>(smem + C::kOffQ);             // [row][kDP / 8]
    uint2* q_frag = reinterpret_cast<uint2*>(smem + C::kOffFrag);          // [tile][step][lane]

    griddep_launch_dependents();
    if (!kFull)                                 // the columns that no copy writes are zeros
        for (int i = tid; i < C::kRing / 16; i += C::kThreads) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
    griddep_wait();
    Passes<C::kRows> passes(a, cta);            // (the first warp's)
    if (warp == 0) {
        passes.next(a, &s_pass[0], lane);
        passes.next(a, &s_pass[1], lane);
    }
    __syncthreads();

    // this lane's share of a half's copies: 16 bytes of codes (or, where a row is
    // not whole sixteens, 8) and of scales (16 keys' are D bytes)
    const int chunk = kFull || D % 32 == 0 ? 16 : 8, per_row = D / 2 / chunk, chunks = kHalf * per_row;
    int to[kFull ? 1 : 4];
#pragma unroll
    for (int i = 0; i < (kFull ? 1 : 4); i++) {
        const int c = lane + 32 * i;
        to[i] = (c / per_row) * C::kRowBytes + (c % per_row) * chunk;
    }
    const int sf_half = lane >> 4, sf_at = (lane & 7) * 16;
    const uint32_t sf_to = sf_half * C::kHalfBytes + 2 * C::kCodes + (lane >> 3 & 1 ? C::kScales : 0) + sf_at;
    const uint8_t* const sf_base = (lane >> 3 & 1 ? prm.v_sf : prm.k_sf) + sf_at;
    const float k_g = *a.k_g, v_g = *a.v_g;
    const int key_row = (g >> 1) + 4 * (g & 1);            // key of a half that is row g of its S^T (and 8 + it)
    const int page_mask = (1 << prm.page_shift) - 1;

    // chunks of this warp in a pass
    auto chunks_of = [&](const Pass& x) {
        const int n = x.valid && x.ke > x.kb ? (x.ke - x.kb + kChunk - 1) / kChunk : 0;
        return n > warp ? (n - warp + C::kWarps - 1) / C::kWarps : 0;
    };
    // page ids of the halves of 16 chunks of this warp from chunk i on, a lane each
    auto load_ids = [&](const Pass& x, int i, int n) {
        const int c = i + (lane >> 1), k = x.kb + (warp + c * C::kWarps) * kChunk + (lane & 1) * kHalf;
        return c < n && k < x.ke ? x.table[k >> prm.page_shift] : -1;
    };
    // Copies of chunk i of a pass into a stage.  A page that the cache does not
    // have is zeros; a half past the pass's end is masked as a whole.
    auto copy = [&](const Pass& x, int i, int ids, int stage) {
        const int k0 = x.kb + (warp + i * C::kWarps) * kChunk;
        const uint32_t st = ring_addr + stage * C::kStageBytes;
        const int row0 = (x.hk << prm.page_shift) + (k0 & page_mask);      // (of the page; the second half's: 16 on, or 0)
        const int row1 = (x.hk << prm.page_shift) + ((k0 + kHalf) & page_mask);
        const uint32_t id0 = __shfl_sync(0xffffffffu, ids, 2 * (i & 15)), id1 = __shfl_sync(0xffffffffu, ids, 2 * (i & 15) + 1);
        const bool real0 = id0 < (uint32_t)prm.pages, real1 = id1 < (uint32_t)prm.pages;
        const uint32_t page0 = real0 ? id0 : 0u, page1 = real1 ? id1 : 0u;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const uint64_t at = (uint64_t)(h ? page1 : page0) * prm.page_stride + (uint32_t)((h ? row1 : row0) * (D / 2));
            const bool real = h ? real1 : real0;
            const uint32_t sh = st + h * C::kHalfBytes + to[0];
            const uint8_t* ck = prm.k + lane * chunk + at;
            const uint8_t* cv = prm.v + lane * chunk + at;
            if (kFull) {
                const int n = real ? 16 : 0;
                copy16<0>(sh, ck, n);
                if (kDP == 128) copy16<512>(sh, ck, n);
                copy16<0>(sh + C::kCodes, cv, n);
                if (kDP == 128) copy16<512>(sh + C::kCodes, cv, n);
            } else if (chunk == 16) {
#pragma unroll
                for (int y = 0; y < (kDP == 128 ? 2 : 1); y++)
                    if (lane + 32 * y < chunks) {
                        copy16<0>(sh + to[kFull ? 0 : y] - to[0], ck + 512 * y, real ? 16 : 0);
                        copy16<0>(sh + C::kCodes + to[kFull ? 0 : y] - to[0], cv + 512 * y, real ? 16 : 0);
                    }
            } else {
#pragma unroll
                for (int y = 0; y < (kDP == 128 ? 4 : 2); y++)
                    if (lane + 32 * y < chunks) {
                        copy8(sh + to[kFull ? 0 : y] - to[0], ck + 256 * y, real ? 8 : 0);
                        copy8(sh + C::kCodes + to[kFull ? 0 : y] - to[0], cv + 256 * y, real ? 8 : 0);
                    }
            }
        }
        if (sf_at < D)
            copy16<0>(st + sf_to, sf_base + (uint64_t)(sf_half ? page1 : page0) * prm.sf_stride + (uint32_t)((sf_half ? row1 : row0) * nb),
                      (sf_half ? real1 : real0) ? 16 : 0);
        copies_end();
    };
    // Q's rows of a pass, a share of each thread
    auto load_q = [&](const Pass& x, uint4* v) {
#pragma unroll
        for (int y = 0; y < C::kQVecs; y++) {
            const int i = tid + y * C::kThreads, row = i / (kDP / 8), col = 8 * (i % (kDP / 8)), r = x.r0 + row;
            v[y] = make_uint4(0, 0, 0, 0);
            if (x.valid && row < C::kRows && r < x.rows && col < D) {
                const int t = r / a.group;
                v[y] = *reinterpret_cast<const uint4*>(prm.q + (int64_t)(x.tok0 + t) * prm.ldq +
                                                       (int64_t)(x.hk * a.group + r - t * a.group) * prm.hq + col);
            }
        }
    };
    auto store_q = [&](const uint4* v) {
#pragma unroll
        for (int y = 0; y < C::kQVecs; y++)
            if (tid + y * C::kThreads < C::kRows * (kDP / 8)) q_rows[tid + y * C::kThreads] = v[y];
    };

    // The ring runs through the passes: while a pass's last chunks are worked on
    // and joined, the first ones of the next are on their way.
    int stage_in = 0, stage_out = 0, ahead = 0;            // next stage to fill, to read; stages filled
    int issue_i = 0, issue_n, ids, ids_next;
    bool in_next = false;                                  // what is issued is of the next pass
    issue_n = chunks_of(s_pass[0]);
    ids = load_ids(s_pass[0], 0, issue_n);
    {
        uint4 v[C::kQVecs];
        load_q(s_pass[0], v);
        store_q(v);
    }
    __syncthreads();
    int x_pass = 0;
#pragma unroll 1
    for (;; x_pass = x_pass == 2 ? 0 : x_pass + 1) {
        const Pass& cur = s_pass[x_pass];
        const Pass& nxt = s_pass[x_pass == 2 ? 0 : x_pass + 1];
        if (!cur.valid) break;
        const int mine = chunks_of(cur), next_n = chunks_of(nxt);
        if (in_next) in_next = false;                      // (issue_i, issue_n and ids are this pass's)
        ids_next = load_ids(nxt, 0, next_n);
        auto issue = [&]() {
            if (issue_i == issue_n && !in_next) {
                in_next = true;
                issue_i = 0;
                issue_n = next_n;
                ids = ids_next;
            }
            if (issue_i == issue_n) return;
            const Pass& from = in_next ? nxt : cur;
            if (issue_i && (issue_i & 15) == 0) ids = load_ids(from, issue_i, issue_n);
            copy(from, issue_i++, ids, stage_in);
            stage_in = stage_in + 1 == C::kStages ? 0 : stage_in + 1;
            ahead++;
        };
#pragma unroll 1
        for (int y = ahead; y < C::kStages; y++) issue();

        // Q of the pass: row g of tile n, columns kDP / 4 * j .. of this lane
        uint32_t q[kNT == 1 ? 2 * kSteps : 1];
        float cf[kNT][2];
#pragma unroll
        for (int n = 0; n < kNT; n++) {
            uint32_t raw[kDP / 8];                         // this lane's kDP / 4 columns
            float amax = 0.0f;
#pragma unroll
            for (int x = 0; x < kDP / 32; x++) {
                const uint4 y = q_rows[(8 * n + g) * (kDP / 8) + j * (kDP / 32) + x];
                raw[4 * x] = y.x, raw[4 * x + 1] = y.y, raw[4 * x + 2] = y.z, raw[4 * x + 3] = y.w;
            }
#pragma unroll
            for (int x = 0; x < kDP / 8; x++) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(raw[x])), fabsf(bf16_hi(raw[x]))));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // times 2^(141 - e), e the largest's biased exponent: it is then
            // 2^14 .. 2^15; and back in the row's factor.  A negative scale's sign
            // goes into Q; a zero scale is any tiny factor (no 0 * inf where masked).
            const int e = max((int)(__float_as_uint(amax) >> 23), 15);
            const float up = __uint_as_float((uint32_t)(268 - e) << 23 | (__float_as_uint(a.scale) & 0x80000000u));
            const float down = __uint_as_float((uint32_t)(e - 14) << 23);
#pragma unroll
            for (int x = 0; x < kDP / 8; x++) raw[x] = cvt_f16x2(bf16_lo(raw[x]) * up, bf16_hi(raw[x]) * up);
            if (kNT == 1) {
#pragma unroll
                for (int x = 0; x < kDP / 8; x++) q[kNT == 1 ? x : 0] = raw[x];
            } else if (warp == n) {
#pragma unroll
                for (int s = 0; s < kSteps; s++) q_frag[(n * kSteps + s) * 32 + lane] = make_uint2(raw[2 * s], raw[2 * s + 1]);
            }
            const float c = fmaxf(fabsf(a.scale) * kLog2e * k_g * down, 1.17549435e-38f);
            cf[n][0] = __shfl_sync(0xffffffffu, c, 8 * j);
            cf[n][1] = __shfl_sync(0xffffffffu, c, 8 * j + 4);
        }
        if (kNT > 1) __syncthreads();

        // nm: kLift - m; top: the score from which m moves
        float o[kNT][kSteps][4], m[kNT][2], nm[kNT][2], limit[kNT][2], l[kNT][2];
#pragma unroll
        for (int n = 0; n < kNT; n++) {
#pragma unroll
            for (int s = 0; s < kSteps; s++) o[n][s][0] = o[n][s][1] = o[n][s][2] = o[n][s][3] = 0.0f;
#pragma unroll
            for (int y = 0; y < 2; y++) m[n][y] = limit[n][y] = -INFINITY, nm[n][y] = l[n][y] = 0.0f;
        }
        const int lo_all = cur.lo_all, hi_all = cur.hi_all;
        int kc = cur.kb + warp * kChunk;                   // first key of the chunk
#pragma unroll 1
        for (int i = 0; i < mine; i++, kc += C::kWarps * kChunk) {
            if (C::kStages == 3 && ahead == 3) copies_wait<2>();
            else if (ahead >= 2) copies_wait<1>();
            else copies_wait<0>();
            __syncwarp();
#pragma unroll 1
            for (int h0 = 0; h0 < 2; h0 += kH) {
                const uint8_t* st = ring + stage_out * C::kStageBytes + h0 * C::kHalfBytes;
                const int k0 = kc + h0 * kHalf;
                const bool edge = k0 < lo_all || k0 + kH * kHalf > hi_all;
                // ---- S^T = K Q^T
                float s[kH][kNT][4];
#pragma unroll
                for (int h = 0; h < kH; h++) {
                    const uint8_t* sk = st + h * C::kHalfBytes;
                    uint32_t w[2][kDP / 32];               // codes of keys key_row and 8 + key_row
                    __half2 sc[2];                         // their scales (128 columns: of two blocks)
#pragma unroll
                    for (int y = 0; y < 2; y++) {
                        const int key = key_row + 8 * y;
                        const uint8_t* sf = sk + 2 * C::kCodes + key * nb;
                        if (kDP == 128) {
                            const uint4 x = *reinterpret_cast<const uint4*>(sk + key * C::kRowBytes + j * 16);
                            w[y][0] = x.x, w[y][1] = x.y, w[y][kDP / 32 - 2] = x.z, w[y][kDP / 32 - 1] = x.w;
                            uint32_t b;
                            if (kFull) {
                                b = *reinterpret_cast<const uint16_t*>(sf + 2 * j);
                            } else {
                                b = 2 * j < nb ? sf[2 * j] : 0u;
                                b |= 2 * j + 1 < nb ? (uint32_t)sf[2 * j + 1] << 8 : 0u;
                            }
                            sc[y] = as_half2(e4m3x2_to_f16x2(b));
                        } else {
                            const uint2 x = *reinterpret_cast<const uint2*>(sk + key * C::kRowBytes + j * 8);
                            w[y][0] = x.x, w[y][1] = x.y;
                            sc[y] = as_half2(e4m3x2_to_f16x2(j < nb ? sf[j] : 0u));
                        }
                    }
#pragma unroll
                    for (int n = 0; n < kNT; n++) s[h][n][0] = s[h][n][1] = s[h][n][2] = s[h][n][3] = 0.0f;
#pragma unroll
                    for (int x = 0; x < kDP / 32; x++) {   // a word of codes: two MMAs
                        uint32_t f[2][4];
#pragma unroll
                        for (int y = 0; y < 2; y++) {
                            e2m1x8_to_f16x2(w[y][x], f[y]);
                            const __half2 z = kDP == 128 && x >= 2 ? __high2half2(sc[y]) : __low2half2(sc[y]);
#pragma unroll
                            for (int u = 0; u < 4; u++) f[y][u] = as_u32(__hmul2(as_half2(f[y][u]), z));
                        }
#pragma unroll
                        for (int u = 0; u < 2; u++) {
                            const uint32_t fa[4] = {f[0][2 * u], f[1][2 * u], f[0][2 * u + 1], f[1][2 * u + 1]};
#pragma unroll
                            for (int n = 0; n < kNT; n++) {
                                if (kNT == 1) {
                                    mma16816(s[h][n], fa, q[kNT == 1 ? 4 * x + 2 * u : 0], q[kNT == 1 ? 4 * x + 2 * u + 1 : 0]);
                                } else {
                                    const uint2 b = q_frag[(n * kSteps + 2 * x + u) * 32 + lane];
                                    mma16816(s[h][n], fa, b.x, b.y);
                                }
                            }
                        }
                    }
                }
                // ---- softmax
                if (edge) {
#pragma unroll
                    for (int h = 0; h < kH; h++) {
#pragma unroll
                        for (int n = 0; n < kNT; n++) {
#pragma unroll
                            for (int y = 0; y < 4; y++) {
                                const int pos = cur.pos0 + (cur.r0 + 8 * n + 2 * j + (y & 1)) / a.group;
                                const int key = k0 + h * kHalf + key_row + 8 * (y >> 1);
                                const bool seen = key <= pos && key < cur.key_end && (!a.window || key > pos - a.window);
                                if (!seen) s[h][n][y] = -INFINITY;
                            }
                        }
                    }
                }
                bool up = false;
#pragma unroll
                for (int n = 0; n < kNT; n++) {
#pragma unroll
                    for (int y = 0; y < 2; y++) {
                        float top = fmaxf(s[0][n][y], s[0][n][y + 2]);
                        if (kH == 2) top = fmaxf(top, fmaxf(s[kH - 1][n][y], s[kH - 1][n][y + 2]));
                        up |= top > limit[n][y];
                    }
                }
                if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                    for (int n = 0; n < kNT; n++) {
#pragma unroll
                        for (int y = 0; y < 2; y++) {
                            float top = fmaxf(s[0][n][y], s[0][n][y + 2]);
                            if (kH == 2) top = fmaxf(top, fmaxf(s[kH - 1][n][y], s[kH - 1][n][y + 2]));
#pragma unroll
                            for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                            top = fmaxf(top * cf[n][y], m[n][y]);
                            const float f = m[n][y] == -INFINITY ? 0.0f : ex2(m[n][y] - top);
                            m[n][y] = top;
                            nm[n][y] = top == -INFINITY ? 0.0f : kLift - top;
                            limit[n][y] = (top + kLazy) / cf[n][y];
                            l[n][y] *= f;
#pragma unroll
                            for (int x = 0; x < kSteps; x++) {
                                o[n][x][y] *= f;
                                o[n][x][y + 2] *= f;
                            }
                        }
                    }
                }
                uint32_t pt[kH][kNT][2];
#pragma unroll
                for (int h = 0; h < kH; h++) {
#pragma unroll
                    for (int n = 0; n < kNT; n++) {
                        float e[4];
#pragma unroll
                        for (int y = 0; y < 4; y++) {
                            e[y] = ex2(fmaf(s[h][n][y], cf[n][y & 1], nm[n][y & 1]));
                            l[n][y & 1] += e[y];
                        }
                        pt[h][n][0] = transpose8x8(cvt_f16x2(e[0], e[1]));
                        pt[h][n][1] = transpose8x8(cvt_f16x2(e[2], e[3]));
                    }
                }
                // ---- O^T += V^T P^T: keys j, j + 4 and j + 8, j + 12 of a half, columns kDP / 8 * g ..
                constexpr int kVW = kDP / 64;              // words of a key's codes
#pragma unroll
                for (int h = 0; h < kH; h++) {
                    const uint8_t* sv = st + h * C::kHalfBytes + C::kCodes;
                    const uint8_t* sf = sv + C::kCodes + C::kScales;
                    uint32_t v[4][kVW];
                    __half2 vs[2];
                    const int blk = kDP == 128 ? g : g >> 1;
                    uint32_t b[4];
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        const int key = j + 4 * u;
                        if (kVW == 2) {
                            const uint2 x = *reinterpret_cast<const uint2*>(sv + key * C::kRowBytes + g * 8);
                            v[u][0] = x.x, v[u][kVW - 1] = x.y;
                        } else {
                            v[u][0] = *reinterpret_cast<const uint32_t*>(sv + key * C::kRowBytes + g * 4);
                        }
                        b[u] = kFull || blk < nb ? sf[key * nb + blk] : 0u;
                    }
                    if (edge) {                            // a value that no row sees may be anything
                        const int lo = cur.lo - k0 - h * kHalf, ke = cur.ke - k0 - h * kHalf;
#pragma unroll
                        for (int u = 0; u < 4; u++)
                            if (j + 4 * u < lo || j + 4 * u >= ke) b[u] = 0u;
                    }
                    vs[0] = as_half2(e4m3x2_to_f16x2(__byte_perm(b[0], b[1], 0x3340)));
                    vs[1] = as_half2(e4m3x2_to_f16x2(__byte_perm(b[2], b[3], 0x3340)));
#pragma unroll
                    for (int y = 0; y < kVW; y++) {
                        uint32_t even[2][4], odd[2][4];    // two keys side by side, of even and odd columns
#pragma unroll
                        for (int u = 0; u < 2; u++) {
                            const uint32_t x0 = v[2 * u][y], x1 = v[2 * u + 1][y];
                            e2m1x8_to_f16x2((x0 & 0x0f0f0f0fu) | (x1 << 4 & 0xf0f0f0f0u), even[u]);
                            e2m1x8_to_f16x2((x0 >> 4 & 0x0f0f0f0fu) | (x1 & 0xf0f0f0f0u), odd[u]);
                        }
#pragma unroll
                        for (int x = 0; x < 4; x++) {
                            uint32_t f[4];
#pragma unroll
                            for (int u = 0; u < 2; u++) {
                                f[2 * u] = as_u32(__hmul2(as_half2(even[u][x]), vs[u]));
                                f[2 * u + 1] = as_u32(__hmul2(as_half2(odd[u][x]), vs[u]));
                            }
#pragma unroll
                            for (int n = 0; n < kNT; n++) mma16816(o[n][4 * y + x], f, pt[h][n][0], pt[h][n][1]);
                        }
                    }
                }
            }
            __syncwarp();                                  // the stage has been read
            stage_out = stage_out + 1 == C::kStages ? 0 : stage_out + 1;
            ahead--;
            issue();
        }

        // ---- the warps' shares of the pass together
        const int r0 = cur.r0, rows = cur.rows, tok0 = cur.tok0, hk = cur.hk;
        const bool whole = cur.parts == 1;
        float* part = a.partials + (2 * cta + (cur.cta0 == cta ? 1 : 0)) * kAttnSlotFloats;
        uint4 q_next[C::kQVecs];
        load_q(nxt, q_next);
        if (warp == 0) passes.next(a, &s_pass[x_pass == 0 ? 2 : x_pass - 1], lane);
#pragma unroll
        for (int n = 0; n < kNT; n++) {
#pragma unroll
            for (int y = 0; y < 2; y++) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[n][y] += __shfl_xor_sync(0xffffffffu, l[n][y], x);
                if (g == 0) m_all[warp * C::kRows + 8 * n + 2 * j + y] = make_float2(m[n][y], l[n][y]);
            }
        }
#pragma unroll
        for (int n0 = 0; n0 < kNT; n0 += C::kJoin) {
            if (n0) __syncthreads();
#pragma unroll
            for (int n = n0; n < n0 + C::kJoin; n++) {
#pragma unroll
                for (int y = 0; y < 2; y++) {
                    float4* to4 = reinterpret_cast<float4*>(o_all + warp * C::kWarpO + ((n - n0) * 4 + j) * C::kLine + y * kDP +
                                                            g * (kDP / 8));
#pragma unroll
                    for (int x = 0; x < kSteps; x += 2)
                        to4[x / 2] = make_float4(o[n][x][y], o[n][x][y + 2], o[n][x + 1][y], o[n][x + 1][y + 2]);
                }
            }
            __syncthreads();
            // a thread adds two columns of a row over the warps
            for (int x = tid; x < C::kJoin * 8 * (kDP / 2); x += C::kThreads) {
                const int rr = x / (kDP / 2), col = 2 * (x % (kDP / 2)), r = r0 + 8 * n0 + rr;
                if (r >= rows || col >= D) continue;
                const float* from = o_all + (rr >> 1) * C::kLine + (rr & 1) * kDP + col;
                float2 ml[C::kWarps], acc = make_float2(0.0f, 0.0f);
                float top = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int y = 0; y < C::kWarps; y++) {
                    ml[y] = m_all[y * C::kRows + 8 * n0 + rr];
                    top = fmaxf(top, ml[y].x);
                }
                const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
                for (int y = 0; y < C::kWarps; y++) {
                    const float f = ex2(ml[y].x - ref);
                    const float2 e = *reinterpret_cast<const float2*>(from + y * C::kWarpO);
                    sum += ml[y].y * f;
                    acc.x += e.x * f;
                    acc.y += e.y * f;
                }
                const int t = r / a.group, head = hk * a.group + r - t * a.group;
                if (whole) {
                    const float inv = sum == 0.0f ? 0.0f : v_g / sum;
                    *reinterpret_cast<uint32_t*>(a.out + (int64_t)(tok0 + t) * a.ldo + (int64_t)head * a.ho + col) =
                        sum == 0.0f ? 0u : cvt_bf16x2(acc.x * inv, acc.y * inv);
                    if (col == 0 && a.lse)
                        a.lse[(int64_t)(tok0 + t) * a.heads + head] =
                            sum == 0.0f ? -INFINITY : (top - kLift + log2f(sum)) * 0.6931471805599453f;
                } else {
                    __stcg(reinterpret_cast<float2*>(part + r * kDP + col), acc);
                    if (col == 0) __stcg(reinterpret_cast<float2*>(part + kAttnSlotRows * kDP + 2 * r), make_float2(top, sum));
                }
            }
        }
        store_q(q_next);
        const int cta0 = cur.cta0, parts = cur.parts;
        const bool join = !whole && cur.last;
        __syncthreads();                                   // the next pass's rows; this one's O have been read
        if (!join) continue;

        // ---- a shared item: the last of its CTAs adds the parts up
        int* ticket = a.tickets + cta0 * 8;
        if (tid == 0) {
            s_last = atom_add_acq_rel(ticket, 1) == parts - 1;
            if (s_last) *ticket = 0;
        }
        __syncthreads();
        const bool mine_to_join = s_last;
        __syncthreads();
        if (!mine_to_join) continue;
        // part i of the item is in slot 2 (cta0 + i), the first in 2 cta0 + 1
        auto slot_of = [&](int i) { return a.partials + (2 * (cta0 + i) + (i == 0 ? 1 : 0)) * kAttnSlotFloats; };
        for (int x = tid; x < rows * (kDP / 2); x += C::kThreads) {
            const int r = x / (kDP / 2), col = 2 * (x % (kDP / 2));
            if (col >= D) continue;
            const int t = r / a.group, head = hk * a.group + r - t * a.group;
            float top = -INFINITY, sum = 0.0f;
            float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll 1
            for (int i0 = 0; i0 < parts; i0 += 8) {
                float2 ml[8], e[8];
#pragma unroll
                for (int u = 0; u < 8; u++) {
                    const float* from = slot_of(min(i0 + u, parts - 1));
                    ml[u] = __ldcg(reinterpret_cast<const float2*>(from + kAttnSlotRows * kDP + 2 * r));
                    e[u] = __ldcg(reinterpret_cast<const float2*>(from + r * kDP + col));
                    if (i0 + u >= parts) ml[u] = make_float2(-INFINITY, 0.0f);
                }
                float most = top;
#pragma unroll
                for (int u = 0; u < 8; u++) most = fmaxf(most, ml[u].x);
                const float f0 = top == -INFINITY ? 0.0f : ex2(top - most);
                acc.x *= f0;
                acc.y *= f0;
                sum *= f0;
                top = most;
#pragma unroll
                for (int u = 0; u < 8; u++) {
                    if (ml[u].y == 0.0f) continue;         // no key of this part
                    const float f = ml[u].x == -INFINITY ? 0.0f : ex2(ml[u].x - top);
                    acc.x += f * e[u].x;
                    acc.y += f * e[u].y;
                    sum += f * ml[u].y;
                }
            }
            const float inv = sum == 0.0f ? 0.0f : v_g / sum;
            *reinterpret_cast<uint32_t*>(a.out + (int64_t)(tok0 + t) * a.ldo + (int64_t)head * a.ho + col) =
                sum == 0.0f ? 0u : cvt_bf16x2(acc.x * inv, acc.y * inv);
            if (col == 0 && a.lse)
                a.lse[(int64_t)(tok0 + t) * a.heads + head] =
                    sum == 0.0f ? -INFINITY : (top - kLift + log2f(sum)) * 0.6931471805599453f;
        }
    }
    copies_wait<0>();
    if (a.cu_end) {
        // the rows past the step's last token, a warp to a row
        const int vecs = D / 8, n = a.heads * vecs;
        for (int64_t t = max(*a.cu_end, 0) + cta + (int)gridDim.x * warp; t < a.tokens; t += gridDim.x * C::kWarps) {
            for (int x = lane; x < n; x += 32) {
                const int h = x / vecs;
                *reinterpret_cast<uint4*>(a.out + t * a.ldo + h * a.ho + 8 * (x - h * vecs)) = make_uint4(0, 0, 0, 0);
            }
            if (a.lse)
                for (int h = lane; h < a.heads; h += 32) a.lse[t * a.heads + h] = -INFINITY;
        }
    }
}

template <int kDP, int kNT, bool kFull>
cudaError_t launch4(const Params4& p, int ctas, cudaStream_t stream)
{
    using C = Cfg4<kDP, kNT>;
    static int attr_set_for_device[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && !attr_set_for_device[dev]) {
        e = cudaFuncSetAttribute(attn4_kernel<kDP, kNT, kFull>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        attr_set_for_device[dev] = 1;
    }
    return launch_programmatic(attn4_kernel<kDP, kNT, kFull>, dim3((unsigned)ctas), dim3(C::kThreads), C::kSmem, stream, p);
}

// Rows of a request, on average: one tile of 8, two, or passes of four.
template <int kDP, bool kFull>
cudaError_t launch_rows(const Params4& p, int64_t rows, int ctas, cudaStream_t stream)
{
    return rows <= 8    ? launch4<kDP, 1, kFull>(p, ctas, stream)
           : rows <= 16 ? launch4<kDP, 2, kFull>(p, ctas, stream)
                        : launch4<kDP, 4, kFull>(p, ctas, stream);
}

}  // namespace

cudaError_t launch_attn4(const AttnArgs& args, const nvfp4_kv4_cache_t& cache, const __nv_bfloat16* q, int64_t ldq,
                         int64_t hq, int64_t requests, int num_sms, cudaStream_t stream)
{
    Params4 p = {};
    p.a = args;
    p.k = cache.k;
    p.v = cache.v;
    p.k_sf = cache.k_sf;
    p.v_sf = cache.v_sf;
    p.page_stride = (uint32_t)cache.page_stride;
    p.sf_stride = (uint32_t)cache.sf_stride;
    p.q = q;
    p.ldq = ldq;
    p.hq = hq;
    p.pages = (int)cache.pages;
    while ((1 << p.page_shift) < cache.page_size) p.page_shift++;
    const int ctas = num_sms < kAttnMaxCtas ? num_sms : kAttnMaxCtas;
    const int64_t rows = (args.tokens + requests - 1) / requests * args.group;
    const int d = args.head_dim;
    return d == 128  ? launch_rows<128, true>(p, rows, ctas, stream)
           : d > 64  ? launch_rows<128, false>(p, rows, ctas, stream)
           : d == 64 ? launch_rows<64, true>(p, rows, ctas, stream)
                     : launch_rows<64, false>(p, rows, ctas, stream);
}

}  // namespace nvfp4
