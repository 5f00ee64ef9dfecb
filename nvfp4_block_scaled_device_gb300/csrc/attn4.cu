// Attention over the 4-bit cache, on warp-level MMAs:
//   s_j = scale * q.k_j over the keys j a row sees, out = sum_j softmax_j(s) v_j,
// with k_j = E2M1 code * E4M3 scale * *k_g, v_j likewise.
//
// A decode step is few rows against many keys: 72 bytes of keys and as many of
// values a key of 128 columns, each read once, and what has to be done for them
// is to turn codes into numbers.  So nothing of them goes back to shared or tensor
// memory, where tcgen05.mma would take them from: every warp has its own ring of chunks of
// 32 keys (cp.async), turns a chunk's codes into the fragments of mma.m16n8k16 in
// registers (cvt of two codes to two halves, times the scale: six bits of
// significand, exact in half precision) and multiplies, for each half of the chunk,
//   S^T = K Q^T      16 keys x 8 rows at a time, over 16 columns
//   O^T += V^T P^T   16 columns x 8 rows at a time, over the 16 keys
// so that 8 rows, not 16, fill an instruction.  The order of a product's inner
// index is free as long as both operands have it: a lane takes 32 columns of a
// key in a row (one 16-byte read), and of the values 16 columns of four keys;
// P^T comes out of S^T by transposing its 8 x 8 blocks (movmatrix).
//   Softmax: 2^(c s - m), c = scale * log2(e) * *k_g, statistics and sums in
// binary32; m only moves when a score has outgrown it by 2^8, which one vote per
// chunk finds out.  P is rounded to half precision, 2^-11 relative, and carried
// 2^6 above 1 so that what is below 2^-20 of the largest loses bits only.  Q is
// scaled by a power of two to the top of half precision's range (its bf16 bits
// fit down to 2^-28 of the row's largest).
//
// The work is cut for CTAs and warps in one of two ways:
//   shares of warps  each warp a contiguous share of its CTA's items on the
//                    schedule's second axis (attn.h), whatever the items' lengths; what
//                    several warps have of an item is added up at the CTA's end;
//   passes together  all warps of a CTA take the chunks of its part of an item in
//                    turn, on the first axis, and are joined at the part's end; an item
//                    of more rows than a warp holds takes several passes.
// Parts of an item that several CTAs have are joined by the last of them, in CTA
// order.  No CTA waits for another, and the results do not depend on who is first.
//
// What bounds it (40 query heads on 8 kv heads of 128 columns): HBM in the steady
// state -- twice the keys of one request of 131071 and one of 65537 take 37.5 us
// more for 248 MB, 6.6 TB/s -- where 32 keys are 430 instructions of a warp, 1.3 us for
// the 16 of an SM, against 1.66 us for their bytes (with the bytes of the codes taken
// apart by shifts, 550 instructions and the binding limit).  Beside that some 15 us
// pass from the launch to the end: 4 to 7 until the first keys are there (the
// schedule, the block table, Q, the keys, one after the other, and every warp's
// ring at once), 4 for the spread of the warps' ends, 2 to add up their shares, 3 for
// the parts of other CTAs.  These two requests 53 us; 64 requests of 200 to 8192
// keys 39 (bf16: 95); one of 333 keys 6.9.  With 9 to 16 rows a request 40 (64
// requests of 200 to 4000 keys, 3 tokens each), with 17 to 32, where two warps of a
// scheduler wait for one another's results (255 registers: 8 warps an SM; code for the
// tiles that are there alone gave nothing), 95 (64 of 200 to 8192, 1 to 4 tokens
// each, and the launches that decide about bf16 pages).
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
static_assert(kChunk * kChunksOfTile == kAttnKeys, "chunks of the schedule");
constexpr float kLazy = 8.0f;          // log2 of the growth that P may carry
constexpr float kLift = 6.0f;          // log2 of P at m
constexpr float kLog2e = 1.4426950408889634f;

template <int kDP, int kNT>
struct Cfg4 {
    static constexpr int kWarps = kNT == 1 ? 16 : 8;
    static constexpr int kStages = kNT == 1 ? 2 : 3;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kRows = 8 * kNT;
    // halves of a chunk worked on together (two tiles: 64 requests of 2 tokens 60.5 us,
    // 63.5 with one after the other; four do not have the registers for it)
    static constexpr int kAtOnce = kNT <= 2 ? 2 : 1;
    static constexpr int kRowBytes = kDP / 2;
    static constexpr int kCodes = kHalf * kRowBytes;             // of K or V of half a chunk
    static constexpr int kScales = kHalf * kDP / 16;
    static constexpr int kHalfBytes = 2 * (kCodes + kScales);    // K, V, scales of K, scales of V
    static constexpr int kStageBytes = 2 * kHalfBytes;
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    // O of all warps for kJoin tiles of 8 rows: two rows and 4 words of padding a
    // line (or a warp's own lanes, one vector after the other)
    static constexpr int kJoin = 16 / kWarps;
    static constexpr int kLine = 2 * kDP + 4;
    static constexpr int kWarpO = kJoin * 4 * kLine;             // floats
    static_assert(kNT == 4 || kWarpO >= kRows * kDP, "a warp's O");
    static constexpr int kOffO = kRing;
    static constexpr int kOffQ = kOffO + kWarps * kWarpO * 4;    // Q's rows (bf16), then (kNT > 1) its fragments
    static constexpr int kOffFrag = kOffQ + kRows * kDP * 2;
    static constexpr int kOffM = kOffFrag + (kNT > 1 ? kNT * (kDP / 16) * 32 * 8 : 0);
    static constexpr int kSmemTogether = kOffM + kWarps * kRows * 2 * 4;
    // Shares of warps.  kNT <= 2: Q in registers, and what a warp leaves for
    // another (its O) where O is above.  4: Q's fragments of each warp in shared
    // memory, and what a warp leaves in its ring, which has to be as large, or (with
    // another part to come) in a part of the CTA's slots that rows do not reach.
    static constexpr bool kLeaveInRing = kNT == 4;
    static constexpr int kOwnStages = kLeaveInRing ? 4 : kStages;
    static constexpr int kOwnRing = kWarps * kOwnStages * kStageBytes;
    static constexpr int kFrags = kNT * (kDP / 16) * 32;         // uint2
    static constexpr int kOffOwnM = kLeaveInRing ? kOwnRing + kWarps * kFrags * 8 : kOffM;
    static constexpr int kSmemOwn = kOffOwnM + kWarps * kRows * 2 * 4;
    static_assert(!kLeaveInRing || kOwnStages * kStageBytes >= kRows * kDP * 4, "a warp's O");
    static constexpr int kSmem = kSmemOwn > kSmemTogether ? kSmemOwn : kSmemTogether;
    static constexpr int kMostRing = kOwnRing > kRing ? kOwnRing : kRing;
    static constexpr int kQVecs = kRows * kDP / 8 / kThreads > 0 ? kRows * kDP / 8 / kThreads : 1;
    static_assert(kSmem <= 232448 - 4096, "shared memory per block");
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
// 16 (8) bytes of global memory into shared memory, kDst and kSrc on from the
// addresses; `real` 0: zeros instead.
template <int kDst = 0, int kSrc = 0>
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, uint32_t real)
{
    asm volatile("cp.async.cg.shared.global [%0 + %3], [%1 + %4], 16, %2;" ::"r"(dst), "l"(src), "r"(real), "n"(kDst), "n"(kSrc)
                 : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const uint8_t* src, uint32_t real)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(real) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
// (x - m) * f + kLift of two rows, two operations in one instruction.
__device__ __forceinline__ float2 exponent2(float x0, float x1, const float* minus_m, const float* f)
{
    float2 d;
    asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n"
        " mov.b64 a, {%6, %7};\n mov.b64 c, {%8, %8};\n fma.rn.f32x2 d, d, a, c;\n mov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(x0), "f"(x1), "f"(minus_m[0]), "f"(minus_m[1]), "f"(f[0]), "f"(f[1]), "f"(kLift));
    return d;
}
// Log of a row's sum of 2^(score - m + kLift), to base e.
__device__ __forceinline__ float log_sum(float m, float l)
{
    return l == 0.0f ? -INFINITY : (m - kLift + log2f(l)) * 0.6931471805599453f;
}

// What a warp has of up to 8 kNT rows: a lane has, of rows 2j and 2j + 1 of each
// tile (j = lane % 4), kDP / 8 columns of O, and their statistics.
template <int kDP, int kNT>
struct Rows {
    float o[kNT][kDP / 16][4];                 // two columns: one of rows 2j, 2j + 1, then the next of them
    // maximum (of the scores without their factor: the difference to it is right
    // for scores of any size; from join_sums() on with it), minus that (0 where there is none)
    float m[kNT][2], nm[kNT][2];
    float limit[kNT][2];                       // the score from which the maximum moves
    float l[kNT][2];                           // sum over this lane's keys
    float cf[kNT][2];                          // the row's factor of the scores

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int n = 0; n < kNT; n++) {
#pragma unroll
            for (int s = 0; s < kDP / 16; s++) o[n][s][0] = o[n][s][1] = o[n][s][2] = o[n][s][3] = 0.0f;
#pragma unroll
            for (int y = 0; y < 2; y++) m[n][y] = limit[n][y] = -INFINITY, nm[n][y] = l[n][y] = 0.0f;
        }
    }
    // The sums of a row's lanes, and the maxima as log2.
    __device__ __forceinline__ void join_sums()
    {
#pragma unroll
        for (int n = 0; n < kNT; n++) {
#pragma unroll
            for (int y = 0; y < 2; y++) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[n][y] += __shfl_xor_sync(0xffffffffu, l[n][y], x);
                m[n][y] *= cf[n][y];
            }
        }
    }
};

// One tile's Q in fragments: raw holds this lane's kDP / 4 columns (from kDP / 4
// * j) of row g as bf16 and becomes f16 for the MMAs.  Scaled by 2^(141 - e), e
// the row's largest biased exponent, which brings that to 2^14 .. 2^15; the
// factor of the row's scores (for the rows of this lane's accumulators) takes it
// back.  A negative scale's sign goes into Q; a zero scale is any tiny factor (no
// 0 * inf where masked).
template <int kDP>
__device__ __forceinline__ void make_q(uint32_t* raw, float scale, float k_g, float* cf, int j)
{
    float amax = 0.0f;
#pragma unroll
    for (int x = 0; x < kDP / 8; x++) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(raw[x])), fabsf(bf16_hi(raw[x]))));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int e = max((int)(__float_as_uint(amax) >> 23), 15);
    const float up = __uint_as_float((uint32_t)(268 - e) << 23 | (__float_as_uint(scale) & 0x80000000u));
    const float down = __uint_as_float((uint32_t)(e - 14) << 23);
#pragma unroll
    for (int x = 0; x < kDP / 8; x++) raw[x] = cvt_f16x2(bf16_lo(raw[x]) * up, bf16_hi(raw[x]) * up);
    const float c = fmaxf(fabsf(scale) * kLog2e * k_g * down, 1.17549435e-38f);
    cf[0] = __shfl_sync(0xffffffffu, c, 8 * j);
    cf[1] = __shfl_sync(0xffffffffu, c, 8 * j + 4);
}

// Which keys rows see.
struct Seen {
    int pos0, r0, group;         // position of row r of the tiles: pos0 + (r0 + r) / group
    int lo, ke, window;          // some row sees keys lo .. ke - 1, none one past
};

// kH halves of a chunk at `st`, keys k0 ..: scores, softmax, products.  kEdge:
// some row does not see all of them (code of its own: the branches around each
// mask cost more than the masks).  q(n, x): fragment x of tile n's Q.
template <int kDP, int kNT, bool kFull, int kH, bool kEdge, typename Q>
__device__ __forceinline__ void work_halves(const uint8_t* st, int k0, const Seen& seen, int nb, Rows<kDP, kNT>& w, Q&& q,
                                            int g, int j)
{
    using C = Cfg4<kDP, kNT>;
    constexpr int kSteps = kDP / 16;
    const int key_row = (g >> 1) + 4 * (g & 1);            // key of a half that is row g of its S^T (and 8 + it)
    // ---- S^T = K Q^T
    float s[kH][kNT][4];
#pragma unroll
    for (int h = 0; h < kH; h++) {
        const uint8_t* sk = st + h * C::kHalfBytes;
        uint32_t code[2][kDP / 32];                        // of keys key_row and 8 + key_row
        __half2 sc[2];                                     // their scales (128 columns: of two blocks)
#pragma unroll
        for (int y = 0; y < 2; y++) {
            const int key = key_row + 8 * y;
            const uint8_t* sf = sk + 2 * C::kCodes + key * nb;
            if (kDP == 128) {
                const uint4 x = *reinterpret_cast<const uint4*>(sk + key * C::kRowBytes + j * 16);
                code[y][0] = x.x, code[y][1] = x.y, code[y][kDP / 32 - 2] = x.z, code[y][kDP / 32 - 1] = x.w;
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
                code[y][0] = x.x, code[y][1] = x.y;
                sc[y] = as_half2(e4m3x2_to_f16x2(j < nb ? sf[j] : 0u));
            }
        }
#pragma unroll
        for (int n = 0; n < kNT; n++) s[h][n][0] = s[h][n][1] = s[h][n][2] = s[h][n][3] = 0.0f;
#pragma unroll
        for (int x = 0; x < kDP / 32; x++) {               // a word of codes: two MMAs
            uint32_t f[2][4];
#pragma unroll
            for (int y = 0; y < 2; y++) {
                e2m1x8_to_f16x2(code[y][x], f[y]);
                const __half2 z = kDP == 128 && x >= 2 ? __high2half2(sc[y]) : __low2half2(sc[y]);
#pragma unroll
                for (int u = 0; u < 4; u++) f[y][u] = as_u32(__hmul2(as_half2(f[y][u]), z));
            }
#pragma unroll
            for (int u = 0; u < 2; u++) {
                const uint32_t fa[4] = {f[0][2 * u], f[1][2 * u], f[0][2 * u + 1], f[1][2 * u + 1]};
#pragma unroll
                for (int n = 0; n < kNT; n++) {
                    const uint2 b = q(n, 2 * x + u);
                    mma16816(s[h][n], fa, b.x, b.y);
                }
            }
        }
    }
    // ---- softmax
    if (kEdge) {
#pragma unroll
        for (int h = 0; h < kH; h++) {
#pragma unroll
            for (int n = 0; n < kNT; n++) {
#pragma unroll
                for (int y = 0; y < 4; y++) {
                    const int pos = seen.pos0 + (seen.r0 + 8 * n + 2 * j + (y & 1)) / seen.group;
                    const int key = k0 + h * kHalf + key_row + 8 * (y >> 1);
                    if (key > pos || key >= seen.ke || (seen.window && key <= pos - seen.window)) s[h][n][y] = -INFINITY;
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
            up |= top > w.limit[n][y];
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
                top = fmaxf(top, w.m[n][y]);
                const bool none = top == -INFINITY;
                const float f = w.m[n][y] == -INFINITY ? 0.0f : ex2((w.m[n][y] - top) * w.cf[n][y]);
                w.m[n][y] = top;
                w.nm[n][y] = none ? 0.0f : -top;
                w.limit[n][y] = none ? -INFINITY : __fadd_rd(top, __fdividef(kLazy, w.cf[n][y]));
                w.l[n][y] *= f;
#pragma unroll
                for (int x = 0; x < kSteps; x++) {
                    w.o[n][x][y] *= f;
                    w.o[n][x][y + 2] *= f;
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
            for (int y = 0; y < 4; y += 2) {
                const float2 x = exponent2(s[h][n][y], s[h][n][y + 1], w.nm[n], w.cf[n]);
                e[y] = ex2(x.x);
                e[y + 1] = ex2(x.y);
                w.l[n][0] += e[y];
                w.l[n][1] += e[y + 1];
            }
            pt[h][n][0] = transpose8x8(cvt_f16x2(e[0], e[1]));
            pt[h][n][1] = transpose8x8(cvt_f16x2(e[2], e[3]));
        }
    }
    // ---- O^T += V^T P^T: keys j, j + 4 and j + 8, j + 12 of a half, columns kDP / 8 * g ..
    constexpr int kVW = kDP / 64;                          // words of a key's codes
#pragma unroll
    for (int h = 0; h < kH; h++) {
        const uint8_t* sv = st + h * C::kHalfBytes + C::kCodes;
        const uint8_t* sf = sv + C::kCodes + C::kScales;
        uint32_t v[4][kVW], b[4];
        const int blk = kDP == 128 ? g : g >> 1;
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
        if (kEdge) {                                       // a value that no row sees may be anything
            const int lo = seen.lo - k0 - h * kHalf, ke = seen.ke - k0 - h * kHalf;
#pragma unroll
            for (int u = 0; u < 4; u++)
                if (j + 4 * u < lo || j + 4 * u >= ke) b[u] = 0u;
        }
        const __half2 vs[2] = {as_half2(e4m3x2_to_f16x2(__byte_perm(b[0], b[1], 0x3340))),
                               as_half2(e4m3x2_to_f16x2(__byte_perm(b[2], b[3], 0x3340)))};
#pragma unroll
        for (int y = 0; y < kVW; y++) {
            uint32_t even[2][4], odd[2][4];                // two keys side by side, of even and odd columns
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
                for (int n = 0; n < kNT; n++) mma16816(w.o[n][4 * y + x], f, pt[h][n][0], pt[h][n][1]);
            }
        }
    }
}

// A warp's ring of chunks, and the copies into it.  Every copy() is followed by
// a release() or, at a part's start, by as many copies as stages are free: with a
// commit for each of them, real or not, the oldest chunk is there when all but
// kStages - 1 commits are complete.
template <int kDP, int kNT, bool kFull, int kStages>
struct Ring {
    using C = Cfg4<kDP, kNT>;
    const Params4& prm;
    uint8_t* base;
    uint32_t addr;
    int lane, D, chunks;                       // copies of a half's codes
    bool whole16;                              // ... of 16 bytes (8 where a row is not whole sixteens)
    int to[kFull ? 1 : 4];
    uint32_t sf_to;
    const uint8_t* k_at;                       // this lane's first bytes of page 0: codes of K and V, scales
    const uint8_t* v_at;
    const uint8_t* sf_at;
    int in = 0, out = 0;                       // stages to fill and to read next, in bytes
    int ahead = 0;                             // filled ones

    __device__ __forceinline__ Ring(const Params4& prm, uint8_t* base, int lane, int D) : prm(prm), base(base), lane(lane), D(D)
    {
        addr = smem_u32(base);
        whole16 = kFull || D % 32 == 0;
        const int chunk = whole16 ? 16 : 8, per_row = D / 2 / chunk;
        chunks = kHalf * per_row;
#pragma unroll
        for (int i = 0; i < (kFull ? 1 : 4); i++) {
            const int c = lane + 32 * i;
            to[i] = (c / per_row) * C::kRowBytes + (c % per_row) * chunk;
        }
        k_at = prm.k + lane * chunk;
        v_at = prm.v + lane * chunk;
        // 16 keys' scales are D bytes: lanes 0-7 and 8-15 K's and V's of the first half, then the second's
        const bool of_v = lane >> 3 & 1;
        sf_to = (lane >> 4) * C::kHalfBytes + 2 * C::kCodes + (of_v ? C::kScales : 0) + (lane & 7) * 16;
        sf_at = (of_v ? prm.v_sf : prm.k_sf) + (lane & 7) * 16;
    }
    __device__ __forceinline__ static int next(int at) { return kStages == 2 ? C::kStageBytes - at : at == (kStages - 1) * C::kStageBytes ? 0 : at + C::kStageBytes; }
    // Page ids of the halves of 16 chunks, `stride` keys apart, from key k on:
    // a lane each; none from ke on.
    __device__ __forceinline__ int load_ids(const int32_t* table, int k, int stride, int ke) const
    {
        k += (lane >> 1) * stride + (lane & 1) * kHalf;
        return k < ke ? table[k >> prm.page_shift] : -1;
    }
    // Copies of the chunk of keys k0 .., kv head hk, into the next stage; the ids
    // of its pages are in lanes 2i and 2i + 1.  A page that the cache does not have
    // is zeros; a half past the keys' end is masked as a whole.
    __device__ __forceinline__ void copy(int k0, int hk, int ids, int i)
    {
        const uint32_t st = addr + in;
        const int page_mask = (1 << prm.page_shift) - 1, head = hk << prm.page_shift;
        uint32_t page[2], row[2], size[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const uint32_t id = __shfl_sync(0xffffffffu, ids, 2 * i + h);
            size[h] = id < (uint32_t)prm.pages ? 16 : 0;
            page[h] = size[h] ? id : 0u;
            row[h] = head + ((k0 + kHalf * h) & page_mask);
            const uint64_t at = (uint64_t)page[h] * prm.page_stride + row[h] * (uint32_t)(D / 2);
            const uint8_t* ck = k_at + at;
            const uint8_t* cv = v_at + at;
            const uint32_t sh = st + h * C::kHalfBytes + to[0];
            if (kFull) {
                copy16(sh, ck, size[h]);
                if (kDP == 128) copy16<512, 512>(sh, ck, size[h]);
                copy16<C::kCodes>(sh, cv, size[h]);
                if (kDP == 128) copy16<C::kCodes + 512, 512>(sh, cv, size[h]);
            } else if (whole16) {
#pragma unroll
                for (int y = 0; y < (kDP == 128 ? 2 : 1); y++)
                    if (lane + 32 * y < chunks) {
                        copy16(sh - to[0] + to[kFull ? 0 : y], ck + 512 * y, size[h]);
                        copy16<C::kCodes>(sh - to[0] + to[kFull ? 0 : y], cv + 512 * y, size[h]);
                    }
            } else {
#pragma unroll
                for (int y = 0; y < (kDP == 128 ? 4 : 2); y++)
                    if (lane + 32 * y < chunks) {
                        copy8(sh - to[0] + to[kFull ? 0 : y], ck + 256 * y, size[h] / 2);
                        copy8(sh - to[0] + C::kCodes + to[kFull ? 0 : y], cv + 256 * y, size[h] / 2);
                    }
            }
        }
        const bool second = lane >> 4;
        if ((kFull && kDP == 128) || (lane & 7) * 16 < D)
            copy16(st + sf_to,
                   sf_at + (uint64_t)(second ? page[1] : page[0]) * prm.sf_stride + (second ? row[1] : row[0]) * (uint32_t)(D / 16),
                   second ? size[1] : size[0]);
        in = next(in);
        ahead++;
    }
    // The oldest chunk, once it is there.
    __device__ __forceinline__ const uint8_t* wait()
    {
        copies_wait<kStages - 1>();
        __syncwarp();
        return base + out;
    }
    __device__ __forceinline__ void release()
    {
        __syncwarp();
        out = next(out);
        ahead--;
    }
};

// The parts of an item that CTAs share, added up by threads [thread0, thread0 +
// threads) of the last of them: part i is in slot 2 (cta0 + i), the first in 2 cta0 + 1.
// A thread adds four columns of a row, of kX rows at a time, kB parts of each at a
// time: their reads are on their way together.
template <int kDP, int kX, int kB>
__device__ __forceinline__ void join_some(const AttnArgs& a, int thread0, int threads, int cta0, int parts, int rows, int tok0,
                                          int hk, float v_g)
{
    auto slot_of = [&](int i) { return a.partials + (2 * (cta0 + i) + (i == 0 ? 1 : 0)) * kAttnSlotFloats; };
    const int n = rows * (kDP / 4);
#pragma unroll 1
    for (int x0 = (int)threadIdx.x - thread0; x0 < n; x0 += kX * threads) {
        float top[kX], sum[kX];
        float4 acc[kX];
#pragma unroll
        for (int y = 0; y < kX; y++) {
            top[y] = -INFINITY;
            sum[y] = 0.0f;
            acc[y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll 1
        for (int i0 = 0; i0 < parts; i0 += kB) {
            float2 ml[kX][kB];
            float4 e[kX][kB];
#pragma unroll
            for (int y = 0; y < kX; y++) {
                const int x = x0 + y * threads, r = x / (kDP / 4), col = 4 * (x % (kDP / 4));
#pragma unroll
                for (int u = 0; u < kB; u++) {
                    ml[y][u] = make_float2(-INFINITY, 0.0f);
                    e[y][u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (i0 + u < parts && x < n) {
                        const float* from = slot_of(i0 + u);
                        ml[y][u] = __ldcg(reinterpret_cast<const float2*>(from + kAttnSlotRows * kDP + 2 * r));
                        e[y][u] = __ldcg(reinterpret_cast<const float4*>(from + r * kDP + col));
                    }
                }
            }
#pragma unroll
            for (int y = 0; y < kX; y++) {
                float most = top[y];
#pragma unroll
                for (int u = 0; u < kB; u++) most = fmaxf(most, ml[y][u].x);
                const float f0 = top[y] == -INFINITY ? 0.0f : ex2(top[y] - most);
                acc[y].x *= f0, acc[y].y *= f0, acc[y].z *= f0, acc[y].w *= f0;
                sum[y] *= f0;
                top[y] = most;
#pragma unroll
                for (int u = 0; u < kB; u++) {
                    if (ml[y][u].y == 0.0f) continue;      // no key of this part
                    const float f = ml[y][u].x == -INFINITY ? 0.0f : ex2(ml[y][u].x - top[y]);
                    acc[y].x += f * e[y][u].x;
                    acc[y].y += f * e[y][u].y;
                    acc[y].z += f * e[y][u].z;
                    acc[y].w += f * e[y][u].w;
                    sum[y] += f * ml[y][u].y;
                }
            }
        }
#pragma unroll
        for (int y = 0; y < kX; y++) {
            const int x = x0 + y * threads, r = x / (kDP / 4), col = 4 * (x % (kDP / 4));
            if (x >= n || col >= a.head_dim) continue;
            const int t = r / a.group, head = hk * a.group + r - t * a.group;
            const float inv = sum[y] == 0.0f ? 0.0f : v_g / sum[y];
            *reinterpret_cast<uint2*>(a.out + (int64_t)(tok0 + t) * a.ldo + (int64_t)head * a.ho + col) =
                sum[y] == 0.0f ? make_uint2(0u, 0u)
                               : make_uint2(cvt_bf16x2(acc[y].x * inv, acc[y].y * inv), cvt_bf16x2(acc[y].z * inv, acc[y].w * inv));
            if (col == 0 && a.lse)
                a.lse[(int64_t)(tok0 + t) * a.heads + head] = log_sum(top[y], sum[y]);
        }
    }
}
template <int kDP>
__device__ __forceinline__ void join_parts(const AttnArgs& a, int thread0, int threads, int cta0, int parts, int rows, int tok0,
                                           int hk, float v_g)
{
    if (parts <= 3)
        join_some<kDP, 4, 3>(a, thread0, threads, cta0, parts, rows, tok0, hk, v_g);
    else
        join_some<kDP, 1, 12>(a, thread0, threads, cta0, parts, rows, tok0, hk, v_g);
}

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

// ------------------------------------------------ passes of all warps together
template <int kDP, int kNT, bool kFull>
__device__ __forceinline__ void passes_together(const Params4& prm, uint8_t* smem, int cta)
{
    using C = Cfg4<kDP, kNT>;
    constexpr int kSteps = kDP / 16;           // MMAs over a key's columns; of 16 columns of O
    __shared__ int s_last;
    __shared__ Pass s_pass[3];
    const AttnArgs& a = prm.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
    const int D = kFull ? kDP : a.head_dim, nb = D / 16;
    float* o_all = reinterpret_cast<float*>(smem + C::kOffO);
    float2* m_all = reinterpret_cast<float2*>(smem + C::kOffM);            // [warp][row] m, l
    uint4* q_rows = reinterpret_cast<uint4*>(smem + C::kOffQ);             // [row][kDP / 8]
    uint2* q_frag = reinterpret_cast<uint2*>(smem + C::kOffFrag);          // [tile][step][lane]

    Passes<C::kRows> passes(a, cta);            // (the first warp's)
    if (warp == 0) {
        passes.next(a, &s_pass[0], lane);
        passes.next(a, &s_pass[1], lane);
    }
    __syncthreads();

    const float k_g = *a.k_g, v_g = *a.v_g;
    // chunks of this warp in a pass
    auto chunks_of = [&](const Pass& x) {
        const int n = x.valid && x.ke > x.kb ? (x.ke - x.kb + kChunk - 1) / kChunk : 0;
        return n > warp ? (n - warp + C::kWarps - 1) / C::kWarps : 0;
    };
    constexpr int kStride = C::kWarps * kChunk;            // a warp's chunks are this many keys apart
    Ring<kDP, kNT, kFull, C::kStages> ring(prm, smem + warp * (C::kStages * C::kStageBytes), lane, D);
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
    int issue_i = 0, issue_n = chunks_of(s_pass[0]), ids, ids_next;
    bool in_next = false;                                  // what is issued is of the next pass
    auto ids_of = [&](const Pass& x, int i) { return ring.load_ids(x.table, x.kb + (warp + i * C::kWarps) * kChunk, kStride, x.ke); };
    ids = issue_n ? ids_of(s_pass[0], 0) : 0;
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
        ids_next = next_n ? ids_of(nxt, 0) : 0;
        auto issue = [&]() {
            if (issue_i == issue_n && !in_next) {
                in_next = true;
                issue_i = 0;
                issue_n = next_n;
                ids = ids_next;
            }
            if (issue_i < issue_n) {
                const Pass& from = in_next ? nxt : cur;
                if (issue_i && (issue_i & 15) == 0) ids = ids_of(from, issue_i);
                ring.copy(from.kb + (warp + issue_i * C::kWarps) * kChunk, from.hk, ids, issue_i & 15);
                issue_i++;
            }
            copies_end();
        };
#pragma unroll 1
        for (int y = ring.ahead; y < C::kStages; y++) issue();

        // Q of the pass: row g of tile n, columns kDP / 4 * j .. of this lane
        Rows<kDP, kNT> w;
        uint32_t q[kNT == 1 ? kDP / 8 : 1];
#pragma unroll
        for (int n = 0; n < kNT; n++) {
            uint32_t raw[kDP / 8];
#pragma unroll
            for (int x = 0; x < kDP / 32; x++) {
                const uint4 y = q_rows[(8 * n + g) * (kDP / 8) + j * (kDP / 32) + x];
                raw[4 * x] = y.x, raw[4 * x + 1] = y.y, raw[4 * x + 2] = y.z, raw[4 * x + 3] = y.w;
            }
            make_q<kDP>(raw, a.scale, k_g, w.cf[n], j);
            if (kNT == 1) {
#pragma unroll
                for (int x = 0; x < kDP / 8; x++) q[kNT == 1 ? x : 0] = raw[x];
            } else if (warp == n) {
#pragma unroll
                for (int s = 0; s < kSteps; s++) q_frag[(n * kSteps + s) * 32 + lane] = make_uint2(raw[2 * s], raw[2 * s + 1]);
            }
        }
        if (kNT > 1) __syncthreads();
        w.clear();
        const Seen seen = {cur.pos0, cur.r0, a.group, cur.lo, cur.ke, a.window};
        const int lo_all = cur.lo_all, hi_all = cur.hi_all;
        int kc = cur.kb + warp * kChunk;                   // first key of the chunk
#pragma unroll 1
        for (int i = 0; i < mine; i++, kc += kStride) {
            const uint8_t* st = ring.wait();
            auto frag = [&](int n, int x) {
                return kNT == 1 ? make_uint2(q[kNT == 1 ? 2 * x : 0], q[kNT == 1 ? 2 * x + 1 : 0]) : q_frag[(n * kSteps + x) * 32 + lane];
            };
#pragma unroll 1
            for (int h = 0; h < 2; h += C::kAtOnce) {
                const int k = kc + h * kHalf;
                const bool edge = k < lo_all || k + C::kAtOnce * kHalf > hi_all;
                if (edge)
                    work_halves<kDP, kNT, kFull, C::kAtOnce, true>(st + h * C::kHalfBytes, k, seen, nb, w, frag, g, j);
                else
                    work_halves<kDP, kNT, kFull, C::kAtOnce, false>(st + h * C::kHalfBytes, k, seen, nb, w, frag, g, j);
            }
            ring.release();
            issue();
        }

        // ---- the warps' shares of the pass together
        const int r0 = cur.r0, rows = cur.rows, tok0 = cur.tok0, hk = cur.hk;
        const bool whole = cur.parts == 1;
        float* part = a.partials + (2 * cta + (cur.cta0 == cta ? 1 : 0)) * kAttnSlotFloats;
        uint4 q_next[C::kQVecs];
        load_q(nxt, q_next);
        if (warp == 0) passes.next(a, &s_pass[x_pass == 0 ? 2 : x_pass - 1], lane);
        w.join_sums();
        if (g == 0) {
#pragma unroll
            for (int n = 0; n < kNT; n++) {
#pragma unroll
                for (int y = 0; y < 2; y++)
                    m_all[warp * C::kRows + 8 * n + 2 * j + y] = make_float2(w.m[n][y], w.l[n][y]);
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
                        to4[x / 2] = make_float4(w.o[n][x][y], w.o[n][x][y + 2], w.o[n][x + 1][y], w.o[n][x + 1][y + 2]);
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
                        a.lse[(int64_t)(tok0 + t) * a.heads + head] = log_sum(top, sum);
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
        join_parts<kDP>(a, 0, C::kThreads, cta0, parts, rows, tok0, hk, v_g);
    }
}

// ------------------------------------------------------- shares of warps
// The part of an item that a warp works on, in its shared memory (this and the
// next one).
struct Work {
    int valid;
    int tok0, rows, pos0, hk;
    int s, item;             // the item's first unit, its units
    int a, b, chunks;        // chunks a .. b - 1 of the item's are this CTA's
    int x0, x1;              // x0 .. x1 - 1 are this warp's
    int lo, lo_all, hi_all;  // as Pass's
    int kb, ke, n;           // keys of its chunks that rows see, chunks
    const int32_t* table;
};

// A warp's walk over the items of its CTA's share of the schedule's second axis.
struct Walk {
    QTile t;
    int qt, hk, s;           // the next item: its QTile's number, kv head, first unit
};

// An item that this CTA shares with others: [0] with the CTAs before it, [1] one
// that begins here.
struct Share {
    int valid, cta0, parts, rows, tok0, hk, last;
};

template <int kDP, int kNT, bool kFull>
__device__ __forceinline__ void own_shares(const Params4& prm, uint8_t* smem, int cta, Share* s_share)
{
    using C = Cfg4<kDP, kNT>;
    constexpr int kSteps = kDP / 16;
    __shared__ Work s_work[C::kWarps][2];
    __shared__ Walk s_walk[C::kWarps];
    const AttnArgs& a = prm.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
    const int D = kFull ? kDP : a.head_dim, Hkv = a.kv_heads, nb = D / 16;
    // what a warp leaves for an earlier one: O in its lanes' order, [tile, vector]
    // [lane][4] floats; its maxima and sums [warp][row]
    __shared__ float4* s_left[C::kWarps];
    float2* const left_ml = reinterpret_cast<float2*>(smem + C::kOffOwnM);
    uint2* const frags = reinterpret_cast<uint2*>(smem + C::kOwnRing) + warp * C::kFrags + lane;   // (kNT 4)
    const ScheduleHead* head = a.sched;
    const QTile* tiles = schedule_tiles(head);

    // The CTA's units u0 .. u1 - 1 (its bounds moved to the edge of an item that they
    // would cut too near it: the warps share what that leaves, or the last one would
    // have up to eight chunks more than the others), this warp's v0 .. v1 - 1.
    const int per = head->per_cta4, units = head->units4, n_tiles = head->qtiles, begin = head->first4[cta];
    const QTile start = head->start4[cta];
    const int after = min(cta + 1, kAttnMaxCtas - 1), begin1 = head->first4[after];      // (read at once with the rest)
    const QTile start1 = head->start4[after];
    auto snapped = [&](int u, const QTile& t, int i) {
        const int item = kItemUnits4 + kChunksOfTile * t.tiles, s = units4_before(t.unit0, Hkv, i);
        const int at = s + (u - s) / item * item;          // the item that it cuts
        return at + snap_unit4(u - at, item);
    };
    const int raw0 = min(cta * per, units), raw1 = min(raw0 + per, units);
    const int u0 = raw0 < units ? snapped(raw0, start, begin) : units;
    const int u1 = raw1 < units ? snapped(raw1, start1, begin1) : units;
    const int len = u1 - u0;
    auto bound = [&](int w) { return u0 + len * w / C::kWarps; };
    const int v0 = bound(warp), v1 = bound(warp + 1);
    const bool final_warp = warp == C::kWarps - 1;
    const float k_g = *a.k_g, v_g = *a.v_g;

    Walk& walk = s_walk[warp];
    const bool any = len > 0;
    if (any) {
        int qt = begin, s = units4_before(start.unit0, Hkv, begin);
        QTile t = start;
        if (v0 >= s + (kItemUnits4 + kChunksOfTile * t.tiles) * Hkv) {
            // a later QTile of the CTA's: the last that begins at or below v0
            for (int base = begin + 1;; base += 32) {
                const int i = base + lane;
                const int at = i < n_tiles ? units4_before(tiles[i].unit0, Hkv, i) : 0x7fffffff;
                const int k = __popc(__ballot_sync(0xffffffffu, at <= v0));
                qt = base + k - 1;
                if (k < 32) break;
            }
            t = tiles[qt];
            s = units4_before(t.unit0, Hkv, qt);
        }
        const int item = kItemUnits4 + kChunksOfTile * t.tiles, hk = (v0 - s) / item;
        if (lane == 0) walk = Walk{t, qt, hk, s + hk * item};
        __syncwarp();
    }
    // The warp's next part into *out.
    auto next = [&](Work* out) {
        Work x;
        x.valid = 0;
        const int end = final_warp ? u1 : v1;
        QTile t = walk.t;
        int qt = walk.qt, hk = walk.hk, s = walk.s;
        while (any && s < end) {
            const int chunks = kChunksOfTile * t.tiles, item = kItemUnits4 + chunks;
            x.a = min(max(u0 - s - kItemUnits4, 0), chunks);
            x.b = min(max(u1 - s - kItemUnits4, 0), chunks);
            x.x0 = warp == 0 ? x.a : min(max(v0 - s - kItemUnits4, x.a), x.b);
            x.x1 = final_warp ? x.b : min(max(v1 - s - kItemUnits4, x.a), x.b);
            if (x.x1 > x.x0) {
                x.valid = 1;
                x.tok0 = t.tok0;
                x.rows = t.n_tok * a.group;
                x.pos0 = t.pos0;
                x.hk = hk;
                x.s = s;
                x.item = item;
                x.chunks = chunks;
                x.lo = a.window ? max(t.pos0 + 1 - a.window, 0) : 0;
                x.lo_all = a.window ? max(t.pos0 + t.n_tok - a.window, 0) : 0;
                const int key0 = t.tile0 * kAttnKeys;
                x.kb = max(key0 + x.x0 * kChunk, x.lo & ~(kChunk - 1));
                x.ke = min(key0 + x.x1 * kChunk, t.kv_end);
                x.hi_all = min(t.pos0 + 1, x.ke);
                x.n = x.ke > x.kb ? (x.ke - x.kb + kChunk - 1) / kChunk : 0;
                x.table = a.block_table + t.req * a.table_ld;
            }
            s += item;
            if (++hk == Hkv) {
                hk = 0;
                qt++;
                if (s < end) t = tiles[qt];
            }
            if (x.valid) break;
        }
        __syncwarp();                                      // (every lane has read what this replaces)
        if (lane == 0) {
            *out = x;
            walk = Walk{t, qt, hk, s};
        }
        __syncwarp();
    };

    Ring<kDP, kNT, kFull, C::kOwnStages> ring(prm, smem + warp * (C::kOwnStages * C::kStageBytes), lane, D);
    Rows<kDP, kNT> w;
    next(&s_work[warp][0]);
    // the next chunk to copy, of this part or (in_next) the next; chunks whose
    // pages' ids are in `ids`, from the issue_i-th on
    int issue_k = 0, issue_ke = 0, issue_hk = 0, issue_i = 0, issue_left = 0, ids = 0;
    bool in_next = false;
    if (s_work[warp][0].valid) {
        const Work& x = s_work[warp][0];
        issue_k = x.kb;
        issue_ke = x.ke;
        issue_hk = x.hk;
        if (x.n) ids = ring.load_ids(x.table, x.kb, kChunk, x.ke);
        issue_left = min(x.n, 16);
    }
    int at = 0;
    bool pending = false;
    // The rows of *this warp* are the CTA's part of the item: out, or to the CTA's slot.
    auto finish = [&](const Work& x) {
        const bool whole = x.a == 0 && x.b == x.chunks;
        float* part = a.partials + (2 * cta + (x.a == 0 ? 1 : 0)) * kAttnSlotFloats;
#pragma unroll
        for (int n = 0; n < kNT; n++) {
#pragma unroll
            for (int y = 0; y < 2; y++) {
                const int r = 8 * n + 2 * j + y, col = g * (kDP / 8);
                if (r >= x.rows) continue;
                if (whole) {
                    const int t = r / a.group, hd = x.hk * a.group + r - t * a.group;
                    const bool none = w.l[n][y] == 0.0f;
                    const float inv = none ? 0.0f : v_g / w.l[n][y];
                    uint32_t v[kSteps];
#pragma unroll
                    for (int i = 0; i < kSteps; i++) v[i] = none ? 0u : cvt_bf16x2(w.o[n][i][y] * inv, w.o[n][i][y + 2] * inv);
                    uint4* out = reinterpret_cast<uint4*>(a.out + (int64_t)(x.tok0 + t) * a.ldo + (int64_t)hd * a.ho + col);
#pragma unroll
                    for (int i = 0; i < kSteps / 4; i++)
                        if (kFull || col + 8 * i < D) out[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    if (g == 0 && a.lse) a.lse[(int64_t)(x.tok0 + t) * a.heads + hd] = log_sum(w.m[n][y], w.l[n][y]);
                } else {
#pragma unroll
                    for (int i = 0; i < kSteps; i += 2)
                        __stcg(reinterpret_cast<float4*>(part + r * kDP + col) + i / 2,
                               make_float4(w.o[n][i][y], w.o[n][i][y + 2], w.o[n][i + 1][y], w.o[n][i + 1][y + 2]));
                    if (g == 0)
                        __stcg(reinterpret_cast<float2*>(part + kAttnSlotRows * kDP + 2 * r), make_float2(w.m[n][y], w.l[n][y]));
                }
            }
        }
        if (!whole && lane == 0) {
            int c0 = x.s / per, c1 = (x.s + x.item - 1) / per;
            if (snap_unit4((c0 + 1) * per - x.s, x.item) == 0) c0++;
            if (c1 > c0 && snap_unit4(c1 * per - x.s, x.item) == x.item) c1--;
            s_share[x.a == 0 ? 1 : 0] = Share{1, c0, c1 - c0 + 1, x.rows, x.tok0, x.hk, 0};
        }
        return whole ? 0 : x.a == 0 ? 2 : 1;
    };
    // Tickets for the CTA's parts (bits 0 and 1 of `which`) that this warp has written:
    // as soon as it has nothing else to do, not when all are ready.
    auto tickets = [&](int which) {
        __syncwarp();
        if (lane < 2 && (which >> lane & 1)) {
            Share& x = s_share[lane];
            int* ticket = a.tickets + x.cta0 * 8;
            x.last = atom_add_acq_rel(ticket, 1) == x.parts - 1;
            if (x.last) *ticket = 0;
        }
    };
    int written = 0;
    if (s_work[warp][0].valid) {
#pragma unroll 1
        for (;; at ^= 1) {
            const Work& cur = s_work[warp][at];
            const Work& nxt = s_work[warp][at ^ 1];
            // Q of the item: row g of tile n, columns kDP / 4 * j .. of this lane
            uint32_t q[C::kLeaveInRing ? 1 : kNT][kDP / 8];
            auto load_q = [&](int n, uint32_t* raw) {
                const int r = 8 * n + g, t = r / a.group;
                const __nv_bfloat16* src = prm.q + (int64_t)(cur.tok0 + t) * prm.ldq +
                                           (int64_t)(cur.hk * a.group + r - t * a.group) * prm.hq + j * (kDP / 4);
#pragma unroll
                for (int x = 0; x < kDP / 32; x++) {
                    uint4 y = make_uint4(0, 0, 0, 0);
                    if (r < cur.rows && (kFull || j * (kDP / 4) + 8 * x < D)) y = *reinterpret_cast<const uint4*>(src + 8 * x);
                    raw[4 * x] = y.x, raw[4 * x + 1] = y.y, raw[4 * x + 2] = y.z, raw[4 * x + 3] = y.w;
                }
            };
            if (!C::kLeaveInRing) {
#pragma unroll
                for (int n = 0; n < kNT; n++) load_q(n, q[C::kLeaveInRing ? 0 : n]);
            }
            next(&s_work[warp][at ^ 1]);
            const int next_ids = nxt.valid && nxt.n ? ring.load_ids(nxt.table, nxt.kb, kChunk, nxt.ke) : 0;
            in_next = false;                               // (what has been issued of the next part is now this one's)
            auto issue = [&]() {
                if (issue_left == 0) {                     // the next ids: of this part, or of the next
                    if (issue_k >= issue_ke && !in_next && nxt.valid) {
                        in_next = true;
                        issue_k = nxt.kb;
                        issue_ke = nxt.ke;
                        issue_hk = nxt.hk;
                        ids = next_ids;
                    } else if (issue_k < issue_ke) {
                        ids = ring.load_ids((in_next ? nxt : cur).table, issue_k, kChunk, issue_ke);
                    }
                    issue_left = min(max((issue_ke - issue_k + kChunk - 1) / kChunk, 0), 16);
                    issue_i = 0;
                }
                if (issue_left) {
                    ring.copy(issue_k, issue_hk, ids, issue_i++);
                    issue_k += kChunk;
                    issue_left--;
                }
                copies_end();
            };
#pragma unroll 1
            for (int y = ring.ahead; y < C::kOwnStages; y++) issue();
#pragma unroll
            for (int n = 0; n < kNT; n++) {
                uint32_t* raw = q[C::kLeaveInRing ? 0 : n];
                if (C::kLeaveInRing) load_q(n, raw);
                make_q<kDP>(raw, a.scale, k_g, w.cf[n], j);
                if (C::kLeaveInRing) {
#pragma unroll
                    for (int x = 0; x < kSteps; x++) frags[32 * (n * kSteps + x)] = make_uint2(raw[2 * x], raw[2 * x + 1]);
                }
            }
            w.clear();
            const Seen seen = {cur.pos0, 0, a.group, cur.lo, cur.ke, a.window};
            const int lo_all = cur.lo_all, hi_all = cur.hi_all;
            int k0 = cur.kb;
#pragma unroll 1
            for (int i = cur.n; i > 0; i--, k0 += kChunk) {
                const uint8_t* st = ring.wait();
                auto frag = [&](int n, int x) {
                    const uint32_t* raw = q[C::kLeaveInRing ? 0 : n];
                    return C::kLeaveInRing ? frags[32 * (n * kSteps + x)] : make_uint2(raw[2 * x], raw[2 * x + 1]);
                };
#pragma unroll 1
                for (int h = 0; h < 2; h += C::kAtOnce) {
                    const int k = k0 + h * kHalf;
                    const bool edge = k < lo_all || k + C::kAtOnce * kHalf > hi_all;
                    if (edge)
                        work_halves<kDP, kNT, kFull, C::kAtOnce, true>(st + h * C::kHalfBytes, k, seen, nb, w, frag, g, j);
                    else
                        work_halves<kDP, kNT, kFull, C::kAtOnce, false>(st + h * C::kHalfBytes, k, seen, nb, w, frag, g, j);
                }
                ring.release();
                issue();
            }
            w.join_sums();
            if (cur.x0 > cur.a) {                          // the part began in an earlier warp, which will add this
                float* left = reinterpret_cast<float*>(smem + C::kOffO) + warp * C::kWarpO;
                if (C::kLeaveInRing) {
                    constexpr int kSpare = (kAttnSlotRows - C::kRows) / C::kRows;      // warps to a slot, behind its rows
                    static_assert(!C::kLeaveInRing || 2 * kSpare >= C::kWarps, "room in the CTA's slots");
                    left = nxt.valid ? a.partials + (2 * cta + warp / kSpare) * kAttnSlotFloats + (1 + warp % kSpare) * C::kRows * kDP
                                     : reinterpret_cast<float*>(smem + warp * (C::kOwnStages * C::kStageBytes));
                }
                float4* to4 = reinterpret_cast<float4*>(left) + lane;
                if (C::kLeaveInRing && lane == 0) s_left[warp] = reinterpret_cast<float4*>(left);
#pragma unroll
                for (int n = 0; n < kNT; n++) {
#pragma unroll
                    for (int i = 0; i < kSteps; i++)
                        to4[32 * (n * kSteps + i)] = make_float4(w.o[n][i][0], w.o[n][i][1], w.o[n][i][2], w.o[n][i][3]);
#pragma unroll
                    for (int y = 0; y < 2; y++)
                        if (g == 0) left_ml[warp * C::kRows + 8 * n + 2 * j + y] = make_float2(w.m[n][y], w.l[n][y]);
                }
            } else if (cur.x1 == cur.b) {
                written |= finish(cur);
            } else {
                pending = true;                            // goes on in the warps behind
                break;
            }
            if (!nxt.valid) break;
        }
    }
    if (written) tickets(written);
    __syncthreads();
    if (pending) {
        const Work& x = s_work[warp][at];
        int reached = x.x1;
#pragma unroll 1
        for (int o = warp + 1; reached < x.b; o++) {
            const int to = o == C::kWarps - 1 ? x.b : min(max(bound(o + 1) - x.s - kItemUnits4, x.a), x.b);
            if (to == reached) continue;
            reached = to;
            const float4* from = (C::kLeaveInRing ? s_left[o] : reinterpret_cast<const float4*>(smem + C::kOffO + o * C::kWarpO * 4)) + lane;
#pragma unroll
            for (int n = 0; n < kNT; n++) {
                float f0[2], f1[2];
#pragma unroll
                for (int y = 0; y < 2; y++) {
                    const float2 ml = left_ml[o * C::kRows + 8 * n + 2 * j + y];
                    const float top = fmaxf(w.m[n][y], ml.x), ref = top == -INFINITY ? 0.0f : top;
                    f0[y] = ex2(w.m[n][y] - ref);
                    f1[y] = ex2(ml.x - ref);
                    w.m[n][y] = top;
                    w.l[n][y] = w.l[n][y] * f0[y] + ml.y * f1[y];
                }
#pragma unroll
                for (int i = 0; i < kSteps; i++) {
                    const float4 e = from[32 * (n * kSteps + i)];
                    w.o[n][i][0] = w.o[n][i][0] * f0[0] + e.x * f1[0];
                    w.o[n][i][1] = w.o[n][i][1] * f0[1] + e.y * f1[1];
                    w.o[n][i][2] = w.o[n][i][2] * f0[0] + e.z * f1[0];
                    w.o[n][i][3] = w.o[n][i][3] * f0[1] + e.w * f1[1];
                }
            }
        }
        written = finish(x);
        if (written) tickets(written);
    }
    __syncthreads();
    // (the CTA that ends last often has both to join: half of its threads each)
    const bool join0 = s_share[0].valid && s_share[0].last, join1 = s_share[1].valid && s_share[1].last;
    if (!join0 && !join1) return;
    const int half = C::kThreads / 2, second = join0 && join1 ? tid >= half : join1;
    const Share& x = s_share[second];
    join_parts<kDP>(a, join0 && join1 && second ? half : 0, join0 && join1 ? half : C::kThreads, x.cta0, x.parts, x.rows, x.tok0,
                    x.hk, v_g);
}

template <int kDP, int kNT, bool kFull>
__global__ void __launch_bounds__(Cfg4<kDP, kNT>::kThreads, 1) attn4_kernel(const __grid_constant__ Params4 prm)
{
    using C = Cfg4<kDP, kNT>;
    extern __shared__ __align__(128) uint8_t smem[];
    const AttnArgs& a = prm.a;
    const int cta = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    griddep_launch_dependents();
    if (!kFull)                                 // the columns that no copy writes are zeros
        for (int i = threadIdx.x; i < C::kMostRing / 16; i += C::kThreads)
            reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x < 3) {                      // what every warp reads first, on its way into L2 meanwhile
        const ScheduleHead* h = a.sched;
        const void* at = threadIdx.x == 0 ? (const void*)h : threadIdx.x == 1 ? (const void*)&h->first4[cta] : (const void*)&h->start4[cta];
        asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
    }
    griddep_wait();
    if (a.skip_few && !a.sched->few_passes) return;
    __shared__ Share s_share[2];
    if (threadIdx.x < 2) s_share[threadIdx.x].valid = 0;
    __syncthreads();
    // Shares of warps where there is an item for each CTA, or a long one: one join at
    // the end, whatever the items' lengths (us, with the shares and with all warps on
    // one item at a time: 40 requests of 200 to 8000 keys 31 and 48, 28 of 200 to 4000
    // 21.7 and 25.7, 20 of 100 to 4000 16.4 and 18.7, 16 of 1000 to 3000 -- 128 items on
    // 152 CTAs -- 19.2 and 19.2).  Else all warps at once on a CTA's one part, which is
    // joined faster (a request of 333 keys 9.3 and 6.6, 8 of 2000 15.5 and 12.2).
    const int64_t items = (int64_t)a.sched->qtiles * a.kv_heads;
    const int per = a.sched->per_cta4;
    if (per > 0 && a.sched->most_tokens * a.group <= C::kRows && (items >= (int)gridDim.x || per >= 256))
        own_shares<kDP, kNT, kFull>(prm, smem, cta, s_share);
    else
        passes_together<kDP, kNT, kFull>(prm, smem, cta);
    copies_wait<0>();
    if (a.cu_end) {
        // the rows past the step's last token, a warp to a row
        const int vecs = a.head_dim / 8, n = a.heads * vecs;
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

// By the rows of a request: one tile of 8, two, or passes of four.
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
    // the same number of tokens for each request where that is possible; else some
    // have more than the average
    const bool even = args.tokens % requests == 0;
    const int64_t rows = (args.tokens + requests - 1) / requests * args.group * (even ? 1 : 2);
    const int d = args.head_dim;
    return d == 128  ? launch_rows<128, true>(p, rows, ctas, stream)
           : d > 64  ? launch_rows<128, false>(p, rows, ctas, stream)
           : d == 64 ? launch_rows<64, true>(p, rows, ctas, stream)
                     : launch_rows<64, false>(p, rows, ctas, stream);
}

}  // namespace nvfp4
