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

constexpr int kGroupKeys = 16;
constexpr float kLazy = 8.0f;          // log2 of the growth that P may carry
constexpr float kLift = 6.0f;          // log2 of P at m
constexpr float kLog2e = 1.4426950408889634f;

template <int kDP, int kNT>
struct Cfg4 {
    static constexpr int kWarps = kNT == 1 ? 16 : 8;
    static constexpr int kStages = kNT == 1 ? 4 : 6;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kRows = 8 * kNT;
    static constexpr int kRowBytes = kDP / 2;
    static constexpr int kCodes = kGroupKeys * kRowBytes;        // of K or V
    static constexpr int kScales = kGroupKeys * kDP / 16;
    static constexpr int kStageBytes = 2 * (kCodes + kScales);   // K, V, scales of K, scales of V
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    // O of all warps for kJoin tiles of 8 rows: two rows and 4 words of padding a line
    static constexpr int kJoin = 16 / kWarps;
    static constexpr int kLine = 2 * kDP + 4;
    static constexpr int kWarpO = kJoin * 4 * kLine;             // floats
    static constexpr int kOffO = kRing;
    static constexpr int kOffQ = kOffO + kWarps * kWarpO * 4;    // Q fragments (kNT > 1)
    static constexpr int kOffM = kOffQ + (kNT > 1 ? kNT * (kDP / 16) * 32 * 8 : 0);
    static constexpr int kSmem = kOffM + kWarps * kRows * 2 * 4 + 2 * kRows * 4;
    static_assert(kSmem <= 232448 - 1024, "shared memory per block");
};

struct Params4 {
    AttnArgs a;
    const uint8_t* k;
    const uint8_t* v;
    const uint8_t* k_sf;
    const uint8_t* v_sf;
    int64_t page_stride, sf_stride;
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
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t y;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
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
// n bytes of global memory into shared memory; `real` 0: zeros instead.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t real)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real) : "memory");
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

template <int kDP, int kNT>
__global__ void __launch_bounds__(Cfg4<kDP, kNT>::kThreads, 1) attn4_kernel(const __grid_constant__ Params4 prm)
{
    using C = Cfg4<kDP, kNT>;
    constexpr int kSteps = kDP / 16;           // MMAs over a key's columns; of 16 columns of O
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_last;
    const AttnArgs& a = prm.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
    const int cta = blockIdx.x, D = a.head_dim, nb = D / 16;
    uint8_t* ring = smem + warp * (C::kStages * C::kStageBytes);
    const uint32_t ring_addr = smem_u32(ring);
    float* o_all = reinterpret_cast<float*>(smem + C::kOffO);
    float* m_all = reinterpret_cast<float*>(smem + C::kOffM);              // [warp][row][m, l]
    float* ml_row = m_all + C::kWarps * C::kRows * 2;                      // [row][m, l] of the piece
    uint2* q_frag = reinterpret_cast<uint2*>(smem + C::kOffQ);             // [tile][step][lane]

    griddep_launch_dependents();
    if (D < kDP)                                // the columns that no copy writes are zeros
        for (int i = tid; i < C::kRing / 16; i += C::kThreads) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
    griddep_wait();
    __syncthreads();

    // this lane's chunks of a group's codes: 16 bytes each where a row is whole
    // chunks, else 8
    const int chunk = D % 32 == 0 ? 16 : 8, per_row = D / 2 / chunk, chunks = kGroupKeys * per_row;
    int to[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int c = lane + 32 * i;
        to[i] = (c / per_row) * C::kRowBytes + (c % per_row) * chunk;
    }
    const float k_g = *a.k_g, v_g = *a.v_g;
    const float c_all = a.scale * kLog2e;
    const int key_row = (g >> 1) + 4 * (g & 1);            // key of a group that is row g of its S^T (and 8 + it)

    Pieces pieces(a, cta);
    Piece p;
    while (pieces.next(p)) {
        const int rows = p.n_tok * a.group;
        const int32_t* table = a.block_table + p.req * a.table_ld;
        const int key_end = min((p.tile0 + p.n) * kAttnKeys, p.kv_end);
        float* part = a.partials + (2 * cta + (p.cta0 == cta ? 1 : 0)) * kAttnSlotFloats;
        const bool whole = p.parts == 1;
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += C::kRows) {
            const int t0 = r0 / a.group, t1 = (min(rows, r0 + C::kRows) - 1) / a.group;
            // keys lo .. hi - 1: some row of the pass sees them; lo_all .. hi_all - 1: all do
            const int hi = min(p.pos0 + t1 + 1, p.kv_end), hi_all = min(p.pos0 + t0 + 1, p.kv_end);
            const int lo = a.window ? max(p.pos0 + t0 + 1 - a.window, 0) : 0;
            const int lo_all = a.window ? max(p.pos0 + t1 + 1 - a.window, 0) : 0;
            const int kb = max(p.tile0 * kAttnKeys, lo) & ~(kGroupKeys - 1), ke = min(key_end, hi);
            const int groups = ke > kb ? (ke - kb + kGroupKeys - 1) / kGroupKeys : 0;
            const int mine = groups > warp ? (groups - warp + C::kWarps - 1) / C::kWarps : 0;

            // the page ids of this warp's next 32 groups, a lane each
            int ids = 0;
            auto fetch = [&](int i) {
                if (i < mine) {
                    if ((i & 31) == 0) {
                        const int k = kb + (warp + (i + lane) * C::kWarps) * kGroupKeys;
                        ids = i + lane < mine ? table[k >> prm.page_shift] : 0;
                    }
                    const int page = __shfl_sync(0xffffffffu, ids, i & 31);
                    const int k = kb + (warp + i * C::kWarps) * kGroupKeys;
                    const bool ok = page >= 0 && page < prm.pages;
                    const int64_t pg = ok ? page : 0;
                    const int row = (p.hk << prm.page_shift) + (k & ((1 << prm.page_shift) - 1));
                    const uint8_t* ck = prm.k + pg * prm.page_stride + (int64_t)row * (D / 2);
                    const uint8_t* cv = prm.v + pg * prm.page_stride + (int64_t)row * (D / 2);
                    const uint32_t st = ring_addr + (i % C::kStages) * C::kStageBytes;
                    if (chunk == 16) {
#pragma unroll
                        for (int x = 0; x < (kDP == 128 ? 2 : 1); x++)
                            if (lane + 32 * x < chunks) {
                                copy16(st + to[x], ck + (lane + 32 * x) * 16, ok ? 16 : 0);
                                copy16(st + C::kCodes + to[x], cv + (lane + 32 * x) * 16, ok ? 16 : 0);
                            }
                    } else {
#pragma unroll
                        for (int x = 0; x < (kDP == 128 ? 4 : 2); x++)
                            if (lane + 32 * x < chunks) {
                                copy8(st + to[x], ck + (lane + 32 * x) * 8, ok ? 8 : 0);
                                copy8(st + C::kCodes + to[x], cv + (lane + 32 * x) * 8, ok ? 8 : 0);
                            }
                    }
                    // 16 keys' scales are D bytes
                    const bool is_v = lane >= 16;
                    if ((lane & 15) < nb)
                        copy16(st + 2 * C::kCodes + (is_v ? C::kScales : 0) + (lane & 15) * 16,
                               (is_v ? prm.v_sf : prm.k_sf) + pg * prm.sf_stride + (int64_t)row * nb + (lane & 15) * 16,
                               ok ? 16 : 0);
                }
                copies_end();
            };
#pragma unroll
            for (int i = 0; i < C::kStages - 1; i++) fetch(i);

            // Q of the pass: row g of tile n, columns kDP / 4 * j .. of this lane
            uint32_t q[2 * kSteps];                        // (kNT 1; else in shared memory)
            float cf[kNT][2];
#pragma unroll
            for (int n = 0; n < kNT; n++) {
                const int r = r0 + 8 * n + g, t = r / a.group;
                const bool here = r < rows;
                uint32_t raw[kDP / 8];                     // this lane's kDP / 4 columns
                const __nv_bfloat16* src =
                    prm.q + (int64_t)(p.tok0 + t) * prm.ldq + (int64_t)(p.hk * a.group + r - t * a.group) * prm.hq + j * (kDP / 4);
                float amax = 0.0f;
#pragma unroll
                for (int x = 0; x < kDP / 32; x++) {
                    uint4 y = make_uint4(0, 0, 0, 0);
                    if (here && j * (kDP / 4) + 8 * x < D) y = *reinterpret_cast<const uint4*>(src + 8 * x);
                    raw[4 * x] = y.x, raw[4 * x + 1] = y.y, raw[4 * x + 2] = y.z, raw[4 * x + 3] = y.w;
                }
#pragma unroll
                for (int x = 0; x < kDP / 8; x++) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(raw[x])), fabsf(bf16_hi(raw[x]))));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                // times 2^(141 - e), e the largest's biased exponent: it is then
                // 2^14 .. 2^15; and back in the row's factor
                const int e = max((int)(__float_as_uint(amax) >> 23), 15);
                const float up = __uint_as_float((uint32_t)(268 - e) << 23), down = __uint_as_float((uint32_t)(e - 14) << 23);
                uint32_t f[kDP / 8];
#pragma unroll
                for (int x = 0; x < kDP / 8; x++) f[x] = cvt_f16x2(bf16_lo(raw[x]) * up, bf16_hi(raw[x]) * up);
                if (kNT == 1) {
#pragma unroll
                    for (int x = 0; x < kDP / 8; x++) q[x] = f[x];
                } else if (warp == 0) {
#pragma unroll
                    for (int s = 0; s < kSteps; s++) q_frag[(n * kSteps + s) * 32 + lane] = make_uint2(f[2 * s], f[2 * s + 1]);
                }
                const float c = c_all * k_g * down;
                cf[n][0] = __shfl_sync(0xffffffffu, c, 8 * j);
                cf[n][1] = __shfl_sync(0xffffffffu, c, 8 * j + 4);
            }
            if (kNT > 1) __syncthreads();

            float o[kNT][kSteps][4], m[kNT][2], l[kNT][2];
#pragma unroll
            for (int n = 0; n < kNT; n++) {
#pragma unroll
                for (int s = 0; s < kSteps; s++) o[n][s][0] = o[n][s][1] = o[n][s][2] = o[n][s][3] = 0.0f;
                m[n][0] = m[n][1] = -INFINITY;
                l[n][0] = l[n][1] = 0.0f;
            }
#pragma unroll 1
            for (int i = 0; i < mine; i++) {
                copies_wait<C::kStages - 2>();
                __syncwarp();
                const uint8_t* st = ring + (i % C::kStages) * C::kStageBytes;
                const uint8_t* sf = st + 2 * C::kCodes;
                const int k0 = kb + (warp + i * C::kWarps) * kGroupKeys;
                const bool edge = k0 < lo_all || k0 + kGroupKeys > hi_all || k0 + kGroupKeys > key_end;
                // ---- S^T = K Q^T
                uint32_t w[2][kDP / 32];                   // codes of keys key_row and 8 + key_row
                uint32_t sc[2][kDP / 64];                  // their scales, twice each
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int key = key_row + 8 * h;
                    if (kDP == 128) {
                        const uint4 x = *reinterpret_cast<const uint4*>(st + key * C::kRowBytes + j * 16);
                        w[h][0] = x.x, w[h][1] = x.y, w[h][kDP / 32 - 2] = x.z, w[h][kDP / 32 - 1] = x.w;
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2*>(st + key * C::kRowBytes + j * 8);
                        w[h][0] = x.x, w[h][1] = x.y;
                    }
#pragma unroll
                    for (int b = 0; b < kDP / 64; b++) {
                        const int blk = j * (kDP / 64) + b;
                        const uint32_t y = blk < nb ? sf[key * nb + blk] : 0u;
                        sc[h][b] = e4m3x2_to_f16x2(y * 0x101u);
                    }
                }
                float s[kNT][4];
#pragma unroll
                for (int n = 0; n < kNT; n++) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
                for (int x = 0; x < kSteps; x++) {
                    uint32_t f[4];
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const uint32_t y = w[h][x >> 1] >> (16 * (x & 1)), z = sc[h][x / 4];
                        f[h] = mul_f16x2(e2m1x2_to_f16x2(y & 0xffu), z);
                        f[2 + h] = mul_f16x2(e2m1x2_to_f16x2(y >> 8 & 0xffu), z);
                    }
#pragma unroll
                    for (int n = 0; n < kNT; n++) {
                        if (kNT == 1) {
                            mma16816(s[n], f, q[2 * x], q[2 * x + 1]);
                        } else {
                            const uint2 b = q_frag[(n * kSteps + x) * 32 + lane];
                            mma16816(s[n], f, b.x, b.y);
                        }
                    }
                }
                // ---- softmax
#pragma unroll
                for (int n = 0; n < kNT; n++) {
#pragma unroll
                    for (int y = 0; y < 4; y++) s[n][y] *= cf[n][y & 1];
                }
                if (edge) {
#pragma unroll
                    for (int n = 0; n < kNT; n++) {
#pragma unroll
                        for (int y = 0; y < 4; y++) {
                            const int pos = p.pos0 + (r0 + 8 * n + 2 * j + (y & 1)) / a.group;
                            const int key = k0 + key_row + 8 * (y >> 1);
                            const bool seen = key <= pos && key < key_end && (!a.window || key > pos - a.window);
                            if (!seen) s[n][y] = -INFINITY;
                        }
                    }
                }
                bool up = false;
#pragma unroll
                for (int n = 0; n < kNT; n++) {
#pragma unroll
                    for (int y = 0; y < 2; y++) {
                        const float top = fmaxf(s[n][y], s[n][y + 2]);
                        up |= top > m[n][y] + kLazy;
                    }
                }
                if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                    for (int n = 0; n < kNT; n++) {
#pragma unroll
                        for (int y = 0; y < 2; y++) {
                            float top = fmaxf(s[n][y], s[n][y + 2]);
#pragma unroll
                            for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                            top = fmaxf(top, m[n][y]);
                            const float f = m[n][y] == -INFINITY ? 0.0f : ex2(m[n][y] - top);
                            m[n][y] = top;
                            l[n][y] *= f;
#pragma unroll
                            for (int x = 0; x < kSteps; x++) {
                                o[n][x][y] *= f;
                                o[n][x][y + 2] *= f;
                            }
                        }
                    }
                }
                uint32_t pt[kNT][2];
#pragma unroll
                for (int n = 0; n < kNT; n++) {
                    float e[4];
#pragma unroll
                    for (int y = 0; y < 4; y++) {
                        const float ms = m[n][y & 1] == -INFINITY ? 0.0f : m[n][y & 1];
                        e[y] = ex2(s[n][y] - ms + kLift);
                        l[n][y & 1] += e[y];
                    }
                    pt[n][0] = transpose8x8(cvt_f16x2(e[0], e[1]));
                    pt[n][1] = transpose8x8(cvt_f16x2(e[2], e[3]));
                }
                // ---- O^T += V^T P^T: keys j, j + 4 and j + 8, j + 12, columns kDP / 8 * g ..
                constexpr int kVW = kDP / 64;              // words of a key's codes
                const uint8_t* sv = st + C::kCodes;
                uint32_t v[4][kVW], vs[2];
                {
                    const int blk = kDP == 128 ? g : g >> 1;
                    uint32_t b[4];
#pragma unroll
                    for (int h = 0; h < 4; h++) {
                        const int key = j + 4 * h;
                        if (kVW == 2) {
                            const uint2 x = *reinterpret_cast<const uint2*>(sv + key * C::kRowBytes + g * 8);
                            v[h][0] = x.x, v[h][kVW - 1] = x.y;
                        } else {
                            v[h][0] = *reinterpret_cast<const uint32_t*>(sv + key * C::kRowBytes + g * 4);
                        }
                        b[h] = blk < nb ? sf[C::kScales + key * nb + blk] : 0u;
                        // a value that no row sees may be anything
                        if (edge && (k0 + key < lo || k0 + key >= ke)) b[h] = 0u;
                    }
                    vs[0] = e4m3x2_to_f16x2(b[0] | b[1] << 8);
                    vs[1] = e4m3x2_to_f16x2(b[2] | b[3] << 8);
                }
#pragma unroll
                for (int y = 0; y < kVW; y++) {
                    uint32_t even[2], odd[2];              // codes of two keys side by side, of even and odd columns
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const uint32_t x0 = v[2 * h][y], x1 = v[2 * h + 1][y];
                        even[h] = (x0 & 0x0f0f0f0fu) | (x1 << 4 & 0xf0f0f0f0u);
                        odd[h] = (x0 >> 4 & 0x0f0f0f0fu) | (x1 & 0xf0f0f0f0u);
                    }
#pragma unroll
                    for (int x = 0; x < 4; x++) {
                        uint32_t f[4];
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            f[2 * h] = mul_f16x2(e2m1x2_to_f16x2(even[h] >> 8 * x & 0xffu), vs[h]);
                            f[2 * h + 1] = mul_f16x2(e2m1x2_to_f16x2(odd[h] >> 8 * x & 0xffu), vs[h]);
                        }
#pragma unroll
                        for (int n = 0; n < kNT; n++) mma16816(o[n][4 * y + x], f, pt[n][0], pt[n][1]);
                    }
                }
                __syncwarp();                              // the stage has been read
                fetch(i + C::kStages - 1);
            }

            // ---- the warps' shares of the pass together
#pragma unroll
            for (int n = 0; n < kNT; n++) {
#pragma unroll
                for (int y = 0; y < 2; y++) {
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) l[n][y] += __shfl_xor_sync(0xffffffffu, l[n][y], x);
                    if (g == 0)
                        reinterpret_cast<float2*>(m_all)[warp * C::kRows + 8 * n + 2 * j + y] = make_float2(m[n][y], l[n][y]);
                }
            }
            __syncthreads();
            if (tid < C::kRows) {
                float top = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int x = 0; x < C::kWarps; x++) top = fmaxf(top, m_all[2 * (x * C::kRows + tid)]);
                const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
                for (int x = 0; x < C::kWarps; x++) {
                    const float2 ml = reinterpret_cast<const float2*>(m_all)[x * C::kRows + tid];
                    sum += ml.y * ex2(ml.x - ref);
                }
                reinterpret_cast<float2*>(ml_row)[tid] = make_float2(top, sum);
            }
            __syncthreads();
#pragma unroll
            for (int n0 = 0; n0 < kNT; n0 += C::kJoin) {
#pragma unroll
                for (int n = n0; n < n0 + C::kJoin; n++) {
#pragma unroll
                    for (int y = 0; y < 2; y++) {
                        const float top = ml_row[2 * (8 * n + 2 * j + y)];
                        const float f = m[n][y] == -INFINITY ? 0.0f : ex2(m[n][y] - top);
                        float4* to4 = reinterpret_cast<float4*>(o_all + warp * C::kWarpO + ((n - n0) * 4 + j) * C::kLine +
                                                                y * kDP + g * (kDP / 8));
#pragma unroll
                        for (int x = 0; x < kSteps; x += 2) {
                            // (what a warp without a key of this row has is not to be counted, whatever it is)
                            to4[x / 2] = f == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                                                   : make_float4(o[n][x][y] * f, o[n][x][y + 2] * f, o[n][x + 1][y] * f,
                                                                 o[n][x + 1][y + 2] * f);
                        }
                    }
                }
                __syncthreads();
                // a thread adds two columns of a row over the warps
                for (int x = tid; x < C::kJoin * 8 * (kDP / 2); x += C::kThreads) {
                    const int rr = x / (kDP / 2), col = 2 * (x % (kDP / 2)), r = r0 + 8 * n0 + rr;
                    if (r >= rows || col >= D) continue;
                    const float* from = o_all + (rr >> 1) * C::kLine + (rr & 1) * kDP + col;
                    float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int y = 0; y < C::kWarps; y++) {
                        const float2 e = *reinterpret_cast<const float2*>(from + y * C::kWarpO);
                        acc.x += e.x;
                        acc.y += e.y;
                    }
                    if (whole) {
                        const float sum = ml_row[2 * (8 * n0 + rr) + 1];
                        const float inv = sum == 0.0f ? 0.0f : v_g / sum;
                        const int t = r / a.group;
                        *reinterpret_cast<uint32_t*>(a.out + (int64_t)(p.tok0 + t) * a.ldo +
                                                     (int64_t)(p.hk * a.group + r - t * a.group) * a.ho + col) =
                            sum == 0.0f ? 0u : cvt_bf16x2(acc.x * inv, acc.y * inv);
                    } else {
                        __stcg(reinterpret_cast<float2*>(part + r * kDP + col), acc);
                    }
                }
                __syncthreads();
            }
            if (tid < C::kRows && r0 + tid < rows) {
                const int r = r0 + tid, t = r / a.group;
                const float2 ml = reinterpret_cast<const float2*>(ml_row)[tid];
                if (!whole)
                    __stcg(reinterpret_cast<float2*>(part + kAttnSlotRows * kDP + 2 * r), ml);
                else if (a.lse)
                    a.lse[(int64_t)(p.tok0 + t) * a.heads + p.hk * a.group + r - t * a.group] =
                        ml.y == 0.0f ? -INFINITY : (ml.x - kLift + log2f(ml.y)) * 0.6931471805599453f;
            }
        }
        if (whole) continue;

        // ---- a shared item: the last of its CTAs adds the parts up
        __syncthreads();
        int* ticket = a.tickets + p.cta0 * 8;
        if (tid == 0) {
            s_last = atom_add_acq_rel(ticket, 1) == p.parts - 1;
            if (s_last) *ticket = 0;
        }
        __syncthreads();
        if (!s_last) continue;
        // part i of the item is in slot 2 (cta0 + i), the first in 2 cta0 + 1
        auto slot_of = [&](int i) { return a.partials + (2 * (p.cta0 + i) + (i == 0 ? 1 : 0)) * kAttnSlotFloats; };
        for (int x = tid; x < rows * (kDP / 2); x += C::kThreads) {
            const int r = x / (kDP / 2), col = 2 * (x % (kDP / 2));
            if (col >= D) continue;
            const int t = r / a.group, head = p.hk * a.group + r - t * a.group;
            float top = -INFINITY, sum = 0.0f;
            float2 acc = make_float2(0.0f, 0.0f);
            for (int i0 = 0; i0 < p.parts; i0 += 8) {
                float2 ml[8], e[8];
#pragma unroll
                for (int u = 0; u < 8; u++) {
                    const float* from = slot_of(min(i0 + u, p.parts - 1));
                    ml[u] = __ldcg(reinterpret_cast<const float2*>(from + kAttnSlotRows * kDP + 2 * r));
                    e[u] = __ldcg(reinterpret_cast<const float2*>(from + r * kDP + col));
                    if (i0 + u >= p.parts) ml[u] = make_float2(-INFINITY, 0.0f);
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
            *reinterpret_cast<uint32_t*>(a.out + (int64_t)(p.tok0 + t) * a.ldo + (int64_t)head * a.ho + col) =
                sum == 0.0f ? 0u : cvt_bf16x2(acc.x * inv, acc.y * inv);
            if (col == 0 && a.lse)
                a.lse[(int64_t)(p.tok0 + t) * a.heads + head] =
                    sum == 0.0f ? -INFINITY : (top - kLift + log2f(sum)) * 0.6931471805599453f;
        }
        __syncthreads();                                   // (s_last)
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

template <int kDP, int kNT>
cudaError_t launch4(const Params4& p, int ctas, cudaStream_t stream)
{
    using C = Cfg4<kDP, kNT>;
    static int attr_set_for_device[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && !attr_set_for_device[dev]) {
        e = cudaFuncSetAttribute(attn4_kernel<kDP, kNT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        attr_set_for_device[dev] = 1;
    }
    return launch_programmatic(attn4_kernel<kDP, kNT>, dim3((unsigned)ctas), dim3(C::kThreads), C::kSmem, stream, p);
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
    p.page_stride = cache.page_stride;
    p.sf_stride = cache.sf_stride;
    p.q = q;
    p.ldq = ldq;
    p.hq = hq;
    p.pages = (int)cache.pages;
    while ((1 << p.page_shift) < cache.page_size) p.page_shift++;
    const int ctas = num_sms < kAttnMaxCtas ? num_sms : kAttnMaxCtas;
    // rows of a request, on average: one tile of 8, two, or passes of four
    const int64_t rows = (args.tokens + requests - 1) / requests * args.group;
    if (cache.head_dim > 64)
        return rows <= 8    ? launch4<128, 1>(p, ctas, stream)
               : rows <= 16 ? launch4<128, 2>(p, ctas, stream)
                            : launch4<128, 4>(p, ctas, stream);
    return rows <= 8    ? launch4<64, 1>(p, ctas, stream)
           : rows <= 16 ? launch4<64, 2>(p, ctas, stream)
                        : launch4<64, 4>(p, ctas, stream);
}

}  // namespace nvfp4
