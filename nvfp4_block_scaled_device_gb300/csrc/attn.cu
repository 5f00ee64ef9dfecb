// Causal attention with grouped heads on the tensor cores, over packed
// prompts or the paged cache:
//   s_j = scale * q.k_j over the keys j a row sees, out = sum_j softmax_j(s) v_j.
//
// One pass over the keys per work item (the schedule in attn.h): row tiles of
// 128 rows -- the query heads of one kv head for consecutive tokens, so a key
// tile is read once for the whole group -- against key tiles of 128 keys.
//   S = Q K^T      tcgen05.mma kind::f16 (bf16, fp32 accumulation), operands
//                  in shared memory (TMA, 128-byte swizzle), S in tensor memory
//   P = 2^(c s - c m), c = scale * log2(e), m a running row maximum: one row
//                  per thread, S read from and P (bf16) written to tensor
//                  memory, the row's sum of P kept in fp32
//   O += P V       tcgen05.mma with P from tensor memory, V in shared memory
//                  (as stored, keys by columns: the MMA's N-major form), O in
//                  tensor memory
// m only moves when a row's maximum has risen by more than 2^8 (kLazy) since
// m was set: P stays below 2^8, its bf16 rounding is relative, and O is
// rescaled a few times per row instead of at every key tile.
//
// Two softmax warpgroups work on two tiles at a time, so that the tensor
// pipe multiplies for one while the other is in its softmax.  An item with
// more than 128 rows has two row tiles, one per warpgroup, on the same keys;
// one with at most 128 rows (decoding) gives the even key tiles to the first
// and the odd ones to the second, which the first merges at the end.
//
// Items are cut at CTA boundaries (equal key tiles per CTA).  A CTA's part of
// a shared item goes to the workspace as fp32 (O, m, l); the CTA whose warp
// takes a part's last ticket adds the parts up in CTA order (the same result
// whatever the order of arrival).  No CTA waits for another.
//
// Warps: 0-3 and 4-7 softmax and epilogue; 8 and 9 the MMAs of the first and
// the second warpgroup (one warp's instruction stream for both would take
// longer than the MMAs themselves); 10 K/V copies; 11 Q copies and the keys'
// end (below).
//
// Rows past the last key of an item's last tile hold other requests' rows,
// pages' unused rows or nothing at all.  Their scores are masked, and warp 11
// zeroes the V rows before the tile is multiplied, so that NaN or infinities
// there cannot reach a sum as 0 * NaN.
//
// The softmax is one small loop over 64 keys at a time: the warps of a CTA run
// four different programs, and code that is run only now and then (masks, a
// risen maximum, an item's end) is fetched from far when it is; unrolled
// copies of it cost thousands of cycles an item.
#include "attn.h"
#include "common.cuh"
#include "internal.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 384;
constexpr int kWarpMma = 8, kWarpKV = 10, kWarpQ = 11;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColS = 256;      // + 128 * warpgroup; P of 64 keys over the first 32 columns of their S
constexpr float kLazy = 8.0f;                   // log2 of the growth that P may carry
constexpr int kRegsSoftmax = 192, kRegsOther = 120;
static_assert(2 * kRegsSoftmax + kRegsOther <= 3 * 168, "the block's registers at launch");

constexpr int kMaxStages = 10;
constexpr int kJoin = 8;                        // vectors of a shared item's parts under way per lane

struct Ctrl {
    uint64_t kv_full[kMaxStages], kv_empty[kMaxStages], v_end[kMaxStages];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_half[2], p_full[2], o_half[2], o_full[2], o_free[2];
    uint64_t ml_full[4];
    uint64_t turn[2][4];
    uint64_t teardown;
    uint32_t tmem_base;
    int abort_flag;
    uint32_t issued;                            // ring stages whose copies have begun
    float m[kAttnRows], l[kAttnRows];           // second warpgroup's statistics (merge)
};

template <int kDP>   // columns of a head, padded: 64 or 128
struct Cfg {
    static constexpr int kTileBytes = 128 * kDP * 2;
    static constexpr int kStages = kDP == 128 ? 5 : 10;
    static constexpr int kHalves = kDP / 64;    // 64-column halves, 16 KB each
    static constexpr int kOffRing = 2 * kTileBytes;
    static constexpr int kOffCtrl = kOffRing + kStages * kTileBytes;
    static constexpr int kSmemBytes = kOffCtrl + (int)sizeof(Ctrl) + 1024;
    static_assert(kSmemBytes <= 232448, "shared memory per block");
    static_assert(kStages <= kMaxStages, "barriers");
};

struct Params {
    CUtensorMap map_q, map_k, map_v;
    AttnArgs a;
};

// ------------------------------------------------------------ instructions
// Instruction descriptor, kind::f16: fp32 D, bf16 A and B, M = 128; B of the
// second product is N-major (bit 16).
__host__ __device__ constexpr uint32_t idesc_of(int n, bool b_n_major)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_n_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((128u >> 4) << 24);
}

// The tensor-core products of one step, each issued by one elected lane of the
// converged warp from a single asm block (see stage_issue_1sm).
// S = Q K^T: operands as 128-byte swizzled rows, K-major; K = 16 columns an
// MMA, 64-column halves 16 KB apart.
template <int kDP>
__device__ __forceinline__ void issue_qk(uint32_t s, uint32_t q_lo, uint32_t k_lo, uint32_t hi, uint32_t idesc)
{
    if (kDP == 128)
        asm volatile(
        "{\n .reg .pred e, pf, pt;\n .reg .b32 r, x, y;\n .reg .b64 da, db;\n"
        " elect.sync r|e, 0xffffffff;\n setp.eq.b32 pt, 0, 0;\n setp.ne.b32 pf, 0, 0;\n"
        " add.u32 x, %1, 0; add.u32 y, %2, 0; mov.b64 da, {x, %3}; mov.b64 db, {y, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pf;\n"
        " add.u32 x, %1, 2; add.u32 y, %2, 2; mov.b64 da, {x, %3}; mov.b64 db, {y, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pt;\n"
        " add.u32 x, %1, 4; add.u32 y, %2, 4; mov.b64 da, {x, %3}; mov.b64 db, {y, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pt;\n"
        " add.u32 x, %1, 6; add.u32 y, %2, 6; mov.b64 da, {x, %3}; mov.b64 db, {y, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pt;\n"
        " add.u32 x, %1, 1024; add.u32 y, %2, 1024; mov.b64 da, {x, %3}; mov.b64 db, {y, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pt;\n"
        " add.u32 x, %1, 1026; add.u32 y, %2, 1026; mov.b64 da, {x, %3}; mov.b64 db, {y, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pt;\n"
        " add.u32 x, %1, 1028; add.u32 y, %2, 1028; mov.b64 da, {x, %3}; mov.b64 db, {y, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pt;\n"
        " add.u32 x, %1, 1030; add.u32 y, %2, 1030; mov.b64 da, {x, %3}; mov.b64 db, {y, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pt;\n"
        "}\n" ::"r"(s), "r"(q_lo), "r"(k_lo), "r"(hi), "r"(idesc)
        : "memory");
    else
        asm volatile(
        "{\n .reg .pred e, pf, pt;\n .reg .b32 r, x, y;\n .reg .b64 da, db;\n"
        " elect.sync r|e, 0xffffffff;\n setp.eq.b32 pt, 0, 0;\n setp.ne.b32 pf, 0, 0;\n"
        " add.u32 x, %1, 0; add.u32 y, %2, 0; mov.b64 da, {x, %3}; mov.b64 db, {y, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pf;\n"
        " add.u32 x, %1, 2; add.u32 y, %2, 2; mov.b64 da, {x, %3}; mov.b64 db, {y, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pt;\n"
        " add.u32 x, %1, 4; add.u32 y, %2, 4; mov.b64 da, {x, %3}; mov.b64 db, {y, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pt;\n"
        " add.u32 x, %1, 6; add.u32 y, %2, 6; mov.b64 da, {x, %3}; mov.b64 db, {y, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pt;\n"
        "}\n" ::"r"(s), "r"(q_lo), "r"(k_lo), "r"(hi), "r"(idesc)
        : "memory");
}
// O += P V over 64 keys: P in tensor memory (8 columns for 16 keys), V as
// stored (N-major; 16 keys are 2 KB).
__device__ __forceinline__ void issue_pv(uint32_t o, uint32_t p, uint32_t v_lo, uint32_t hi, uint32_t idesc,
                                         uint32_t acc)
{
    asm volatile(
        "{\n .reg .pred e, p, pt;\n .reg .b32 r, x, y;\n .reg .b64 db;\n"
        " elect.sync r|e, 0xffffffff;\n setp.eq.b32 pt, 0, 0;\n setp.ne.b32 p, %5, 0;\n"
        " add.u32 x, %2, 0; mov.b64 db, {x, %3}; add.u32 y, %1, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], db, %4, p;\n"
        " add.u32 x, %2, 128; mov.b64 db, {x, %3}; add.u32 y, %1, 8;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], db, %4, pt;\n"
        " add.u32 x, %2, 256; mov.b64 db, {x, %3}; add.u32 y, %1, 16;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], db, %4, pt;\n"
        " add.u32 x, %2, 384; mov.b64 db, {x, %3}; add.u32 y, %1, 24;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], db, %4, pt;\n"
        "}\n" ::"r"(o), "r"(p), "r"(v_lo), "r"(hi), "r"(idesc), "r"(acc)
        : "memory");
}

// One poll, without waiting (warp-uniform).
__device__ __forceinline__ bool mbar_test_warp(uint32_t bar, uint32_t parity)
{
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                            int w)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v)
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = __uint_as_float(r[i]);
}
// 32 columns of 16 rows in the layout of the warp-level MMAs' accumulators:
// v[4i + 2b + x] is row lane / 4 + 8b, column 8i + 2 (lane % 4) + x.
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, float* v)
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = __uint_as_float(r[i]);
}
// 4 x 4 transpose among four lanes: lane q's a[m] becomes lane m's a[q].
__device__ __forceinline__ void quad_transpose(uint32_t* a, int q)
{
    const bool b0 = q & 1, b1 = q & 2;
    uint32_t x = __shfl_xor_sync(0xffffffffu, b0 ? a[0] : a[1], 1);
    uint32_t y = __shfl_xor_sync(0xffffffffu, b0 ? a[2] : a[3], 1);
    (b0 ? a[0] : a[1]) = x;
    (b0 ? a[2] : a[3]) = y;
    x = __shfl_xor_sync(0xffffffffu, b1 ? a[0] : a[2], 2);
    y = __shfl_xor_sync(0xffffffffu, b1 ? a[1] : a[3], 2);
    (b1 ? a[0] : a[2]) = x;
    (b1 ? a[1] : a[3]) = y;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two binary32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
        " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
        " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ int atom_add_acq_rel(int* p, int v)
{
    int old;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

// The MMA warp's waits: mbar_wait_warp with less code around the poll.
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status, int site)
{
    if (mbar_test_warp(bar, parity)) return true;
    const uint32_t t0 = (uint32_t)clock64();
    while (!mbar_poll_warp<false>(bar, parity)) {
        const bool late = (uint32_t)clock64() - t0 > 0xE0000000u;      // about 2 s
        if (__any_sync(0xffffffffu, late || *abort_flag)) {
            if (late && *abort_flag == 0) atomicCAS(status, 0, kErrTimeout * 100 + site);
            *abort_flag = 1;
            return false;
        }
    }
    return true;
}

// Waits for the ring's stage use `use` to be full.  A warp that leaves uses to
// the other MMA warp has not seen their phases end, and a parity wait is only
// right from the phase before on: so first the copies of this use have begun,
// which they do once the stage's use before has been consumed.
__device__ __forceinline__ bool wait_use(const volatile uint32_t* issued, uint32_t use, uint32_t bar, uint32_t parity,
                                         volatile int* abort_flag, int* status, int site)
{
    if (__any_sync(0xffffffffu, (int32_t)(*issued - use) <= 0)) {
        const uint32_t t0 = (uint32_t)clock64();
        while (__any_sync(0xffffffffu, (int32_t)(*issued - use) <= 0)) {
            const bool late = (uint32_t)clock64() - t0 > 0xE0000000u;
            if (__any_sync(0xffffffffu, late || *abort_flag)) {
                if (late && *abort_flag == 0) atomicCAS(status, 0, kErrTimeout * 100 + site);
                *abort_flag = 1;
                return false;
            }
        }
    }
    return wait_on(bar, parity, abort_flag, status, site);
}

__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// What is done to a row's 128 scores in tensor memory before the softmax reads
// them: the sign of a negative scale, -inf at keys outside lw .. h - 1.
__device__ __forceinline__ void edit_scores(uint32_t taddr, bool negate, int h, int lw)
{
#pragma unroll 1
    for (int x = 0; x < 128; x += 32) {
        const uint32_t seen = low_bits(h - x) & ~low_bits(lw - x);
        if (!negate && __all_sync(0xffffffffu, seen == ~0u)) continue;
        float s[32];
        tmem_ld32(taddr + x, s);
        tmem_ld_wait();
        uint32_t r[32];
#pragma unroll
        for (int k = 0; k < 32; k++)
            r[k] = (seen >> k) & 1u ? __float_as_uint(s[k]) ^ (negate ? 0x80000000u : 0u) : 0xff800000u;
        tmem_st32(taddr + x, r);
    }
    tmem_st_wait();
}

// P of 64 keys: e = 2^(c s + mc) as bf16 pairs; returns the sum of e.
__device__ __forceinline__ float exp_scores(const float* s, float c, float mc, uint32_t* r)
{
    float2 sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
    for (int y = 0; y < 32; y++) {
        float2 e = fma2(make_float2(s[2 * y], s[2 * y + 1]), make_float2(c, c), make_float2(mc, mc));
        e.x = ex2(e.x);
        e.y = ex2(e.y);
        sum[y & 1] = add2(sum[y & 1], e);
        r[y] = cvt_bf16x2(e.x, e.y);
    }
    sum[0] = add2(sum[0], sum[1]);
    return sum[0].x + sum[0].y;
}

__device__ __forceinline__ float max_scores(const float* s)
{
    float x[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int k = 4; k < 60; k += 8) {
#pragma unroll
        for (int y = 0; y < 4; y++) x[y] = max3(x[y], s[k + 2 * y], s[k + 2 * y + 1]);
    }
#pragma unroll
    for (int y = 0; y < 4; y++) x[y] = fmaxf(x[y], s[60 + y]);
    return fmaxf(max3(x[0], x[1], x[2]), x[3]);
}

// ------------------------------------------------------------------ pieces
// A CTA's share of one item.
struct Piece {
    int tok0, n_tok, req, pos0, kv_end, kv_row;   // of its QTile
    int hk;              // kv head
    int tile0, n;        // key tiles tile0 .. tile0 + n - 1
    bool two;            // two row tiles
    int cta0, parts;     // first CTA of the item and how many share it

    // Tiles lo .. hi - 1 of the piece that rows of row tile j see (one at
    // least, so that rows that see no key are written too).
    __device__ __forceinline__ void range(int j, int row_tokens, int window, int& lo, int& hi) const
    {
        lo = 0;
        hi = n;
        if (!two) return;
        const int first = pos0 + j * row_tokens, last = pos0 + min(n_tok, (j + 1) * row_tokens) - 1;
        const int lo_key = window ? max(first + 1 - window, 0) : 0, hi_key = min(last + 1, kv_end);
        lo = min(max(lo_key / kAttnKeys - tile0, 0), n - 1);
        hi = min(max((hi_key - 1) / kAttnKeys + 1 - tile0, lo + 1), n);
    }
};

// The pieces of CTA `cta` in order; every warp of the CTA walks them alike.
// kAhead: the next QTile is fetched while the current one is worked on.
template <bool kAhead>
struct Pieces {
    const int4* table;
    int u, end, per_cta, qt, kv_heads, row_tokens;
    int4 f0, f1, f2;     // QTile qt, or (kAhead) the one that comes next

    __device__ __forceinline__ Pieces(const AttnArgs& a, int cta)
    {
        const ScheduleHead* s = a.sched;
        table = reinterpret_cast<const int4*>(schedule_tiles(s));
        kv_heads = a.kv_heads;
        row_tokens = row_tile_tokens(a.group);
        const int4* start = reinterpret_cast<const int4*>(&s->start[cta]);
        f0 = start[0];
        f1 = start[1];
        f2 = start[2];
        qt = s->first[cta];
        const int units = s->units;
        per_cta = s->per_cta;
        u = cta * per_cta < units ? cta * per_cta : units;
        end = units - u < per_cta ? units : u + per_cta;
    }
    __device__ __forceinline__ void fetch()
    {
        qt++;
        f0 = table[3 * qt];
        f1 = table[3 * qt + 1];
        f2 = table[3 * qt + 2];
    }
    __device__ __forceinline__ bool next(Piece& p)
    {
        while (u < end) {
            int rel = u - f2.x;
            if (!kAhead && rel == (kItemUnits + f1.w) * kv_heads) {
                fetch();
                rel = 0;
            }
            const int tiles = f1.w, item = kItemUnits + tiles;
            p.hk = rel / item;
            const int r0 = rel - p.hk * item, r1 = min(end - u, item - r0) + r0;   // the CTA's units of the item
            const int k0 = max(snap_unit(r0, item) - kItemUnits, 0);
            p.n = max(snap_unit(r1, item) - kItemUnits, 0) - k0;
            p.tok0 = f0.x;
            p.n_tok = f0.y;
            p.req = f0.z;
            p.pos0 = f0.w;
            p.kv_end = f1.x;
            p.kv_row = f1.y;
            p.tile0 = f1.z + k0;
            p.two = f0.y > row_tokens;
            p.cta0 = 0;
            p.parts = 1;
            if (p.n < tiles) {                           // shared with other CTAs
                const int i0 = u - r0;                   // the item's first unit
                int c0 = i0 / per_cta, c1 = (i0 + item - 1) / per_cta;
                if (snap_unit((c0 + 1) * per_cta - i0, item) == 0) c0++;
                if (c1 > c0 && snap_unit(c1 * per_cta - i0, item) == item) c1--;
                p.cta0 = c0;
                p.parts = c1 - c0 + 1;
            }
            u += r1 - r0;
            if (kAhead && rel + (r1 - r0) == item * kv_heads && u < end) fetch();
            if (p.n > 0) return true;
        }
        return false;
    }
};

// A key tile's position in the ring: tile g of the CTA has its keys in stage
// 2g % kStages, its values in the next.
template <int kStages>
__device__ __forceinline__ uint32_t stage_of(uint32_t use, uint32_t* parity)
{
    const uint32_t turn = use / kStages;
    *parity = turn & 1u;
    return use - turn * kStages;
}

template <int kDP>
__global__ void __launch_bounds__(kThreads, 1) attn_kernel(const __grid_constant__ Params prm)
{
    using C = Cfg<kDP>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw_addr);
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + C::kOffCtrl);
    volatile int* abort_flag = &ctrl->abort_flag;
    const AttnArgs& a = prm.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x;
    int* status = a.status;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; s++) {
            mbar_init(smem_u32(&ctrl->kv_full[s]), 1);
            mbar_init(smem_u32(&ctrl->kv_empty[s]), 2);      // both MMA warps
            mbar_init(smem_u32(&ctrl->v_end[s]), 1);
        }
        mbar_init(smem_u32(&ctrl->q_full), 1);
        mbar_init(smem_u32(&ctrl->q_empty), 2);
        for (int j = 0; j < 2; j++) {
            mbar_init(smem_u32(&ctrl->s_full[j]), 1);
            mbar_init(smem_u32(&ctrl->p_half[j]), 4);
            mbar_init(smem_u32(&ctrl->p_full[j]), 4);
            mbar_init(smem_u32(&ctrl->o_half[j]), 1);
            mbar_init(smem_u32(&ctrl->o_full[j]), 1);
            mbar_init(smem_u32(&ctrl->o_free[j]), 4);
        }
        for (int w = 0; w < 4; w++) {
            mbar_init(smem_u32(&ctrl->ml_full[w]), 1);
            mbar_init(smem_u32(&ctrl->turn[0][w]), 1);
            mbar_init(smem_u32(&ctrl->turn[1][w]), 1);
        }
        mbar_init(smem_u32(&ctrl->teardown), 2);
        ctrl->abort_flag = 0;
        ctrl->issued = 0;
        fence_barrier_init();
    }
    if (warp == kWarpKV && lane == 0) {
        prefetch_tmap(&prm.map_k);
        prefetch_tmap(&prm.map_v);
    }
    if (warp == kWarpQ && lane == 0) prefetch_tmap(&prm.map_q);
    if (warp == kWarpMma) {
        tmem_alloc(smem_u32(&ctrl->tmem_base), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctrl->tmem_base;
    griddep_launch_dependents();
    griddep_wait();                  // schedule, Q, K, V, outputs, workspace: after the previous kernel
    Piece p;

    if (warp >= 8) {
        Pieces<true> pieces(a, cta);
        setmaxnreg_dec<kRegsOther>();
        if (warp == kWarpKV) {
            // ------------------------------------------------ K/V copies
            const bool paged = a.block_table != nullptr;
            const int ppt = paged ? kAttnKeys / a.page_size : 1;       // pages of a key tile
            uint32_t use = 0;
            uint32_t issued = 0, issued_ph = 0;   // stages with copies under way, and whose phase
            bool ok = true;
            while (ok && pieces.next(p)) {
                const int* table = paged ? a.block_table + (int64_t)p.req * a.table_ld : nullptr;
                int lo[2], hi[2];
                for (int j = 0; j < 2; j++) p.range(j, row_tile_tokens(a.group), a.window, lo[j], hi[j]);
                for (int i = 0; i < p.n && ok; i++) {
                    const int key0 = (p.tile0 + i) * kAttnKeys;
                    const int valid = min(kAttnKeys, max(p.kv_end - key0, 0));
                    const int pages = paged ? (valid + a.page_size - 1) / a.page_size : 0;
                    int page = 0;
                    if (lane < pages) page = __ldg(table + (key0 / a.page_size) + lane);
                    for (int kv = 0; kv < 2; kv++, use++) {
                        uint32_t ph;
                        const uint32_t s = stage_of<kStages>(use, &ph);
                        if (!mbar_wait_warp(smem_u32(&ctrl->kv_empty[s]), ph ^ 1u, abort_flag, status, 41)) {
                            ok = false;
                            break;
                        }
                        if (lane == 0) *(volatile uint32_t*)&ctrl->issued = use + 1;
                        const CUtensorMap* map = kv ? &prm.map_v : &prm.map_k;
                        const uint32_t dst = base + C::kOffRing + s * C::kTileBytes;
                        // an item's last values go through warp 11
                        const uint32_t bar =
                            smem_u32(kv && valid < kAttnKeys ? &ctrl->v_end[s] : &ctrl->kv_full[s]);
                        const uint32_t bytes =
                            paged ? (uint32_t)(pages * a.page_size * kDP * 2) : (uint32_t)C::kTileBytes;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(bar, bytes);
                            // only one MMA warp will use it
                            if (!p.two || i < lo[0] || i >= hi[0] || i < lo[1] || i >= hi[1])
                                mbar_arrive(smem_u32(&ctrl->kv_empty[s]));
                        }
                        __syncwarp();
                        if (paged) {
                            // box b: half b / ppt of page b % ppt (at most 16)
                            const int b = lane, half = b / ppt, pg = b - half * ppt;
                            const int id = __shfl_sync(0xffffffffu, page, pg);
                            if (half < C::kHalves && pg < pages)
                                tma_load_4d(dst + half * 16384 + pg * a.page_size * 128, map, bar, half * 64, 0, p.hk,
                                            id);
                        } else if (lane < C::kHalves) {
                            tma_load_3d(dst + lane * 16384, map, bar, lane * 64, p.hk, p.kv_row + key0);
                        }
                        __syncwarp();
                        issued |= 1u << s;
                        issued_ph = (issued_ph & ~(1u << s)) | (ph << s);
                    }
                }
            }
            if (!ok && lane == 0) {
                // stopped early: let the copies under way land before the
                // CTA's shared memory goes away (bounded).  Values that end
                // an item complete on v_end, which has its own phases:
                // waiting on both for either phase costs time only here
                for (int s = 0; s < kStages; s++)
                    if (issued & (1u << s)) {
                        mbar_wait_teardown(smem_u32(&ctrl->kv_full[s]), (issued_ph >> s) & 1u);
                        mbar_wait_teardown(smem_u32(&ctrl->v_end[s]), 0);
                        mbar_wait_teardown(smem_u32(&ctrl->v_end[s]), 1);
                    }
            }
            __syncwarp();
        } else if (warp == kWarpQ) {
            // ------------------- Q copies, and values past the last key
            uint32_t n = 0, tile = 0, ends = 0;    // items, key tiles; ends: bit s = phase of v_end[s]
            bool ok = true;
            const int row_tokens = row_tile_tokens(a.group), rows = a.group * row_tokens;
            const uint32_t bar = smem_u32(&ctrl->q_full);
            while (pieces.next(p)) {
                if (!mbar_wait_warp(smem_u32(&ctrl->q_empty), (n & 1u) ^ 1u, abort_flag, status, 42)) {
                    ok = false;
                    break;
                }
                const int boxes = (p.two ? 2 : 1) * C::kHalves;
                if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(boxes * rows * 128));
                __syncwarp();
                if (lane < boxes) {
                    const int j = lane / C::kHalves, half = lane - j * C::kHalves;
                    tma_load_3d(base + j * C::kTileBytes + half * 16384, &prm.map_q, bar, half * 64, p.hk * a.group,
                                p.tok0 + j * row_tokens);
                }
                __syncwarp();
                n++;
                tile += p.n;
                const int valid = min(kAttnKeys, max(p.kv_end - (p.tile0 + p.n - 1) * kAttnKeys, 0));
                if (valid == kAttnKeys) continue;
                uint32_t ph;
                const uint32_t s = stage_of<kStages>(2 * (tile - 1) + 1, &ph);
                if (!mbar_wait_warp<true>(smem_u32(&ctrl->v_end[s]), (ends >> s) & 1u, abort_flag, status, 43)) {
                    ok = false;
                    break;
                }
                ends ^= 1u << s;
                uint8_t* v = smem + C::kOffRing + s * C::kTileBytes;
                const int vec = (kAttnKeys - valid) * 8;          // 16-byte vectors of a half's rows
                for (int x = lane; x < vec * C::kHalves; x += 32) {
                    const int half = x / vec, y = x - half * vec;
                    *reinterpret_cast<uint4*>(v + half * 16384 + valid * 128 + y * 16) = make_uint4(0, 0, 0, 0);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctrl->kv_full[s]));
            }
            if (!ok && n > 0 && lane == 0) mbar_wait_teardown(bar, (n - 1) & 1u);
            __syncwarp();
        } else {
            // ------------------------------------------------------- MMA
            // Warp 8 + j issues warpgroup j's products: S of a key tile, then
            // its O once P is there, then the next S into the same columns,
            // across items too.  Two row tiles: both warps use every key
            // tile; one row tile: warp j the tiles j, j + 2, ...  Either way
            // a stage is free after two commits on it.
            const int j = warp - kWarpMma;
            const uint64_t kdesc0 = make_smem_desc(base, 16, 1024, 2);       // K-major: 8-row groups 1 KB apart
            const uint64_t vdesc0 = make_smem_desc(base, 16384, 1024, 2);    // N-major: 64-column halves 16 KB
                                                                             // apart, 8-key groups 1 KB apart
            constexpr uint32_t kIdescS = idesc_of(128, false), kIdescO = idesc_of(kDP, true);
            const uint32_t k_hi = (uint32_t)(kdesc0 >> 32), v_hi = (uint32_t)(vdesc0 >> 32);
            const uint32_t q_lo = (uint32_t)kdesc0;
            const uint32_t ring_k = q_lo + (C::kOffRing >> 4), ring_v = (uint32_t)vdesc0 + (C::kOffRing >> 4);
            const uint32_t full0 = smem_u32(&ctrl->kv_full[0]), empty0 = smem_u32(&ctrl->kv_empty[0]);
            const uint32_t ts = tmem + kColS + 128u * j, to = tmem + kColO + 128u * j;
            const uint32_t s_full = smem_u32(&ctrl->s_full[j]), o_full = smem_u32(&ctrl->o_full[j]);
            const uint32_t p_half = smem_u32(&ctrl->p_half[j]), p_full = smem_u32(&ctrl->p_full[j]);
            const uint32_t o_half = smem_u32(&ctrl->o_half[j]);
            const uint32_t q_empty = smem_u32(&ctrl->q_empty);
            uint32_t use = 0;                      // stages used by the items before
            uint32_t qph = 0, pph = 0, oph = 1;    // phases: Q, P, O free (nothing to wait for at first)
            bool ok = true;
            while (ok && pieces.next(p)) {
                int first, end;
                p.range(j, row_tile_tokens(a.group), a.window, first, end);
                const int by = p.two ? 1 : 2;
                if (!p.two) first = j;
                uint32_t kph;                      // stage of the warp's next K, its phase; V is in the stage after
                uint32_t ks = stage_of<kStages>(use + 2 * first, &kph);
                const uint32_t qt = q_lo + (p.two && j ? C::kTileBytes >> 4 : 0);
                if (!wait_on(smem_u32(&ctrl->q_full), qph, abort_flag, status, 44)) break;
                qph ^= 1u;
                if (first >= end && lane == 0) mbar_arrive(q_empty);     // no tile for this warp
                for (int i = first; i < end; i += by) {
                    const uint32_t ku = use + 2u * (uint32_t)i;
                    if (!wait_use(&ctrl->issued, ku, full0 + 8u * ks, kph, abort_flag, status, 45)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    issue_qk<kDP>(ts, qt, ring_k + ks * (C::kTileBytes >> 4), k_hi, kIdescS);
                    mma_commit_warp(s_full);
                    mma_commit_warp(empty0 + 8u * ks);
                    if (i + by >= end) mma_commit_warp(q_empty);
                    const bool wrap = ks + 1 == kStages;
                    const uint32_t vs = wrap ? 0 : ks + 1, vph = wrap ? kph ^ 1u : kph;
                    // the accumulator's previous item has been read
                    if (i == first) {
                        if (!wait_on(smem_u32(&ctrl->o_free[j]), oph, abort_flag, status, 47)) {
                            ok = false;
                            break;
                        }
                        oph ^= 1u;
                    }
                    const uint32_t v_lo = ring_v + vs * (C::kTileBytes >> 4);
                    if (!wait_use(&ctrl->issued, ku + 1, full0 + 8u * vs, vph, abort_flag, status, 46) ||
                        !wait_on(p_half, pph, abort_flag, status, 48)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    issue_pv(to, ts, v_lo, v_hi, kIdescO, i != first);
                    mma_commit_warp(o_half);
                    if (!wait_on(p_full, pph, abort_flag, status, 49)) {
                        ok = false;
                        break;
                    }
                    pph ^= 1u;
                    tc_fence_after();
                    issue_pv(to, ts + 64, v_lo + (64 * 128 >> 4), v_hi, kIdescO, 1u);
                    mma_commit_warp(o_full);
                    mma_commit_warp(empty0 + 8u * vs);
                    ks += 2 * by;
                    if (ks >= kStages) {
                        ks -= kStages;
                        kph ^= 1u;
                    }
                }
                use += 2u * (uint32_t)p.n;
            }
            // every MMA issued has completed before teardown
            mma_commit_warp(smem_u32(&ctrl->teardown));
            if (lane == 0) mbar_wait_teardown(smem_u32(&ctrl->teardown), 0);
            __syncwarp();
        }
    } else {
        // ------------------------------------------- softmax and epilogue
        setmaxnreg_inc<kRegsSoftmax>();
        Pieces<false> pieces(a, cta);
        const int j = warp >> 2, w = warp & 3;
        const int row = w * 32 + lane;
        const int row_tokens = row_tile_tokens(a.group);
        const int tk = row / a.group, g = row - tk * a.group;    // this thread's token and head in a row tile
        const uint32_t lane_addr = tmem + ((uint32_t)(w * 32) << 16);
        const uint32_t ts = lane_addr + kColS + 128 * j, to = lane_addr + kColO + 128 * j;
        const bool negate = a.scale < 0.0f;
        // a zero scale: any tiny factor gives equal probabilities, without 0 * inf at masked keys
        const float c = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1.17549435e-38f);
        const float lazy = kLazy / c;
        uint32_t s_cnt = 0, ml_cnt = 0, t_cnt = 0;
        bool ok = true;
        while (ok && pieces.next(p)) {
            int first, end, first_o, end_o;                      // tiles of this warpgroup, of the other
            p.range(j, row_tokens, a.window, first, end);
            p.range(1 - j, row_tokens, a.window, first_o, end_o);
            const int by = p.two ? 1 : 2;
            if (!p.two) first = j;
            const int t = (p.two && j ? row_tokens : 0) + tk;    // token of the item
            const bool mine = tk < row_tokens && t < p.n_tok;
            const bool any = __any_sync(0xffffffffu, mine);
            const int pos = p.pos0 + t;
            const int hi = mine ? min(pos + 1, p.kv_end) : 0;      // keys lo .. hi - 1
            const int lo = mine && a.window ? max(pos + 1 - a.window, 0) : 0;
            float m = -INFINITY, l = 0.0f;
            if (first >= end) continue;      // the second warpgroup of a single key tile
            for (int i = first; i < end; i += by) {
                if (!mbar_wait_warp(smem_u32(&ctrl->s_full[j]), s_cnt & 1u, abort_flag, status, 50)) {
                    ok = false;
                    break;
                }
                s_cnt++;
                const bool both = p.two && i >= first_o && i < end_o;
                if (both) {
                    // the two warpgroups' exponentials in turn (per pair of
                    // warps): together they would wait for the tensor pipe
                    // together, and leave it idle together
                    if (!mbar_wait_warp(smem_u32(&ctrl->turn[j][w]), (t_cnt & 1u) ^ (j ? 0u : 1u), abort_flag, status,
                                        54)) {
                        ok = false;
                        break;
                    }
                    t_cnt++;
                }
                if (any) {
                    tc_fence_after();
                    const int key0 = (p.tile0 + i) * kAttnKeys;
                    if (negate || __any_sync(0xffffffffu, mine && (hi < key0 + kAttnKeys || lo > key0)))
                        edit_scores(ts, negate, hi - key0, lo - key0);
                }
#pragma unroll 1
                for (int half = 0; half < 2 && ok; half++) {     // 64 keys at a time
                    if (any) {
                        float s[64];
                        uint32_t r[32];
                        float mc, sum;
                        for (;;) {
                            tmem_ld32(ts + 64 * half, s);
                            tmem_ld32(ts + 64 * half + 32, s + 32);
                            tmem_ld_wait();
                            // P with the m in use, their maximum beside it;
                            // where that has outgrown m (and at an item's
                            // first keys) m moves and P is formed again: S is
                            // still there
                            mc = m == -INFINITY ? 0.0f : -m * c;
                            const float mx = max_scores(s);
                            sum = exp_scores(s, c, mc, r);
                            const bool up = mine && (mx > m + lazy || (m == -INFINITY && mx > m));
                            if (!__any_sync(0xffffffffu, up)) break;
                            const float m1 = up ? mx : m;
                            if (i > first || half) {
                                // rescale what has been summed with the old
                                // maximum: the P V of the tiles before is
                                // complete, as S is; that of the first half
                                // has a signal
                                const float f = up ? ex2((m - m1) * c) : 1.0f;
                                l *= f;
                                if (half && !mbar_wait_warp(smem_u32(&ctrl->o_half[j]), (s_cnt - 1) & 1u, abort_flag, status,
                                                            51)) {
                                    ok = false;
                                    break;
                                }
                                tc_fence_after();
#pragma unroll 1
                                for (int k = 0; k < kDP / 16; k++) {
                                    float o[16];
                                    tmem_ld16(to + 16 * k, o);
                                    tmem_ld_wait();
                                    uint32_t q[16];
#pragma unroll
                                    for (int y = 0; y < 16; y++) q[y] = __float_as_uint(f == 0.0f ? 0.0f : o[y] * f);
                                    tmem_st16(to + 16 * k, q);
                                }
                            }
                            m = m1;
                        }
                        tmem_st32(ts + 64 * half, r);
                        l += sum;
                        tmem_st_wait();
                        tc_fence_before();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(smem_u32(half ? &ctrl->p_full[j] : &ctrl->p_half[j]));
                        if (both && !half) mbar_arrive(smem_u32(&ctrl->turn[1 - j][w]));
                    }
                }
            }
            if (!ok) break;

            // ---- the item's end: O in tensor memory, m and l here
            const bool merge = !p.two && p.n > 1;       // both warpgroups hold a share of the same rows
            if (!mbar_wait_warp(smem_u32(&ctrl->o_full[j]), (s_cnt - 1) & 1u, abort_flag, status, 52)) break;
            tc_fence_after();
            if (merge && j == 1) {
                ctrl->m[row] = m;
                ctrl->l[row] = l;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctrl->ml_full[w]));   // warp w of the other takes over
                continue;
            }
            float f0 = 1.0f, f1 = 0.0f;
            if (merge) {
                if (!mbar_wait_warp(smem_u32(&ctrl->ml_full[w]), ml_cnt & 1u, abort_flag, status, 53)) break;
                ml_cnt++;
                tc_fence_after();
                const float mb = ctrl->m[row], lb = ctrl->l[row];
                const float mm = fmaxf(m, mb), ms = mm == -INFINITY ? 0.0f : mm;
                f0 = ex2((m - ms) * c);
                f1 = ex2((mb - ms) * c);
                l = l * f0 + lb * f1;
                m = mm;
            }
            const float m2 = m * c;                              // log2 of e^(largest score)
            const bool whole = p.parts == 1;
            const bool none = l == 0.0f;                         // the row sees no key
            const int head = p.hk * a.group + g;
            const int64_t tok = p.tok0 + t;
            if (any && whole) {
                // rows in the accumulator layout, four lanes to a row: 64
                // contiguous bytes of 8 rows a store (a row a lane would be
                // 16 bytes of 32 rows, four times the accesses)
                const float inv = none ? 0.0f : 1.0f / l;
                const uint32_t valid = __ballot_sync(0xffffffffu, mine);
                const int64_t at = tok * a.ldo + head * a.ho;
#pragma unroll 1
                for (int h = 0; h < 2; h++) {                    // rows 16h .. 16h + 15 of the warp
                    float fa[2], fb[2];
                    __nv_bfloat16* out[2];
                    bool live[2];
#pragma unroll
                    for (int b = 0; b < 2; b++) {
                        const int r = 16 * h + 8 * b + (lane >> 2);
                        fa[b] = __shfl_sync(0xffffffffu, f0 * inv, r);
                        fb[b] = __shfl_sync(0xffffffffu, f1 * inv, r);
                        out[b] = a.out + __shfl_sync(0xffffffffu, at, r) + 8 * (lane & 3);
                        live[b] = (valid >> r) & 1u;
                    }
                    if ((valid >> (16 * h)) == 0) break;         // (the rows of an item are its first)
#pragma unroll 1
                    for (int k = 0; k < kDP; k += 64) {          // 64 columns at a time
                        float o[32];
                        const uint32_t at_h = ((uint32_t)(16 * h) << 16) + k;
                        tmem_ld_rows(to + at_h, o);
                        tmem_ld_rows(to + at_h + 32, o + 16);
                        tmem_ld_wait();
#pragma unroll
                        for (int x = 0; x < 32; x++) o[x] = fa[(x >> 1) & 1] == 0.0f ? 0.0f : o[x] * fa[(x >> 1) & 1];
                        if (merge) {
                            float o1[32];
                            tmem_ld_rows(to + 128 + at_h, o1);
                            tmem_ld_rows(to + 128 + at_h + 32, o1 + 16);
                            tmem_ld_wait();
#pragma unroll
                            for (int x = 0; x < 32; x++)
                                o[x] += fb[(x >> 1) & 1] == 0.0f ? 0.0f : o1[x] * fb[(x >> 1) & 1];
                        }
#pragma unroll
                        for (int y = 0; y < 2; y++) {
#pragma unroll
                            for (int b = 0; b < 2; b++) {
                                uint32_t x[4];
#pragma unroll
                                for (int i = 0; i < 4; i++)
                                    x[i] = cvt_bf16x2(o[16 * y + 4 * i + 2 * b], o[16 * y + 4 * i + 2 * b + 1]);
                                quad_transpose(x, lane & 3);
                                const int col = k + 32 * y;
                                if (live[b] && col + 8 * (lane & 3) < a.head_dim)
                                    *reinterpret_cast<uint4*>(out[b] + col) = make_uint4(x[0], x[1], x[2], x[3]);
                            }
                        }
                    }
                }
                if (mine && a.lse)
                    a.lse[tok * a.heads + head] = none ? -INFINITY : (m2 + log2f(l)) * 0.6931471805599453f;
            } else if (any) {
                float* part = a.partials + (2 * cta + (p.cta0 == cta ? 1 : 0)) * kAttnSlotFloats;
                const int srow = (p.two ? j * kAttnRows : 0) + row;
#pragma unroll 1
                for (int k = 0; k < kDP / 32; k++) {
                    float o[32];
                    tmem_ld32(to + 32 * k, o);
                    tmem_ld_wait();
                    if (merge) {
                        float o1[32];
                        tmem_ld32(to + 128 + 32 * k, o1);
                        tmem_ld_wait();
#pragma unroll
                        for (int y = 0; y < 32; y++) o[y] = (f0 == 0.0f ? 0.0f : o[y] * f0) + (f1 == 0.0f ? 0.0f : o1[y] * f1);
                    }
                    if (!mine) continue;
#pragma unroll
                    for (int y = 0; y < 8; y++)
                        __stcg(reinterpret_cast<float4*>(part) + (8 * k + y) * kAttnSlotRows + srow,
                               make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]));
                }
                if (mine) {
                    __stcg(part + kAttnSlotRows * kDP + srow, m2);
                    __stcg(part + kAttnSlotRows * (kDP + 1) + srow, l);
                }
            }
            // the accumulators may be overwritten
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&ctrl->o_free[j]));
                if (merge) mbar_arrive(smem_u32(&ctrl->o_free[1]));
            }
            if (whole || !any) continue;

            // ---- a shared item: the last of its CTAs adds the parts up, per warp
            __syncwarp();
            int* ticket = a.tickets + (p.cta0 * 2 + (p.two ? j : 0)) * 4 + w;
            int last = 0;
            if (lane == 0) last = atom_add_acq_rel(ticket, 1) == p.parts - 1;   // (after the warp's stores: cumulative)
            last = __shfl_sync(0xffffffffu, last, 0);
            if (!last) continue;
            if (lane == 0) *ticket = 0;
            const int row0 = (p.two ? j * kAttnRows : 0) + w * 32;   // the warp's first row in a slot
            const int rows = __popc(__ballot_sync(0xffffffffu, mine));
            // part i of the item is in slot 2 (cta0 + i), the first in 2 cta0 + 1
            const float* const part0 = a.partials + (2 * p.cta0 + 1) * kAttnSlotFloats;
            auto part_of = [&](int i) { return part0 + (i == 0 ? 0 : 2 * i - 1) * kAttnSlotFloats; };
            const int my = row0 + min(lane, rows - 1);
            float mall = -INFINITY, lall = 0.0f;
#pragma unroll 4
            for (int i = 0; i < p.parts; i++) mall = fmaxf(mall, __ldcg(part_of(i) + kAttnSlotRows * kDP + my));
            const float ms = mall == -INFINITY ? 0.0f : mall;
#pragma unroll 4
            for (int i = 0; i < p.parts; i++) {
                const float* part = part_of(i) + kAttnSlotRows * kDP + my;
                lall += __ldcg(part + kAttnSlotRows) * ex2(__ldcg(part) - ms);
            }
            if (mine && a.lse)
                a.lse[tok * a.heads + head] = lall == 0.0f ? -INFINITY : (mall + log2f(lall)) * 0.6931471805599453f;
            const float inv = lall == 0.0f ? 0.0f : 1.0f / lall;
            const int64_t at = tok * a.ldo + head * a.ho;
            // lane l takes the 4-column vectors l, l + 32, ... of the rows'
            // vectors (row fastest), kJoin of them at a time
            const int vecs = rows * (a.head_dim / 4);
            const int dv = 32 / rows, dr = 32 - dv * rows;
            int v = lane / rows, r = lane - v * rows;
            for (int b = lane; b - lane < vecs; b += 32 * kJoin) {
                float4 acc[kJoin];
                int vv[kJoin], rr[kJoin];
#pragma unroll
                for (int y = 0; y < kJoin; y++) {
                    const bool in = b + 32 * y < vecs;
                    vv[y] = in ? v : 0;
                    rr[y] = in ? r : 0;
                    v += dv;
                    r += dr;
                    if (r >= rows) {
                        r -= rows;
                        v++;
                    }
                    acc[y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
#pragma unroll 2
                for (int i = 0; i < p.parts; i++) {
                    const float* part = part_of(i);
                    const float f = ex2(__ldcg(part + kAttnSlotRows * kDP + my) - ms) * inv;
#pragma unroll
                    for (int y = 0; y < kJoin; y++) {
                        const float4 o = __ldcg(reinterpret_cast<const float4*>(part) + vv[y] * kAttnSlotRows + row0 + rr[y]);
                        const float fy = __shfl_sync(0xffffffffu, f, rr[y]);
                        acc[y].x += fy * o.x;
                        acc[y].y += fy * o.y;
                        acc[y].z += fy * o.z;
                        acc[y].w += fy * o.w;
                    }
                }
#pragma unroll
                for (int y = 0; y < kJoin; y++) {
                    const int64_t ar = __shfl_sync(0xffffffffu, at, rr[y]);
                    const bool none_r = __shfl_sync(0xffffffffu, inv, rr[y]) == 0.0f;
                    const uint2 w2 = make_uint2(cvt_bf16x2(acc[y].x, acc[y].y), cvt_bf16x2(acc[y].z, acc[y].w));
                    if (b + 32 * y < vecs)
                        *reinterpret_cast<uint2*>(a.out + ar + 4 * vv[y]) = none_r ? make_uint2(0u, 0u) : w2;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int kDP>
cudaError_t launch(const Params& p, int num_sms, cudaStream_t stream)
{
    static int attr_set_for_device[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && !attr_set_for_device[dev]) {
        e = cudaFuncSetAttribute(attn_kernel<kDP>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<kDP>::kSmemBytes);
        if (e != cudaSuccess) return e;
        attr_set_for_device[dev] = 1;
    }
    return launch_programmatic(attn_kernel<kDP>, dim3((unsigned)num_sms), dim3(kThreads), Cfg<kDP>::kSmemBytes, stream,
                               p);
}

}  // namespace

cudaError_t launch_attn(const CUtensorMap& map_q, const CUtensorMap& map_k, const CUtensorMap& map_v,
                        const AttnArgs& args, int num_sms, cudaStream_t stream)
{
    Params p;
    p.map_q = map_q;
    p.map_k = map_k;
    p.map_v = map_v;
    p.a = args;
    const int ctas = num_sms < kAttnMaxCtas ? num_sms : kAttnMaxCtas;
    return args.head_dim > 64 ? launch<128>(p, ctas, stream) : launch<64>(p, ctas, stream);
}

}  // namespace nvfp4
