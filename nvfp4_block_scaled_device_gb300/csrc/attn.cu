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
// Two softmax warpgroups work on two row tiles at a time, 64 keys a step, each
// with two halves of S (one is multiplied while the other is in its softmax).
// An item with more than 128 rows has two row tiles, one per warpgroup, on the
// same keys; one with at most 128 rows (decoding) gives the even key tiles to
// the first and the odd ones to the second, which the first merges at the end.
//
// Items are cut at CTA boundaries (equal key tiles per CTA).  A CTA's part of
// a shared item goes to the workspace as fp32 (O, m, l); the CTA whose warp
// takes a part's last ticket adds the parts up in CTA order (the same result
// whatever the order of arrival).  No CTA waits for another.
//
// Warps: 0-3 and 4-7 softmax and epilogue; 8 and 9 the MMAs of the first and
// the second warpgroup; 10 K/V copies; 11 Q copies and the keys' end (next).
//
// Rows past the last key of an item's last tile hold other requests' rows,
// pages' unused rows or nothing at all, and so may rows before a window's
// first key.  Their scores are masked, and warp 11 zeroes the V rows before
// the tile is multiplied, so that NaN or infinities there cannot reach a sum
// as 0 * NaN.
//
// What bounds it (40 query heads on 8 kv heads of 128 columns, 2070 MHz):
//   - Few rows, many keys: HBM.  Two requests of 65537 and more keys, 879 MB of
//     cache: 138 us, 6.35 TB/s.  Many short ones add the start of each CTA
//     (4-5 us until the first S) and the items' ends: 64 requests of 200 to 8192
//     keys 95 us, 5.8 TB/s.
//   - Long prompts: the tensor pipe and what keeps it from running.  A prompt of
//     8192: 505 to 530 us from run to run, 1.3 PFLOP/s.  128 keys against two row tiles take about
//     3000 cycles.  The products take 2560 of them: Q K^T of 64 keys reads Q
//     again (48 KB of shared memory for 384 cycles, where the arithmetic would
//     take 256), P V 256.  S of 128 keys would not read Q twice, but fills
//     tensor memory with one S a warpgroup: 587 us (where this took 524), as a
//     warpgroup then waits for its own products.  The rest is latency from P's
//     arrival to the next S, and 5000-6000 cycles at an item's end.
//   - Short prompts: those ends and the start.  17 tokens take 6.8 us.
// The warps of a CTA run four different programs, which drive each other out of
// the instruction cache; every program's repeated path is kept short.  With
// loops written out, waits with their own time limits and divisions in the walk
// over the items (110 KB of code instead of 81) the prompt of 8192 took 525 us
// where it then took 508, the 64 requests 104 and 98.
#include "attn.h"
#include "common.cuh"
#include "internal.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 384;
constexpr int kWarpMma = 8, kWarpKV = 10, kWarpQ = 11;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColS = 256;      // + 128 * warpgroup; P of 64 keys over the first 32 columns of their S
constexpr int kStep = 64;                       // keys of a step
constexpr float kLazy = 8.0f;                   // log2 of the growth that P may carry
constexpr int kRegsSoftmax = 192, kRegsOther = 120;
static_assert(2 * kRegsSoftmax + kRegsOther <= 3 * 168, "the block's registers at launch");

constexpr int kMaxStages = 10;

struct Ctrl {
    uint64_t kv_full[kMaxStages], kv_empty[kMaxStages], v_end[kMaxStages];
    uint64_t q_full, q_empty;
    uint64_t s_full[2][2], p_full[2][2], o_full[2][2];   // of a warpgroup's even and odd steps
    uint64_t o_free[2];
    uint64_t ml_full[4];
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

// How a tile of keys or values lies in its 128-row stage.  The usual layout:
// 64-column halves 16 KB apart, rows in order; a step is 64 rows in a row.
// kFold, for pages of 16 rows of 128 columns: a page's both halves in one copy,
// [page][half][16 rows][64 columns], as a copy costs about 60 cycles beside 4
// per 128 bytes and two copies of 2 KB a page keep HBM waiting (64 requests of
// 200 to 8192 keys: 144 us in two copies, 104 in one).  Step h is then
// the eight rows 8h .. 8h + 7 of each page: 8-row groups at one distance, which
// is all that a descriptor can say.
template <bool kFold>
struct Layout {
    static constexpr uint32_t kHalf = kFold ? 2048 : 16384;       // bytes between 64-column halves,
    static constexpr uint32_t kGroup = kFold ? 4096 : 1024;       // a step's 8-row groups,
    static constexpr uint32_t kStepAt = kFold ? 1024 : 8192;      // a tile's two steps
    __device__ static uint32_t row(int r) { return kFold ? (uint32_t)(r >> 4) * 4096u + (r & 15) * 128u : r * 128u; }
    // First key of 8-key group g of step h (from its tile's first key).
    __device__ static int key(int h, int g) { return kFold ? 16 * g + 8 * h : kStep * h + 8 * g; }
};

template <int kValue>
struct Int {
    static constexpr int value = kValue;
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
// converged warp from a single asm block (see stage_issue_1sm), and what its
// completion signals.
// S = Q K^T (N = 64 keys): operands as 128-byte swizzled rows, K-major; K = 16
// columns an MMA, Q's 64-column halves 16 KB apart, K's kHalf bytes.
template <int kDP, uint32_t kHalf>
__device__ __forceinline__ void issue_qk(uint32_t s, uint32_t q_lo, uint32_t q_hi, uint32_t k_lo, uint32_t k_hi,
                                         uint32_t idesc, uint32_t bar)
{
    constexpr uint32_t kB = kHalf >> 4;
    if (kDP == 128)
        asm volatile(
        "{\n .reg .pred e, pf, pt;\n .reg .b32 r, x, y;\n .reg .b64 da, db;\n"
        " elect.sync r|e, 0xffffffff;\n setp.eq.b32 pt, 0, 0;\n setp.ne.b32 pf, 0, 0;\n"
        " add.u32 x, %1, 0; add.u32 y, %2, 0; mov.b64 da, {x, %3}; mov.b64 db, {y, %6};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pf;\n"
        " add.u32 x, %1, 2; add.u32 y, %2, 2; mov.b64 da, {x, %3}; mov.b64 db, {y, %6};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pt;\n"
        " add.u32 x, %1, 4; add.u32 y, %2, 4; mov.b64 da, {x, %3}; mov.b64 db, {y, %6};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pt;\n"
        " add.u32 x, %1, 6; add.u32 y, %2, 6; mov.b64 da, {x, %3}; mov.b64 db, {y, %6};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pt;\n"
        " add.u32 x, %1, 1024; add.u32 y, %2, %7; mov.b64 da, {x, %3}; mov.b64 db, {y, %6};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pt;\n"
        " add.u32 x, %1, 1026; add.u32 y, %2, %8; mov.b64 da, {x, %3}; mov.b64 db, {y, %6};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pt;\n"
        " add.u32 x, %1, 1028; add.u32 y, %2, %9; mov.b64 da, {x, %3}; mov.b64 db, {y, %6};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pt;\n"
        " add.u32 x, %1, 1030; add.u32 y, %2, %10; mov.b64 da, {x, %3}; mov.b64 db, {y, %6};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pt;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n"
        "}\n" ::"r"(s), "r"(q_lo), "r"(k_lo), "r"(q_hi), "r"(idesc), "r"(bar), "r"(k_hi),
        "n"(kB), "n"(kB + 2), "n"(kB + 4), "n"(kB + 6)
        : "memory");
    else
        asm volatile(
        "{\n .reg .pred e, pf, pt;\n .reg .b32 r, x, y;\n .reg .b64 da, db;\n"
        " elect.sync r|e, 0xffffffff;\n setp.eq.b32 pt, 0, 0;\n setp.ne.b32 pf, 0, 0;\n"
        " add.u32 x, %1, 0; add.u32 y, %2, 0; mov.b64 da, {x, %3}; mov.b64 db, {y, %6};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pf;\n"
        " add.u32 x, %1, 2; add.u32 y, %2, 2; mov.b64 da, {x, %3}; mov.b64 db, {y, %6};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pt;\n"
        " add.u32 x, %1, 4; add.u32 y, %2, 4; mov.b64 da, {x, %3}; mov.b64 db, {y, %6};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pt;\n"
        " add.u32 x, %1, 6; add.u32 y, %2, 6; mov.b64 da, {x, %3}; mov.b64 db, {y, %6};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, pt;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n"
        "}\n" ::"r"(s), "r"(q_lo), "r"(k_lo), "r"(q_hi), "r"(idesc), "r"(bar), "r"(k_hi)
        : "memory");
}
// O += P V over 64 keys: P in tensor memory (8 columns for 16 keys), V as
// stored (N-major; 16 keys are 2 KB).
template <uint32_t kGroup>
__device__ __forceinline__ void issue_pv(uint32_t o, uint32_t p, uint32_t v_lo, uint32_t hi, uint32_t idesc,
                                         uint32_t acc, uint32_t bar)
{
    constexpr uint32_t kMma = 2 * kGroup >> 4;       // 16 keys on
    asm volatile(
        "{\n .reg .pred e, p, pt;\n .reg .b32 r, x, y;\n .reg .b64 db;\n"
        " elect.sync r|e, 0xffffffff;\n setp.eq.b32 pt, 0, 0;\n setp.ne.b32 p, %5, 0;\n"
        " add.u32 x, %2, 0; mov.b64 db, {x, %3}; add.u32 y, %1, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], db, %4, p;\n"
        " add.u32 x, %2, %7; mov.b64 db, {x, %3}; add.u32 y, %1, 8;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], db, %4, pt;\n"
        " add.u32 x, %2, %8; mov.b64 db, {x, %3}; add.u32 y, %1, 16;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], db, %4, pt;\n"
        " add.u32 x, %2, %9; mov.b64 db, {x, %3}; add.u32 y, %1, 24;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], db, %4, pt;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%6];\n"
        "}\n" ::"r"(o), "r"(p), "r"(v_lo), "r"(hi), "r"(idesc), "r"(acc), "r"(bar), "n"(kMma), "n"(2 * kMma), "n"(3 * kMma)
        : "memory");
}

// Arrival of the warp (its lane 0), without a branch around it.
__device__ __forceinline__ void mbar_arrive_warp(uint32_t bar, int lane)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.eq.s32 p, %1, 0;\n @p mbarrier.arrive.shared::cta.b64 _, [%0];\n}" ::"r"(bar), "r"(lane)
        : "memory");
}

// One look (warp-uniform): test_wait, as try_wait may suspend the warp.
__device__ __forceinline__ bool mbar_test_warp(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n vote.sync.all.pred p, p, 0xffffffff;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
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

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                            int w, int v)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v)
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

// The waits of this kernel (converged, bounded by 2 to 4 seconds: %clock_hi
// counts 2^32 cycles).  Less code than mbar_wait_warp at each of some twenty
// places: a failure only notes where, and wait_failed reports it at the end.
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, const volatile int* abort_flag, int& failed, int site)
{
    if (mbar_test_warp(bar, parity)) return true;
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .u32 t0, t, a;\n mov.u32 t0, %%clock_hi;\n"
        "POLL_%=:\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " vote.sync.all.pred p, p, 0xffffffff;\n"
        " @p bra.uni DONE_%=;\n"
        " ld.volatile.shared.u32 a, [%3];\n"
        " mov.u32 t, %%clock_hi;\n"
        " sub.u32 t, t, t0;\n"
        " setp.lt.u32 q, t, 2;\n"
        " setp.eq.and.u32 q, a, 0, q;\n"
        " vote.sync.all.pred q, q, 0xffffffff;\n"
        " @q bra.uni POLL_%=;\n"
        "DONE_%=:\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(smem_u32((const void*)abort_flag))
        : "memory");
    if (!ok) failed = site;
    return ok != 0;
}

// After a wait that failed: the CTA's other warps give up too; a wait that ran
// out (not one that another's failure ended) is recorded.
__device__ __forceinline__ void wait_failed(volatile int* abort_flag, int* status, int site)
{
    if (*abort_flag == 0) atomicCAS(status, 0, kErrTimeout * 100 + site);
    *abort_flag = 1;
}

// Waits for the ring's stage use `use` to be full.  A warp that leaves uses to
// the other MMA warp has not seen their phases end, and a parity wait is only
// right from the phase before on: so first the copies of this use have begun,
// which they do once the stage's use before has been consumed.
__device__ __forceinline__ bool wait_use(const volatile uint32_t* issued, uint32_t use, uint32_t bar, uint32_t parity,
                                         const volatile int* abort_flag, int& failed, int site)
{
    const uint32_t t0 = (uint32_t)(clock64() >> 32);
    while (__any_sync(0xffffffffu, (int32_t)(*issued - use) <= 0)) {
        if (__any_sync(0xffffffffu, (uint32_t)(clock64() >> 32) - t0 >= 2u || *abort_flag)) {
            failed = site;
            return false;
        }
    }
    return wait_on(bar, parity, abort_flag, failed, site);
}

__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// What is done to a row's scores of step h of a key tile in tensor memory before
// the softmax reads them: the sign of a negative scale, -inf at keys outside
// lo .. hi - 1 (from the tile's first key).
template <bool kFold>
__device__ __forceinline__ void edit_scores(uint32_t taddr, bool negate, int h, int lo, int hi)
{
#pragma unroll 1
    for (int x = 0; x < kStep; x += 32) {
        uint32_t seen;
        if (kFold) {
            seen = 0;
#pragma unroll 1
            for (int g = 0; g < 4; g++) {
                const int key = Layout<true>::key(h, x / 8 + g);
                seen |= ((low_bits(hi - key) & ~low_bits(lo - key)) & 0xffu) << (8 * g);
            }
        } else {
            const int key = kStep * h + x;
            seen = low_bits(hi - key) & ~low_bits(lo - key);
        }
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
    int tok0, n_tok, req, pos0, kv_end;   // of its QTile
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
    // Keys live0 .. live1 - 1 of key tile i are live: the others precede every
    // row's window, or follow the item's last key.
    __device__ __forceinline__ void live(int i, int window, int& live0, int& live1) const
    {
        const int key0 = (tile0 + i) * kAttnKeys;
        live0 = window ? min(max(pos0 + 1 - window - key0, 0), kAttnKeys) : 0;
        live1 = min(kAttnKeys, max(kv_end - key0, 0));
    }
};

// The pieces of CTA `cta` in order; every warp of the CTA walks them alike.
// The next QTile is fetched while the current one is worked on.
struct Pieces {
    const int4* table;
    int u, end, per_cta, qt, kv_heads, row_tokens;
    int hk, r0;          // the next piece: its kv head, units of its item before it
    int4 f0, f1;         // ... and QTile (number qt)

    __device__ __forceinline__ Pieces(const AttnArgs& a, int cta)
    {
        const ScheduleHead* s = a.sched;
        table = reinterpret_cast<const int4*>(schedule_tiles(s));
        kv_heads = a.kv_heads;
        row_tokens = a.row_tokens;
        const int4* start = reinterpret_cast<const int4*>(&s->start[cta]);
        f0 = start[0];
        f1 = start[1];
        qt = s->first[cta];
        const int units = s->units;
        per_cta = s->per_cta;
        u = cta * per_cta < units ? cta * per_cta : units;
        end = units - u < per_cta ? units : u + per_cta;
        const uint32_t rel = (uint32_t)(u - f1.w), item = (uint32_t)(kItemUnits + f1.z);
        hk = (int)(rel / item);
        r0 = (int)(rel - hk * item);
    }
    __device__ __forceinline__ bool next(Piece& p)
    {
        while (u < end) {
            const int tiles = f1.z, item = kItemUnits + tiles;
            const int r1 = min(end - u + r0, item);      // the CTA's units of the item: r0 .. r1 - 1
            const int k0 = max(snap_unit(r0, item) - kItemUnits, 0);
            p.n = max(snap_unit(r1, item) - kItemUnits, 0) - k0;
            p.hk = hk;
            p.tok0 = f0.x;
            p.n_tok = f0.y;
            p.req = f0.z;
            p.pos0 = f0.w;
            p.kv_end = f1.x;
            p.tile0 = f1.y + k0;
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
            r0 = r1;
            if (r1 == item) {
                r0 = 0;
                if (++hk == kv_heads) {
                    hk = 0;
                    if (u < end) {
                        qt++;
                        f0 = table[2 * qt];
                        f1 = table[2 * qt + 1];
                    }
                }
            }
            if (p.n > 0) return true;
        }
        return false;
    }
};

// The ring's order within an item of n key tiles: K0 K1 V0 K2 V1 ... K(n-1)
// V(n-2) V(n-1).  Values are needed a softmax later than their keys; fetched
// right behind them they would hold a stage for that time (with 5 stages of 32
// KB that leaves too little under way for HBM's latency).
__device__ __forceinline__ uint32_t use_of_k(int i) { return i == 0 ? 0u : 2u * i - 1u; }
__device__ __forceinline__ uint32_t use_of_v(int i, int n) { return i == n - 1 ? 2u * n - 1u : 2u * i + 2u; }

// Stage and phase parity of the ring's use `use`.
template <int kStages>
__device__ __forceinline__ uint32_t stage_of(uint32_t use, uint32_t* parity)
{
    const uint32_t turn = use / kStages;
    *parity = turn & 1u;
    return use - turn * kStages;
}

template <int kDP, bool kFold>
__global__ void __launch_bounds__(kThreads, 1) attn_kernel(const __grid_constant__ Params prm)
{
    using C = Cfg<kDP>;
    using L = Layout<kFold>;
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
            for (int x = 0; x < 2; x++) {
                mbar_init(smem_u32(&ctrl->s_full[j][x]), 1);
                mbar_init(smem_u32(&ctrl->p_full[j][x]), 4);
                mbar_init(smem_u32(&ctrl->o_full[j][x]), 1);
            }
            mbar_init(smem_u32(&ctrl->o_free[j]), 4);
        }
        for (int w = 0; w < 4; w++) mbar_init(smem_u32(&ctrl->ml_full[w]), 1);
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
    int failed = 0;                  // the wait that failed

    if (warp >= 8) {
        Pieces pieces(a, cta);
        setmaxnreg_dec<kRegsOther>();
        if (warp == kWarpKV) {
            // ------------------------------------------------ K/V copies
            const bool paged = a.block_table != nullptr;
            const int ppt = paged ? kAttnKeys / a.page_size : 1;       // pages of a key tile
            const uint32_t page_bytes = paged ? (uint32_t)(a.page_size * kDP * 2) : (uint32_t)C::kTileBytes;
            // a copy per lane: half `half` of the tile's page pg (at most 16 copies; kFold: whole pages)
            const int half = kFold ? 0 : lane / ppt, pg = lane - half * ppt;
            const uint32_t copy_at = base + C::kOffRing + (kFold ? lane * 4096u : half * 16384u + pg * a.page_size * 128u);
            uint32_t use = 0, s = 0, ph = 1;      // the ring's next use, its stage, the phase of that stage's use before
            bool ok = true;
            while (ok && pieces.next(p)) {
                const int* table = paged ? a.block_table + (int64_t)p.req * a.table_ld : nullptr;
                int lo[2], hi[2], live0, live1, unused;
                for (int j = 0; j < 2; j++) p.range(j, a.row_tokens, a.window, lo[j], hi[j]);
                // tiles from .. to - 1 are both MMA warps', the others one's
                const int from = p.two ? max(lo[0], lo[1]) : p.n, to = min(hi[0], hi[1]);
                p.live(0, a.window, live0, unused);
                p.live(p.n - 1, a.window, unused, live1);
                const int last_pages = paged ? (live1 + a.page_size - 1) / a.page_size : 1;
                // this lane's page of tiles i - 1, i, i + 1
                auto page_of = [&](int i) {
                    const int at = (p.tile0 + i) * ppt + pg;
                    return paged && i < p.n && at * a.page_size < p.kv_end ? table[at] : 0;
                };
                int page0 = 0, page1 = page_of(0), page2 = page_of(1);
#pragma unroll 1
                for (int x = 0; x < 2 * p.n + 2; x++) {
                    // keys of tile i, then values of tile i - 1
                    const int kv = x & 1, i = (x >> 1) - kv, id = kv ? page0 : page1;
                    if (kv) {
                        page0 = page1;
                        page1 = page2;
                        page2 = page_of(i + 3);
                    }
                    if (i < 0 || i == p.n) continue;
                    if (!wait_on(smem_u32(&ctrl->kv_empty[s]), ph, abort_flag, failed, 41)) {
                        ok = false;
                        break;
                    }
                    const bool last = i == p.n - 1;
                    const int pages = last ? last_pages : ppt;
                    // an item's first and last values go through warp 11
                    const bool edge = kv && ((i == 0 && live0 > 0) || (last && live1 < kAttnKeys));
                    const uint32_t bar = smem_u32(edge ? &ctrl->v_end[s] : &ctrl->kv_full[s]);
                    if (lane == 0) {
                        *(volatile uint32_t*)&ctrl->issued = use + 1;
                        mbar_arrive_expect_tx(bar, pages * page_bytes);
                        if (i < from || i >= to) mbar_arrive(smem_u32(&ctrl->kv_empty[s]));   // only one MMA warp's
                    }
                    __syncwarp();
                    const CUtensorMap* map = kv ? &prm.map_v : &prm.map_k;
                    const uint32_t dst = copy_at + s * C::kTileBytes;
                    if (half < C::kHalves && pg < pages) {
                        if (kFold) tma_load_5d(dst, map, bar, 0, 0, 0, p.hk, id);
                        else if (paged) tma_load_4d(dst, map, bar, half * 64, 0, p.hk, id);
                        // (packed: the request's first row is its key 0)
                        else tma_load_3d(dst, map, bar, half * 64, p.hk, p.tok0 - p.pos0 + (p.tile0 + i) * kAttnKeys);
                    }
                    __syncwarp();
                    use++;
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok && lane == 0) {
                // stopped early: let the copies under way land before the
                // CTA's shared memory goes away (bounded).  Values that end
                // an item complete on v_end, which has its own phases:
                // waiting on both for either phase costs time only here
                for (uint32_t u = use < kStages ? 0u : use - kStages; u < use; u++) {
                    uint32_t uph;
                    const uint32_t us = stage_of<kStages>(u, &uph);
                    mbar_wait_teardown(smem_u32(&ctrl->kv_full[us]), uph);
                    mbar_wait_teardown(smem_u32(&ctrl->v_end[us]), 0);
                    mbar_wait_teardown(smem_u32(&ctrl->v_end[us]), 1);
                }
            }
            __syncwarp();
        } else if (warp == kWarpQ) {
            // ------------------------ Q copies, and the ends of the values
            uint32_t n = 0, use = 0, ends = 0;     // items, uses of the ring; ends: bit s = phase of v_end[s]
            bool ok = true;
            const int row_tokens = a.row_tokens, rows = a.group * row_tokens;
            const uint32_t bar = smem_u32(&ctrl->q_full);
            while (pieces.next(p)) {
                if (!wait_on(smem_u32(&ctrl->q_empty), (n & 1u) ^ 1u, abort_flag, failed, 42)) {
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
                // the first tile's values before every row's window, the last's past the last key
                for (int i = 0; i < p.n && ok; i = i < p.n - 1 ? p.n - 1 : p.n) {
                    int live0, live1;
                    p.live(i, a.window, live0, live1);
                    if (live0 == 0 && live1 == kAttnKeys) continue;
                    uint32_t ph;
                    const uint32_t s = stage_of<kStages>(use + use_of_v(i, p.n), &ph);
                    if (!wait_on(smem_u32(&ctrl->v_end[s]), (ends >> s) & 1u, abort_flag, failed, 43)) {
                        ok = false;
                        break;
                    }
                    ends ^= 1u << s;
                    uint8_t* v = smem + C::kOffRing + s * C::kTileBytes;
                    // four rows at a time, eight lanes to a row (the item's last
                    // product waits for this)
                    for (int r = live0 > 0 ? lane >> 3 : live1 + (lane >> 3); r < kAttnKeys; r += 4) {
                        if (r >= live0 && r < live1) continue;
                        uint8_t* at = v + L::row(r) + (lane & 7) * 16;
#pragma unroll
                        for (int half = 0; half < C::kHalves; half++)
                            *reinterpret_cast<uint4*>(at + half * L::kHalf) = make_uint4(0, 0, 0, 0);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&ctrl->kv_full[s]));
                }
                if (!ok) break;
                use += 2u * (uint32_t)p.n;
            }
            if (!ok && n > 0 && lane == 0) mbar_wait_teardown(bar, (n - 1) & 1u);
            __syncwarp();
        } else {
            // ------------------------------------------------------- MMA
            // Warp 8 + j issues warpgroup j's products, across items too: for
            // each half of a key tile the last tile's P V, once P is there,
            // then this tile's S over it (they share columns).  Two row tiles: both
            // warps use every key tile; one row tile: warp j the tiles j,
            // j + 2, ... (a stage is free after two arrivals: both warps', or
            // the one warp's and the copying warp's own).
            const int j = warp - kWarpMma;
            const uint64_t qdesc0 = make_smem_desc(base, 16, 1024, 2);                  // K-major
            const uint64_t kdesc0 = make_smem_desc(base, 16, L::kGroup, 2);             // K-major
            const uint64_t vdesc0 = make_smem_desc(base, L::kHalf, L::kGroup, 2);       // N-major
            constexpr uint32_t kIdescS = idesc_of(kStep, false), kIdescO = idesc_of(kDP, true);
            constexpr uint32_t kStepDesc = L::kStepAt >> 4;
            const uint32_t q_hi = (uint32_t)(qdesc0 >> 32), k_hi = (uint32_t)(kdesc0 >> 32), v_hi = (uint32_t)(vdesc0 >> 32);
            const uint32_t q_lo = (uint32_t)qdesc0;
            const uint32_t ring_k = (uint32_t)kdesc0 + (C::kOffRing >> 4), ring_v = (uint32_t)vdesc0 + (C::kOffRing >> 4);
            const uint32_t full0 = smem_u32(&ctrl->kv_full[0]), empty0 = smem_u32(&ctrl->kv_empty[0]);
            const uint32_t ts = tmem + kColS + 128u * j, to = tmem + kColO + 128u * j;
            const uint32_t s_full = smem_u32(&ctrl->s_full[j][0]), o_full = smem_u32(&ctrl->o_full[j][0]);
            const uint32_t p_full = smem_u32(&ctrl->p_full[j][0]), o_free = smem_u32(&ctrl->o_free[j]);
            const uint32_t q_full = smem_u32(&ctrl->q_full), q_empty = smem_u32(&ctrl->q_empty);
            uint32_t use = 0;                      // stages used by the items before
            uint32_t qph = 0, oph = 1;             // phases: Q, O free (nothing to wait for at first)
            // A key tile's two steps use the first and the second half of S (and
            // of everything that alternates).  What lies between a tile's last
            // product and the next tile's first is on the path that bounds
            // long prompts (the tensor pipe is idle there): the keys' and
            // values' barriers are looked at while the products before run,
            // with test_wait (prompt of 8192 524 us; with try_wait, which
            // suspends where a phase is not complete, 564).
            bool pend = false;                     // the last tile's P V are still to be issued:
            uint32_t v_use = 0, v_st = 0, v_ph = 0, v_first = 0;   // V's use, stage, phase; the item's first tile
            bool v_ok = false;                     // V was there
            uint32_t tph = 0, t_cnt = 0;           // the phase of the last tile's barriers; tiles
            uint32_t safe = 0;                     // this warp has waited for the stage's last use, from this use on
            auto there = [&](uint32_t u, uint32_t st, uint32_t ph) {
                const volatile uint32_t* issued = &ctrl->issued;
                if ((int32_t)(u - safe) < 0 && __any_sync(0xffffffffu, (int32_t)(*issued - u) <= 0))
                    return false;
                return mbar_test_warp(full0 + 8u * st, ph);
            };
            auto ready_v = [&]() {
                if (v_ok) return true;
                if (v_first) {                     // the accumulator's last item has been read
                    if (!wait_on(o_free, oph, abort_flag, failed, 47)) return false;
                    oph ^= 1u;
                }
                return wait_use(&ctrl->issued, v_use, full0 + 8u * v_st, v_ph, abort_flag, failed, 46);
            };
            bool fresh = false, k_ok = false, more = true;    // the item's first tile; its keys are there; items to come
            bool pass = false;                                // an item without a tile for this warp
            int i = 0, end = 0, by = 1, n = 0;                // the next tile to multiply, the item's
            uint32_t qt = 0, ku = 0, ks = 0, kph = 0;
            for (;;) {
                if (i >= end && more && !pass) {              // the next item
                    use += 2u * (uint32_t)n;
                    more = pieces.next(p);
                    if (more) {
                        p.range(j, a.row_tokens, a.window, i, end);
                        by = p.two ? 1 : 2;
                        if (!p.two) i = j;
                        n = p.n;
                        // (it leaves some to the other)
                        if (!p.two || i > 0 || end < n) safe = use + 2u * (uint32_t)n + kStages;
                        qt = q_lo + (p.two && j ? C::kTileBytes >> 4 : 0);
                        ku = use + use_of_k(i);
                        ks = stage_of<kStages>(ku, &kph);
                        fresh = true;
                        k_ok = false;
                        pass = i >= end;
                    }
                }
                if (pass) {
                    // No tile for this warp, it only passes Q on.  Not while it
                    // holds values that the ring may need for the other's keys:
                    // it waits with nothing pending.
                    bool q_there = mbar_test_warp(q_full, qph);
                    if (!q_there && !pend) {
                        if (!wait_on(q_full, qph, abort_flag, failed, 44)) break;
                        q_there = true;
                    }
                    if (q_there) {
                        qph ^= 1u;
                        mbar_arrive_warp(q_empty, lane);
                        pass = false;
                        continue;
                    }
                }
                // What goes out now: the last tile's P V, and the next tile's S
                // over them if its operands are there (waited for only when
                // nothing else is left).
                bool s_too = i < end;
                if (s_too && !k_ok) {
                    s_too = (!fresh || mbar_test_warp(q_full, qph)) && there(ku, ks, kph);
                    if (!s_too && !pend) {
                        if ((fresh && !wait_on(q_full, qph, abort_flag, failed, 44)) ||
                            !wait_use(&ctrl->issued, ku, full0 + 8u * ks, kph, abort_flag, failed, 45))
                            break;
                        s_too = true;
                    }
                }
                if (!s_too && !pend) break;                   // all done
                if (pend && !ready_v()) break;
                const uint32_t k = ring_k + ks * (C::kTileBytes >> 4), k_empty = empty0 + 8u * ks;
                const uint32_t v = ring_v + v_st * (C::kTileBytes >> 4), v_empty = empty0 + 8u * v_st;
                const uint32_t first = v_first;
                bool ok = true;
#pragma unroll 1
                for (uint32_t h = 0; h < 2; h++) {
                    if (pend) {
                        ok = wait_on(p_full + 8u * h, tph, abort_flag, failed, 48);
                        if (!ok) break;
                    }
                    tc_fence_after();
                    if (pend) {
                        issue_pv<L::kGroup>(to, ts + 64u * h, v + h * kStepDesc, v_hi, kIdescO, h | (first ^ 1u),
                                            o_full + 8u * h);
                        if (h) mma_commit_warp(v_empty);
                    }
                    if (!s_too) continue;
                    issue_qk<kDP, L::kHalf>(ts + 64u * h, qt, q_hi, k + h * kStepDesc, k_hi, kIdescS, s_full + 8u * h);
                    if (h) {
                        mma_commit_warp(k_empty);
                        if (i >= end) mma_commit_warp(q_empty);
                    } else {
                        v_use = use + use_of_v(i, n);
                        v_st = stage_of<kStages>(v_use, &v_ph);
                        v_first = fresh ? 1u : 0u;
                        v_ok = !fresh && there(v_use, v_st, v_ph);
                        if (fresh) qph ^= 1u;
                        fresh = false;
                        i += by;
                        ku = use + use_of_k(i);
                        ks = stage_of<kStages>(ku, &kph);
                        k_ok = i < end && there(ku, ks, kph);
                    }
                }
                if (!ok) break;
                pend = s_too;
                if (s_too) tph = t_cnt++ & 1u;
            }
            // every MMA issued has completed before teardown
            mma_commit_warp(smem_u32(&ctrl->teardown));
            if (lane == 0) mbar_wait_teardown(smem_u32(&ctrl->teardown), 0);
            __syncwarp();
        }
    } else {
        // ------------------------------------------- softmax and epilogue
        setmaxnreg_inc<kRegsSoftmax>();
        Pieces pieces(a, cta);
        const int j = warp >> 2, w = warp & 3;
        const int row = w * 32 + lane;
        const int row_tokens = a.row_tokens;
        const int tk = row / a.group, g = row - tk * a.group;    // this thread's token and head in a row tile
        const uint32_t lane_addr = tmem + ((uint32_t)(w * 32) << 16);
        const uint32_t ts = lane_addr + kColS + 128 * j, to = lane_addr + kColO + 128 * j;
        const uint32_t s_full = smem_u32(&ctrl->s_full[j][0]), p_full = smem_u32(&ctrl->p_full[j][0]);
        const uint32_t o_full = smem_u32(&ctrl->o_full[j][0]);
        const bool negate = a.scale < 0.0f;
        // a zero scale: any tiny factor gives equal probabilities, without 0 * inf at masked keys
        const float c = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1.17549435e-38f);
        const float lazy = kLazy / c;
        uint32_t cnt = 0, ml_cnt = 0;      // steps done
        bool ok = true;
        while (ok && pieces.next(p)) {
            int first, end;                                      // tiles of this warpgroup
            p.range(j, row_tokens, a.window, first, end);
            const int by = p.two ? 1 : 2;
            if (!p.two) first = j;
            const int t = (p.two && j ? row_tokens : 0) + tk;    // token of the item
            const bool mine = tk < row_tokens && t < p.n_tok;
            const bool any = __any_sync(0xffffffffu, mine);
            const int pos = p.pos0 + t;
            const int hi = mine ? min(pos + 1, p.kv_end) : 0;      // keys lo .. hi - 1
            const int lo = mine && a.window ? max(pos + 1 - a.window, 0) : 0;
            // keys that every row of the warp sees (edits are needed beyond)
            const int hi_all = __reduce_min_sync(0xffffffffu, mine ? hi : 0x7fffffff);
            const int lo_all = __reduce_max_sync(0xffffffffu, lo);
            // keys that no row of the warp sees: below and from
            const int lo_any = __reduce_min_sync(0xffffffffu, mine ? lo : 0x7fffffff);
            const int hi_any = __reduce_max_sync(0xffffffffu, hi);
            float m = -INFINITY, l = 0.0f;
            if (first >= end) continue;      // the second warpgroup of a single key tile
#pragma unroll 1
            for (int x = 0; x < 2 * (end - first); x += by == 1 || (x & 1) == 0 ? 1 : 3, cnt++) {
                // step x: 64 keys; its barriers and columns alternate
                const uint32_t buf = cnt & 1u, ph = (cnt >> 1) & 1u;
                if (!wait_on(s_full + 8u * buf, ph, abort_flag, failed, 50)) {
                    ok = false;
                    break;
                }
                if (any) {
                    tc_fence_after();
                    // the tile's first key; keys that the step reaches from there
                    const int h = x & 1, key0 = p.tile0 * kAttnKeys + 2 * first * kStep + (x - h) * kStep;
                    if (key0 + L::key(h, 0) >= hi_any || key0 + L::key(h, 7) + 8 <= lo_any) {
                        // none of the step's keys: P = 0
                        uint32_t r[32];
#pragma unroll
                        for (int y = 0; y < 32; y++) r[y] = 0u;
                        tmem_st32(ts + 64 * buf, r);
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        mbar_arrive_warp(p_full + 8u * buf, lane);
                        continue;
                    }
                    if (negate || hi_all < key0 + L::key(h, 7) + 8 || lo_all > key0 + L::key(h, 0))
                        edit_scores<kFold>(ts + 64 * buf, negate, h, lo - key0, hi - key0);
                    float s[kStep];
                    uint32_t r[32];
                    float mc, sum;
                    for (;;) {
                        tmem_ld32(ts + 64 * buf, s);
                        tmem_ld32(ts + 64 * buf + 32, s + 32);
                        tmem_ld_wait();
                        // P with the m in use, the step's maximum beside it;
                        // where that has outgrown m (and at an item's first
                        // keys) m moves and P is formed again: S is still there
                        mc = m == -INFINITY ? 0.0f : -m * c;
                        const float mx = max_scores(s);
                        sum = exp_scores(s, c, mc, r);
                        const bool up = mine && (mx > m + lazy || (m == -INFINITY && mx > m));
                        if (!__any_sync(0xffffffffu, up)) break;
                        const float m1 = up ? mx : m;
                        if (x > 0) {
                            // rescale what has been summed with the old
                            // maximum, once the last P V is complete
                            const float f = up ? ex2((m - m1) * c) : 1.0f;
                            l *= f;
                            if (!wait_on(o_full + 8u * (buf ^ 1u), ((cnt - 1) >> 1) & 1u, abort_flag, failed, 51)) {
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
                    if (!ok) break;
                    tmem_st32(ts + 64 * buf, r);
                    l += sum;
                    tmem_st_wait();
                    tc_fence_before();
                }
                __syncwarp();
                mbar_arrive_warp(p_full + 8u * buf, lane);
            }
            if (!ok) break;

            // ---- the item's end: O in tensor memory, m and l here
            const bool merge = !p.two && p.n > 1;       // both warpgroups hold a share of the same rows
            if (!wait_on(o_full + 8u * ((cnt - 1) & 1u), ((cnt - 1) >> 1) & 1u, abort_flag, failed, 52)) break;
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
                if (!wait_on(smem_u32(&ctrl->ml_full[w]), ml_cnt & 1u, abort_flag, failed, 53)) break;
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
                const uint32_t valid = __ballot_sync(0xffffffffu, mine), zero = __ballot_sync(0xffffffffu, none);
                const int64_t at = tok * a.ldo + head * a.ho;
#pragma unroll 1
                for (int x = 0; x < 2 * (kDP / 32); x++) {       // 16 rows, 32 columns at a time
                    const int h = 16 * (x & 1), col = 32 * (x >> 1);
                    if (valid >> h == 0) continue;               // (the rows of an item are its first)
                    float o[16], o1[16];
                    const uint32_t from = ((uint32_t)h << 16) + col;
                    tmem_ld_rows(to + from, o);
                    if (merge) tmem_ld_rows(to + 128 + from, o1);
                    tmem_ld_wait();
#pragma unroll
                    for (int b = 0; b < 2; b++) {
                        const int r = h + 8 * b + (lane >> 2);
                        const float fa = __shfl_sync(0xffffffffu, f0 * inv, r), fb = __shfl_sync(0xffffffffu, f1 * inv, r);
                        __nv_bfloat16* out = a.out + __shfl_sync(0xffffffffu, at, r) + col + 8 * (lane & 3);
                        uint32_t w4[4];
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            float e0 = o[4 * i + 2 * b] * fa, e1 = o[4 * i + 2 * b + 1] * fa;
                            if (merge) {
                                e0 += o1[4 * i + 2 * b] * fb;
                                e1 += o1[4 * i + 2 * b + 1] * fb;
                            }
                            w4[i] = (zero >> r) & 1u ? 0u : cvt_bf16x2(e0, e1);
                        }
                        quad_transpose(w4, lane & 3);
                        if ((valid >> r) & 1u && col + 8 * (lane & 3) < a.head_dim)
                            *reinterpret_cast<uint4*>(out) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
                    }
                }
                if (mine && a.lse)
                    a.lse[tok * a.heads + head] = none ? -INFINITY : (m2 + log2f(l)) * 0.6931471805599453f;
            } else if (any) {
                float* part = a.partials + (2 * cta + (p.cta0 == cta ? 1 : 0)) * kAttnSlotFloats;
                const int srow = (p.two ? j * kAttnRows : 0) + row;
#pragma unroll 1
                for (int k = 0; k < kDP; k += 16) {
                    float o[16];
                    tmem_ld16(to + k, o);
                    tmem_ld_wait();
                    if (merge) {
                        float o1[16];
                        tmem_ld16(to + 128 + k, o1);
                        tmem_ld_wait();
#pragma unroll
                        for (int y = 0; y < 16; y++) o[y] = o[y] * f0 + o1[y] * f1;
                    }
                    if (!mine) continue;
#pragma unroll
                    for (int y = 0; y < 4; y++)
                        __stcg(reinterpret_cast<float4*>(part) + (k / 4 + y) * kAttnSlotRows + srow,
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
            __syncwarp();                    // the other CTAs' parts, acquired by lane 0, for every lane
            if (lane == 0) *ticket = 0;
            // rows in turn over the lanes, `share` lanes to a row with every
            // share-th 4-column vector each
            const int rows = __popc(__ballot_sync(0xffffffffu, mine));
            const int share = rows <= 4 ? 8 : rows <= 8 ? 4 : rows <= 16 ? 2 : 1;
            const int r = lane & (32 / share - 1), sub = lane / (32 / share);
            const int srow = (p.two ? j * kAttnRows : 0) + w * 32 + r;
            // part i of the item is in slot 2 (cta0 + i), the first in 2 cta0 + 1
            const float* const stat = a.partials + kAttnSlotRows * kDP + srow;
            auto slot_of = [&](int i) { return (2 * (p.cta0 + i) + (i == 0 ? 1 : 0)) * kAttnSlotFloats; };
            // maximum and sum over the parts: each of a row's lanes takes
            // every share-th part (a read of another CTA's words takes 1-2
            // thousand cycles: few rounds of many)
            float mall = -INFINITY, lall = 0.0f;
#pragma unroll 1
            for (int i0 = sub; i0 < p.parts; i0 += 4 * share) {
                float mi[4], li[4], top = mall;
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    const int i = i0 + u * share;
                    mi[u] = i < p.parts ? __ldcg(stat + slot_of(i)) : -INFINITY;
                    li[u] = i < p.parts ? __ldcg(stat + slot_of(i) + kAttnSlotRows) : 0.0f;
                }
#pragma unroll
                for (int u = 0; u < 4; u++) top = fmaxf(top, mi[u]);
                const float ref = top == -INFINITY ? 0.0f : top;
                lall *= ex2(mall - ref);
#pragma unroll
                for (int u = 0; u < 4; u++) lall += li[u] * ex2(mi[u] - ref);
                mall = top;
            }
#pragma unroll 1
            for (int x = 32 / share; x < 32; x <<= 1) {
                const float mo = __shfl_xor_sync(0xffffffffu, mall, x), lo = __shfl_xor_sync(0xffffffffu, lall, x);
                const float top = fmaxf(mall, mo), ref = top == -INFINITY ? 0.0f : top;
                lall = lall * ex2(mall - ref) + lo * ex2(mo - ref);
                mall = top;
            }
            const float ms = mall == -INFINITY ? 0.0f : mall;
            const float inv = lall == 0.0f ? 0.0f : 1.0f / lall;
            const int64_t at = __shfl_sync(0xffffffffu, tok * a.ldo + head * a.ho, r);
            const int64_t lse_at = __shfl_sync(0xffffffffu, tok * a.heads + head, r);
            if (a.lse && r < rows && sub == 0)
                a.lse[lse_at] = lall == 0.0f ? -INFINITY : (mall + log2f(lall)) * 0.6931471805599453f;
            if (r >= rows) continue;
            const int vecs = a.head_dim / 4;
            auto join = [&](auto vecs_at_once, auto parts_at_once) {
                constexpr int kV = decltype(vecs_at_once)::value, kP = decltype(parts_at_once)::value;
#pragma unroll 1
                for (int v0 = sub; v0 < vecs; v0 += kV * share) {
                    float4 acc[kV];
#pragma unroll
                    for (int y = 0; y < kV; y++) acc[y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
                    for (int i0 = 0; i0 < p.parts; i0 += kP) {
                        float f[kP];
                        float4 e[kP][kV];
#pragma unroll
                        for (int u = 0; u < kP; u++) {
                            const int i = min(i0 + u, p.parts - 1);
                            f[u] = i0 + u < p.parts ? __ldcg(stat + slot_of(i)) : -INFINITY;
                            const float4* o = reinterpret_cast<const float4*>(a.partials + slot_of(i)) + srow;
#pragma unroll
                            for (int y = 0; y < kV; y++)
                                e[u][y] = __ldcg(o + min(v0 + y * share, vecs - 1) * kAttnSlotRows);
                        }
#pragma unroll
                        for (int u = 0; u < kP; u++) {
                            f[u] = ex2(f[u] - ms) * inv;
#pragma unroll
                            for (int y = 0; y < kV; y++) {
                                acc[y].x += f[u] * e[u][y].x;
                                acc[y].y += f[u] * e[u][y].y;
                                acc[y].z += f[u] * e[u][y].z;
                                acc[y].w += f[u] * e[u][y].w;
                            }
                        }
                    }
#pragma unroll
                    for (int y = 0; y < kV; y++)
                        if (v0 + y * share < vecs)
                            *reinterpret_cast<uint2*>(a.out + at + 4 * (v0 + y * share)) =
                                lall == 0.0f ? make_uint2(0u, 0u)
                                             : make_uint2(cvt_bf16x2(acc[y].x, acc[y].y), cvt_bf16x2(acc[y].z, acc[y].w));
                }
            };
            if (share == 1) join(Int<8>(), Int<2>());
            else join(Int<4>(), Int<4>());
        }
    }
    if (failed) wait_failed(abort_flag, status, failed);
    if (a.cu_end) {
        // the rows past the step's last token, a warp to a row (by warps as
        // they come to the end)
        const int vecs = a.head_dim / 8, n = a.heads * vecs;
        for (int64_t t = max(*a.cu_end, 0) + cta + (int)gridDim.x * warp; t < a.tokens; t += gridDim.x * (kThreads / 32)) {
            for (int x = lane; x < n; x += 32) {
                const int h = x / vecs;
                *reinterpret_cast<uint4*>(a.out + t * a.ldo + h * a.ho + 8 * (x - h * vecs)) = make_uint4(0, 0, 0, 0);
            }
            if (a.lse)
                for (int h = lane; h < a.heads; h += 32) a.lse[t * a.heads + h] = -INFINITY;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int kDP, bool kFold>
cudaError_t launch(const Params& p, int num_sms, cudaStream_t stream)
{
    static int attr_set_for_device[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && !attr_set_for_device[dev]) {
        e = cudaFuncSetAttribute(attn_kernel<kDP, kFold>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<kDP>::kSmemBytes);
        if (e != cudaSuccess) return e;
        attr_set_for_device[dev] = 1;
    }
    return launch_programmatic(attn_kernel<kDP, kFold>, dim3((unsigned)num_sms), dim3(kThreads), Cfg<kDP>::kSmemBytes,
                               stream, p);
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
    if (args.fold) return launch<128, true>(p, ctas, stream);
    return args.head_dim > 64 ? launch<128, false>(p, ctas, stream) : launch<64, false>(p, ctas, stream);
}

}  // namespace nvfp4
