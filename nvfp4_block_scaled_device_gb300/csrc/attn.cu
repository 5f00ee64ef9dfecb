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
// Warps: 0-3 and 4-7 softmax and epilogue, 8 MMA, 9 K/V copies, 10 Q copies,
// 11 the keys' end (below).
//
// Rows past the last key of an item's last tile hold other requests' rows,
// pages' unused rows or nothing at all.  Their scores are masked, and warp 11
// zeroes the V rows before the tile is multiplied, so that NaN or infinities
// there cannot reach a sum as 0 * NaN.
#include <string.h>

#include "attn.h"
#include "common.cuh"
#include "internal.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 384;
constexpr int kWarpMma = 8, kWarpKV = 9, kWarpQ = 10, kWarpEnd = 11;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColS = 256;      // + 128 * warpgroup
constexpr float kLazy = 8.0f;                   // log2 of the growth that P may carry
constexpr int kRegsSoftmax = 216, kRegsOther = 72;
static_assert(2 * kRegsSoftmax + kRegsOther <= 3 * 168, "the block's registers at launch");

constexpr int kMaxStages = 10;

struct Ctrl {
    uint64_t kv_full[kMaxStages], kv_empty[kMaxStages], v_end[kMaxStages];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2], o_full[2], o_free[2];
    uint64_t ml_full[4];
    uint64_t teardown;
    uint32_t tmem_base;
    int abort_flag;
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

// The warp-wide form of the other kernels: the converged warp executes, one
// elected lane issues.  kSteps MMAs of K = 16.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b32 r;\n"
        " setp.ne.b32 p, %4, 0;\n"
        " elect.sync r|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b32 r;\n"
        " setp.ne.b32 p, %4, 0;\n"
        " elect.sync r|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
        "}\n" ::"r"(d), "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
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

// ------------------------------------------------------------------ pieces
// A CTA's share of one item.
struct Piece {
    QTile q;
    int hk;              // kv head
    int tile0, n;        // key tiles tile0 .. tile0 + n - 1
    bool two;            // two row tiles
    int cta0, parts;     // first CTA of the item and how many share it
};

// The pieces of CTA `cta` in order; every warp of the CTA walks them alike.
struct Pieces {
    const ScheduleHead* s;
    int64_t u, end, per_cta;
    int qt;
    int kv_heads, row_tokens;

    __device__ __forceinline__ Pieces(const AttnArgs& a, int cta)
    {
        s = a.sched;
        kv_heads = a.kv_heads;
        row_tokens = row_tile_tokens(a.group);
        const int64_t units = s->units;
        per_cta = s->per_cta;
        u = cta * per_cta;
        end = u + per_cta < units ? u + per_cta : units;
        qt = u < end ? s->first[cta] : 0;
    }
    __device__ __forceinline__ bool next(Piece& p)
    {
        if (u >= end) return false;
        const int4* e = reinterpret_cast<const int4*>(schedule_tiles(s) + qt);
        const int4 e0 = e[0], e1 = e[1], e2 = e[2];
        p.q.tok0 = e0.x;
        p.q.n_tok = e0.y;
        p.q.req = e0.z;
        p.q.pos0 = e0.w;
        p.q.kv_end = e1.x;
        p.q.kv_row = e1.y;
        p.q.tiles = e1.w;
        const int64_t unit0 = (int64_t)(uint32_t)e2.x | ((int64_t)e2.y << 32);
        const int rel = (int)(u - unit0), tiles = e1.w;
        p.hk = rel / tiles;
        const int k0 = rel - p.hk * tiles;
        const int64_t left = end - u;
        p.n = left < tiles - k0 ? (int)left : tiles - k0;
        p.tile0 = e1.z + k0;
        p.two = e0.y > row_tokens;
        const int64_t i0 = u - k0;                   // the item's first unit
        const int64_t c0 = i0 / per_cta, c1 = (i0 + tiles - 1) / per_cta;
        p.cta0 = (int)c0;
        p.parts = (int)(c1 - c0) + 1;
        u += p.n;
        if (rel + p.n == tiles * kv_heads) qt++;
        return true;
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
            mbar_init(smem_u32(&ctrl->kv_empty[s]), 1);
            mbar_init(smem_u32(&ctrl->v_end[s]), 1);
        }
        mbar_init(smem_u32(&ctrl->q_full), 1);
        mbar_init(smem_u32(&ctrl->q_empty), 1);
        for (int j = 0; j < 2; j++) {
            mbar_init(smem_u32(&ctrl->s_full[j]), 1);
            mbar_init(smem_u32(&ctrl->p_full[j]), 4);
            mbar_init(smem_u32(&ctrl->o_full[j]), 1);
            mbar_init(smem_u32(&ctrl->o_free[j]), 4);
        }
        for (int w = 0; w < 4; w++) mbar_init(smem_u32(&ctrl->ml_full[w]), 1);
        mbar_init(smem_u32(&ctrl->teardown), 1);
        ctrl->abort_flag = 0;
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
    Pieces pieces(a, cta);
    Piece p;

    if (warp >= 8) {
        setmaxnreg_dec<kRegsOther>();
        if (warp == kWarpKV) {
            // ------------------------------------------------ K/V copies
            const bool paged = a.block_table != nullptr;
            const int ppt = paged ? kAttnKeys / a.page_size : 1;       // pages of a key tile
            uint32_t use = 0;
            uint32_t issued = 0, issued_ph = 0;   // stages with copies under way, and whose phase
            bool ok = true;
            while (ok && pieces.next(p)) {
                const int* table = paged ? a.block_table + (int64_t)p.q.req * a.table_ld : nullptr;
                for (int i = 0; i < p.n && ok; i++) {
                    const int key0 = (p.tile0 + i) * kAttnKeys;
                    const int valid = min(kAttnKeys, max(p.q.kv_end - key0, 0));
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
                        const CUtensorMap* map = kv ? &prm.map_v : &prm.map_k;
                        const uint32_t dst = base + C::kOffRing + s * C::kTileBytes;
                        // an item's last values go through warp 11
                        const uint32_t bar =
                            smem_u32(kv && valid < kAttnKeys ? &ctrl->v_end[s] : &ctrl->kv_full[s]);
                        const uint32_t bytes =
                            paged ? (uint32_t)(pages * a.page_size * kDP * 2) : (uint32_t)C::kTileBytes;
                        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
                        __syncwarp();
                        if (paged) {
                            // box b: half b / ppt of page b % ppt (at most 16)
                            const int b = lane, half = b / ppt, pg = b - half * ppt;
                            const int id = __shfl_sync(0xffffffffu, page, pg);
                            if (half < C::kHalves && pg < pages)
                                tma_load_4d(dst + half * 16384 + pg * a.page_size * 128, map, bar, half * 64, 0, p.hk,
                                            id);
                        } else if (lane < C::kHalves) {
                            tma_load_3d(dst + lane * 16384, map, bar, lane * 64, p.hk, p.q.kv_row + key0);
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
            // --------------------------------------------------- Q copies
            uint32_t n = 0;
            bool ok = true;
            const int rows = a.group * row_tile_tokens(a.group);
            while (pieces.next(p)) {
                if (!mbar_wait_warp(smem_u32(&ctrl->q_empty), (n & 1u) ^ 1u, abort_flag, status, 42)) {
                    ok = false;
                    break;
                }
                const int boxes = (p.two ? 2 : 1) * C::kHalves;
                const uint32_t bar = smem_u32(&ctrl->q_full);
                if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(boxes * rows * 128));
                __syncwarp();
                if (lane < boxes) {
                    const int j = lane / C::kHalves, half = lane - j * C::kHalves;
                    tma_load_3d(base + j * C::kTileBytes + half * 16384, &prm.map_q, bar, half * 64, p.hk * a.group,
                                p.q.tok0 + j * row_tile_tokens(a.group));
                }
                __syncwarp();
                n++;
            }
            if (!ok && n > 0 && lane == 0) mbar_wait_teardown(smem_u32(&ctrl->q_full), (n - 1) & 1u);
            __syncwarp();
        } else if (warp == kWarpEnd) {
            // ----------------------------------- values past the last key
            uint32_t tile = 0, ends = 0;       // ends: bit s = phase of v_end[s]
            while (pieces.next(p)) {
                tile += p.n;
                const int key0 = (p.tile0 + p.n - 1) * kAttnKeys;
                const int valid = min(kAttnKeys, max(p.q.kv_end - key0, 0));
                if (valid == kAttnKeys) continue;
                uint32_t ph;
                const uint32_t s = stage_of<kStages>(2 * (tile - 1) + 1, &ph);
                if (!mbar_wait_warp<true>(smem_u32(&ctrl->v_end[s]), (ends >> s) & 1u, abort_flag, status, 43)) break;
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
        } else {
            // ------------------------------------------------------- MMA
            const uint64_t kdesc0 = make_smem_desc(base, 16, 1024, 2);              // K-major: 8-row groups 1 KB apart
            const uint64_t vdesc0 = make_smem_desc(base, 16384, 1024, 2);           // N-major: 64-column halves 16 KB
                                                                                    // apart, 8-key groups 1 KB apart
            constexpr uint32_t kIdescS = idesc_of(128, false), kIdescO = idesc_of(kDP, true);
            uint32_t tile = 0, np = 0;                  // key tiles and pieces done
            uint32_t p_cnt[2] = {0, 0}, o_cnt[2] = {0, 0};
            bool ok = true;
            while (ok && pieces.next(p)) {
                const int N = p.two ? 2 * p.n : p.n;
                if (!mbar_wait_warp(smem_u32(&ctrl->q_full), np & 1u, abort_flag, status, 44)) break;
                np++;
                // step n: warpgroup n & 1, key tile n / 2 (two row tiles) or n
                auto issue_s = [&](int n) {
                    const int j = n & 1, i = p.two ? n >> 1 : n;
                    uint32_t ph;
                    const uint32_t s = stage_of<kStages>(2 * (tile + i), &ph);
                    if (!mbar_wait_warp(smem_u32(&ctrl->kv_full[s]), ph, abort_flag, status, 45)) return false;
                    tc_fence_after();
                    const uint64_t qd = kdesc0 + ((p.two && j ? C::kTileBytes : 0) >> 4);
                    const uint64_t kd = kdesc0 + ((C::kOffRing + s * C::kTileBytes) >> 4);
#pragma unroll
                    for (int k = 0; k < kDP / 16; k++) {
                        const uint32_t off = (uint32_t)((k >> 2) * 16384 + (k & 3) * 32) >> 4;
                        mma_ss(tmem + kColS + 128 * j, qd + off, kd + off, kIdescS, k != 0);
                    }
                    if (!p.two || j) mma_commit_warp(smem_u32(&ctrl->kv_empty[s]));
                    mma_commit_warp(smem_u32(&ctrl->s_full[j]));
                    if (n == N - 1) mma_commit_warp(smem_u32(&ctrl->q_empty));
                    return true;
                };
                auto issue_o = [&](int n) {
                    const int j = n & 1, i = p.two ? n >> 1 : n;
                    uint32_t ph;
                    const uint32_t s = stage_of<kStages>(2 * (tile + i) + 1, &ph);
                    if (!mbar_wait_warp(smem_u32(&ctrl->kv_full[s]), ph, abort_flag, status, 46)) return false;
                    if (n < 2) {
                        // the accumulator's previous item has been read
                        if (o_cnt[j] > 0 && !mbar_wait_warp(smem_u32(&ctrl->o_free[j]), (o_cnt[j] - 1) & 1u, abort_flag,
                                                            status, 47))
                            return false;
                        o_cnt[j]++;
                    }
                    if (!mbar_wait_warp(smem_u32(&ctrl->p_full[j]), p_cnt[j] & 1u, abort_flag, status, 48)) return false;
                    p_cnt[j]++;
                    tc_fence_after();
                    const uint64_t vd = vdesc0 + ((C::kOffRing + s * C::kTileBytes) >> 4);
#pragma unroll
                    for (int k = 0; k < kAttnKeys / 16; k++)
                        mma_ts(tmem + kColO + 128 * j, tmem + kColS + 128 * j + 8 * k, vd + ((k * 2048) >> 4), kIdescO,
                               n >= 2 || k != 0);
                    if (!p.two || j) mma_commit_warp(smem_u32(&ctrl->kv_empty[s]));
                    mma_commit_warp(smem_u32(&ctrl->o_full[j]));
                    return true;
                };
                ok = issue_s(0) && (N < 2 || issue_s(1));
                for (int n = 0; n < N && ok; n++) ok = issue_o(n) && (n + 2 >= N || issue_s(n + 2));
                tile += p.n;
            }
            // every MMA issued has completed before teardown
            mma_commit_warp(smem_u32(&ctrl->teardown));
            if (lane == 0) mbar_wait_teardown(smem_u32(&ctrl->teardown), 0);
            __syncwarp();
        }
    } else {
        // ------------------------------------------- softmax and epilogue
        setmaxnreg_inc<kRegsSoftmax>();
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
        uint32_t s_cnt = 0, ml_cnt = 0;
        bool ok = true;
        while (ok && pieces.next(p)) {
            const int N = p.two ? 2 * p.n : p.n;
            const int t = (p.two && j ? row_tokens : 0) + tk;    // token of the item
            const bool mine = tk < row_tokens && t < p.q.n_tok;
            const bool any = __any_sync(0xffffffffu, mine);
            const int pos = p.q.pos0 + t;
            const int hi = mine ? min(pos + 1, p.q.kv_end) : 0;      // keys lo .. hi - 1
            const int lo = mine && a.window ? max(pos + 1 - a.window, 0) : 0;
            float m = -INFINITY, l = 0.0f;
            if (j >= N) continue;            // the second warpgroup of a single key tile
            for (int n = j; n < N; n += 2) {
                const int i = p.two ? n >> 1 : n;
                if (!mbar_wait_warp(smem_u32(&ctrl->s_full[j]), s_cnt & 1u, abort_flag, status, 50)) {
                    ok = false;
                    break;
                }
                s_cnt++;
                if (any) {
                    tc_fence_after();
                    float s[128];
#pragma unroll
                    for (int k = 0; k < 4; k++) tmem_ld32(ts + 32 * k, s + 32 * k);
                    tmem_ld_wait();
                    if (negate) {
#pragma unroll
                        for (int k = 0; k < 128; k++) s[k] = -s[k];
                    }
                    const int key0 = (p.tile0 + i) * kAttnKeys;
                    const int h = hi - key0, lw = lo - key0;
                    if (__any_sync(0xffffffffu, mine && (h < kAttnKeys || lw > 0))) {
#pragma unroll
                        for (int k = 0; k < 128; k++) s[k] = k < h && k >= lw ? s[k] : -INFINITY;
                    }
                    float x[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                    for (int k = 4; k < 124; k += 8) {
#pragma unroll
                        for (int y = 0; y < 4; y++) x[y] = max3(x[y], s[k + 2 * y], s[k + 2 * y + 1]);
                    }
#pragma unroll
                    for (int y = 0; y < 4; y++) x[y] = fmaxf(x[y], s[124 + y]);
                    const float mx = fmaxf(max3(x[0], x[1], x[2]), x[3]);
                    const bool up = mine && (mx > m + lazy || (m == -INFINITY && mx > m));
                    if (__any_sync(0xffffffffu, up)) {
                        const float m1 = up ? mx : m;
                        if (n >= 2) {
                            // rescale what has been summed with the old maximum
                            const float f = up ? ex2((m - m1) * c) : 1.0f;
                            l *= f;
                            if (!mbar_wait_warp(smem_u32(&ctrl->o_full[j]), (s_cnt - 2) & 1u, abort_flag, status, 51)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
#pragma unroll 1
                            for (int k = 0; k < kDP / 32; k++) {
                                float o[32];
                                tmem_ld32(to + 32 * k, o);
                                tmem_ld_wait();
                                uint32_t r[32];
#pragma unroll
                                for (int y = 0; y < 32; y++) r[y] = __float_as_uint(f == 0.0f ? 0.0f : o[y] * f);
                                tmem_st32(to + 32 * k, r);
                            }
                        }
                        m = m1;
                    }
                    const float mc = m == -INFINITY ? 0.0f : -m * c;
                    float2 sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        uint32_t r[32];
#pragma unroll
                        for (int y = 0; y < 32; y++) {
                            float2 e = fma2(make_float2(s[64 * k + 2 * y], s[64 * k + 2 * y + 1]), make_float2(c, c),
                                            make_float2(mc, mc));
                            e.x = ex2(e.x);
                            e.y = ex2(e.y);
                            sum[y & 1] = add2(sum[y & 1], e);
                            r[y] = cvt_bf16x2(e.x, e.y);
                        }
                        tmem_st32(ts + 32 * k, r);
                    }
                    sum[0] = add2(sum[0], sum[1]);
                    l += sum[0].x + sum[0].y;
                    tmem_st_wait();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctrl->p_full[j]));
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
            const int64_t tok = p.q.tok0 + t;
            if (any) {
                const float inv = whole ? (none ? 0.0f : 1.0f / l) : 1.0f;
                const int slot = 2 * cta + (p.cta0 == cta ? 1 : 0);
                float* part = a.partials + slot * kAttnSlotFloats;
                const int srow = (p.two ? j * kAttnRows : 0) + row;
#pragma unroll 1
                for (int k = 0; k < kDP / 32; k++) {
                    float o[32];
                    tmem_ld32(to + 32 * k, o);
                    tmem_ld_wait();
                    if (merge) {
                        float o1[32];
                        tmem_ld32(lane_addr + kColO + 128 + 32 * k, o1);
                        tmem_ld_wait();
#pragma unroll
                        for (int y = 0; y < 32; y++) o[y] = o[y] * f0 + o1[y] * f1;
                    }
                    if (!mine) continue;
                    if (whole) {
                        __nv_bfloat16* out = a.out + tok * a.ldo + head * a.ho + 32 * k;
#pragma unroll
                        for (int y = 0; y < 4; y++) {
                            uint4 v;
                            v.x = cvt_bf16x2(none ? 0.0f : o[8 * y] * inv, none ? 0.0f : o[8 * y + 1] * inv);
                            v.y = cvt_bf16x2(none ? 0.0f : o[8 * y + 2] * inv, none ? 0.0f : o[8 * y + 3] * inv);
                            v.z = cvt_bf16x2(none ? 0.0f : o[8 * y + 4] * inv, none ? 0.0f : o[8 * y + 5] * inv);
                            v.w = cvt_bf16x2(none ? 0.0f : o[8 * y + 6] * inv, none ? 0.0f : o[8 * y + 7] * inv);
                            if (32 * k + 8 * y < a.head_dim) *reinterpret_cast<uint4*>(out + 8 * y) = v;
                        }
                    } else {
#pragma unroll
                        for (int y = 0; y < 8; y++)
                            __stcg(reinterpret_cast<float4*>(part) + (8 * k + y) * kAttnSlotRows + srow,
                                   make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]));
                    }
                }
                if (mine && whole && a.lse)
                    a.lse[tok * a.heads + head] = none ? -INFINITY : (m2 + log2f(l)) * 0.6931471805599453f;
                if (mine && !whole) {
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
            __threadfence();
            __syncwarp();
            int* ticket = a.tickets + (p.cta0 * 2 + (p.two ? j : 0)) * 4 + w;
            int last = 0;
            if (lane == 0) last = atom_add_acq_rel(ticket, 1) == p.parts - 1;
            last = __shfl_sync(0xffffffffu, last, 0);
            if (!last) continue;
            __threadfence();
            if (lane == 0) *ticket = 0;
            const int row0 = (p.two ? j * kAttnRows : 0) + w * 32;   // the warp's first row in a slot
            const int rows = __popc(__ballot_sync(0xffffffffu, mine));
            auto part_of = [&](int i) {
                const int cc = p.cta0 + i;
                return a.partials + (int64_t)(2 * cc + (i == 0 ? 1 : 0)) * kAttnSlotFloats;
            };
            float mall = -INFINITY, lall = 0.0f;
            if (mine) {
                for (int i = 0; i < p.parts; i++)
                    mall = fmaxf(mall, __ldcg(part_of(i) + kAttnSlotRows * kDP + row0 + lane));
                const float ms = mall == -INFINITY ? 0.0f : mall;
                for (int i = 0; i < p.parts; i++)
                    lall += __ldcg(part_of(i) + kAttnSlotRows * (kDP + 1) + row0 + lane) *
                            ex2(__ldcg(part_of(i) + kAttnSlotRows * kDP + row0 + lane) - ms);
                if (a.lse) a.lse[tok * a.heads + head] = lall == 0.0f ? -INFINITY : (mall + log2f(lall)) * 0.6931471805599453f;
            }
            // 4 columns of a row per lane
            const int vecs = rows * (a.head_dim / 4);
            for (int b = 0; b < vecs; b += 32) {
                const int x = min(b + lane, vecs - 1);
                const int v = x / rows, r = x - v * rows;
                const float mr = __shfl_sync(0xffffffffu, mall, r), lr = __shfl_sync(0xffffffffu, lall, r);
                const int64_t tr = __shfl_sync(0xffffffffu, tok, r);
                const int hr = __shfl_sync(0xffffffffu, head, r);
                const float ms = mr == -INFINITY ? 0.0f : mr;
                float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
                for (int i = 0; i < p.parts; i++) {
                    const float* part = part_of(i);
                    const float f = ex2(__ldcg(part + kAttnSlotRows * kDP + row0 + r) - ms);
                    const float4 o = __ldcg(reinterpret_cast<const float4*>(part) + v * kAttnSlotRows + row0 + r);
                    acc.x += f * o.x;
                    acc.y += f * o.y;
                    acc.z += f * o.z;
                    acc.w += f * o.w;
                }
                const float inv = lr == 0.0f ? 0.0f : 1.0f / lr;
                const bool zero = lr == 0.0f;
                uint2 v2;
                v2.x = cvt_bf16x2(zero ? 0.0f : acc.x * inv, zero ? 0.0f : acc.y * inv);
                v2.y = cvt_bf16x2(zero ? 0.0f : acc.z * inv, zero ? 0.0f : acc.w * inv);
                if (b + lane < vecs) *reinterpret_cast<uint2*>(a.out + tr * a.ldo + hr * a.ho + 4 * v) = v2;
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
