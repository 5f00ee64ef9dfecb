// The walk over the attention's schedule (attn.h) that its kernels share: which
// part of which item a CTA works on next.
#pragma once

#include "attn.h"

namespace nvfp4 {
namespace {

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

__device__ __forceinline__ int atom_add_acq_rel(int* p, int v)
{
    int old;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

}  // namespace
}  // namespace nvfp4
