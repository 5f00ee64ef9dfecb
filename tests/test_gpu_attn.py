"""GPU tests of the attention operators (step tables, cache append, packed
prompts, paged cache) against plain forms: the tables and the cache bit for
bit, attention against binary64 within the bounds of _attn.py."""
import math

import numpy as np
import pytest
import torch

from _attn import check, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_device_gb300 as m
    return m


@pytest.fixture(scope="module")
def ws(nv):
    return nv.workspace(nv.attn_workspace_bytes())


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def plan_reference(ctx, q, P, table, free, cursor, tokens):
    """The step's tables by plain loops."""
    table = table.copy()
    R = len(q)
    cu, pos, slot = [0], np.zeros(tokens, np.int32), np.full(tokens, -1, np.int32)
    for r in range(R):
        cu.append(cu[-1] + q[r])
    for r in range(R):
        for j in range(-(-ctx[r] // P), -(-(ctx[r] + q[r]) // P)):
            if j < table.shape[1]:
                table[r, j] = free[cursor] if cursor < len(free) else -1
            cursor += 1
        for t in range(q[r]):
            p, i = ctx[r] + t, cu[r] + t
            pos[i] = p
            page = table[r, p // P] if p // P < table.shape[1] else -1
            if page >= 0:
                slot[i] = page * P + p % P
    return np.array(cu), pos, slot, table, cursor


def lengths(rng, R, lo, hi):
    return [int(x) for x in rng.integers(lo, hi + 1, R)]


# ---------------------------------------------------------------------- plan
@pytest.mark.parametrize("R,q_lo,q_hi,c_lo,c_hi,P,pad", [
    (1, 1, 1, 0, 0, 16, 0), (1, 0, 0, 5, 5, 16, 3), (1, 1000, 1000, 0, 0, 16, 0), (3, 0, 2, 0, 40, 16, 1),
    (64, 1, 1, 100, 4096, 16, 0), (33, 0, 70, 0, 300, 32, 9), (513, 0, 9, 0, 200, 64, 100),
    (1025, 1, 1, 0, 129, 128, 0), (8192, 0, 2, 0, 100, 16, 0), (2, 9000, 9001, 15, 17, 128, 5)])
def test_plan(nv, R, q_lo, q_hi, c_lo, c_hi, P, pad):
    rng = np.random.default_rng(R * 31 + P)
    q, ctx = lengths(rng, R, q_lo, q_hi), lengths(rng, R, c_lo, c_hi)
    have, need = [-(-c // P) for c in ctx], [-(-(c + n) // P) for c, n in zip(ctx, q)]
    tokens = max(1, sum(q) + pad)
    ids = rng.permutation(sum(need) + 7).astype(np.int32)
    table = np.full((R, max(need) + 2), -1, np.int32)
    at = 0
    for r in range(R):
        table[r, :have[r]] = ids[at:at + have[r]]
        at += have[r]
    free, cursor = ids[at:], 4
    exp = plan_reference(ctx, q, P, table, free, cursor, tokens)
    plan = nv.AttnPlan(R, tokens, 8, 2, page_size=P, block_table=torch.from_numpy(table).cuda())
    for _ in range(2):                              # a second call on the same inputs gives the same tables
        nv.nvfp4_attn_plan(plan, i32(q), i32(ctx), torch.from_numpy(free).cuda(), i32([cursor]))
    torch.cuda.synchronize()
    assert nv.device_status() == 0
    for name, got, want in (("cu_q", plan.cu_q, exp[0]), ("pos", plan.pos, exp[1]), ("slot", plan.slot, exp[2]),
                            ("table", plan.block_table, exp[3]), ("cursor", plan.cursor, [exp[4]]),
                            ("kv_len", plan.kv_len, np.add(ctx, q))):
        assert np.array_equal(got.cpu().numpy(), want), name


def test_plan_without_cache_or_free_list(nv):
    q = [3, 0, 7]
    plan = nv.AttnPlan(3, 12, 8, 2)
    nv.nvfp4_attn_plan(plan, i32(q))
    assert plan.cu_q.tolist() == [0, 3, 3, 10] and plan.kv_len.tolist() == q
    assert plan.pos.tolist() == [0, 1, 2] + list(range(7)) + [0, 0]
    # tables managed by the caller: read, not written; table rows wider apart than their columns
    wide = torch.arange(30, dtype=torch.int32, device="cuda").reshape(3, 10)
    plan = nv.AttnPlan(3, 10, 8, 2, page_size=16, block_table=wide[:, :4])
    before = wide.clone()
    nv.nvfp4_attn_plan(plan, i32(q), i32([16, 3, 40]))
    assert torch.equal(wide, before)
    assert plan.slot.tolist() == [16, 17, 18] + [22 * 16 + 8 + t for t in range(7)]
    assert nv.device_status() == 0


def test_plan_errors_are_recorded(nv):
    bad = 100 + 31
    # a negative length counts as zero
    plan = nv.AttnPlan(3, 8, 8, 2)
    nv.nvfp4_attn_plan(plan, i32([2, -5, 3]))
    assert plan.cu_q.tolist() == [0, 2, 2, 5] and nv.device_status() == bad
    # more tokens than rows: dropped
    plan = nv.AttnPlan(2, 4, 8, 2)
    nv.nvfp4_attn_plan(plan, i32([3, 3]))
    assert plan.cu_q.tolist() == [0, 3, 4] and plan.kv_len.tolist() == [3, 1] and nv.device_status() == bad
    # the free list runs out: entries and slots -1, the cursor counts what was asked for
    plan = nv.AttnPlan(2, 64, 8, 2, page_size=16, block_table=4)
    nv.nvfp4_attn_plan(plan, i32([32, 32]), free_pages=i32([7, 9, 5]))
    assert plan.block_table.tolist() == [[7, 9, -1, -1], [5, -1, -1, -1]]
    assert plan.slot.tolist() == [7 * 16 + t for t in range(16)] + [9 * 16 + t for t in range(16)] + \
        [5 * 16 + t for t in range(16)] + [-1] * 16
    assert plan.cursor.item() == 4 and nv.device_status() == bad
    # a request longer than its table
    plan = nv.AttnPlan(1, 48, 8, 2, page_size=16, block_table=2)
    nv.nvfp4_attn_plan(plan, i32([48]), free_pages=i32([1, 2, 3]))
    assert plan.block_table.tolist() == [[1, 2]] and plan.slot.tolist()[32:] == [-1] * 16
    assert nv.device_status() == bad
    # no errors left behind
    plan = nv.AttnPlan(1, 4, 8, 2)
    nv.nvfp4_attn_plan(plan, i32([4]))
    assert nv.device_status() == 0


# -------------------------------------------------------------------- append
@pytest.mark.parametrize("T,Hkv,D,P,layout", [(1, 1, 16, 16, "slices"), (17, 8, 128, 16, "slices"),
                                              (333, 3, 96, 32, "heads_first"), (1000, 20, 64, 64, "slices"),
                                              (6, 2, 128, 128, "interleaved"), (2049, 8, 104, 64, "interleaved")])
def test_append(nv, T, Hkv, D, P, layout):
    g = torch.Generator("cuda").manual_seed(T + D)
    pages = -(-T // P) + 3
    rnd = lambda *s: torch.randint(-2 ** 15, 2 ** 15, s, dtype=torch.int16, device="cuda", generator=g).view(torch.bfloat16)
    if layout == "heads_first":                     # [heads, tokens, columns] in memory
        k, v = rnd(Hkv, T, D).transpose(0, 1), rnd(Hkv, T, D).transpose(0, 1)
    else:                                           # column slices of one projection
        x = rnd(T, (2 * Hkv + 3) * D)
        k, v = x[:, D:(Hkv + 1) * D].unflatten(1, (Hkv, D)), x[:, (Hkv + 1) * D:(2 * Hkv + 1) * D].unflatten(1, (Hkv, D))
    if layout == "interleaved":
        both = rnd(pages, 2, Hkv, P, D)
        cache = nv.KVCache(both[:, 0], both[:, 1])
    else:
        cache = nv.KVCache(rnd(pages, Hkv, P, D), rnd(pages, Hkv, P, D))
    bits = lambda t: t.contiguous().view(torch.int16)
    ek, ev = bits(cache.k).clone(), bits(cache.v).clone()
    slot = torch.randperm(pages * P, device="cuda", generator=g)[:T]
    slot[T // 2] = -1 if T > 1 else slot[T // 2]
    ok = slot >= 0
    page, row = slot[ok] // P, slot[ok] % P
    ek[page, :, row], ev[page, :, row] = bits(k)[ok], bits(v)[ok]
    plan = nv.AttnPlan(1, T, Hkv, Hkv, page_size=P, block_table=pages)
    plan.slot.copy_(slot)
    nv.nvfp4_kv_append(k, v, plan, cache)
    assert torch.equal(bits(cache.k), ek) and torch.equal(bits(cache.v), ev)
    assert nv.device_status() == 0


def test_append_slot_outside_the_cache_is_skipped(nv):
    k = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    cache = nv.KVCache(*(torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    plan = nv.AttnPlan(1, 4, 2, 2, page_size=16, block_table=3)
    for bad in (48, -2, 2 ** 31 - 1):
        cache.k.zero_()
        plan.slot.copy_(i32([47, bad, -1, 0]))
        nv.nvfp4_kv_append(k, k, plan, cache)
        assert cache.k.float().sum().item() == 2 * 2 * 64 and nv.device_status() == 100 + 32


# -------------------------------------------------------------------- prompt
def rows(gen, T, H, D, layout, std=1.0):
    """bf16 [T, H, D] in one of several memory orders."""
    r = lambda *s: (torch.randn(s, device="cuda", generator=gen) * std).to(torch.bfloat16)
    if layout == "heads_first":
        return r(H, T, D).transpose(0, 1)
    if layout == "padded":
        return r(T, H, D + 24)[:, :, 8:8 + D]
    return r(T, H, D)


def run_prompt(nv, ws, lens, H, Hkv, D, window=0, layout="plain", pad=0, std=1.5, scale=None, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed + sum(lens) + D)
    T = sum(lens) + pad
    q, k, v = (rows(gen, T, h, D, layout, s) for h, s in ((H, std), (Hkv, std), (Hkv, 1.0)))
    out = rows(gen, T, H, D, layout)
    out.fill_(7.0)
    lse = torch.full((T, H), 7.0, device="cuda")
    plan = nv.AttnPlan(len(lens), T, H, Hkv, window=window)
    nv.nvfp4_attn_plan(plan, i32(lens))
    nv.nvfp4_attn_prompt(q, k, v, plan, out, ws, scale=scale, lse=lse)
    torch.cuda.synchronize()
    assert nv.device_status() == 0
    at = 0
    for n in lens:
        sl = slice(at, at + n)
        if not n:
            continue
        ref = reference(q[sl].double(), k[sl].double(), v[sl].double(), 0, D ** -0.5 if scale is None else scale, window)
        check(out[sl], lse[sl], ref[0], ref[1], ref[2], f"prompt {lens} H={H}/{Hkv} D={D} window={window} rows {sl}")
        at += n
    assert (out[at:] == 7.0).all() and (lse[at:] == 7.0).all()       # padding rows are not written
    return out


@pytest.mark.parametrize("lens", [[1], [2], [17], [127], [128], [129], [255, 1], [1, 1, 1], [0, 5, 0, 130, 0],
                                  [300, 77, 499], [1025], [640, 0, 2]])
@pytest.mark.parametrize("H,Hkv,D", [(40, 8, 128), (4, 4, 64)])
def test_prompt_lengths(nv, ws, lens, H, Hkv, D):
    if sum(lens) == 0:
        pytest.skip("no rows")
    run_prompt(nv, ws, lens, H, Hkv, D)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (7, 1), (28, 4), (64, 8), (9, 3), (33, 1), (128, 1), (130, 2), (20, 20)])
@pytest.mark.parametrize("D", [128, 64, 96, 16, 72, 120])
def test_prompt_heads(nv, ws, H, Hkv, D):
    run_prompt(nv, ws, [70, 139], H, Hkv, D, pad=3)


@pytest.mark.parametrize("window", [1, 2, 63, 128, 129, 200, 5000])
@pytest.mark.parametrize("H,Hkv,D", [(10, 2, 128), (2, 2, 64)])
def test_prompt_window(nv, ws, window, H, Hkv, D):
    run_prompt(nv, ws, [700, 3, 131], H, Hkv, D, window=window)


@pytest.mark.parametrize("layout", ["heads_first", "padded"])
@pytest.mark.parametrize("H,Hkv,D", [(10, 2, 128), (6, 6, 64), (5, 1, 80)])
def test_prompt_layouts(nv, ws, layout, H, Hkv, D):
    run_prompt(nv, ws, [33, 200, 1], H, Hkv, D, layout=layout, pad=2)


def test_prompt_scores_of_all_sizes(nv, ws):
    for std, scale in ((0.01, None), (8.0, None), (1.0, 0.0), (1.0, -0.3), (3.0, 0.02)):
        run_prompt(nv, ws, [150, 61], 10, 2, 64, std=std, scale=scale)


def test_prompt_rising_scores_and_large_values(nv, ws):
    """Scores that rise along the keys (the running maximum moves at every
    key) and fall, over several tiles."""
    T, D = 900, 64
    gen = torch.Generator("cuda").manual_seed(3)
    for sign in (1.0, -1.0):
        q = torch.ones(T, 2, D, device="cuda").to(torch.bfloat16)
        ramp = torch.linspace(-6, 6, T, device="cuda")[:, None, None] * sign
        k = (ramp + 0.01 * torch.randn(T, 2, D, device="cuda", generator=gen)).to(torch.bfloat16)
        v = (1000 * torch.randn(T, 2, D, device="cuda", generator=gen)).to(torch.bfloat16)
        out, lse = torch.empty_like(q), torch.empty(T, 2, device="cuda")
        plan = nv.AttnPlan(1, T, 2, 2)
        nv.nvfp4_attn_plan(plan, i32([T]))
        nv.nvfp4_attn_prompt(q, k, v, plan, out, ws, lse=lse)
        ref = reference(q.double(), k.double(), v.double(), 0, D ** -0.5)
        check(out, lse, *ref, "rising scores")


def test_prompt_neighbours_do_not_reach_each_other(nv, ws):
    """A request full of NaN, infinities and the type's extremes next to
    others: the others' outputs are bit for bit what they are without it."""
    lens, H, Hkv, D = [130, 45, 300], 10, 2, 128
    gen = torch.Generator("cuda").manual_seed(9)
    T = sum(lens)
    q, k, v = (rows(gen, T, h, D, "plain") for h in (H, Hkv, Hkv))
    plan = nv.AttnPlan(3, T, H, Hkv)
    nv.nvfp4_attn_plan(plan, i32(lens))
    outs = []
    for poison in (None, math.nan, math.inf, -math.inf, torch.finfo(torch.bfloat16).min):
        kk, vv, qq = k.clone(), v.clone(), q.clone()
        if poison is not None:
            for t in (kk, vv, qq):
                t[130:175] = poison
        out = torch.empty_like(q)
        nv.nvfp4_attn_prompt(qq, kk, vv, plan, out, ws)
        outs.append(out)
    for o in outs[1:]:
        assert torch.equal(o[:130], outs[0][:130]) and torch.equal(o[175:], outs[0][175:])


# --------------------------------------------------------------------- paged
def make_paged(nv, gen, rng, ctx, q, Hkv, D, P, spare=2, interleaved=False, fill=math.nan, cols=None):
    """A cache whose live rows are random and all others `fill`; the table's
    unused entries point at pages full of `fill`."""
    need = [-(-(c + n) // P) for c, n in zip(ctx, q)]
    pages = sum(need) + spare
    shape = (pages, 2, Hkv, P, D)
    if interleaved:
        both = torch.full(shape, fill, dtype=torch.bfloat16, device="cuda")
        kc, vc = both[:, 0], both[:, 1]
    else:
        kc, vc = (torch.full((pages, Hkv, P, D), fill, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ids = rng.permutation(pages).astype(np.int32)
    width = max(max(need), cols or 1)
    table = np.full((len(q), width), ids[-1] if spare else -1, np.int32)
    at = 0
    live = []
    for r, (c, n) in enumerate(zip(ctx, q)):
        table[r, :need[r]] = ids[at:at + need[r]]
        at += need[r]
        kv = [(torch.randn(c + n, Hkv, D, device="cuda", generator=gen) * s).to(torch.bfloat16) for s in (1.5, 1.0)]
        for dst, src in zip((kc, vc), kv):
            for j in range(need[r]):
                part = src[j * P:(j + 1) * P]
                dst[int(table[r, j]), :, :part.shape[0]] = part.transpose(0, 1)
        live.append(kv)
    return nv.KVCache(kc, vc), torch.from_numpy(table).cuda(), live


def run_paged(nv, ws, ctx, q, H, Hkv, D, P, window=0, layout="plain", pad=0, seed=0, **more):
    gen = torch.Generator("cuda").manual_seed(seed + sum(q) + D)
    rng = np.random.default_rng(seed + P)
    cache, table, live = make_paged(nv, gen, rng, ctx, q, Hkv, D, P, **more)
    T = sum(q) + pad
    qq, out = rows(gen, T, H, D, layout, 1.5), rows(gen, T, H, D, layout)
    out.fill_(7.0)
    lse = torch.full((T, H), 7.0, device="cuda")
    plan = nv.AttnPlan(len(q), T, H, Hkv, page_size=P, block_table=table, window=window)
    nv.nvfp4_attn_plan(plan, i32(q), i32(ctx))
    nv.nvfp4_attn_paged(qq, cache, plan, out, ws, lse=lse)
    torch.cuda.synchronize()
    assert nv.device_status() == 0
    at = 0
    for r, (c, n) in enumerate(zip(ctx, q)):
        sl = slice(at, at + n)
        k, v = (x.double() for x in live[r])
        if n:
            ref = reference(qq[sl].double(), k, v, c, D ** -0.5, window)
            check(out[sl], lse[sl], *ref, f"paged ctx={c} q={n} H={H}/{Hkv} D={D} P={P} window={window}")
        at += n
    assert (out[at:] == 7.0).all() and (lse[at:] == 7.0).all()
    return out, lse


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("ctx,q", [([0], [1]), ([1], [1]), ([15], [1]), ([16], [1]), ([127], [1]), ([128], [1]),
                                   ([333], [1]), ([0, 500, 3, 129], [1, 1, 1, 1]), ([1000], [17]), ([77], [130]),
                                   ([2000, 0, 64], [1, 70, 0]), ([5, 900], [300, 1])])
def test_paged_lengths(nv, ws, ctx, q, P):
    run_paged(nv, ws, ctx, q, 40, 8, 128, P)


@pytest.mark.parametrize("H,Hkv,D", [(1, 1, 128), (7, 1, 64), (28, 4, 128), (64, 8, 96), (9, 3, 16), (128, 1, 128),
                                     (130, 2, 72), (20, 20, 64)])
def test_paged_heads(nv, ws, H, Hkv, D):
    run_paged(nv, ws, [700, 31, 4], [1, 3, 150], H, Hkv, D, 32, pad=2)


@pytest.mark.parametrize("window", [1, 16, 100, 128, 300, 4000])
def test_paged_window(nv, ws, window):
    run_paged(nv, ws, [1500, 90, 0], [1, 140, 33], 10, 2, 128, 16, window=window)


@pytest.mark.parametrize("D", [128, 64])
def test_many_short_items_after_a_longer_one(nv, ws, D):
    """Items of a single key tile are one MMA warp's alone: the other passes
    many of them in a row, whatever it still has to do for the item before."""
    H, Hkv = 8, 4
    lens = [200, 3, 1, 5, 2, 64, 7, 1, 1, 2] * 30
    gen = torch.Generator("cuda").manual_seed(D)
    T = sum(lens)
    q, k, v = (rows(gen, T, h, D, "plain", 1.5) for h in (H, Hkv, Hkv))
    out, lse = torch.empty_like(q), torch.empty(T, H, device="cuda")
    plan = nv.AttnPlan(len(lens), T, H, Hkv)
    nv.nvfp4_attn_plan(plan, i32(lens))
    nv.nvfp4_attn_prompt(q, k, v, plan, out, ws, lse=lse)
    torch.cuda.synchronize()
    assert nv.device_status() == 0
    at = 0
    for n in lens:
        sl = slice(at, at + n)
        check(out[sl], lse[sl], *reference(q[sl].double(), k[sl].double(), v[sl].double(), 0, D ** -0.5), f"rows {sl}")
        at += n
    rng = np.random.default_rng(D)
    ctx = [int(c) for c in rng.choice([3, 9, 40, 70, 100, 300, 700], 400, p=[.2, .2, .2, .1, .1, .1, .1])]
    run_paged(nv, ws, ctx, [1] * len(ctx), H, Hkv, D, 16, seed=D)


@pytest.mark.parametrize("P,D", [(16, 128), (64, 128), (16, 64), (128, 80)])
@pytest.mark.parametrize("window", [1, 40, 129, 700])
def test_paged_rows_before_the_window(nv, ws, window, P, D):
    """Cached rows that have left every row's window may hold anything (their
    pages may be another request's by now)."""
    gen, rng = torch.Generator("cuda").manual_seed(window + D), np.random.default_rng(P)
    ctx, q, H, Hkv = [1500, 90, 2, 4111], [1, 33, 5, 1], 10, 2
    cache, table, live = make_paged(nv, gen, rng, ctx, q, Hkv, D, P)
    for r, c in enumerate(ctx):
        for at in range(max(c + 1 - window, 0)):
            for t in (cache.k, cache.v):
                t[int(table[r, at // P]), :, at % P] = math.nan if at % 2 else math.inf
    T = sum(q)
    qq = rows(gen, T, H, D, "plain", 1.5)
    out, lse = torch.empty_like(qq), torch.empty(T, H, device="cuda")
    plan = nv.AttnPlan(len(q), T, H, Hkv, page_size=P, block_table=table, window=window)
    nv.nvfp4_attn_plan(plan, i32(q), i32(ctx))
    nv.nvfp4_attn_paged(qq, cache, plan, out, ws, lse=lse)
    torch.cuda.synchronize()
    assert nv.device_status() == 0
    at = 0
    for r, (c, n) in enumerate(zip(ctx, q)):
        k, v = (x.double() for x in live[r])
        ref = reference(qq[at:at + n].double(), k, v, c, D ** -0.5, window)
        check(out[at:at + n], lse[at:at + n], *ref, f"rows before the window, ctx={c}")
        at += n


@pytest.mark.parametrize("layout,interleaved", [("heads_first", True), ("padded", False)])
def test_paged_layouts(nv, ws, layout, interleaved):
    run_paged(nv, ws, [300, 12], [5, 64], 10, 2, 96, 64, layout=layout, interleaved=interleaved)


def test_paged_ragged_batches(nv, ws):
    rng = np.random.default_rng(2)
    for R, c_hi, q_hi in ((150, 900, 1), (40, 2500, 9), (7, 9000, 40)):
        ctx, q = [int(x) for x in np.exp(rng.uniform(0, np.log(c_hi), R))], lengths(rng, R, 0, q_hi)
        run_paged(nv, ws, ctx, q, 10, 2, 128, 16, seed=R)


def test_paged_long_context(nv, ws):
    """Few rows, a long axis: one request's keys spread over the whole GPU."""
    run_paged(nv, ws, [70001], [1], 10, 2, 128, 64)
    run_paged(nv, ws, [33333, 40000], [1, 2], 8, 8, 64, 16)


def test_paged_empty_rows(nv, ws):
    """Rows whose window lies past the block table's last page see no key:
    out 0, lse -inf."""
    H, Hkv, D, P = 10, 2, 64, 16
    gen, rng = torch.Generator("cuda").manual_seed(1), np.random.default_rng(1)
    for n in (60, 300):
        cache, table, live = make_paged(nv, gen, rng, [0], [32], Hkv, D, P)
        plan = nv.AttnPlan(1, n, H, Hkv, page_size=P, block_table=table, window=8)
        q = rows(gen, n, H, D, "plain")
        out, lse = torch.full_like(q, 7.0), torch.full((n, H), 7.0, device="cuda")
        nv.nvfp4_attn_plan(plan, i32([n]), i32([0]))
        assert nv.device_status() == 100 + 31
        nv.nvfp4_attn_paged(q, cache, plan, out, ws, lse=lse)
        k, v = (x.double() for x in live[0])
        check(out, lse, *reference(q.double(), k, v, 0, D ** -0.5, window=8), "rows without keys")
        assert (out[39:] == 0).all() and torch.isneginf(lse[39:]).all()


def test_paged_bad_pages_count_as_zeros(nv, ws):
    H, Hkv, D, P = 10, 2, 128, 16
    gen, rng = torch.Generator("cuda").manual_seed(5), np.random.default_rng(5)
    cache, table, live = make_paged(nv, gen, rng, [300], [1], Hkv, D, P)
    k, v = (x.double() for x in live[0])
    for j, bad in ((0, -1), (7, cache.pages), (18, 2 ** 31 - 1)):
        table[0, j] = bad
        for x in (k, v):
            x[j * P:(j + 1) * P] = 0
    plan = nv.AttnPlan(1, 1, H, Hkv, page_size=P, block_table=table)
    q = rows(gen, 1, H, D, "plain")
    out, lse = torch.empty_like(q), torch.empty(1, H, device="cuda")
    nv.nvfp4_attn_plan(plan, i32([1]), i32([300]))
    nv.device_status()
    nv.nvfp4_attn_paged(q, cache, plan, out, ws, lse=lse)
    torch.cuda.synchronize()
    check(out, lse, *reference(q.double(), k, v, 300, D ** -0.5), "bad pages")


def test_paged_far_pages(nv, ws):
    """Pages beyond 2^31 elements from the cache's start."""
    H, Hkv, D, P = 10, 2, 128, 64
    pages = 2 ** 31 // (Hkv * P * D) + 40
    cache = nv.KVCache.empty(pages, Hkv, P, D)
    gen = torch.Generator("cuda").manual_seed(6)
    n = 10
    table = torch.arange(pages - n, pages, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    for c in (cache.k, cache.v):
        c[pages - n:] = torch.randn(n, Hkv, P, D, device="cuda", generator=gen).to(torch.bfloat16)
    L = n * P - 5
    plan = nv.AttnPlan(1, 3, H, Hkv, page_size=P, block_table=table)
    q, kn, vn = (rows(gen, 3, h, D, "plain") for h in (H, Hkv, Hkv))
    nv.nvfp4_attn_plan(plan, i32([3]), i32([L - 3]))
    nv.nvfp4_kv_append(kn, vn, plan, cache)
    out, lse = torch.empty_like(q), torch.empty(3, H, device="cuda")
    nv.nvfp4_attn_paged(q, cache, plan, out, ws, lse=lse)
    k, v = (c[table[0].long()].transpose(1, 2).reshape(-1, Hkv, D)[:L].double() for c in (cache.k, cache.v))
    assert torch.equal(k[L - 3:], kn.double()) and torch.equal(v[L - 3:], vn.double())
    check(out, lse, *reference(q.double(), k, v, L - 3, D ** -0.5), "far pages")


# ------------------------------------------------------- together, streams
def test_prefill_in_chunks_equals_one_prompt(nv, ws):
    """A prompt in uneven chunks over the cache, another request decoding
    beside it, against binary64 over the whole prompt."""
    H, Hkv, D, P, L = 10, 2, 128, 32, 431
    gen = torch.Generator("cuda").manual_seed(8)
    q, k, v = (rows(gen, L, h, D, "plain", 1.5) for h in (H, Hkv, Hkv))
    cache = nv.KVCache.empty(40, Hkv, P, D)
    free = torch.randperm(40, device="cuda", generator=gen).to(torch.int32)
    table = torch.full((2, 16), -1, dtype=torch.int32, device="cuda")
    cursor = i32([0])
    ref = reference(q.double(), k.double(), v.double(), 0, D ** -0.5)
    at = 0
    for n in (1, 130, 200, 3, 97):
        other = (rows(gen, 1, h, D, "plain") for h in (H, Hkv, Hkv))
        qs, ks, vs = (torch.cat([x[at:at + n], o]) for x, o in zip((q, k, v), other))
        plan = nv.AttnPlan(2, n + 1, H, Hkv, page_size=P, block_table=table)
        done = 0 if at == 0 else at
        nv.nvfp4_attn_plan(plan, i32([n, 1]), i32([done, {0: 0, 1: 1, 131: 2, 331: 3, 334: 4}[at]]), free, cursor)
        cursor = plan.cursor
        nv.nvfp4_kv_append(ks, vs, plan, cache)
        out, lse = torch.empty_like(qs), torch.empty(n + 1, H, device="cuda")
        nv.nvfp4_attn_paged(qs, cache, plan, out, ws, lse=lse)
        check(out[:n], lse[:n], *(x[at:at + n] for x in ref), f"chunk at {at}")
        at += n
    assert nv.device_status() == 0 and at == L


def test_graph_replay_with_new_lengths(nv):
    """One captured step replayed with other lengths, on a side stream;
    bit-identical to the eager calls, twice."""
    H, Hkv, D, P, R, T = 10, 2, 128, 16, 5, 64
    gen = torch.Generator("cuda").manual_seed(4)
    cache0 = torch.randn(2, 400, Hkv, P, D, device="cuda", generator=gen).to(torch.bfloat16)
    cache = nv.KVCache(cache0[0].clone(), cache0[1].clone())
    q, k, v = (rows(gen, T, h, D, "plain") for h in (H, Hkv, Hkv))
    table = torch.randperm(400, device="cuda", generator=gen).to(torch.int32).reshape(R, 80)
    plan = nv.AttnPlan(R, T, H, Hkv, page_size=P, block_table=table)
    ws = nv.workspace(nv.attn_workspace_bytes())
    ql, cl = i32([1] * R), i32([50] * R)
    out, lse = torch.zeros_like(q), torch.zeros(T, H, device="cuda")

    def step():
        nv.nvfp4_attn_plan(plan, ql, cl)
        nv.nvfp4_kv_append(k, v, plan, cache)
        nv.nvfp4_attn_paged(q, cache, plan, out, ws, lse=lse)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            step()
    for lens in (([1, 1, 1, 1, 1], [1000, 3, 0, 200, 1279]), ([40, 0, 2, 1, 21], [1, 700, 5, 1200, 90])):
        got = []
        for how in ("graph", "eager", "graph"):
            ql.copy_(i32(lens[0]))
            cl.copy_(i32(lens[1]))
            out.zero_()
            lse.zero_()
            cache.k.copy_(cache0[0])
            cache.v.copy_(cache0[1])
            torch.cuda.synchronize()
            with torch.cuda.stream(stream):
                g.replay() if how == "graph" else step()
            stream.synchronize()
            got.append((out.clone(), lse.clone(), cache.k.clone()))
        for other in got[1:]:
            assert all(torch.equal(a, b) for a, b in zip(got[0], other))
        assert out[:sum(lens[0])].abs().sum() > 0
    assert nv.device_status() == 0
