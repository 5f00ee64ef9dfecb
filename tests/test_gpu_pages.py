"""GPU tests of the page operators: forked requests, the free list, pages moved
together, and the copies, against plain Python over lists."""
import numpy as np
import pytest
import torch

from _kv4 import random_cache4
from test_gpu_attn import i32

pytestmark = pytest.mark.gpu

REPORTED = 100 + 34


@pytest.fixture(scope="module")
def nv():
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_device_gb300 as m
    return m


def table_of(ctx, page, cols, pages, rng, ld=None):
    """A table whose requests hold scattered pages; the ids that are free."""
    ids = rng.permutation(pages).astype(np.int32)
    table, at = np.full((len(ctx), ld or cols), -7, np.int32), 0
    for r, c in enumerate(ctx):
        n = -(-c // page)
        table[r, :n] = ids[at:at + n]
        at += n
    return table, ids[at:]


def on_gpu(nv, table, ctx, page, pages, cols):
    return nv.PageTable(torch.from_numpy(table.copy()).cuda()[:, :cols], i32(list(ctx)), page, pages)


# -------------------------------------------------------------------- fork
def fork_reference(table, ctx, page, cols, src, dst, free, cursor, pages):
    table, ctx, copies, bad = table.copy(), list(ctx), [], False
    R = len(ctx)
    for i, (a, b) in enumerate(zip(src, dst)):
        if not (0 <= a < R and 0 <= b < R) or b in src or b in dst[:i] or not 0 <= ctx[a] <= page * cols:
            copies.append((-1, -1))
            bad = True
            continue
        full, rest = divmod(ctx[a], page)
        new = np.full(cols, -1, np.int32)
        new[:full] = table[a, :full]
        pair = (-1, -1)
        if rest:
            if cursor < len(free) and 0 <= free[cursor] < pages:
                pair = (int(table[a, full]), int(free[cursor]))
                new[full] = free[cursor]
            else:
                bad = True
            cursor += 1
        table[b, :cols], ctx[b] = new, ctx[a]
        copies.append(pair)
    return table, ctx, copies, cursor, bad


def check_fork(nv, table, ctx, page, cols, pages, src, dst, free, cursor=0, in_place=False, captured=False):
    t = on_gpu(nv, table, ctx, page, pages, cols)
    n = len(src)
    cs, cd = i32([5] * n), i32([5] * n)
    cur = i32([cursor])
    out = cur if in_place else i32([99])
    call = lambda: nv.nvfp4_pages_fork(t, i32_src, i32_dst, free_dev, cur, out, cs, cd)
    i32_src, i32_dst, free_dev = i32(list(src)), i32(list(dst)), i32(list(map(int, free)))
    nv.device_status()
    if captured:
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            call()
        graph.replay()
    else:
        call()
    torch.cuda.synchronize()
    new, lens, copies, at, bad = fork_reference(table, ctx, page, cols, list(src), list(dst), free, cursor, pages)
    assert out.item() == at and t.ctx_len.tolist() == lens
    whole = t.block_table._base if t.block_table._base is not None else t.block_table
    assert np.array_equal(whole.cpu().numpy(), new)
    assert list(zip(cs.tolist(), cd.tolist())) == copies
    assert nv.device_status() == (REPORTED if bad else 0)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("parents,children,page,ctx_hi,ld", [(1, 1, 16, 40, 0), (1, 8, 16, 777, 3), (64, 8, 16, 3000, 0),
                                                             (5, 3, 128, 1000, 1), (1000, 3, 64, 300, 0)])
def test_fork(nv, parents, children, page, ctx_hi, ld, in_place, captured):
    rng = np.random.default_rng(parents + page)
    n = parents * children
    ctx = np.zeros(parents + n, np.int64)
    order = rng.permutation(parents + n)
    ctx[order[:parents]] = rng.integers(0, ctx_hi + 1, parents)
    ctx[order[0]] = page * 2                                  # a last page that is full: nothing to copy
    ctx[order[parents:]] = rng.integers(0, 50, n)             # what the children were before
    cols = -(-max(ctx_hi, 2 * page) // page) + 1
    pages = int(sum(-(-c // page) for c in ctx)) + n + 4
    table, free = table_of(ctx, page, cols, pages, rng, cols + ld)
    check_fork(nv, table, ctx, page, cols, pages, np.repeat(order[:parents], children).tolist(), order[parents:].tolist(),
               free, 2, in_place, captured)


def test_fork_of_a_long_request(nv):
    """Rows of more than one segment."""
    rng = np.random.default_rng(1)
    ctx = [16 * 2500 + 5, 0, 0, 0]
    table, free = table_of(ctx, 16, 3000, 2600, rng)
    check_fork(nv, table, ctx, 16, 3000, 2600, [0, 0, 0], [3, 1, 2], free)


def test_fork_leaves_out_what_it_cannot_do(nv):
    rng = np.random.default_rng(2)
    ctx = [20, 5, 33, 16 * 4, 16 * 4 + 1, 0, 0, 0, -3]
    table, free = table_of([max(0, min(c, 64)) for c in ctx], 16, 4, 40, rng)
    for src, dst in (([0, 0], [5, 5]),                        # one destination twice: the first pair has it
                     ([0, 5], [5, 6]),                        # a destination that is a source
                     ([1], [1]),                              # itself
                     ([9, 0, -1], [5, 9, 6]), ([0], [-1]),    # requests that do not exist
                     ([4, 3], [5, 6]),                        # a length that the row cannot hold; a full one
                     ([8, 2], [5, 6]),                        # a negative length
                     ([0, 1, 2], [5, 6, 7])):
        check_fork(nv, table, ctx, 16, 4, 40, src, dst, free)
    for count in (0, 1, 2):                                   # pages run out
        check_fork(nv, table, ctx, 16, 4, 40, [0, 1, 2], [5, 6, 7], free[:count])
    check_fork(nv, table, ctx, 16, 4, 40, [0, 1, 2], [5, 6, 7], [int(free[0]), 40, -5])    # ids that are no pages
    check_fork(nv, table, ctx, 16, 4, 40, [], [], free, 3)
    with pytest.raises(ValueError):
        nv.nvfp4_pages_fork(on_gpu(nv, table, ctx, 16, 40, 4), i32([0]), i32([5, 6]), i32([1]), None, None, i32([0]), i32([0]))


def test_fork_of_everything(nv):
    """8192 requests, half of them the children of the other half."""
    rng = np.random.default_rng(3)
    ctx = [int(c) for c in rng.integers(0, 40, 4096)] + [0] * 4096
    pages = sum(-(-c // 16) for c in ctx) + 4096
    table, free = table_of(ctx, 16, 3, pages, rng)
    check_fork(nv, table, ctx, 16, 3, pages, list(range(4096)), (4096 + rng.permutation(4096)).tolist(), free)


# -------------------------------------------------------------------- free
def check_free(nv, table, ctx, page, cols, pages, mode, bad=False, captured=False):
    """mode: 'list', 'compact' or 'in place'."""
    t = on_gpu(nv, table, ctx, page, pages, cols)
    free, count = i32([-9] * pages), i32([-9])
    args = []
    if mode != "list":
        out = t.block_table if mode == "in place" else torch.full_like(t.block_table, -9)
        args = [out, i32([-9] * (pages // 2)), i32([-9] * (pages // 2))]
    nv.device_status()
    if captured:
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            nv.nvfp4_pages_free(t, free, count, *args)
        graph.replay()
    else:
        nv.nvfp4_pages_free(t, free, count, *args)
    torch.cuda.synchronize()
    assert nv.device_status() == (REPORTED if bad else 0)
    rows = [table[r, :min(cols, -(-max(c, 0) // page))].tolist() for r, c in enumerate(ctx)]
    used = {p for row in rows for p in row if 0 <= p < pages}
    n = pages - len(used)
    assert count.item() == n
    pad = lambda x, k: list(x) + [-1] * (k - len(x))
    if mode == "list":
        assert free.tolist() == pad([p for p in range(pages) if p not in used], pages)
    else:
        moves = list(zip(sorted(p for p in used if p >= len(used)), [p for p in range(len(used)) if p not in used]))
        to = dict(moves)
        assert free.tolist() == pad(range(len(used), pages), pages)
        assert args[1].tolist() == pad([a for a, _ in moves], pages // 2)
        assert args[2].tolist() == pad([b for _, b in moves], pages // 2)
        assert args[0].tolist() == [pad([to.get(p, p) for p in row], cols) for row in rows]
    if mode != "in place":
        assert np.array_equal(t.block_table.cpu().numpy(), table[:, :cols])
    assert t.ctx_len.tolist() == list(ctx)


@pytest.mark.parametrize("mode", ["list", "compact", "in place"])
@pytest.mark.parametrize("R,page,ctx_hi,spare,shared,ld", [
    (1, 16, 0, 1, 0, 0), (1, 16, 1, 0, 0, 0), (3, 128, 500, 5, 1, 2), (64, 16, 4096, 70, 20, 0), (64, 32, 900, 1000, 5, 1),
    (8192, 16, 60, 3000, 500, 0), (5, 16, 16 * 2500, 77, 2, 0)])
def test_free(nv, R, page, ctx_hi, spare, shared, ld, mode):
    rng = np.random.default_rng(R + page)
    ctx = [int(c) for c in rng.integers(0, ctx_hi + 1, R)]
    ctx[0] = ctx_hi
    cols = -(-ctx_hi // page) + 1
    pages = sum(-(-c // page) for c in ctx) + spare
    table, _ = table_of(ctx, page, cols, pages, rng, cols + ld)
    for _ in range(shared):                                   # some requests share their first pages
        a, b = rng.integers(0, R, 2)
        n = min(-(-ctx[a] // page), -(-ctx[b] // page)) // 2
        table[b, :n] = table[a, :n]
    for r in rng.integers(0, R, R // 4):                      # some have ended
        ctx[r] = 0
    check_free(nv, table, ctx, page, cols, pages, mode, captured=R == 64)


@pytest.mark.parametrize("mode", ["list", "compact"])
@pytest.mark.parametrize("pages", [1, 2, 31, 32, 33, 255, 256, 257, 2 ** 20])
def test_free_at_the_sizes_of_its_words(nv, pages, mode):
    rng = np.random.default_rng(pages)
    for n in {0, 1, pages // 2, pages - 1, pages} if pages < 1000 else {pages // 3}:
        cols = 4096 if pages > 1000 else 64
        held = rng.permutation(pages)[:n].astype(np.int32)
        R = max(1, -(-n // cols))
        table = np.full((R, cols), -7, np.int32)
        table.flat[:n] = held
        check_free(nv, table, [16 * min(cols, max(0, n - r * cols)) for r in range(R)], 16, cols, pages, mode)


@pytest.mark.parametrize("mode", ["list", "compact", "in place"])
def test_entries_that_are_no_pages_and_lengths_too_long(nv, mode):
    table = np.array([[3, -1, 9], [40, 2, 2 ** 31 - 1], [-2 ** 31, 5, 6]], np.int32)
    check_free(nv, table, [48, 48, 48], 16, 3, 40, mode, bad=True)
    table = np.array([[3, 4, 9], [7, 2, 11]], np.int32)
    check_free(nv, table, [49, 16], 16, 3, 12, mode, bad=True)
    check_free(nv, table, [-1, 16], 16, 3, 12, mode, bad=True)


# -------------------------------------------------------------------- copy
def cache_of(nv, kind, pages, heads, page, dim, gen, gap):
    if kind == "bf16":
        make = lambda: torch.randn(pages, gap, heads, page, dim, device="cuda", generator=gen).bfloat16()[:, 0]
        return nv.KVCache(make(), make())
    c = random_cache4(nv, gen, pages, heads, page, dim)
    wide = lambda t: t.new_zeros((pages, gap, *t.shape[1:]))[:, 0].copy_(t)
    return nv.KVCache4(wide(c.k), wide(c.v), wide(c.k_sf), wide(c.v_sf), c.k_g, c.v_g)


def planes(c):
    return [t for t in (c.k, c.v, getattr(c, "k_sf", None), getattr(c, "v_sf", None)) if t is not None]


@pytest.mark.parametrize("kinds,heads,page,dim,gap,n", [
    (["bf16"], 1, 16, 16, 1, 1), (["bf16", "4", "bf16"], 8, 16, 128, 1, 9), (["4"], 3, 32, 96, 2, 300),
    (["bf16"] * 40, 2, 16, 64, 1, 20), (["bf16"], 5, 128, 80, 3, 17), (["4"] * 17, 1, 16, 16, 1, 6)])
def test_copy(nv, kinds, heads, page, dim, gap, n):
    pages = 2 * n + 5
    gen = torch.Generator("cuda").manual_seed(n)
    caches = [cache_of(nv, k, pages, heads, page, dim, gen, gap) for k in kinds]
    rng = np.random.default_rng(n)
    ids = rng.permutation(pages)
    src, dst = rng.integers(0, n, n), ids[ids >= n][:n]       # sources again and again, destinations once
    src, dst = src.astype(np.int32), dst.astype(np.int32)
    src[rng.random(n) < 0.3] = -1
    dst[src < 0] = -1
    want = [[t.clone() for t in planes(c)] for c in caches]
    for c in want:
        for t in c:
            for a, b in zip(src, dst):
                if a >= 0:
                    t[b] = t[a].clone()
    nv.nvfp4_pages_copy(caches, torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda())
    torch.cuda.synchronize()
    for c, w in zip(caches, want):
        for t, x in zip(planes(c), w):
            assert torch.equal(t, x)
            whole = t._base if t._base is not None else t     # what lies between the pages is as it was
            assert gap == 1 or "4" not in kinds or not whole[:, 1:].any()
    assert nv.device_status() == 0


def test_copy_of_pages_that_are_none(nv):
    c = nv.KVCache(*(torch.randn(4, 1, 16, 64, device="cuda").bfloat16() for _ in range(2)))
    for src, dst in (([4], [0]), ([0], [4]), ([-1], [2]), ([2], [-1]), ([-2], [1]), ([2 ** 31 - 1], [1])):
        want = c.k.clone()
        nv.nvfp4_pages_copy(c, i32(src + [0]), i32(dst + [3]))
        want[3] = want[0]
        assert torch.equal(c.k, want) and nv.device_status() == REPORTED
    nv.nvfp4_pages_copy(c, i32([]), i32([]))
    nv.nvfp4_pages_copy([c], i32([-1, -1]), i32([-1, -1]))
    assert torch.equal(c.k, want) and nv.device_status() == 0
    with pytest.raises(ValueError):
        nv.nvfp4_pages_copy(c, i32([0]), i32([1, 2]))
    with pytest.raises(ValueError):
        nv.nvfp4_pages_copy([c, nv.KVCache.empty(5, 1, 16, 64)], i32([0]), i32([1]))


def test_a_server_that_forks_ends_and_moves(nv):
    """The calls as a server makes them: steps, forks, requests that end, the
    free list made anew, the cache moved together.  Each request's rows are
    followed by their contents."""
    rng = np.random.default_rng(11)
    R, page, pages, cols, Hkv, D = 12, 16, 150, 12, 2, 64
    cache = nv.KVCache(*(torch.zeros(pages, Hkv, page, D, device="cuda").bfloat16() for _ in range(2)))
    table = torch.full((R, cols), -1, dtype=torch.int32, device="cuda")
    ctx = i32([0] * R)
    held = nv.PageTable(table, ctx, page, pages)
    free, count = i32(list(range(pages))), i32([pages])
    cursor = i32([0])
    rows = [[] for _ in range(R)]                             # each request's tokens, as numbers
    token = 0
    moves = [i32([0] * (pages // 2)) for _ in range(2)]
    for step in range(30):
        q = [int(rng.integers(1, 20)) if len(x) + 20 < page * cols and rng.random() < 0.8 else 0 for x in rows]
        T = sum(q) + 1
        plan = nv.AttnPlan(R, T, Hkv, Hkv, page_size=page, block_table=table)
        nv.nvfp4_attn_plan(plan, i32(q), ctx, free, cursor)
        cursor = plan.cursor
        x = (torch.arange(token, token + T, device="cuda") % 251).bfloat16()[:, None, None].expand(T, Hkv, D).contiguous()
        nv.nvfp4_kv_append(x, x, plan, cache)
        for r in range(R):
            rows[r] += [(token + i) % 251 for i in range(q[r])]
            token += q[r]
        token += 1
        ctx.add_(i32(q))
        ended = [r for r in range(R) if rng.random() < 0.25]
        for r in ended:
            rows[r] = []
            ctx[r] = 0
        live = [r for r in range(R) if rows[r]]
        if ended and live:                                    # children in the rows of those that ended
            n = int(rng.integers(1, len(ended) + 1))
            src = [live[int(rng.integers(len(live)))] for _ in range(n)]
            cs, cd = i32([0] * n), i32([0] * n)
            nv.nvfp4_pages_fork(held, i32(src), i32(ended[:n]), free, cursor, cursor, cs, cd)
            nv.nvfp4_pages_copy([cache], cs, cd)
            for a, b in zip(src, ended):
                rows[b] = list(rows[a])
        if step % 3 == 2:
            nv.nvfp4_pages_free(held, free, count, table, *moves)
            nv.nvfp4_pages_copy(cache, *moves)
        else:
            nv.nvfp4_pages_free(held, free, count)
        cursor = i32([0])
        torch.cuda.synchronize()
        assert nv.device_status() == 0
        ids, lens = table.tolist(), ctx.tolist()
        assert lens == [len(x) for x in rows]
        for r in range(R):
            got = [cache.k[ids[r][p // page], 1, p % page, 3].item() for p in range(0, lens[r], 7)]
            assert got == rows[r][::7], (step, r)
        used = {p for r in range(R) for p in ids[r][:-(-lens[r] // page)]}
        assert count.item() == pages - len(used)
        assert step % 3 != 2 or max(used, default=-1) < len(used)
