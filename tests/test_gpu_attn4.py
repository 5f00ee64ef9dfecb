"""GPU tests of the attention over the 4-bit cache against binary64 over the
values that its codes and scales stand for."""
import numpy as np
import pytest
import torch

from _attn import LSE_ABS, LSE_REL, OUT_P, reference
from _kv4 import decode, random_cache4
from test_gpu_attn import i32, rows
from test_gpu_heads import pages_apart, plan_of

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


# |out - ref| <= 2^-8 |ref| (the output's rounding to bf16, half a step)
#             + p sum_j p_j |v_j| + 2^-31 sum_j |v_j|
# with p = 2^-11 + 2^-11: a probability's rounding to half precision (half a step),
# and the binary32 scores, whose errors stay below 2^-15 as in _attn.py (code times
# scale is exact; q's bits too, down to 2^-28 of its row's largest).  Probabilities
# are carried 2^6 above the largest, so one below 2^-20 of it lies among half
# precision's subnormals, 2^-24 apart: off by 2^-25 / 2^6 = 2^-31 of the largest at
# most, and the sum that they are divided by is no smaller than that.  Through the
# bf16 pages p is OUT_P, that kernel's.
P_HALF = 2.0 ** -11 + 2.0 ** -11


def check(out, lse, ref, mag, ref_lse, p, vals, what=""):
    err = (out.double() - ref).abs()
    tiny = 2.0 ** -31 * vals.abs().sum(0).max() if len(vals) else 0.0
    bad = ~(err <= 2.0 ** -8 * ref.abs() + p * mag + tiny + 1e-30)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist(), out[tuple(bad.nonzero()[0])].item(),
                           ref[tuple(bad.nonzero()[0])].item())
    if lse is not None:
        same = (lse.double() == ref_lse) | ((lse.double() - ref_lse).abs() <= LSE_ABS + LSE_REL * ref_lse.abs())
        assert same.all(), (what, (~same).nonzero()[0].tolist())


def values(cache):
    return decode(cache.k, cache.k_sf) * cache.k_g.double(), decode(cache.v, cache.v_sf) * cache.v_g.double()


def run(nv, ws, ctx, q_len, H, Hkv, D, page, window=0, layout="plain", pad=0, scale=None, seed=0, expanded=False,
        std=1.0, apart=False, k_g=2.0 ** -6, check_it=True, dirty=True):
    gen = torch.Generator("cuda").manual_seed(seed + sum(ctx) + D)
    pages = sum(-(-(c + n) // page) for c, n in zip(ctx, q_len)) + 3
    cache = random_cache4(nv, gen, pages, Hkv, page, D, k_g)
    plan = plan_of(nv, q_len, ctx, H, Hkv, page, pages, window, pad)
    if dirty:                                                 # rows that nobody sees: NaN scales
        seen = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
        for r, (c, n) in enumerate(zip(ctx, q_len)):
            at = torch.arange(max(0, c - window + 1) if window else 0, c + n if n else 0, device="cuda")
            seen[plan.block_table[r].long()[at // page], at % page] = True
        for sf in (cache.k_sf, cache.v_sf):
            sf.copy_(torch.where(seen[:, None, :, None], sf, 0x7f))
    cache = pages_apart(nv, cache) if apart else cache
    T = plan.tokens
    q = rows(gen, T, H, D, layout, std)
    out, lse = rows(gen, T, H, D, layout), torch.full((T, H), 7.0, device="cuda")
    out.fill_(7.0)
    scratch = nv.KVCache(*(torch.full((pages, Hkv, page, D), float("nan"), device="cuda").bfloat16() for _ in range(2))) \
        if expanded else None
    nv.nvfp4_attn_paged4(q, cache, plan, out, ws, scale=scale, lse=lse, expanded=scratch)
    torch.cuda.synchronize()
    assert nv.device_status() == 0
    assert not ws[:8192].any()                                # the tickets are back at zero
    if not check_it:
        return out, lse
    k, v = values(cache)
    at = 0
    for r, (c, n) in enumerate(zip(ctx, q_len)):
        if n:
            pos = torch.arange(c + n, device="cuda")
            pg, row = plan.block_table[r].long()[pos // page], pos % page
            keys, vals = (x[pg, :, row].nan_to_num() for x in (k, v))     # (the rows that are NaN are not seen)
            ref = reference(q[at:at + n].double(), keys, vals, c, D ** -0.5 if scale is None else scale, window)
            check(out[at:at + n], lse[at:at + n], *ref, OUT_P if expanded else P_HALF, vals,
                  f"request {r}: {n} behind {c}")
        at += n
    assert (out[at:] == 7.0).all() and (lse[at:] == 7.0).all()
    return out, lse


@pytest.mark.parametrize("ctx", [[0], [1], [15], [16], [127], [128], [129], [5, 0, 300, 17], [4000, 1], [777] * 20])
@pytest.mark.parametrize("H,Hkv,D,page", [(40, 8, 128, 16), (4, 4, 64, 64)])
def test_single_tokens(nv, ws, ctx, H, Hkv, D, page):
    run(nv, ws, ctx, [1] * len(ctx), H, Hkv, D, page)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (7, 1), (28, 4), (9, 3), (16, 1), (33, 1), (128, 1), (20, 20)])
@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128])
def test_heads(nv, ws, H, Hkv, D):
    run(nv, ws, [70, 139, 0], [1, 1, 1], H, Hkv, D, 32, pad=2)


@pytest.mark.parametrize("expanded", [False, True])
@pytest.mark.parametrize("ctx,q_len", [([100, 0], [2, 3]), ([0], [17]), ([30, 200, 5], [4, 0, 7]), ([0, 64], [130, 300]),
                                       ([1000], [64]), ([333, 0, 10], [1, 90, 1]), ([0], [1])])
@pytest.mark.parametrize("H,Hkv,D,page", [(10, 2, 128, 16), (3, 3, 64, 128), (24, 2, 96, 64)])
def test_several_tokens(nv, ws, ctx, q_len, H, Hkv, D, page, expanded):
    few = sum(q_len) / len(q_len) * (H // Hkv) < 40           # (few rows do not go through the bf16 pages)
    if expanded and few:
        pytest.skip("the same call")
    run(nv, ws, ctx, q_len, H, Hkv, D, page, expanded=expanded)


@pytest.mark.parametrize("expanded", [False, True])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 128, 5000])
def test_windows(nv, ws, window, expanded):
    run(nv, ws, [700, 3, 131], [1, 1, 1] if not expanded else [200, 40, 131], 10, 2, 128, 16, window)
    run(nv, ws, [700, 3, 131], [9, 2, 40], 6, 2, 64, 32, window, expanded=False)
    if expanded:
        run(nv, ws, [700, 3, 131], [90, 60, 140], 10, 2, 128, 64, window, expanded=True)


@pytest.mark.parametrize("ctx,H,Hkv,D,page", [([20000], 8, 1, 128, 64), ([9001, 3], 40, 8, 128, 16), ([30000, 17, 5000], 12, 4, 64, 32),
                                              ([12345], 20, 1, 128, 128), ([10000], 64, 1, 96, 16)])
def test_long_contexts_shared_by_ctas(nv, ws, ctx, H, Hkv, D, page):
    run(nv, ws, ctx, [1] * len(ctx), H, Hkv, D, page)
    run(nv, ws, ctx, [3] * len(ctx), H, Hkv, D, page, window=4000, seed=1)


@pytest.mark.parametrize("H,Hkv,D,page,tokens", [(40, 8, 128, 16, 1), (12, 12, 64, 32, 1), (16, 8, 96, 64, 3), (24, 8, 128, 128, 4),
                                                 (16, 4, 32, 16, 2), (128, 8, 128, 16, 1)])
@pytest.mark.parametrize("kind", ["mixed", "tiny", "empty", "window"])
def test_more_items_than_ctas(nv, ws, H, Hkv, D, page, tokens, kind):
    """Several items to a CTA, cut anywhere between its warps."""
    rng = np.random.default_rng(H + D)
    n = 96 if kind == "tiny" else 72
    ctx = {"mixed": rng.integers(0, 2500, n), "tiny": rng.integers(0, 40, n), "empty": rng.integers(0, 900, n),
           "window": rng.integers(0, 3000, n)}[kind].tolist()
    q = [tokens] * n
    if kind == "empty":                                       # requests without new tokens in between
        q = [0 if rng.random() < 0.2 else int(rng.integers(1, tokens + 1)) for _ in ctx]
    run(nv, ws, ctx, q, H, Hkv, D, page, window=300 if kind == "window" else 0, pad=1)


def test_one_request_of_many_tokens_among_single_ones(nv, ws):
    """Rows of one request that need several passes, where the step's average is a few."""
    ctx = [int(c) for c in np.random.default_rng(3).integers(0, 700, 64)]
    run(nv, ws, ctx, [1] * 20 + [70] + [1] * 43, 10, 2, 128, 16)
    run(nv, ws, ctx, [1] * 63 + [200], 4, 4, 64, 32)


def _through_the_pages(nv, ws, ctx, q_len, H, Hkv, D):
    """Whether a step went through its bf16 pages: bit for bit what the call without them gives, or not."""
    a, b = (run(nv, ws, ctx, q_len, H, Hkv, D, 16, expanded=x) for x in (False, True))
    return not (torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]))


@pytest.mark.parametrize("H,Hkv,D", [(10, 2, 128), (8, 1, 64)])
def test_the_lengths_decide_about_the_bf16_pages(nv, ws, H, Hkv, D):
    ctx = [int(c) for c in np.random.default_rng(4).integers(100, 700, 30)]
    assert not _through_the_pages(nv, ws, ctx, [2] * 29 + [3], H, Hkv, D)          # a few rows each
    assert not _through_the_pages(nv, ws, ctx, [1] * 29 + [9], H, Hkv, D)          # one of two passes among many of one
    assert _through_the_pages(nv, ws, [2000] + ctx[1:], [90] + [1] * 29, H, Hkv, D)    # one of many rows and keys
    assert not _through_the_pages(nv, ws, ctx, [1] * 29 + [0], H, Hkv, D)          # (no more tokens than requests)


@pytest.mark.parametrize("H,Hkv,n", [(40, 8, 200), (28, 4, 40), (32, 32, 400)])
def test_one_request_of_many_passes_decides(nv, ws, H, Hkv, n):
    """Few passes on average, but many for the CTAs that have the one request."""
    ctx = [int(c) for c in np.random.default_rng(6).integers(100, 1000, 64)]
    assert _through_the_pages(nv, ws, ctx, [1] * 20 + [n] + [1] * 43, H, Hkv, 128)
    assert not _through_the_pages(nv, ws, ctx, [1] * 20 + [2] + [1] * 43, H, Hkv, 128)


@pytest.mark.parametrize("H,Hkv,D,page", [(10, 2, 128, 16), (8, 8, 64, 64), (9, 3, 96, 32), (4, 1, 128, 128), (6, 2, 16, 16)])
@pytest.mark.parametrize("ctx,q_len,std", [([0], [70], 1.0), ([3, 1, 0], [60, 50, 90], 4.0), ([3000], [100], 1.0), ([900, 20], [130, 300], 0.1)])
def test_probabilities_through_the_pages(nv, ws, H, Hkv, D, page, ctx, q_len, std):
    """They are rounded to half precision there too: the tolerance of the codes."""
    gen = torch.Generator("cuda").manual_seed(D + sum(ctx))
    pages = sum(-(-(c + n) // page) for c, n in zip(ctx, q_len)) + 3
    cache = random_cache4(nv, gen, pages, Hkv, page, D)
    plan = plan_of(nv, q_len, ctx, H, Hkv, page, pages)
    q = rows(gen, plan.tokens, H, D, "plain", std)
    out, lse = torch.empty_like(q), torch.empty(plan.tokens, H, device="cuda")
    nv.nvfp4_attn_paged4(q, cache, plan, out, ws, lse=lse, expanded=nv.KVCache.empty(pages, Hkv, page, D))
    k, v = values(cache)
    at = 0
    for r, (c, n) in enumerate(zip(ctx, q_len)):
        pos = torch.arange(c + n, device="cuda")
        ids, row = plan.block_table[r].long()[pos // page], pos % page
        ref = reference(q[at:at + n].double(), k[ids, :, row], v[ids, :, row], c, D ** -0.5)
        check(out[at:at + n], lse[at:at + n], *ref, P_HALF, v[ids, :, row], f"request {r}")
        at += n
    assert nv.device_status() == 0


@pytest.mark.parametrize("L,std", [(300, 2e4), (2000, 2e4)])
def test_large_scores_through_the_pages(nv, ws, L, std):
    """Scores of 10^6 to 10^7: a row whose largest is alone gives that key's value (bounds as above)."""
    H, Hkv, D, T = 8, 4, 64, 64
    gen = torch.Generator("cuda").manual_seed(L)
    pages = -(-(L + T) // 16)
    cache = random_cache4(nv, gen, pages, Hkv, 16, D, 2.0 ** 2)
    plan = plan_of(nv, [T], [L], H, Hkv, 16, pages)
    q = (torch.randn(T, H, D, device="cuda", generator=gen) * std).bfloat16()
    out = torch.empty_like(q)
    nv.nvfp4_attn_paged4(q, cache, plan, out, ws, expanded=nv.KVCache.empty(pages, Hkv, 16, D))
    k, v = values(cache)
    at = torch.arange(L + T, device="cuda")
    keys, vals = (x[plan.block_table[0].long()[at // 16], :, at % 16] for x in (k, v))
    alone = 0
    for h in range(H):
        x = q[:, h].double() * D ** -0.5
        seen = at[None] <= L + torch.arange(T, device="cuda")[:, None]
        s = torch.where(seen, x @ keys[:, h // 2].T, -float("inf"))
        top = s.topk(2)
        gap = 2 * D * 2.0 ** -24 * (x.abs() @ keys[:, h // 2].abs().T).max(1).values + 200
        sure = top.values[:, 0] - top.values[:, 1] > gap
        alone += int(sure.sum())
        assert (top.values[sure, 0] > 1e5).all() and top.values.max() < 2 ** 24
        want = vals[top.indices[:, 0], h // 2]
        assert ((out[:, h].double() - want).abs() <= 2.0 ** -8 * want.abs())[sure].all()
    assert alone >= H * T // 2


@pytest.mark.parametrize("window", [0, 1, 60, 1000])
@pytest.mark.parametrize("H,Hkv,D,page", [(10, 2, 128, 16), (8, 8, 64, 64), (9, 3, 96, 32)])
def test_steps_whose_lengths_decide(nv, ws, H, Hkv, D, page, window):
    """With bf16 pages at hand and a few rows per request on average."""
    ctx = [int(c) for c in np.random.default_rng(D).integers(0, 900, 40)]
    for q in ([1] * 39 + [90], [0, 2] * 20, [3] * 39 + [1], [100, 0, 0, 1] + [1] * 36):
        q = [max(n, 1) for n in q] if window else q           # (run()'s rows that nobody sees need a token then)
        run(nv, ws, ctx, q, H, Hkv, D, page, window, pad=3, expanded=True, layout="padded")


def test_a_captured_step_whose_lengths_decide(nv, ws):
    """One graph: replays with many rows for a request and with few, bit for bit the plain
    calls; rows of padding are zeros whichever way was taken."""
    H, Hkv, D, page, R, T = 10, 2, 128, 16, 12, 84
    gen = torch.Generator("cuda").manual_seed(12)
    ctx = [int(c) for c in np.random.default_rng(9).integers(50, 400, R)]
    cache = random_cache4(nv, gen, 400, Hkv, page, D)
    table = plan_of(nv, [T] * R, ctx, H, Hkv, page, 400).block_table
    plan = nv.AttnPlan(R, T, H, Hkv, page_size=page, block_table=table)
    assert T > R and -(-T // R) * (H // Hkv) < 40
    q = torch.randn(T, H, D, device="cuda", generator=gen).bfloat16()
    lens, at, scratch = i32([1] * R), i32(ctx), nv.KVCache.empty(400, Hkv, page, D)
    out, lse = torch.empty_like(q), torch.empty(T, H, device="cuda")

    def step(o, l, e):
        nv.nvfp4_attn_plan(plan, lens, at)
        nv.nvfp4_attn_paged4(q, cache, plan, o, ws, lse=l, zero_padding=True, expanded=e)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    step(out, lse, scratch)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        step(out, lse, scratch)
    for n in ([70] + [1] * 11, [1] * 12, [1] * 11 + [73], [2] * 12, [0] * 12, [84] + [0] * 11):
        lens.copy_(i32(n))
        out.fill_(7.0), lse.fill_(7.0)
        graph.replay()
        plain, codes = ((torch.empty_like(out), torch.empty_like(lse)) for _ in range(2))
        step(*plain, scratch)
        step(*codes, None)
        assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])
        assert torch.equal(out, codes[0]) == (max(n) < 10)
        assert (out[sum(n):] == 0).all() and (lse[sum(n):] == -float("inf")).all()
    assert nv.device_status() == 0 and not ws[:8192].any()


def test_a_plan_without_pages_has_no_second_axis(nv):
    """Only the attention over a paged 4-bit cache reads it; the first axis is that of the step with pages."""
    lens = [300, 1, 40, 7, 0, 129]
    table = torch.arange(120, dtype=torch.int32, device="cuda").view(6, 20)
    plans = [nv.AttnPlan(6, sum(lens), 8, 2), nv.AttnPlan(6, sum(lens), 8, 2, page_size=16, block_table=table)]
    for p in plans:
        nv.nvfp4_attn_plan(p, i32(lens))
    assert nv.device_status() == 0
    plain, paged = (p.schedule.view(torch.int32) for p in plans)
    n, first4 = int(plain[2]), 16 + 256 * 9                   # QTiles; where the second axis' CTAs begin
    assert n == int(paged[2]) > 0
    assert torch.equal(plain[:3], paged[:3]) and torch.equal(plain[16:first4], paged[16:first4])
    at = first4 + 256 * 9
    assert torch.equal(plain[at:at + 8 * n], paged[at:at + 8 * n])
    assert not plain[3:16].any() and not plain[first4:at].any() and paged[3:6].all()


def test_a_share_of_very_long_items(nv, ws):
    run(nv, ws, [170000], [1], 8, 8, 64, 128)
    run(nv, ws, [120000, 90000], [1, 2], 8, 8, 32, 64)


@pytest.mark.parametrize("layout", ["heads_first", "padded"])
@pytest.mark.parametrize("D", [128, 80])
def test_layouts(nv, ws, layout, D):
    run(nv, ws, [33, 200, 1], [1, 1, 1], 10, 2, D, 16, layout=layout, pad=2, apart=True)
    run(nv, ws, [33, 200, 1], [5, 3, 1], 10, 2, D, 16, layout=layout, pad=2, apart=True)


@pytest.mark.parametrize("std,scale,k_g", [(1e-3, None, 2.0 ** -6), (8.0, None, 2.0 ** -6), (1.0, 0.0, 2.0 ** -6),
                                           (1.0, -0.3, 2.0 ** -6), (1.0, None, 0.0123), (1e30, 1e-30, 2.0 ** -6),
                                           (1e-30, 1e29, 2.0 ** -6), (0.0, None, 2.0 ** -6)])
def test_scores_of_all_sizes(nv, ws, std, scale, k_g):
    for expanded, n in ((False, 1), (False, 5), (True, 40)):
        run(nv, ws, [150, 61], [n, n], 10, 2, 64, 16, std=std, scale=scale, k_g=k_g, expanded=expanded)


@pytest.mark.parametrize("q_len", [1, 2, 5])
@pytest.mark.parametrize("L", [300, 9000])
def test_scores_beyond_binary32s_whole_numbers(nv, ws, L, q_len):
    """Scores of 10^9 and more, where neighbours in binary32 are 64 apart: a row whose
    largest score is alone gives that key's value.  The products' sums are off by less
    than D 2^-24 of sum |q_i k_i|; two scores that far apart and 200 more leave e^-200."""
    H, Hkv, D = 8, 4, 64
    gen = torch.Generator("cuda").manual_seed(L)
    pages = -(-(L + q_len) // 16)
    cache = random_cache4(nv, gen, pages, Hkv, 16, D, 2.0 ** 2)
    plan = plan_of(nv, [q_len], [L], H, Hkv, 16, pages)
    q = (torch.randn(q_len, H, D, device="cuda", generator=gen) * 2e7).bfloat16()
    out, lse = torch.empty_like(q), torch.empty(q_len, H, device="cuda")
    nv.nvfp4_attn_paged4(q, cache, plan, out, ws, lse=lse)
    k, v = values(cache)
    at = torch.arange(L + q_len, device="cuda")
    pg, row = plan.block_table[0].long()[at // 16], at % 16
    keys, vals = k[pg, :, row], v[pg, :, row]
    alone = 0
    for t in range(q_len):
        for h in range(H):
            n, x = L + t + 1, q[t, h].double()
            products = keys[:n, h // 2] * x * D ** -0.5
            s = products.sum(1)
            top = s.topk(2)
            gap = 2 * D * 2.0 ** -24 * products.abs().sum(1).max() + 200
            if top.values[0] - top.values[1] < gap:
                continue
            alone += 1
            want = vals[top.indices[0], h // 2]
            assert top.values[0] > 1e9
            assert ((out[t, h].double() - want).abs() <= 2.0 ** -8 * want.abs()).all(), (t, h)
            assert abs(lse[t, h].double() - top.values[0]) <= gap / 2 + 2.0 ** -22 * top.values[0]
    assert alone >= H * q_len // 2


def test_rising_scores(nv, ws):
    """Scores that rise (or fall) along the keys: the running maximum moves at every group."""
    L, D = 1500, 64
    gen = torch.Generator("cuda").manual_seed(4)
    plan = plan_of(nv, [1], [L - 1], 2, 2, 16, 100)
    for sign in (1, -1):
        cache = random_cache4(nv, gen, 100, 2, 16, D, 2.0 ** -2, 2.0)
        cache.k.fill_(0x22 if sign > 0 else 0xaa)              # +-1 times a scale that rises
        at = torch.arange(L, device="cuda")
        cache.k_sf[plan.block_table[0].long()[at // 16], :, at % 16] = (0x10 + at * 0x50 // L).to(torch.uint8)[:, None, None]
        q = torch.ones(1, 2, D, device="cuda").bfloat16()
        out, lse = torch.empty_like(q), torch.empty(1, 2, device="cuda")
        nv.nvfp4_attn_paged4(q, cache, plan, out, ws, lse=lse)
        k, v = values(cache)
        pg, row = plan.block_table[0].long()[at // 16], at % 16
        check(out, lse, *reference(q.double(), k[pg, :, row], v[pg, :, row], L - 1, D ** -0.5), P_HALF, v[pg, :, row])


def test_page_ids_outside_the_cache_are_pages_of_zeros(nv, ws):
    D, page, ctx = 128, 16, 100
    gen = torch.Generator("cuda").manual_seed(5)
    cache = random_cache4(nv, gen, 10, 2, page, D)
    plan = plan_of(nv, [1], [ctx], 10, 2, page, 10)
    plan.block_table[0, 2], plan.block_table[0, 4], plan.block_table[0, 5] = -1, 10, 2 ** 31 - 1
    q = rows(gen, 1, 10, D, "plain")
    out = torch.empty_like(q)
    nv.nvfp4_attn_paged4(q, cache, plan, out, ws)
    k, v = values(cache)
    at = torch.arange(ctx + 1, device="cuda")
    ids = plan.block_table[0].long()[at // page]
    ok = ((ids >= 0) & (ids < 10))[:, None, None]
    keys, vals = (torch.where(ok, x[ids.clamp(0, 9), :, at % page], 0.0) for x in (k, v))
    ref = reference(q.double(), keys, vals, ctx, D ** -0.5)
    check(out, None, *ref, P_HALF, vals)


@pytest.mark.parametrize("window", [0, 20])
def test_rows_past_the_tables_columns(nv, ws, window):
    """Keys that the block table has no column for are seen by no row; with a window some rows see none."""
    D, page = 64, 16
    gen = torch.Generator("cuda").manual_seed(6)
    cache = random_cache4(nv, gen, 8, 2, page, D)
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    plan = nv.AttnPlan(1, 3, 4, 2, page_size=page, block_table=table, window=window)
    k, v = values(cache)
    for ctx in (62, 80, 200):
        nv.nvfp4_attn_plan(plan, i32([3]), i32([ctx]))
        nv.device_status()
        q = rows(gen, 3, 4, D, "plain")
        out, lse = torch.full_like(q, 7.0), torch.full((3, 4), 7.0, device="cuda")
        nv.nvfp4_attn_paged4(q, cache, plan, out, ws, lse=lse)
        at = torch.arange(64, device="cuda")
        keys, vals = (x[at // page, :, at % page] for x in (k, v))
        ref = reference(q.double(), keys, vals, ctx, D ** -0.5, window)
        check(out, lse, *ref, P_HALF, vals)
        if window and ctx == 200:
            assert (out == 0).all() and (lse == -float("inf")).all()


def test_zero_padding(nv, ws):
    for q_len, expanded in (([1, 1], False), ([4, 3], False), ([60, 70], True)):
        gen = torch.Generator("cuda").manual_seed(7)
        cache = random_cache4(nv, gen, 40, 2, 16, 64)
        plan = plan_of(nv, q_len, [30, 50], 10, 2, 16, 40, pad=3)
        q = rows(gen, plan.tokens, 10, 64, "plain")
        scratch = nv.KVCache.empty(40, 2, 16, 64) if expanded else None
        got = []
        for zero in (False, True):
            out, lse = torch.full_like(q, 7.0), torch.full((plan.tokens, 10), 7.0, device="cuda")
            nv.nvfp4_attn_paged4(q, cache, plan, out, ws, lse=lse, zero_padding=zero, expanded=scratch)
            got.append((out, lse))
        n = sum(q_len)
        assert torch.equal(got[0][0][:n], got[1][0][:n]) and torch.equal(got[0][1][:n], got[1][1][:n])
        assert (got[0][0][n:] == 7).all() and (got[1][0][n:] == 0).all() and (got[1][1][n:] == -float("inf")).all()


def test_the_same_every_time_and_beside_the_bf16_attention(nv, ws):
    """Bit for bit, also with the workspace used by the other kernel in between."""
    ctx = [5000, 30, 801, 12000]
    first = run(nv, ws, ctx, [1] * 4, 40, 8, 128, 16)
    cache = nv.KVCache(*(torch.randn(1200, 8, 16, 128, device="cuda").bfloat16() for _ in range(2)))
    plan = plan_of(nv, [1] * 4, ctx, 40, 8, 16, 1200)
    q = torch.randn(4, 40, 128, device="cuda").bfloat16()
    for _ in range(3):
        nv.nvfp4_attn_paged(q, cache, plan, torch.empty_like(q), ws)
        again = run(nv, ws, ctx, [1] * 4, 40, 8, 128, 16, check_it=False)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_a_request_does_not_reach_its_neighbours(nv, ws):
    """NaN in one request's keys and values: the others bit for bit as without."""
    gen = torch.Generator("cuda").manual_seed(8)
    cache = random_cache4(nv, gen, 60, 2, 16, 128)
    ctx = [130, 300, 45]
    plan = plan_of(nv, [1, 1, 1], ctx, 10, 2, 16, 60)
    q = rows(gen, 3, 10, 128, "plain")
    a, b = torch.empty_like(q), torch.empty_like(q)
    nv.nvfp4_attn_paged4(q, cache, plan, a, ws)
    cache.k_sf[plan.block_table[1].long()[3]] = 0x7f
    cache.v_sf[plan.block_table[1].long()[7]] = 0x7f
    nv.nvfp4_attn_paged4(q, cache, plan, b, ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2]) and b[1].isnan().all()


def test_captured_steps_as_the_contexts_grow(nv, ws):
    """Append and attention of decoding steps in a graph, bit for bit the plain calls."""
    H, Hkv, D, page, R, steps = 10, 2, 128, 16, 3, 20
    outs = []
    for captured in (False, True):
        gen = torch.Generator("cuda").manual_seed(9)
        cache = random_cache4(nv, gen, 40, Hkv, page, D)
        plan = nv.AttnPlan(R, R, H, Hkv, page_size=page, block_table=10)
        ctx, one, free = i32([0, 14, 100]), i32([1] * R), i32(list(range(20, 40)))
        plan.block_table[:, :7] = torch.arange(21, device="cuda").view(3, 7)
        kv, q = (torch.zeros(R, h, D, device="cuda").bfloat16() for h in (2 * Hkv, H))
        out = torch.empty_like(q)

        def step():
            nv.nvfp4_attn_plan(plan, one, ctx, free, plan.cursor)
            nv.nvfp4_kv4_append(kv[:, :Hkv], kv[:, Hkv:], plan, cache)
            nv.nvfp4_attn_paged4(q, cache, plan, out, ws)
            ctx.add_(one)
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        if captured:
            with torch.cuda.graph(graph, stream=stream):
                step()
        got = []
        for _ in range(steps):
            for t in (kv, q):
                t.copy_(torch.randn(t.shape, device="cuda", generator=gen))
            graph.replay() if captured else step()
            got.append(out.clone())
        torch.cuda.synchronize()
        assert nv.device_status() == 0
        outs.append(torch.stack(got))
    assert torch.equal(*outs)


def test_refusals(nv, ws):
    q = torch.zeros(2, 4, 64, device="cuda").bfloat16()
    cache = random_cache4(nv, torch.Generator("cuda").manual_seed(1), 4, 2, 16, 64)
    plan = nv.AttnPlan(2, 2, 4, 2, page_size=16, block_table=2)
    for bad, error in ((dict(q=q.float()), ValueError), (dict(q=q.cpu()), ValueError), (dict(out=q[:1]), ValueError),
                       (dict(lse=torch.zeros(2, 3, device="cuda")), ValueError), (dict(ws=ws.cpu()), ValueError),
                       (dict(ws=ws[:100]), nv.NVFP4Error), (dict(scale=float("inf")), nv.NVFP4Error),
                       (dict(expanded=nv.KVCache.empty(5, 2, 16, 64)), nv.NVFP4Error),
                       (dict(expanded=nv.KVCache.empty(4, 2, 32, 64)), nv.NVFP4Error),
                       (dict(plan=nv.AttnPlan(2, 2, 4, 2, page_size=32, block_table=2)), nv.NVFP4Error),
                       (dict(plan=nv.AttnPlan(2, 2, 4, 1, page_size=16, block_table=2)), nv.NVFP4Error)):
        with pytest.raises(error):
            nv.nvfp4_attn_paged4(**{**dict(q=q, cache=cache, plan=plan, out=torch.empty_like(q), ws=ws), **bad})
