"""GPU tests of serving steps one after another: the free list's cursor
advanced in place, and steps of other sizes and lengths on one plan."""
import numpy as np
import pytest
import torch

import synthetic
from _attn import check
from _gpu import dev
from test_gpu_attn import i32, plan_reference, rows
from test_gpu_serving import D, H, HEADS, KV, weights, x_of  # noqa: F401  (weights: the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_device_gb300 as m
    return m


@pytest.mark.parametrize("R,q_hi,P", [(3, 40, 16), (700, 1, 16), (700, 9, 32), (3000, 3, 64)])
@pytest.mark.parametrize("captured", [False, True])
def test_cursor_advanced_in_place(nv, R, q_hi, P, captured):
    """plan.cursor is read and advanced by every step, while another stream's
    products keep the SMs busy (the plan's blocks start one by one)."""
    rng = np.random.default_rng(R + P)
    steps, cols = 6, -(-(6 * q_hi + 40) // P)
    ctx = np.zeros(R, np.int64)
    tokens = R * q_hi
    free = rng.permutation(R * cols).astype(np.int32)
    plan = nv.AttnPlan(R, tokens, 8, 2, page_size=P, block_table=cols)
    plan.cursor.fill_(3)
    q_dev, ctx_dev, free_dev = i32([0] * R), i32([0] * R), torch.from_numpy(free).cuda()
    table, cursor = np.full((R, cols), -1, np.int32), 3
    step = lambda: nv.nvfp4_attn_plan(plan, q_dev, ctx_dev, free_dev, plan.cursor)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    if captured:
        with torch.cuda.graph(graph, stream=stream):
            step()
    a = torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)
    b = torch.empty_like(a)
    torch.cuda.synchronize()
    for _ in range(steps):
        q = rng.integers(0 if q_hi > 1 else 1, q_hi + 1, R)
        q_dev.copy_(i32(q.tolist()))
        ctx_dev.copy_(i32(ctx.tolist()))
        torch.cuda.synchronize()
        for _ in range(8):
            torch.matmul(a, a, out=b)
        with torch.cuda.stream(stream):
            graph.replay() if captured else step()
        torch.cuda.synchronize()
        cu, pos, slot, table, cursor = plan_reference(ctx.tolist(), q.tolist(), P, table, free, cursor, tokens)
        assert plan.cursor.item() == cursor
        assert np.array_equal(plan.block_table.cpu().numpy(), table)
        assert np.array_equal(plan.slot.cpu().numpy(), slot) and np.array_equal(plan.pos.cpu().numpy(), pos)
        assert np.array_equal(plan.cu_q.cpu().numpy(), cu)
        ctx += q
        # (the first 3 pages of the list are skipped: the last requests to open one may find none)
        assert nv.device_status() == (100 + 31 if cursor > len(free) else 0)


@pytest.mark.parametrize("R", [1, 33, 8192])
def test_lengths_far_beyond_the_tables(nv, R):
    """Lengths that are not lengths (2^31 - 1 new tokens each) cost no more than
    the tables have room for: pages for the columns there are, as long as the
    list has some, and a report."""
    cols, huge = 3, 2 ** 31 - 1
    free = i32([7, 9])
    plan = nv.AttnPlan(R, 40, 8, 2, page_size=16, block_table=cols)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for ctx in (None, i32([16] * R), i32([huge] * R)):
        plan.block_table.fill_(-5)
        torch.cuda.synchronize()
        start.record()
        nv.nvfp4_attn_plan(plan, i32([huge] * R), ctx, free)
        end.record()
        torch.cuda.synchronize()
        assert nv.device_status() == 100 + 31 and start.elapsed_time(end) < 50
        have = 0 if ctx is None else min(cols, (int(ctx[0]) + 15) // 16)
        want = np.full((R, cols), -5, np.int64)
        want[:, have:] = -1
        want[0, have:min(cols, have + 2)] = [7, 9][:cols - have]
        assert np.array_equal(plan.block_table.cpu().numpy(), want)
        taken = 2 ** 27 if ctx is None or int(ctx[0]) == huge else (16 + huge + 15) // 16 - 1
        assert plan.cursor.item() == min(huge, R * taken)
        assert plan.cu_q.tolist() == [0] + [40] * R


@pytest.mark.parametrize("R,Hkv,ctx", [(64, 2, 2 ** 30 - 1), (300, 1, 2 ** 29 + 12345), (3, 80, 2 ** 30 - 1)])
def test_a_schedule_too_long_ends_with_a_whole_item(nv, R, Hkv, ctx):
    """Only the step's tables: no attention runs on them."""
    plan = nv.AttnPlan(R, R, 4 * Hkv, Hkv)
    nv.nvfp4_attn_plan(plan, i32([1] * R), i32([ctx] * R))
    assert nv.device_status() == 100 + 31
    units, per_cta, qtiles = plan.schedule.view(torch.int32)[:3].tolist()
    item = 2 + (ctx + 1 + 127) // 128                    # units of one kv head of one request
    assert R * Hkv * item > 2 ** 30
    assert units == 2 ** 30 // item * item and qtiles == R


def test_positions_beyond_the_schedule_are_reported(nv):
    P = 128
    table = torch.zeros((1, 2 ** 30 // P + 1), dtype=torch.int32, device="cuda")
    for heads, ctx, n, status in ((8, 2 ** 30 - 2, 2, 0), (8, 2 ** 30 - 2, 3, 131), (8, 2 ** 30, 1, 131), (0, 2 ** 30, 1, 0)):
        plan = nv.AttnPlan(1, n, 8, 2, page_size=P, block_table=table)
        plan._c.heads = heads                            # (0: tables without a schedule)
        nv.nvfp4_attn_plan(plan, i32([n]), i32([ctx]))
        assert plan.pos.tolist() == [ctx + t for t in range(n)]
        assert plan.slot.tolist() == [(ctx + t) % P for t in range(n)] and nv.device_status() == status


# ------------------------------------------------------------------- padding
@pytest.mark.parametrize("layout", ["plain", "heads_first", "padded"])
@pytest.mark.parametrize("lens,pad", [([5, 0, 130], 1), ([1], 700), ([0, 0], 3), ([300, 2], 0)])
def test_padding_rows_zeroed(nv, layout, lens, pad):
    """Only where asked for: out 0 and lse -inf past the last token, every
    other row (and what lies between the rows) bit for bit as without."""
    H, Hkv, D = 10, 2, 72
    gen = torch.Generator("cuda").manual_seed(pad)
    T = sum(lens) + pad
    q, k, v = (rows(gen, T, h, D, layout) for h in (H, Hkv, Hkv))
    plan, ws = nv.AttnPlan(len(lens), T, H, Hkv), nv.workspace(nv.attn_workspace_bytes())
    nv.nvfp4_attn_plan(plan, i32(lens))
    got = []
    for zero in (False, True):
        out, lse = rows(gen, T, H, D, layout), torch.full((T, H), 7.0, device="cuda")
        whole = out._base if out._base is not None else out
        whole.fill_(7.0)
        nv.nvfp4_attn_prompt(q, k, v, plan, out, ws, lse=lse, zero_padding=zero)
        got.append((whole.clone(), out.clone(), lse))
        if zero:
            out[sum(lens):] = 7.0
            assert torch.equal(whole, got[0][0])
    n = sum(lens)
    assert torch.equal(got[0][1][:n], got[1][1][:n]) and torch.equal(got[0][2][:n], got[1][2][:n])
    assert (got[0][1][n:] == 7.0).all() and (got[0][2][n:] == 7.0).all()
    assert (got[1][1][n:] == 0.0).all() and torch.isneginf(got[1][2][n:]).all()
    assert nv.device_status() == 0


@pytest.mark.parametrize("cached", [True, False])
def test_a_step_does_not_depend_on_the_steps_before(nv, weights, cached):
    """A step with few tokens after one with many (finite, then not) on the
    same buffers gives what it gives on buffers of its own."""
    T, R, page = 150, 3, 16
    cos, sin = (torch.from_numpy(t).cuda() for t in synthetic.rope_tables(T, D))
    norms = [dev(synthetic.norm_weight(80 + i, H)) for i in range(2)]
    small, xs = i32([3, 0, 20]), x_of(T, 601)

    def run(before):
        plan = nv.AttnPlan(R, T, HEADS, KV, **(dict(page_size=page, block_table=10) if cached else {}))
        cache = nv.KVCache(*(torch.zeros(64, KV, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
        layer = ServingLayer(plan, cache if cached else None, weights[0], *norms, cos, sin)
        free = torch.arange(30, dtype=torch.int32, device="cuda")
        out = torch.empty_like(xs)
        for x in before:
            nv.nvfp4_attn_plan(plan, i32([9, 140, 1]), None, free + 30 if cached else None)
            layer.forward(x, out)
        if cached:
            plan.block_table.fill_(-1)
        nv.nvfp4_attn_plan(plan, small, None, free if cached else None)
        layer.forward(xs, out)
        torch.cuda.synchronize()
        return out

    from nvfp4_block_scaled_device_gb300.serving import ServingLayer
    large, broken = 50.0 * x_of(T, 602), x_of(T, 603)
    broken[100] = float("inf")
    alone = run([])
    assert torch.isfinite(alone.float()).all()
    assert torch.equal(run([large]), alone) and torch.equal(run([broken]), alone)
    assert nv.device_status() == 0


@pytest.mark.parametrize("window", [0, 40])
def test_packed_prompts_of_a_step_with_pages(nv, window):
    """Bit for bit as without pages where the block table reaches, and no keys
    past it (reported by the plan)."""
    lens, heads, kv, d, page = [150, 0, 33, 96], 10, 2, 64, 16
    gen = torch.Generator("cuda").manual_seed(window)
    T = sum(lens)
    q, k, v = (rows(gen, T, h, d, "plain", 1.5) for h in (heads, kv, kv))
    got = []
    for cols in (None, 10, 6):                      # none, enough for 150 tokens, for 96
        plan = nv.AttnPlan(len(lens), T, heads, kv, window=window, **({"page_size": page, "block_table": cols} if cols else {}))
        out, lse = torch.empty_like(q), torch.empty(T, heads, device="cuda")
        nv.nvfp4_attn_plan(plan, i32(lens), None, torch.arange(99, dtype=torch.int32, device="cuda") if cols else None)
        assert nv.device_status() == (131 if cols == 6 else 0)
        nv.nvfp4_attn_prompt(q, k, v, plan, out, nv.workspace(nv.attn_workspace_bytes()), lse=lse)
        got.append((out, lse))
    for a, b, c in zip(*got):
        assert torch.equal(a, b) and torch.equal(c[:96], a[:96]) and torch.equal(c[150:], a[150:])
    # the rows past the table: keys up to its end, within their window
    p = torch.arange(150, device="cuda")[:, None]
    j = torch.arange(96, device="cuda")
    seen = (j <= p) & (j > p - window if window else j >= 0)
    for h in range(heads):
        s = (q[:150, h].double() @ k[:96, h // 5].double().T / d ** 0.5).masked_fill(~seen, -float("inf"))
        ref = torch.logsumexp(s, 1)
        w = torch.where(seen, torch.exp(s - ref.clamp(min=-1e300)[:, None]), 0.0)
        check(got[2][0][:150, h], got[2][1][:150, h], w @ v[:96, h // 5].double(), w @ v[:96, h // 5].double().abs(), ref,
              f"head {h}")
