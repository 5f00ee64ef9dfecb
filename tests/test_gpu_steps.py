"""GPU tests of serving steps one after another: the free list's cursor
advanced in place, and steps of other sizes and lengths on one plan."""
import numpy as np
import pytest
import torch

from test_gpu_attn import i32, plan_reference

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
