"""GPU tests of rotary positions outside the tables: every kernel that rotates
takes the nearest table row, bit for bit, and reports it."""
import numpy as np
import pytest
import torch

import synthetic
from _gpu import dev, quantize_gpu
from test_gpu_attn import i32
from test_gpu_serving import D, H, HEADS, KV, weights, x_of  # noqa: F401  (weights: the module's fixture)

pytestmark = pytest.mark.gpu
BAD = 100 + 33


@pytest.fixture(scope="module")
def nv():
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_device_gb300 as m
    return m


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("T,split", [(1, False), (2, False), (1, True), (8, True), (17, False), (17, True), (300, False),
                                     (300, True), (1024, True)])
def test_positions_outside_the_tables(nv, T, split, inverse):
    N, K, P, hd, rd = 1024, 512, 40, 128, 64
    rng = np.random.default_rng(T)
    ws = nv.workspace(256)
    A, W = (quantize_gpu(synthetic.normal(rng, s), ws) for s in ((T, K), (N, K)))
    gws = nv.workspace(nv.gemm_workspace_bytes()) if split else None
    # the tables lie inside larger ones: a row beside them would show in the output
    ct, st = (torch.from_numpy(t).cuda() for t in synthetic.rope_tables(3 * P, rd))
    ct, st = ct[P:2 * P], st[P:2 * P]
    pos = torch.from_numpy(rng.integers(0, P, T).astype(np.int32)).cuda()

    def run(p):
        out = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        nv.nvfp4_gemm_rope(A, W, out, p, ct, st, 0, 6, hd, rd, inverse=inverse, workspace=gws)
        torch.cuda.synchronize()
        return out

    run(pos)
    assert nv.device_status() == 0
    for bad in (P, P + 7, -1, -5, 2 ** 31 - 1, -2 ** 31):
        p = pos.clone()
        p[T // 2] = bad
        got = run(p)
        assert nv.device_status() == BAD and nv.device_status() == 0
        assert torch.equal(got, run(p.clamp(0, P - 1)))


def test_a_request_past_the_rotary_tables(nv, weights):
    """A serving step in which one request has outgrown the tables: reported,
    the other requests' keys, values and queries as without it."""
    from nvfp4_block_scaled_device_gb300.serving import ServingLayer
    P, page = 24, 16
    cos, sin = (torch.from_numpy(t).cuda() for t in synthetic.rope_tables(P, D))
    norms = [dev(synthetic.norm_weight(80 + i, H)) for i in range(2)]
    got = []
    for ctx in ([3, 23], [3, 24], [3, 31], [3, 1000]):
        plan = nv.AttnPlan(2, 2, HEADS, KV, page_size=page, block_table=torch.arange(4, dtype=torch.int32, device="cuda")
                           .reshape(2, 2).contiguous())
        cache = nv.KVCache(*(torch.zeros(4, KV, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
        layer = ServingLayer(plan, cache, weights[0], *norms, cos, sin)
        x, out = x_of(2, 604), torch.empty((2, H), dtype=torch.bfloat16, device="cuda")
        nv.nvfp4_attn_plan(plan, i32([1, 1]), i32(ctx))
        torch.cuda.synchronize()
        assert nv.device_status() == (100 + 31 if ctx[1] >= 32 else 0)        # past its block table
        layer.forward(x, out)
        torch.cuda.synchronize()
        assert nv.device_status() == (BAD if ctx[1] >= P else 0)
        got.append((layer.scratch["qkv"].clone(), cache.k[:2].clone()))
    for qkv, k in got[1:]:
        assert torch.equal(qkv, got[0][0]) and torch.equal(k, got[0][1])
