"""GPU tests of the serving layers: prompts and decode steps through step
tables, cache and attention, each layer's attention against binary64 over the
keys and values it was given, and a captured decode step bit for bit against
the plain one."""
import numpy as np
import pytest
import torch

import synthetic
from _attn import check, reference
from _gpu import dev

pytestmark = pytest.mark.gpu

H, I, HEADS, KV, D, LAYERS = 256, 512, 4, 2, 64, 2


@pytest.fixture(scope="module")
def nv():
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_device_gb300 as m
    return m


@pytest.fixture(scope="module")
def weights(nv):
    ws = nv.workspace(256)
    shapes = (("qkv", (HEADS + 2 * KV) * D, H), ("o", H, HEADS * D), ("gate", I, H), ("up", I, H), ("down", H, I))
    return [{k: nv.quantize_new(dev(synthetic.weight(300 + 10 * layer + j, rows, cols, std=0.2)), ws)
             for j, (k, rows, cols) in enumerate(shapes)} for layer in range(LAYERS)]


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def x_of(tokens, seed):
    return dev(synthetic.activations(tokens, seed=seed, h=H))


class Server:
    """Prompts, then one token per request and step."""

    def __init__(self, nv, weights, prompts, page, steps, window=0):
        from nvfp4_block_scaled_device_gb300.serving import ServingLayer
        self.nv, self.prompts, self.R = nv, prompts, len(prompts)
        need = [-(-(n + steps) // page) for n in prompts]
        pages = sum(need) + 3
        rng = np.random.default_rng(page)
        self.free = torch.from_numpy(rng.permutation(pages).astype(np.int32)).cuda()
        table = torch.full((self.R, max(need)), -1, dtype=torch.int32, device="cuda")
        cos, sin = (torch.from_numpy(t).cuda() for t in synthetic.rope_tables(max(prompts) + steps, D))
        plans = [nv.AttnPlan(self.R, T, HEADS, KV, page_size=page, block_table=table, window=window)
                 for T in (sum(prompts) + 2, self.R)]
        caches = [nv.KVCache.empty(pages, KV, page, D) for _ in weights]
        self.stacks = [(plan, [ServingLayer(plan, cache, w, dev(synthetic.norm_weight(80, H)),
                                            dev(synthetic.norm_weight(81, H)), cos, sin)
                               for cache, w in zip(caches, weights)]) for plan in plans]
        self.ctx, self.one = i32([0] * self.R), i32([1] * self.R)
        self.x = torch.zeros((self.R, H), dtype=torch.bfloat16, device="cuda")
        self.out = torch.empty_like(self.x)

    def run(self, stack, q_len, x, out):
        plan, layers = self.stacks[stack]
        self.nv.nvfp4_attn_plan(plan, q_len, self.ctx, self.free, plan.cursor)
        for layer in layers:
            layer.forward(x, out)
            x = out
        self.ctx.add_(q_len)

    def prefill(self):
        plan = self.stacks[0][0]
        x = x_of(plan.tokens, 500)
        out = torch.empty_like(x)
        self.run(0, i32(self.prompts), x, out)
        self.stacks[1][0].cursor.copy_(plan.cursor)
        return out

    def decode(self):
        self.run(1, self.one, self.x, self.out)


@pytest.mark.parametrize("page,window", [(16, 0), (64, 0), (32, 50)])
def test_steps_against_binary64(nv, weights, page, window):
    prompts, steps = [37, 1, 130], 5
    server = Server(nv, weights, prompts, page, steps, window)
    keys = [[[] for _ in prompts] for _ in weights]
    for step in range(steps):
        q = prompts if step == 0 else [1] * len(prompts)
        if step == 0:
            server.prefill()
        else:
            server.x.copy_(x_of(len(prompts), 510 + step))
            server.decode()
        torch.cuda.synchronize()
        assert nv.device_status() == 0
        for at_layer, layer in enumerate(server.stacks[min(step, 1)][1]):
            rows = layer.scratch["qkv"].view(-1, HEADS + 2 * KV, D)
            got = layer.scratch["attn"].view(-1, HEADS, D)
            at = 0
            for r, n in enumerate(q):
                new = rows[at:at + n].clone()
                keys[at_layer][r].append(new[:, HEADS:])
                kv = torch.cat(keys[at_layer][r]).double()
                ref = reference(new[:, :HEADS].double(), kv[:, :KV], kv[:, KV:], len(kv) - n, D ** -0.5, window)
                check(got[at:at + n], None, *ref, f"step {step} layer {at_layer} request {r}")
                at += n


def test_captured_step_matches_plain_steps(nv, weights):
    prompts, steps = [20, 63, 5], 6
    outs = []
    for captured in (False, True):
        server = Server(nv, weights, prompts, 16, steps)
        got = [server.prefill()]
        if captured:
            ctx, cursor = server.ctx.clone(), server.stacks[1][0].cursor.clone()
            stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.graph(graph, stream=stream):
                server.decode()
            torch.cuda.current_stream().wait_stream(stream)
            assert torch.equal(server.ctx, ctx) and torch.equal(server.stacks[1][0].cursor, cursor)
        for step in range(steps):
            server.x.copy_(x_of(len(prompts), 520 + step))
            graph.replay() if captured else server.decode()
            got.append(server.out.clone())
        torch.cuda.synchronize()
        assert nv.device_status() == 0
        outs.append(got)
    for step, (a, b) in enumerate(zip(*outs)):
        assert torch.equal(a[:sum(prompts)], b[:sum(prompts)]), f"step {step}"


def test_packed_prompts_without_a_cache(nv, weights):
    """A plan without pages gives each layer's attention over the prompts alone."""
    from nvfp4_block_scaled_device_gb300.serving import ServingLayer
    lens = [9, 140, 1]
    T = sum(lens)
    cos, sin = (torch.from_numpy(t).cuda() for t in synthetic.rope_tables(max(lens), D))
    plan = nv.AttnPlan(len(lens), T, HEADS, KV)
    layer = ServingLayer(plan, None, weights[0], dev(synthetic.norm_weight(80, H)), dev(synthetic.norm_weight(81, H)),
                         cos, sin)
    x = x_of(T, 530)
    out = torch.empty_like(x)
    nv.nvfp4_attn_plan(plan, i32(lens))
    layer.forward(x, out)
    torch.cuda.synchronize()
    assert nv.device_status() == 0 and torch.isfinite(out.float()).all()
    rows, got, at = layer.scratch["qkv"].view(T, -1, D), layer.scratch["attn"].view(T, HEADS, D), 0
    for r, n in enumerate(lens):
        new = rows[at:at + n].double()
        ref = reference(new[:, :HEADS], new[:, HEADS:HEADS + KV], new[:, HEADS + KV:], 0, D ** -0.5)
        check(got[at:at + n], None, *ref, f"request {r}")
        at += n


def test_refusals(nv, weights):
    from nvfp4_block_scaled_device_gb300.serving import ServingLayer
    norm = dev(synthetic.norm_weight(80, H))
    cos, sin = (torch.from_numpy(t).cuda() for t in synthetic.rope_tables(8, D))
    with pytest.raises(ValueError):
        ServingLayer(nv.AttnPlan(1, 4, 2 * HEADS, KV), None, weights[0], norm, norm, cos, sin)
    with pytest.raises(ValueError):
        ServingLayer(nv.AttnPlan(1, 4, HEADS, KV), nv.KVCache.empty(2, KV, 16, D), weights[0], norm, norm, cos, sin)
