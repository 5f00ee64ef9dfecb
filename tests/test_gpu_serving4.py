"""GPU tests of serving layers with head norms and a 4-bit cache, and of a server
whose requests fork, end and have their pages moved: each layer's attention
against binary64 over the rows that its cache stands for."""
import numpy as np
import pytest
import torch

import synthetic
from _attn import OUT_P, reference
from _gpu import dev
from test_gpu_attn import i32
from test_gpu_attn4 import P_HALF, check, values
from test_gpu_serving import D, H, HEADS, KV, weights, x_of  # noqa: F401  (weights: the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_device_gb300 as m
    return m


class Server:
    """R rows of a block table; steps of any lengths, as many tokens at most as the plan has."""

    def __init__(self, nv, weights, R, tokens, page, cols, pages, four, norms, halves=False, window=0):
        from nvfp4_block_scaled_device_gb300.serving import ServingLayer
        self.nv, self.R, self.page, self.four = nv, R, page, four
        self.table = torch.full((R, cols), -1, dtype=torch.int32, device="cuda")
        self.ctx, self.free = i32([0] * R), i32(np.random.default_rng(page).permutation(pages).tolist())
        cos, sin = (torch.from_numpy(t).cuda() for t in synthetic.rope_tables(page * cols, D))
        gen = torch.Generator("cuda").manual_seed(17)
        self.norms = [(1 + 0.3 * torch.randn(D, device="cuda", generator=gen)).bfloat16() for _ in range(2)] if norms else [None] * 2
        self.caches = [nv.KVCache4.empty(pages, KV, page, D, 2.0 ** -9, 2.0 ** -9) if four else nv.KVCache.empty(pages, KV, page, D)
                       for _ in weights]
        for c in self.caches:                                 # rows that nobody has written: NaN
            (c.k_sf if four else c.k).fill_(0x7f if four else float("nan"))
            (c.v_sf if four else c.v).fill_(0x7f if four else float("nan"))
        self.window, self.halves, self.rope = window, halves, (cos, sin)
        self.stacks = []
        for T in tokens:
            plan, scratch, layers = nv.AttnPlan(R, T, HEADS, KV, page_size=page, block_table=self.table, window=window), None, []
            for c, w in zip(self.caches, weights):
                layers.append(ServingLayer(plan, c, w, dev(synthetic.norm_weight(80, H)), dev(synthetic.norm_weight(81, H)), cos, sin,
                                           scratch=scratch, q_norm=self.norms[0], k_norm=self.norms[1], halves=halves))
                scratch = layers[0].scratch
            self.stacks.append((plan, layers))
        self.cursor = i32([0])
        self.held = nv.PageTable(self.table, self.ctx, page, pages)

    def step(self, q, x, stack=0, look=True):
        plan, layers = self.stacks[stack]
        out = torch.empty_like(x)
        plan.cursor.copy_(self.cursor)
        self.nv.nvfp4_attn_plan(plan, i32(q), self.ctx, self.free, plan.cursor)
        for at, layer in enumerate(layers):
            before = x.clone()
            layer.forward(x, out)
            if look:
                self.look(q, plan, layer, at, before)
            x = out
        self.ctx.add_(i32(q))
        self.cursor.copy_(plan.cursor)
        torch.cuda.synchronize()
        assert self.nv.device_status() == 0
        return out

    def look(self, q, plan, layer, at, x):
        """The layer's attention against binary64 over what its cache stands for."""
        rows, got = layer.scratch["qkv"].view(-1, HEADS + 2 * KV, D), layer.scratch["attn"].view(-1, HEADS, D)
        cache = self.caches[at]
        k, v = values(cache) if self.four else (cache.k.double(), cache.v.double())
        ctx, first = self.ctx.tolist(), 0
        bf16 = not self.four or layer.scratch["expanded"] is not None
        for r, n in enumerate(q):
            if n:
                pos = torch.arange(ctx[r] + n, device="cuda")
                ids, row = self.table[r].long()[pos // self.page], pos % self.page
                ref = reference(rows[first:first + n, :HEADS].double(), k[ids, :, row], v[ids, :, row], ctx[r], D ** -0.5, self.window)
                check(got[first:first + n], None, *ref, OUT_P if bf16 else P_HALF, v[ids, :, row],
                      f"layer {at} request {r}")
            first += n


@pytest.mark.parametrize("four,norms,halves,page,window", [(True, True, True, 16, 0), (True, False, False, 64, 0),
                                                           (False, True, False, 32, 0), (True, True, False, 32, 50),
                                                           (False, False, True, 16, 0)])
def test_steps(nv, weights, four, norms, halves, page, window):
    prompts = [37, 1, 130]
    s = Server(nv, weights, 3, [sum(prompts) + 2, 3], page, 12, 40, four, norms, halves, window)
    s.step(prompts, x_of(sum(prompts) + 2, 600))
    for i in range(4):
        s.step([1, 1, 1], x_of(3, 610 + i), stack=1)


@pytest.mark.parametrize("window", [0, 70])
def test_a_chunk_among_decoding_requests(nv, weights, window):
    """A few rows per request on average, one request with many: through the bf16 pages,
    bit for bit as nvfp4_attn_paged4 does that; not without them, nor in a step of single tokens."""
    R, page, lens = 12, 16, [300] + [20] * 11
    s = Server(nv, weights, R, [sum(lens), 105], page, 30, 80, True, True, True, window)
    s.step(lens, x_of(sum(lens), 630))
    plan, layers = s.stacks[1]
    assert 105 / R * (HEADS // KV) < 40 and all(layer.expands for layer in layers)
    for i, q in enumerate(([90] + [1] * 11, [1] * 12, [0] + [1] * 11)):
        s.step(q, x_of(105, 631 + i), stack=1)                # (3 rows of padding and more)
        for at, layer in enumerate(layers):
            rows, n = layer.scratch["qkv"].view(-1, HEADS + 2 * KV, D), sum(q)
            if at + 1 < len(layers):
                continue                                      # (the scratch is the last layer's)
            out = [torch.empty(105, HEADS, D, device="cuda").bfloat16() for _ in range(2)]
            pages = nv.KVCache.empty(80, KV, page, D)
            for o, e in zip(out, (pages, None)):
                nv.nvfp4_attn_paged4(rows[:, :HEADS], s.caches[at], plan, o, layer.scratch["ws_attn"], zero_padding=True, expanded=e)
            assert torch.equal(layer.scratch["attn"].view(-1, HEADS, D), out[0])
            assert torch.equal(out[0][:n], out[1][:n]) == (q[0] < 2) and (out[0][n:] == 0).all()


def test_a_layer_without_bf16_pages(nv, weights):
    from nvfp4_block_scaled_device_gb300.serving import ServingLayer
    cos, sin = (torch.from_numpy(t).cuda() for t in synthetic.rope_tables(64, D))
    norm = dev(synthetic.norm_weight(80, H))
    make = lambda R, T, four=True, **f: ServingLayer(
        nv.AttnPlan(R, T, HEADS, KV, page_size=16, block_table=4),
        nv.KVCache4.empty(20, KV, 16, D) if four else nv.KVCache.empty(20, KV, 16, D), weights[0], norm, norm, cos, sin, **f)
    for layer, has in ((make(4, 5), True), (make(4, 4), False), (make(4, 300), True), (make(4, 300, expand=False), False),
                       (make(4, 300, four=False), False)):
        assert layer.expands == has and (layer.scratch["expanded"] is not None) == has
    outs = []                                                 # a prompt straight from the codes
    for expand in (True, False):
        layer = make(1, 50, expand=expand)
        layer.plan.block_table.copy_(i32([[3, 0, 7, 5]]))
        nv.nvfp4_attn_plan(layer.plan, i32([50]), i32([0]))
        x = x_of(50, 640)
        layer.forward(x, torch.empty_like(x))
        rows, got = layer.scratch["qkv"].view(50, -1, D), layer.scratch["attn"].view(50, HEADS, D)
        k, v = values(layer.cache)
        pos = torch.arange(50, device="cuda")
        ids = layer.plan.block_table[0].long()[pos // 16]
        check(got, None, *reference(rows[:, :HEADS].double(), k[ids, :, pos % 16], v[ids, :, pos % 16], 0, D ** -0.5),
              OUT_P if expand else P_HALF, v[ids, :, pos % 16])
        outs.append(got.clone())
    assert not torch.equal(*outs)


@pytest.mark.parametrize("four", [False, True])
def test_what_the_cache_holds(nv, weights, four):
    """Norm, rotation and the write in one pass: what the calls one by one give."""
    s = Server(nv, weights[:1], 2, [20], 16, 4, 10, four, True, True)
    plan, (layer,) = s.stacks[0]
    s.step([11, 9], x_of(20, 620), look=False)
    rows = layer.scratch["qkv"].view(20, -1, D)
    k, v = rows[:, HEADS:HEADS + KV], rows[:, HEADS + KV:]
    out = torch.empty_like(k)
    nv.nvfp4_qk_norm_rope(None, k, None, s.norms[1], plan.pos, *s.rope, k_out=out, halves=True)
    other = nv.KVCache4.empty(10, KV, 16, D, 2.0 ** -9, 2.0 ** -9) if four else nv.KVCache.empty(10, KV, 16, D)
    (nv.nvfp4_kv4_append if four else nv.nvfp4_kv_append)(out, v, plan, other)
    slot = plan.slot.long()
    for name in ("k", "v", "k_sf", "v_sf")[:4 if four else 2]:
        a, b = getattr(s.caches[0], name), getattr(other, name)
        assert torch.equal(a[slot // 16, :, slot % 16], b[slot // 16, :, slot % 16])


@pytest.mark.parametrize("four", [False, True])
def test_requests_that_fork_end_and_move(nv, weights, four):
    rng = np.random.default_rng(5)
    R, page, pages = 8, 16, 60
    s = Server(nv, weights, R, [100, R], page, 10, pages, four, True)
    nvp = [i32([0] * (pages // 2)) for _ in range(2)]
    free, count = i32([0] * pages), i32([0])
    s.step([40, 33, 0, 20, 0, 0, 0, 0], x_of(100, 640))
    live = [0, 1, 3]
    for i in range(8):
        if i == 1:                                            # two children of request 0, one of 3
            src, dst = [0, 0, 3], [2, 4, 7]
            cs, cd = i32([0] * 3), i32([0] * 3)
            nv.nvfp4_pages_fork(s.held, i32(src), i32(dst), s.free, s.cursor, s.cursor, cs, cd)
            nv.nvfp4_pages_copy(s.caches, cs, cd)
            live += dst
            for c in s.caches:                                # a child's rows are its parent's
                for a, b in zip(src, dst):
                    for p in range(int(s.ctx[a])):
                        x, y = (c.k[int(s.table[r, p // page]), :, p % page] for r in (a, b))
                        assert torch.equal(x, y)
        if i in (3, 5):                                       # the parent ends, then a child; the cache is moved together
            gone = 0 if i == 3 else 7
            live.remove(gone)
            s.ctx[gone] = 0
            nv.nvfp4_pages_free(s.held, free, count, s.table, *nvp)
            nv.nvfp4_pages_copy(s.caches, *nvp)
            held = {int(p) for r in live for p in s.table[r, :-(-int(s.ctx[r]) // page)]}
            assert held == set(range(len(held))) and count.item() == pages - len(held)
            s.free, s.cursor = free.clone(), i32([0])
        q = [int(r in live) for r in range(R)]
        s.step(q, x_of(R, 650 + i), stack=1)


def test_captured_decode_steps(nv, weights):
    """A whole step with norms and a 4-bit cache in a graph, as the contexts grow, bit for bit the plain calls."""
    outs = []
    for captured in (False, True):
        s = Server(nv, weights, 3, [70, 3], 16, 10, 40, True, True, True)
        s.step([20, 45, 5], x_of(70, 660), look=False)
        plan, layers = s.stacks[1]
        plan.cursor.copy_(s.cursor)
        one, x, out = i32([1] * 3), torch.zeros(3, H, device="cuda", dtype=torch.bfloat16), torch.empty(3, H, device="cuda").bfloat16()

        def step():
            nv.nvfp4_attn_plan(plan, one, s.ctx, s.free, plan.cursor)
            y = x
            for layer in layers:
                layer.forward(y, out)
                y = out
            s.ctx.add_(one)
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        if captured:
            with torch.cuda.graph(graph, stream=stream):
                step()
        got = []
        for i in range(20):
            x.copy_(x_of(3, 670 + i))
            graph.replay() if captured else step()
            got.append(out.clone())
        torch.cuda.synchronize()
        assert nv.device_status() == 0
        outs.append(torch.stack(got))
    assert torch.equal(*outs)


def test_packed_prompts_without_a_cache(nv, weights):
    from nvfp4_block_scaled_device_gb300.serving import ServingLayer
    lens = [9, 140, 1]
    T = sum(lens)
    cos, sin = (torch.from_numpy(t).cuda() for t in synthetic.rope_tables(200, D))
    w = torch.ones(D, device="cuda").bfloat16()
    plan = nv.AttnPlan(3, T, HEADS, KV)
    layer = ServingLayer(plan, None, weights[0], dev(synthetic.norm_weight(80, H)), dev(synthetic.norm_weight(81, H)), cos, sin,
                         q_norm=w, k_norm=w, halves=True)
    nv.nvfp4_attn_plan(plan, i32(lens))
    x = x_of(T, 690)
    layer.forward(x, torch.empty_like(x))
    rows, got, at = layer.scratch["qkv"].view(T, -1, D), layer.scratch["attn"].view(T, HEADS, D), 0
    for n in lens:
        new = rows[at:at + n].double()
        ref = reference(new[:, :HEADS], new[:, HEADS:HEADS + KV], new[:, HEADS + KV:], 0, D ** -0.5)
        check(got[at:at + n], None, *ref, OUT_P, new[:, HEADS + KV:])
        at += n
    # (normed by ones and rotated: rows of length sqrt(D))
    assert (rows[:, :HEADS].double().pow(2).mean(-1) - 1).abs().max() < 0.02


def test_refusals(nv, weights):
    from nvfp4_block_scaled_device_gb300.serving import ServingLayer
    norm = dev(synthetic.norm_weight(80, H))
    cos, sin = (torch.from_numpy(t).cuda() for t in synthetic.rope_tables(8, D))
    w = torch.ones(D, device="cuda").bfloat16()
    plan = nv.AttnPlan(1, 40, HEADS, KV, page_size=16, block_table=4)
    cache = nv.KVCache4.empty(4, KV, 16, D)
    make = lambda **f: ServingLayer(**{**dict(plan=plan, cache=cache, weights=weights[0], attn_norm=norm, mlp_norm=norm, cos_t=cos,
                                              sin_t=sin), **f})
    layer = make(q_norm=w)
    for bad in (dict(q_norm=w.float()), dict(k_norm=w[:32]), dict(halves=True, cos_t=cos[:, :20], sin_t=sin[:, :20]),
                dict(cache=nv.KVCache4.empty(4, KV, 32, D)), dict(cache=nv.KVCache4.empty(4, KV, 16, 2 * D)),
                dict(scratch={**layer.scratch, "expanded": None}),
                dict(scratch={**layer.scratch, "expanded": nv.KVCache.empty(5, KV, 16, D)})):
        with pytest.raises(ValueError):
            make(**bad)
