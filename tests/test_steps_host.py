"""Host-side tests of what the calls of a serving step refuse (before any CUDA
call: they run on a machine without a GPU)."""
import ctypes

import pytest

from test_attn_host import INVALID, cache, io, nv, step  # noqa: F401  (nv: the module's fixture)

MB = 1 << 20
APART = dict(requests=4, tokens=64, q_len=MB, ctx_len=2 * MB, cu_q=3 * MB, kv_len=4 * MB, pos=5 * MB, slot=6 * MB,
             block_table=7 * MB, schedule=8 * MB, cursor=9 * MB, cursor_out=10 * MB)


@pytest.mark.parametrize("bad", [dict(ctx_len=4 * MB), dict(q_len=4 * MB + 12), dict(ctx_len=3 * MB + 16),
                                 dict(q_len=3 * MB - 12), dict(ctx_len=5 * MB + 252), dict(q_len=6 * MB),
                                 dict(ctx_len=10 * MB - 12)])
def test_lengths_that_are_outputs_are_refused(nv, bad):
    assert nv.lib().nvfp4_attn_plan(step(nv, **{**APART, **bad}), None) == INVALID


@pytest.mark.parametrize("good", [{}, dict(cursor=10 * MB), dict(ctx_len=4 * MB + 16), dict(q_len=3 * MB + 20),
                                  dict(q_len=2 * MB), dict(ctx_len=5 * MB + 256)])
def test_lengths_beside_the_outputs_are_not(nv, good):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are not memory")
    assert nv.lib().nvfp4_attn_plan(step(nv, **{**APART, **good}), None) != INVALID


def test_zero_padding_fits_the_old_struct(nv):
    """The flag lies in what was padding at the struct's end."""
    assert ctypes.sizeof(nv._AttnIOC) == 72 and nv._AttnIOC.zero_padding.offset == 68


class Shape:
    """What the checks look at of a plan or a cache."""

    def __init__(self, **f):
        self.__dict__.update(f)


def test_append_refuses_other_pages(nv):
    """Before it looks at k and v: slots of pages of another size name other rows."""
    for plan, cache in ((16, 32), (128, 64)):
        with pytest.raises(ValueError, match="pages of"):
            nv.nvfp4_kv_append(None, None, Shape(slot=1, page_size=plan, tokens=1), Shape(page_size=cache))


@pytest.mark.parametrize("bad", [dict(page_size=64), dict(kv_heads=4), dict(head_dim=32)])
def test_serving_layer_refuses_a_cache_that_does_not_fit(nv, bad):
    from nvfp4_block_scaled_device_gb300.serving import ServingLayer
    plan = Shape(tokens=4, heads=4, kv_heads=2, page_size=32)
    weights = {k: Shape(rows=r, cols=c) for k, r, c in (("qkv", 512, 256), ("o", 256, 256), ("gate", 512, 256))}
    cache = Shape(**{**dict(page_size=32, kv_heads=2, head_dim=64), **bad})
    with pytest.raises(ValueError, match="does not fit"):
        ServingLayer(plan, cache, weights, None, None, None, None)


def test_plan_refuses_a_table_with_overlapping_rows(nv):
    """Its pitch was taken to be a row's width: rows past the first lay outside the tensor."""
    import torch
    row = torch.zeros((1, 8), dtype=torch.int32)
    for table in (row.expand(4, 8), torch.zeros(14, dtype=torch.int32).as_strided((4, 8), (2, 1))):
        with pytest.raises(ValueError, match="overlap"):
            nv.AttnPlan(4, 4, 8, 2, page_size=16, block_table=table)


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), float("-inf"), 3e38, -3e38])
def test_attention_refuses_scales_that_are_not_finite(nv, scale):
    """They ran as a scale of 0, or as an infinite one."""
    L, ws = nv.lib(), (MB, 1 << 40, None)
    assert L.nvfp4_attn_paged(step(nv), io(nv, scale=scale), cache(nv), *ws) == INVALID
    assert L.nvfp4_attn_prompt(step(nv), io(nv, scale=scale), MB, 256, 128, MB, 256, 128, *ws) == INVALID


@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-38, 2e38])
def test_attention_takes_any_other_scale(nv, scale):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are not memory")
    assert nv.lib().nvfp4_attn_paged(step(nv), io(nv, scale=scale), cache(nv), MB, 1 << 40, None) != INVALID


def layer_scratch(T, heads, N, H):
    import torch
    return {"h": Shape(rows=T, cols=H), "a": Shape(rows=T, cols=heads * 64), "qkv": torch.empty(T, N),
            "x1": torch.empty(T, H), "ws_mlp": torch.empty(1 << 24, dtype=torch.uint8)}


def serving_layer(T, scratch, heads=4):
    from nvfp4_block_scaled_device_gb300.serving import ServingLayer
    plan = Shape(tokens=T, heads=heads, kv_heads=2, page_size=0)
    N = (heads + 4) * 64
    weights = {k: Shape(rows=r, cols=c) for k, r, c in (("qkv", N, 256), ("o", 256, heads * 64), ("gate", 512, 256))}
    return ServingLayer(plan, None, weights, Shape(device="cpu"), None, None, None, scratch=scratch)


def test_serving_layer_refuses_scratch_of_other_sizes(nv):
    """A larger step's rows were written past a smaller one's buffers."""
    serving_layer(8, layer_scratch(8, 4, 512, 256))
    for bad in (layer_scratch(7, 4, 512, 256), layer_scratch(8, 2, 512, 256), layer_scratch(8, 4, 448, 256),
                layer_scratch(8, 4, 512, 192), {**layer_scratch(8, 4, 512, 256), "ws_mlp": layer_scratch(1, 1, 1, 1)["x1"]}):
        with pytest.raises(ValueError, match="other sizes"):
            serving_layer(8, bad)


def test_serving_layer_refuses_rows_that_are_not_the_plan_s(nv):
    """Before anything is launched."""
    import torch
    layer = serving_layer(8, layer_scratch(8, 4, 512, 256))
    x = torch.empty(8, 256)
    for a, b in ((torch.empty(9, 256), torch.empty(9, 256)), (x, torch.empty(7, 256)), (torch.empty(8, 320), x)):
        with pytest.raises(ValueError, match="must be"):
            layer.forward(a, b)
