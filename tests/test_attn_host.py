"""Host-side tests of the attention operators: every refusal happens before
any CUDA call (they run on a machine without a GPU)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def nv():
    from nvfp4_block_scaled_device_gb300 import build
    build.build()
    import nvfp4_block_scaled_device_gb300 as m
    m.lib()
    return m


A = 1 << 20          # a 256-byte aligned address that no call dereferences


def step(nv, **f):
    d = dict(requests=4, tokens=64, q_len=A, ctx_len=None, cu_q=A, kv_len=A, pos=A, page_size=16, block_table=A,
             table_cols=8, table_ld=8, slot=A, free_pages=None, free_count=0, cursor=None, cursor_out=A, heads=10,
             kv_heads=2, window=0, schedule=A, schedule_bytes=1 << 40)
    d.update(f)
    return ctypes.byref(nv._StepC(**d))


def io(nv, **f):
    d = dict(q=A, ldq=1280, hq=128, out=A, ldo=1280, ho=128, lse=A, head_dim=128, scale=0.1)
    d.update(f)
    return ctypes.byref(nv._AttnIOC(**d))


def cache(nv, **f):
    d = dict(k=A, v=A, pages=10, page_size=16, kv_heads=2, head_dim=128, page_stride=2 * 16 * 128)
    d.update(f)
    return ctypes.byref(nv._CacheC(**d))


INVALID, MISALIGNED, WORKSPACE = 1, 2, 5


@pytest.mark.parametrize("bad,status", [
    (dict(requests=0), INVALID), (dict(requests=8193), INVALID), (dict(tokens=0), INVALID),
    (dict(tokens=1 << 31), INVALID), (dict(q_len=None), INVALID), (dict(cu_q=None), INVALID),
    (dict(kv_len=None), INVALID), (dict(page_size=8), INVALID), (dict(page_size=48), INVALID),
    (dict(page_size=256), INVALID), (dict(block_table=None), INVALID), (dict(table_cols=0), INVALID),
    (dict(table_ld=7), INVALID), (dict(table_cols=1 << 28, table_ld=1 << 28), INVALID), (dict(slot=None), INVALID),
    (dict(free_pages=A, free_count=-1), INVALID), (dict(kv_heads=0), INVALID), (dict(kv_heads=3), INVALID),
    (dict(heads=2, kv_heads=4), INVALID), (dict(heads=129, kv_heads=1), INVALID), (dict(window=-1), INVALID),
    (dict(schedule=None), WORKSPACE), (dict(schedule_bytes=16), WORKSPACE), (dict(schedule=A + 64), MISALIGNED),
    (dict(q_len=A + 2), MISALIGNED), (dict(ctx_len=A + 1), MISALIGNED), (dict(cu_q=A + 2), MISALIGNED),
    (dict(pos=A + 2), MISALIGNED), (dict(slot=A + 2), MISALIGNED), (dict(block_table=A + 2), MISALIGNED),
    (dict(free_pages=A + 2, free_count=1), MISALIGNED), (dict(cursor=A + 2), MISALIGNED)])
def test_plan_refusals(nv, bad, status):
    assert nv.lib().nvfp4_attn_plan(step(nv, **bad), None) == status


def test_plan_refuses_null(nv):
    assert nv.lib().nvfp4_attn_plan(None, None) == INVALID


@pytest.mark.parametrize("bad,status", [
    (dict(pages=0), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(page_size=24), INVALID),
    (dict(kv_heads=0), INVALID), (dict(head_dim=136), INVALID), (dict(head_dim=8), INVALID),
    (dict(head_dim=100), INVALID), (dict(page_stride=4088), INVALID), (dict(pages=1 << 28), INVALID),
    (dict(k=A + 8), MISALIGNED), (dict(v=A + 2), MISALIGNED), (dict(page_stride=4100), MISALIGNED)])
def test_cache_refusals(nv, bad, status):
    L = nv.lib()
    assert L.nvfp4_kv_append(A, 256, 128, A, 256, 128, A, 64, cache(nv, **bad), None) == status
    assert L.nvfp4_attn_paged(step(nv), io(nv), cache(nv, **bad), A, 1 << 40, None) == status


def test_append_refusals(nv):
    L = nv.lib()
    call = lambda k=A, ldk=256, hk=128, v=A, ldv=256, hv=128, slot=A, tokens=64: \
        L.nvfp4_kv_append(k, ldk, hk, v, ldv, hv, slot, tokens, cache(nv), None)
    for bad in (dict(k=None), dict(v=None), dict(slot=None), dict(tokens=0), dict(tokens=1 << 31), dict(ldk=120),
                dict(hv=64)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(k=A + 8), dict(v=A + 2), dict(ldk=260), dict(hk=132), dict(slot=A + 2)):
        assert call(**bad) == MISALIGNED, bad
    assert L.nvfp4_kv_append(A, 256, 128, A, 256, 128, A, 64, None, None) == INVALID


IO_BAD = [(dict(q=None), INVALID), (dict(out=None), INVALID), (dict(head_dim=0), INVALID), (dict(head_dim=8), INVALID),
          (dict(head_dim=129), INVALID), (dict(head_dim=256), INVALID), (dict(ldq=64), INVALID), (dict(ho=64), INVALID),
          (dict(q=A + 8), MISALIGNED), (dict(out=A + 2), MISALIGNED), (dict(ldq=1284), MISALIGNED),
          (dict(hq=130), MISALIGNED), (dict(ldo=1284), MISALIGNED), (dict(lse=A + 2), MISALIGNED)]


@pytest.mark.parametrize("bad,status", IO_BAD)
def test_attention_refusals(nv, bad, status):
    L = nv.lib()
    assert L.nvfp4_attn_paged(step(nv), io(nv, **bad), cache(nv), A, 1 << 40, None) == status
    assert L.nvfp4_attn_prompt(step(nv), io(nv, **bad), A, 256, 128, A, 256, 128, A, 1 << 40, None) == status


def test_attention_refuses_what_does_not_fit_together(nv):
    L = nv.lib()
    for bad in (dict(page_size=32), dict(kv_heads=1, page_stride=4096), dict(head_dim=64)):
        assert L.nvfp4_attn_paged(step(nv), io(nv), cache(nv, **bad), A, 1 << 40, None) == INVALID, bad
    assert L.nvfp4_attn_paged(step(nv, page_size=0), io(nv), cache(nv), A, 1 << 40, None) == INVALID
    assert L.nvfp4_attn_paged(step(nv, heads=0), io(nv), cache(nv), A, 1 << 40, None) == INVALID
    assert L.nvfp4_attn_paged(None, io(nv), cache(nv), A, 1 << 40, None) == INVALID
    assert L.nvfp4_attn_paged(step(nv), None, cache(nv), A, 1 << 40, None) == INVALID
    assert L.nvfp4_attn_paged(step(nv), io(nv), None, A, 1 << 40, None) == INVALID
    # a step with cached tokens is not a packed prompt
    assert L.nvfp4_attn_prompt(step(nv, ctx_len=A), io(nv), A, 256, 128, A, 256, 128, A, 1 << 40, None) == INVALID
    assert L.nvfp4_attn_prompt(step(nv), io(nv), None, 256, 128, A, 256, 128, A, 1 << 40, None) == INVALID
    assert L.nvfp4_attn_prompt(step(nv), io(nv), A, 256, 120, A, 256, 128, A, 1 << 40, None) == INVALID
    assert L.nvfp4_attn_prompt(step(nv), io(nv), A, 256, 128, A, 260, 128, A, 1 << 40, None) == MISALIGNED
    for ws, n, status in ((None, 1 << 40, WORKSPACE), (A, 16, WORKSPACE), (A + 128, 1 << 40, MISALIGNED)):
        assert L.nvfp4_attn_paged(step(nv), io(nv), cache(nv), ws, n, None) == status
        assert L.nvfp4_attn_prompt(step(nv), io(nv), A, 256, 128, A, 256, 128, ws, n, None) == status


def test_size_helpers(nv):
    assert nv.attn_workspace_bytes() >= 256
    assert nv.attn_schedule_bytes(0, 1, 1, 1) == 0
    small, large = nv.attn_schedule_bytes(1, 1, 8, 8), nv.attn_schedule_bytes(8192, 16384, 8, 8)
    assert 0 < small <= large


def test_binding_checks_its_tensors(nv):
    with pytest.raises(ValueError):
        nv.KVCache(torch.zeros(2, 2, 16, 64), torch.zeros(2, 2, 16, 64))
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nv._heads_3d(x, "x", 4, 2, 64)                  # not a CUDA tensor
    with pytest.raises(ValueError):
        nv._i32(torch.zeros(3, dtype=torch.int64), 3, "n")
