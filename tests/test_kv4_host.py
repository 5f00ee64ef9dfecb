"""Host-side tests of the head norms, the 4-bit cache and the page operators:
every refusal happens before any CUDA call (they run on a machine without a GPU)."""
import ctypes

import pytest
import torch

from test_attn_host import A, INVALID, MISALIGNED, cache, nv, step  # noqa: F401  (nv: the module's fixture)


def cache4(nv, **f):
    d = dict(k=A, v=A, k_sf=A, v_sf=A, k_g=A, v_g=A, pages=10, page_size=16, kv_heads=2, head_dim=128,
             page_stride=2 * 16 * 64, sf_stride=2 * 16 * 8)
    d.update(f)
    return nv._Cache4C(**d)


def heads(nv, **f):
    d = dict(tokens=64, heads=10, kv_heads=2, head_dim=128, q=A, ldq=1280, hq=128, q_out=A, ldqo=1280, hqo=128, k=A,
             ldk=256, hk=128, k_out=A, ldko=256, hko=128, q_norm=A, k_norm=A, eps=1e-6, pos=A, cos_t=A, sin_t=A,
             table_ld=64, positions=100, rope_dim=128, halves=0, slot=None, v=None, ldv=0, hv=0)
    d.update(f)
    return ctypes.byref(nv._HeadsC(**d))


CACHE4_BAD = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k_sf=None), INVALID), (dict(v_sf=None), INVALID),
    (dict(k_g=None), INVALID), (dict(v_g=None), INVALID), (dict(pages=0), INVALID), (dict(pages=1 << 28), INVALID),
    (dict(page_size=24), INVALID), (dict(page_size=0), INVALID), (dict(kv_heads=0), INVALID),
    (dict(head_dim=136), INVALID), (dict(head_dim=8), INVALID), (dict(head_dim=72), INVALID),
    (dict(page_stride=2032), INVALID), (dict(sf_stride=240), INVALID), (dict(k=A + 8), MISALIGNED),
    (dict(v=A + 4), MISALIGNED), (dict(k_sf=A + 8), MISALIGNED), (dict(v_sf=A + 1), MISALIGNED),
    (dict(k_g=A + 2), MISALIGNED), (dict(v_g=A + 1), MISALIGNED), (dict(page_stride=2056), MISALIGNED),
    (dict(sf_stride=264), MISALIGNED)]


@pytest.mark.parametrize("bad,status", CACHE4_BAD)
def test_cache4_refusals(nv, bad, status):
    L, c = nv.lib(), cache4(nv, **bad)
    assert L.nvfp4_kv4_append(A, 256, 128, A, 256, 128, A, 64, ctypes.byref(c), None) == status
    assert L.nvfp4_kv4_expand(ctypes.byref(c), step(nv), cache(nv), None) == status
    assert L.nvfp4_qk_norm_rope(heads(nv, slot=A, v=A, ldv=256, hv=128, cache4=ctypes.addressof(c)), None) == status


def test_append4_and_expand_refusals(nv):
    L, c = nv.lib(), ctypes.byref(cache4(nv))
    call = lambda k=A, ldk=256, hk=128, v=A, ldv=256, hv=128, slot=A, tokens=64: \
        L.nvfp4_kv4_append(k, ldk, hk, v, ldv, hv, slot, tokens, c, None)
    for bad in (dict(k=None), dict(v=None), dict(slot=None), dict(tokens=0), dict(tokens=1 << 31), dict(ldk=120), dict(hv=64)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(k=A + 8), dict(v=A + 2), dict(ldk=260), dict(hk=132), dict(slot=A + 2)):
        assert call(**bad) == MISALIGNED, bad
    assert L.nvfp4_kv4_append(A, 256, 128, A, 256, 128, A, 64, None, None) == INVALID
    for bad in (dict(pages=11), dict(page_size=32, page_stride=1 << 14), dict(kv_heads=1), dict(head_dim=64), dict(k=None)):
        assert L.nvfp4_kv4_expand(c, step(nv), cache(nv, **bad), None) == INVALID, bad
    assert L.nvfp4_kv4_expand(c, step(nv, page_size=32), cache(nv), None) == INVALID
    assert L.nvfp4_kv4_expand(c, step(nv, window=-1), cache(nv), None) == INVALID
    assert L.nvfp4_kv4_expand(c, None, cache(nv), None) == INVALID
    assert L.nvfp4_kv4_expand(c, step(nv), None, None) == INVALID


@pytest.mark.parametrize("bad,status", [
    (dict(tokens=0), INVALID), (dict(tokens=1 << 31), INVALID), (dict(heads=-1), INVALID),
    (dict(heads=0, kv_heads=0), INVALID), (dict(kv_heads=65536), INVALID), (dict(head_dim=8), INVALID),
    (dict(head_dim=132), INVALID), (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(k=None), INVALID),
    (dict(k_out=None), INVALID), (dict(ldq=64), INVALID), (dict(hko=64), INVALID), (dict(ldqo=2560), INVALID),
    (dict(hko=256), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(cos_t=None), INVALID), (dict(sin_t=None), INVALID),
    (dict(rope_dim=0), INVALID), (dict(rope_dim=130), INVALID), (dict(rope_dim=63), INVALID),
    (dict(rope_dim=72, halves=1), INVALID), (dict(table_ld=63), INVALID), (dict(positions=0), INVALID),
    (dict(positions=1 << 31), INVALID), (dict(q=A + 8), MISALIGNED), (dict(q_out=A + 2), MISALIGNED),
    (dict(k=A + 8), MISALIGNED), (dict(k_out=A + 8), MISALIGNED), (dict(ldk=260), MISALIGNED),
    (dict(q_norm=A + 2), MISALIGNED), (dict(k_norm=A + 8), MISALIGNED), (dict(pos=A + 1), MISALIGNED),
    (dict(cos_t=A + 2), MISALIGNED)])
def test_heads_refusals(nv, bad, status):
    assert nv.lib().nvfp4_qk_norm_rope(heads(nv, **bad), None) == status


def test_heads_refuse_caches_that_do_not_fit(nv):
    L = nv.lib()
    c, c4, none = cache(nv)._obj, cache4(nv), cache(nv, pages=0)._obj
    ok = dict(slot=A, v=A, ldv=256, hv=128)
    assert L.nvfp4_qk_norm_rope(None, None) == INVALID
    for bad in (dict(), dict(cache=ctypes.addressof(c), cache4=ctypes.addressof(c4)),
                dict(cache=ctypes.addressof(c), v=None), dict(cache=ctypes.addressof(c), kv_heads=1),
                dict(cache=ctypes.addressof(c), kv_heads=0), dict(cache4=ctypes.addressof(c4), head_dim=64, rope_dim=64),
                dict(cache=ctypes.addressof(none))):
        assert L.nvfp4_qk_norm_rope(heads(nv, **{**ok, **bad}), None) == INVALID, bad
    for bad in (dict(slot=A + 2), dict(v=A + 8), dict(ldv=260)):
        assert L.nvfp4_qk_norm_rope(heads(nv, **{**ok, "cache": ctypes.addressof(c), **bad}), None) == MISALIGNED, bad


# ------------------------------------------------------------------- pages
B = [A + (i << 24) for i in range(1, 9)]          # addresses far from each other


def pages(nv, **f):
    d = dict(block_table=A, requests=4, table_cols=8, table_ld=8, ctx_len=B[0], page_size=16, pages=100)
    d.update(f)
    return ctypes.byref(nv._PagesC(**d))


PAGES_BAD = [(dict(block_table=None), INVALID), (dict(ctx_len=None), INVALID), (dict(requests=0), INVALID),
             (dict(requests=8193), INVALID), (dict(table_cols=0), INVALID), (dict(table_ld=7), INVALID),
             (dict(pages=0), INVALID), (dict(pages=(1 << 20) + 1), INVALID), (dict(page_size=8), INVALID),
             (dict(table_cols=1 << 27, table_ld=1 << 27), INVALID), (dict(block_table=A + 2), MISALIGNED),
             (dict(ctx_len=B[0] + 1), MISALIGNED)]


@pytest.mark.parametrize("bad,status", PAGES_BAD)
def test_page_table_refusals(nv, bad, status):
    L = nv.lib()
    assert L.nvfp4_pages_fork(pages(nv, **bad), B[1], B[2], 2, B[3], 10, None, None, B[4], B[5], None) == status
    assert L.nvfp4_pages_free(pages(nv, **bad), B[1], B[2], None, 0, None, None, None) == status


def test_fork_refusals(nv):
    L = nv.lib()
    call = lambda src=B[1], dst=B[2], n=2, free=B[3], count=10, cursor=None, out=None, cs=B[4], cd=B[5]: \
        L.nvfp4_pages_fork(pages(nv), src, dst, n, free, count, cursor, out, cs, cd, None)
    for bad in (dict(src=None), dict(dst=None), dict(n=-1), dict(n=5), dict(count=-1), dict(cs=None), dict(cd=None),
                dict(cs=B[1]), dict(cd=B[1] + 4), dict(cs=B[2]), dict(out=B[1]), dict(src=B[0]), dict(dst=A + 8),
                dict(cs=B[0] + 12), dict(out=B[0]), dict(free=A), dict(free=B[4]), dict(free=B[5] - 8),
                dict(cs=B[5] + 4), dict(out=B[4]), dict(out=B[3] + 36), dict(cursor=B[5]), dict(cursor=B[0] + 4),
                dict(cs=A + 8), dict(out=A)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(src=B[1] + 2), dict(dst=B[2] + 1), dict(free=B[3] + 2), dict(cursor=B[6] + 2), dict(out=B[6] + 2),
                dict(cs=B[4] + 2), dict(cd=B[5] + 2)):
        assert call(**bad) == MISALIGNED, bad
    assert L.nvfp4_pages_fork(None, B[1], B[2], 2, B[3], 10, None, None, B[4], B[5], None) == INVALID


def test_free_refusals(nv):
    L = nv.lib()
    call = lambda free=B[1], count=B[2], out=None, ld=8, ms=None, md=None: \
        L.nvfp4_pages_free(pages(nv), free, count, out, ld, ms, md, None)
    for bad in (dict(free=None), dict(count=None), dict(count=B[1] + 396), dict(free=A), dict(count=B[0]),
                dict(out=B[3]), dict(out=B[3], ms=B[4]), dict(out=B[3], ld=7, ms=B[4], md=B[5]),
                dict(out=A + 4, ms=B[4], md=B[5]), dict(out=A, ld=9, ms=B[4], md=B[5]),
                dict(out=B[3], ms=B[4], md=B[4] + 196), dict(out=B[3], ms=B[3], md=B[4]), dict(out=B[0], ms=B[4], md=B[5])):
        assert call(**bad) == INVALID, bad
    for bad in (dict(free=B[1] + 2), dict(count=B[2] + 1), dict(out=B[3] + 2, ms=B[4], md=B[5]),
                dict(out=B[3], ms=B[4] + 2, md=B[5])):
        assert call(**bad) == MISALIGNED, bad


def test_copy_refusals(nv):
    L = nv.lib()

    def call(n_planes=1, pages=100, src=B[1], dst=B[2], n=2, planes=True, **f):
        p = nv._PlaneC(**{**dict(base=A, page_bytes=4096, page_stride=4096), **f})
        return L.nvfp4_pages_copy(ctypes.byref(p) if planes else None, n_planes, pages, src, dst, n, None)
    for bad in (dict(planes=False), dict(n_planes=0), dict(pages=0), dict(pages=1 << 31), dict(n=-1), dict(n=1 << 31),
                dict(src=None), dict(dst=None), dict(base=None), dict(page_bytes=0), dict(page_stride=4080),
                dict(page_bytes=1 << 30, page_stride=1 << 30)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(base=A + 8), dict(page_bytes=4088), dict(page_stride=4104), dict(src=B[1] + 2), dict(dst=B[2] + 2)):
        assert call(**bad) == MISALIGNED, bad


def test_binding_checks_its_tensors(nv):
    u8 = lambda n: torch.zeros(2, 2, 16, n, dtype=torch.uint8)
    with pytest.raises(ValueError):
        nv.KVCache4(u8(32), u8(32), u8(4), u8(4), torch.ones(1), torch.ones(1))        # not CUDA tensors
    with pytest.raises(ValueError):
        nv.PageTable(torch.zeros(4, 8, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), 16, 10)
    with pytest.raises(ValueError):
        nv.nvfp4_qk_norm_rope(torch.zeros(4, 2, 64, dtype=torch.bfloat16), None)
    with pytest.raises(ValueError):
        nv.nvfp4_qk_norm_rope(None, None)
    with pytest.raises(ValueError):
        nv.nvfp4_pages_copy([], torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_attention_refusals(nv):
    from test_attn_host import IO_BAD, WORKSPACE, io
    L, c = nv.lib(), ctypes.byref(cache4(nv))
    for bad, status in CACHE4_BAD:
        assert L.nvfp4_attn_paged4(step(nv), io(nv), ctypes.byref(cache4(nv, **bad)), None, A, 1 << 40, None) == status, bad
    for bad, status in IO_BAD:
        assert L.nvfp4_attn_paged4(step(nv), io(nv, **bad), c, None, A, 1 << 40, None) == status, bad
    for bad in (dict(pages=11), dict(kv_heads=1), dict(head_dim=64), dict(k=None)):
        assert L.nvfp4_attn_paged4(step(nv), io(nv), c, cache(nv, **bad), A, 1 << 40, None) == INVALID, bad
    for s in (step(nv, page_size=0), step(nv, page_size=32), step(nv, heads=0), step(nv, kv_heads=1), None):
        assert L.nvfp4_attn_paged4(s, io(nv), c, None, A, 1 << 40, None) == INVALID
    assert L.nvfp4_attn_paged4(step(nv), None, c, None, A, 1 << 40, None) == INVALID
    assert L.nvfp4_attn_paged4(step(nv), io(nv), None, None, A, 1 << 40, None) == INVALID
    for ws, n, status in ((None, 1 << 40, WORKSPACE), (A, 16, WORKSPACE), (A + 128, 1 << 40, MISALIGNED)):
        assert L.nvfp4_attn_paged4(step(nv), io(nv), c, None, ws, n, None) == status


def test_packed_bytes_are_the_structures(nv):
    values = (1, 2, 3, 4, *range(5, 17), 17, 18, 1e-6, 19, 20, 21, 22, 23, 24, 1, 25, 26, 27, 28, 29, 30)
    assert nv._pack_heads(*values) == bytes(nv._HeadsC(*values))
    io = (1, 2, 3, 4, 5, 6, 7, 64, 0.25, 1)
    assert nv._pack_io(*io) == bytes(nv._AttnIOC(*io))
    assert nv._pack_plane(1, 2, 3) == bytes(nv._PlaneC(1, 2, 3))
