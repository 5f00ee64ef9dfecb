"""GPU tests of the head norms with rotation, and of rows into and out of the
4-bit cache."""
import numpy as np
import pytest
import torch

import oracle
import synthetic
from _gpu import dev, host
from _kv4 import decode, random_cache4
from test_gpu_attn import i32, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_block_scaled_device_gb300 as m
    return m


def tables(n, half, gen):
    angle = torch.rand(n, half, device="cuda", dtype=torch.float64, generator=gen) * 6.3
    return angle.cos().float(), angle.sin().float()


def reference(x, w, eps, pos, cos, sin, rd, halves):
    """float64 result and the magnitude that its binary32 errors scale with."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    mag, D = y.abs(), x.shape[-1]
    if pos is not None:
        p = pos.long().clamp(0, cos.shape[0] - 1)
        c, s = (t[p][:, None, :rd // 2].double() for t in (cos, sin))
        a, b = (slice(D - rd, D - rd // 2), slice(D - rd // 2, D)) if halves else \
            (slice(D - rd, D, 2), slice(D - rd + 1, D, 2))
        z = y.clone()
        z[..., a], z[..., b] = y[..., a] * c - y[..., b] * s, y[..., a] * s + y[..., b] * c
        m = mag.clone()
        m[..., a] = (y[..., a] * c).abs() + (y[..., b] * s).abs()
        m[..., b] = (y[..., a] * s).abs() + (y[..., b] * c).abs()
        y, mag = z, m
    return y, mag


def check(got, ref, mag):
    # 2^-8: the rounding to bf16, half a step.  In binary32: the sum of up to 128
    # squares (8 in a lane, 4 levels of lanes: 12 roundings, of positive terms),
    # the mean, + eps, the reciprocal square root (2 ulp), two products: below
    # 2^-20 of the normed value; the rotation adds two roundings of each product's
    # size: 2^-19 of the sum of magnitudes covers both, after the rounding 2^-18.
    err = (got.double() - ref).abs()
    bad = ~(err <= 2.0 ** -8 * ref.abs() + 2.0 ** -18 * mag + 1e-38)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("T,H,Hkv,D,rd,layout", [
    (1, 40, 8, 128, 128, "plain"), (1, 1, 1, 16, 16, "plain"), (7, 5, 3, 64, 32, "padded"),
    (33, 8, 1, 96, 96, "heads_first"), (130, 20, 20, 80, 48, "plain"), (3, 7, 2, 24, 16, "padded"),
    (2000, 40, 8, 128, 64, "plain"), (5, 3, 0, 128, 128, "plain"), (5, 0, 3, 40, 32, "plain")])
def test_norm_and_rotation(nv, T, H, Hkv, D, rd, layout, halves):
    gen = torch.Generator("cuda").manual_seed(T + D)
    q, k = (rows(gen, T, h, D, layout) if h else None for h in (H, Hkv))
    qn, kn = (torch.randn(D, device="cuda", generator=gen).bfloat16() for _ in range(2))
    cos, sin = tables(50, rd // 2, gen)
    pos = torch.randint(0, 50, (T,), device="cuda", generator=gen).int()
    out = [None if x is None else torch.full_like(x, 7.0) for x in (q, k)]
    nv.nvfp4_qk_norm_rope(q, k, qn, kn, pos, cos, sin, *out, halves=halves, eps=1e-5)
    for x, w, o in ((q, qn, out[0]), (k, kn, out[1])):
        if x is not None:
            check(o, *reference(x, w, 1e-5, pos, cos, sin, rd, halves))
    # in place, the same bits
    nv.nvfp4_qk_norm_rope(q, k, qn, kn, pos, cos, sin, halves=halves, eps=1e-5)
    for x, o in ((q, out[0]), (k, out[1])):
        assert x is None or torch.equal(x, o)
    assert nv.device_status() == 0


@pytest.mark.parametrize("rd", [2, 6, 30, 100, 126])
def test_interleaved_pairs_of_any_width(nv, rd):
    gen = torch.Generator("cuda").manual_seed(rd)
    q, k = rows(gen, 9, 4, 128, "plain"), rows(gen, 9, 2, 128, "plain")
    cos, sin = tables(20, rd // 2 + 3, gen)                   # (an odd pitch, wider than needed)
    pos = torch.arange(9, device="cuda").int()
    want = [reference(x, w, 1e-6, pos, cos, sin, rd, False) for x, w in ((q, None), (k, None))]
    head = q[..., :128 - rd].clone()
    nv.nvfp4_qk_norm_rope(q, k, None, None, pos, cos, sin, rope_dim=rd)
    check(q, *want[0])
    check(k, *want[1])
    assert torch.equal(q[..., :128 - rd], head)               # columns that are not rotated: bit for bit


def test_one_of_the_norms_and_no_rotation(nv):
    gen = torch.Generator("cuda").manual_seed(5)
    q, k = rows(gen, 40, 6, 64, "plain"), rows(gen, 40, 2, 64, "plain")
    q[3, 2] = 0                                               # a row of zeros stays one
    w = torch.randn(64, device="cuda", generator=gen).bfloat16()
    for qn, kn in ((w, None), (None, w), (None, None)):
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        nv.nvfp4_qk_norm_rope(q, k, qn, kn, q_out=qo, k_out=ko)
        for x, n, o in ((q, qn, qo), (k, kn, ko)):
            if n is None:
                assert torch.equal(o, x)
            else:
                check(o, *reference(x, n, 1e-6, None, None, None, 0, False))
    assert (qo[3, 2] == 0).all()


def test_values_that_are_not_finite_stay_in_their_row(nv):
    gen = torch.Generator("cuda").manual_seed(6)
    q, k = rows(gen, 12, 8, 128, "plain"), rows(gen, 12, 4, 128, "plain")
    w = torch.ones(128, device="cuda").bfloat16()
    cos, sin = tables(12, 64, gen)
    pos = torch.arange(12, device="cuda").int()
    clean = torch.empty_like(q)
    nv.nvfp4_qk_norm_rope(q, k, w, w, pos, cos, sin, q_out=clean, k_out=torch.empty_like(k))
    q[4, 3, 17], q[9, 0, 5] = float("nan"), float("inf")
    got = torch.empty_like(q)
    nv.nvfp4_qk_norm_rope(q, k, w, w, pos, cos, sin, q_out=got, k_out=torch.empty_like(k))
    same = torch.ones(12, 8, dtype=torch.bool, device="cuda")
    same[4, 3] = same[9, 0] = False
    assert torch.equal(got[same], clean[same]) and got[4, 3].isnan().all() and got[9, 0].isnan().any()


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("D,rd", [(128, 64), (96, 32), (64, 48), (128, 128)])
def test_an_infinity_in_a_normed_row(nv, D, rd, halves):
    """Its row's mean is infinite: the row becomes 0, NaN at the infinity and, among the
    rotated columns, at its partner; columns that are not rotated keep their zeros' signs."""
    gen = torch.Generator("cuda").manual_seed(D + rd)
    q = rows(gen, 2 * D, 3, D, "plain")
    w = (1 + torch.rand(D, device="cuda", generator=gen)).bfloat16()
    cos, sin = tables(2 * D, rd // 2, gen)
    pos, at = torch.arange(2 * D, device="cuda").int(), torch.arange(D, device="cuda")
    q[at, 1, at], q[D + at, 2, at] = float("inf"), -float("inf")
    q[:, 0, :D - rd] = -0.0
    rot0, half = D - rd, rd // 2
    mate = torch.where(at < rot0, at, torch.where(at < rot0 + half, at + half, at - half) if halves else at ^ 1)
    nan = torch.zeros(q.shape, dtype=torch.bool, device="cuda")
    for first, head in ((0, 1), (D, 2)):
        nan[first + at, head, at] = nan[first + at, head, mate] = True
    gone = torch.zeros(2 * D, 3, dtype=torch.bool, device="cuda")
    gone[:D, 1] = gone[D:, 2] = True
    out = torch.empty_like(q)
    nv.nvfp4_qk_norm_rope(q, None, w, None, pos, cos, sin, q_out=out, halves=halves)
    assert torch.equal(out.isnan(), nan)
    assert ((out == 0) | nan)[gone].all()
    assert (out[:, 0, :rot0].view(torch.int16) == -2 ** 15).all()


@pytest.mark.parametrize("halves", [None, False, True])
@pytest.mark.parametrize("D,rd", [(128, 128), (128, 64), (80, 48)])
def test_rows_whose_squares_are_beyond_binary32(nv, D, rd, halves):
    """Their mean is infinite in binary32, 1 / rms is 0 and so are they, whatever the weights."""
    gen = torch.Generator("cuda").manual_seed(D + rd)
    q = rows(gen, 9, 4, D, "plain")
    w = (1 + 99 * torch.rand(D, device="cuda", generator=gen)).bfloat16()
    big = (1 + torch.rand(5, D, device="cuda", generator=gen)) * torch.tensor([1e19, 1e25, 1e37, 1.2e38, 1.6e38], device="cuda")[:, None]
    q[2:7, 1], q[2:7, 3] = big.bfloat16(), -big.bfloat16()
    cos, sin = tables(9, rd // 2, gen)
    pos = torch.arange(9, device="cuda").int()
    out = torch.empty_like(q)
    rope = {} if halves is None else dict(pos=pos, cos_t=cos, sin_t=sin, halves=halves)
    nv.nvfp4_qk_norm_rope(q, None, w, None, q_out=out, **rope)
    assert (out[2:7, 1] == 0).all() and (out[2:7, 3] == 0).all()
    q[2:7, 1], q[2:7, 3] = 1, 1
    other = torch.empty_like(q)
    nv.nvfp4_qk_norm_rope(q, None, w, None, q_out=other, **rope)
    assert torch.equal(out[:, ::2], other[:, ::2]) and torch.equal(out[:2], other[:2]) and torch.equal(out[7:], other[7:])


def test_rotation_is_that_of_the_projection(nv):
    """Without norms: nvfp4_gemm then this, bit for bit nvfp4_gemm_rope."""
    ws = nv.workspace(256)
    T, D, H, Hkv = 37, 128, 3, 1
    x = nv.quantize_new(dev(synthetic.activations(T, seed=3, h=256)), ws)
    w = nv.quantize_new(dev(synthetic.weight(4, (H + 2 * Hkv) * D, 256)), ws)
    cos, sin = (torch.from_numpy(t).cuda() for t in synthetic.rope_tables(40, 64))
    pos = i32([(7 * t) % 40 for t in range(T)])
    plain, fused = (torch.empty((T, (H + 2 * Hkv) * D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    nv.nvfp4_gemm(x, w, plain)
    nv.nvfp4_gemm_rope(x, w, fused, pos, cos, sin, 0, H + Hkv, D, 64)
    heads = plain.view(T, -1, D)
    nv.nvfp4_qk_norm_rope(heads[:, :H], heads[:, H:H + Hkv], None, None, pos, cos, sin)
    assert torch.equal(plain, fused)


@pytest.mark.parametrize("halves", [False, True])
def test_positions_outside_the_tables(nv, halves):
    gen = torch.Generator("cuda").manual_seed(7)
    q, k = rows(gen, 4, 2, 64, "plain"), rows(gen, 4, 1, 64, "plain")
    cos, sin = tables(10, 32, gen)
    pos = i32([-5, 9, 10, 2 ** 31 - 1])
    ref = reference(q, None, 0, pos, cos, sin, 64, halves)
    nv.device_status()
    nv.nvfp4_qk_norm_rope(q, k, None, None, pos, cos, sin, halves=halves)
    check(q, *ref)
    assert nv.device_status() == 100 + 33


# ------------------------------------------------------------- the 4-bit cache
def plan_of(nv, lens, ctx, heads, kv_heads, page, pages, window=0, pad=0, cols=None):
    """A plan whose block table scatters the requests over the pages."""
    need = [-(-(c + n) // page) for c, n in zip(ctx, lens)]
    rng = np.random.default_rng(sum(need) + page)
    ids = rng.permutation(pages)[:sum(need)]
    table, at = np.full((len(lens), cols or max(max(need), 1)), -1, np.int32), 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += n
    plan = nv.AttnPlan(len(lens), sum(lens) + pad, heads, kv_heads, page_size=page,
                       block_table=torch.from_numpy(table).cuda(), window=window)
    nv.nvfp4_attn_plan(plan, i32(lens), i32(ctx))
    return plan


def pages_apart(nv, cache, gap=2):
    """The same cache with other memory between its pages."""
    wide = lambda t: t.new_empty((t.shape[0], gap, *t.shape[1:])).random_(0, 256)[:, 0].copy_(t)
    return nv.KVCache4(wide(cache.k), wide(cache.v), wide(cache.k_sf), wide(cache.v_sf), cache.k_g, cache.v_g)


@pytest.mark.parametrize("page,Hkv,D,g,apart", [(16, 8, 128, 2.0 ** -6, False), (64, 1, 64, 0.0123, False),
                                                (32, 3, 96, 2.0 ** -9, True), (128, 2, 16, 1.7, False),
                                                (16, 5, 80, 3e-4, True)])
def test_append4_is_the_quantizer(nv, page, Hkv, D, g, apart):
    """Codes and scales bit for bit the oracle's; every other byte of the cache untouched."""
    lens, ctx = [40, 1, 0, 13], [5, 100, 3, 16]
    gen = torch.Generator("cuda").manual_seed(page + D)
    cache = random_cache4(nv, gen, 40, Hkv, page, D, g, 2 * g)
    cache = pages_apart(nv, cache) if apart else cache
    plan = plan_of(nv, lens, ctx, Hkv, Hkv, page, 40, pad=2)
    T = plan.tokens
    k, v = (rows(gen, T, Hkv, D, "padded") for _ in range(2))
    k[3, 0] = 0                                               # blocks of zeros
    k[4] *= 1000                                              # beyond what the scales reach
    v[5] *= 1e-6                                              # below it
    v[6, :, 0] = -0.0
    k[7, 0, 1:16] = torch.tensor([0.25, -0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.0, -0.0, 0.24, 0.26, -5.1, 4.9, 0.5])
    old = [t.clone() for t in (cache.k, cache.v, cache.k_sf, cache.v_sf)]
    nv.nvfp4_kv4_append(k, v, plan, cache)
    slots = plan.slot.tolist()
    for x, gg, codes, sf, oc, osf in ((k, g, cache.k, cache.k_sf, *old[0::2]), (v, 2 * g, cache.v, cache.v_sf, *old[1::2])):
        c, s = oracle.quantize(host(x.reshape(T * Hkv, D)), np.float32(gg))
        c, s = c.reshape(T, Hkv, D // 2), s.reshape(T, Hkv, D // 16)
        for t, sl in enumerate(slots):
            if sl >= 0:
                oc[sl // page, :, sl % page] = torch.from_numpy(c[t]).cuda()
                osf[sl // page, :, sl % page] = torch.from_numpy(s[t]).cuda()
        assert torch.equal(codes, oc) and torch.equal(sf, osf)
    assert nv.device_status() == 0


def test_append4_of_values_that_are_not_finite(nv):
    cache = random_cache4(nv, torch.Generator("cuda").manual_seed(1), 2, 1, 16, 64, 1.0, 1.0)
    plan = plan_of(nv, [3], [0], 1, 1, 16, 2)
    k = torch.ones(3, 1, 64, device="cuda", dtype=torch.bfloat16)
    k[0, 0, 3], k[1, 0, 17], k[2, 0, 40] = float("nan"), float("inf"), -float("inf")
    nv.nvfp4_kv4_append(k, k, plan, cache)
    at = plan.slot.tolist()
    x = decode(cache.k, cache.k_sf)[:, 0]
    row = lambda t: x[at[t] // 16, at[t] % 16]
    one = 6 * 0.171875                                        # a block of ones: the scale is E4M3(1 / 6), the codes 6
    assert row(0)[:16].isnan().all() and (row(0)[16:] == one).all()
    assert row(1)[17] == 2688 and (row(1)[18:32] == 0).all() and (row(1)[32:] == one).all()
    assert row(2)[40] == -2688


@pytest.mark.parametrize("with_heads", [False, True])
@pytest.mark.parametrize("D", [128, 80])
@pytest.mark.parametrize("g", [1.0, 2.0 ** -6, 2.0 ** -11, 0.0123, 2.0 ** -80, 2.0 ** 90, 2.0 ** 115])
def test_append4_of_infinities_and_the_largest_numbers(nv, g, D, with_heads):
    """Whatever the global scale, infinities are the largest bf16 number and what the
    scales do not reach saturates, bit for bit the oracle's; NaN stays in its block."""
    T, Hkv, page, inf = 9, 3, 16, float("inf")
    gen = torch.Generator("cuda").manual_seed(D)
    cache = random_cache4(nv, gen, 4, Hkv, page, D, g, g)
    plan = plan_of(nv, [T], [2], Hkv, Hkv, page, 4)
    x = torch.randn(T, Hkv, D, device="cuda", generator=gen).bfloat16() * min(g, 2.0 ** 100) * 3
    most = torch.finfo(torch.bfloat16).max
    x[0, 0, 5], x[1, 1, 20], x[2, 2, 63] = inf, -inf, most
    x[3, 0, 16:32] = torch.tensor([inf, -inf, most, -most, 1e38, -1e37, 1e36, -1e30, 1e20, 1.0, -1.0, 0.0, -0.0, 1e-3, 1e-30, -1e35])
    x[4, :, ::16], x[5, :, 3::16], x[6] = 1e36, -inf, inf
    x[7, 1, 33], x[7, 1, 34], x[8, 0, 0] = float("nan"), inf, 1e38
    y = x.flip(0).neg().contiguous()                          # (the values: other blocks)
    if with_heads:
        out = torch.empty_like(x)
        nv.nvfp4_qk_norm_rope(None, x, k_out=out, v=y, plan=plan, cache=cache)
        assert torch.equal(out.view(torch.int16), x.view(torch.int16))
    else:
        nv.nvfp4_kv4_append(x, y, plan, cache)
    at = plan.slot.long()
    for rows_in, codes, sf in ((x, cache.k, cache.k_sf), (y, cache.v, cache.v_sf)):
        nan = rows_in.view(T, Hkv, D // 16, 16).isnan().any(-1).cpu()
        c, s = oracle.quantize(host(rows_in.clamp(-most, most).nan_to_num().reshape(T * Hkv, D)), np.float32(g))
        c, s = (torch.from_numpy(z).view(T, Hkv, D // 16, -1).clone() for z in (c, s))
        c[nan], s[nan] = 0, 0x7f
        assert int(nan.sum()) == 1
        assert torch.equal(codes[at // page, :, at % page].cpu().view(T, Hkv, D // 16, 8), c)
        assert torch.equal(sf[at // page, :, at % page].cpu().view(T, Hkv, D // 16, 1), s)


def test_slots_outside_the_cache_are_reported(nv):
    cache = random_cache4(nv, torch.Generator("cuda").manual_seed(2), 2, 2, 16, 64)
    plan = nv.AttnPlan(1, 4, 2, 2, page_size=16, block_table=1)
    old = cache.k.clone()
    x = torch.randn(4, 2, 64, device="cuda").bfloat16()
    for slots, status in (([-1, -1, -1, -1], 0), ([32, -1, -1, -1], 132), ([-2, -1, 2 ** 31 - 1, -1], 132)):
        plan.slot.copy_(i32(slots))
        nv.nvfp4_kv4_append(x, x, plan, cache)
        assert nv.device_status() == status and torch.equal(cache.k, old)


@pytest.mark.parametrize("window", [0, 1, 20])
@pytest.mark.parametrize("page,Hkv,D,k_g,apart", [(16, 8, 128, 2.0 ** -6, False), (32, 2, 96, 0.0123, True),
                                                  (128, 1, 64, 2.0 ** -3, False)])
def test_expand(nv, page, Hkv, D, k_g, apart, window):
    """The rows that a new token sees, in bf16; no other row is touched."""
    lens, ctx = [1, 0, 17, 3], [200, 50, 0, 33]
    gen = torch.Generator("cuda").manual_seed(page + window)
    cache = random_cache4(nv, gen, 60, Hkv, page, D, k_g)
    cache = pages_apart(nv, cache) if apart else cache
    plan = plan_of(nv, lens, ctx, Hkv, Hkv, page, 60, window=window)
    plan.block_table[3, 0] = 60                               # no page of the cache: left out
    out = nv.KVCache(*(torch.full((60, 2, Hkv, page, D), 7.0, device="cuda").bfloat16()[:, 0] for _ in range(2)))
    want = [out.k.clone(), out.v.clone()]
    for x, (codes, sf, g) in enumerate(((cache.k, cache.k_sf, cache.k_g), (cache.v, cache.v_sf, cache.v_g))):
        val = (decode(codes, sf).float() * g).bfloat16()
        for r, (n, c) in enumerate(zip(lens, ctx)):
            for p in range(max(0, c - window + 1) if window else 0, c + n if n else 0):
                pg = int(plan.block_table[r, p // page])
                if pg < 60:
                    want[x][pg, :, p % page] = val[pg, :, p % page]
    nv.nvfp4_kv4_expand(cache, plan, out)
    assert torch.equal(out.k, want[0]) and torch.equal(out.v, want[1])


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("T,H,Hkv,D,page", [(1, 40, 8, 128, 16), (19, 3, 3, 96, 32), (300, 8, 2, 64, 64)])
def test_into_a_cache_in_the_same_pass(nv, T, H, Hkv, D, page, four):
    """Bit for bit the pass and the append after it; q alike, k_out as well where asked for."""
    gen = torch.Generator("cuda").manual_seed(T)
    qkv = rows(gen, T + 1, H + 2 * Hkv, D, "plain")
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    qn, kn = (torch.randn(D, device="cuda", generator=gen).bfloat16() for _ in range(2))
    cos, sin = tables(T + 1, D // 2, gen)
    plan = plan_of(nv, [T], [3], H, Hkv, page, 30, pad=1)
    caches = []
    for _ in range(3):
        g = torch.Generator("cuda").manual_seed(1)
        caches.append(random_cache4(nv, g, 30, Hkv, page, D, 0.01, 0.02) if four else
                      nv.KVCache(*(torch.randn(30, Hkv, page, D, device="cuda", generator=g).bfloat16() for _ in range(2))))
    pos = torch.arange(T + 1, device="cuda").int()
    qo, ko, q2, k2 = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q), torch.empty_like(k)
    nv.nvfp4_qk_norm_rope(q, k, qn, kn, pos, cos, sin, q_out=qo, k_out=ko)
    (nv.nvfp4_kv4_append if four else nv.nvfp4_kv_append)(ko, v, plan, caches[0])
    nv.nvfp4_qk_norm_rope(q, k, qn, kn, pos, cos, sin, q_out=q2, v=v, plan=plan, cache=caches[1])
    nv.nvfp4_qk_norm_rope(q, k, qn, kn, pos, cos, sin, q_out=q2, k_out=k2, v=v, plan=plan, cache=caches[2])
    assert torch.equal(qo, q2) and torch.equal(ko, k2)
    for c in caches[1:]:
        assert torch.equal(c.k, caches[0].k) and torch.equal(c.v, caches[0].v)
        if four:
            assert torch.equal(c.k_sf, caches[0].k_sf) and torch.equal(c.v_sf, caches[0].v_sf)
    assert nv.device_status() == 0


def test_on_another_stream_and_captured(nv):
    gen = torch.Generator("cuda").manual_seed(9)
    q, k = rows(gen, 8, 4, 64, "plain"), rows(gen, 8, 2, 64, "plain")
    w = torch.randn(64, device="cuda", generator=gen).bfloat16()
    cos, sin = tables(8, 32, gen)
    pos = torch.arange(8, device="cuda").int()
    want, got, ko = torch.empty_like(q), torch.empty_like(q), torch.empty_like(k)
    call = lambda out, stream=None: nv.nvfp4_qk_norm_rope(q, k, w, w, pos, cos, sin, q_out=out, k_out=ko, stream=stream)
    call(want)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        call(got)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    got.zero_()
    torch.cuda.synchronize()
    call(got, stream)
    stream.synchronize()
    assert torch.equal(got, want)


def test_refusals(nv):
    x = torch.zeros(4, 2, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(64, device="cuda", dtype=torch.bfloat16)
    cos = torch.zeros(8, 32, device="cuda")
    pos = i32([0, 1, 2, 3])
    cache = random_cache4(nv, torch.Generator("cuda").manual_seed(1), 4, 2, 16, 64)
    plan = nv.AttnPlan(1, 4, 2, 2, page_size=16, block_table=1)
    for bad in (dict(q=x.float()), dict(q=x.cpu()), dict(q=x.transpose(1, 2)), dict(q_norm=w[:32]),
                dict(q_norm=w.float()), dict(pos=pos.long()), dict(pos=pos[:3]), dict(cos_t=cos[:4]),
                dict(sin_t=cos.double()), dict(rope_dim=66), dict(q_out=x[:3]), dict(v=x), dict(cache=cache),
                dict(v=x, cache=cache), dict(v=x[:3], cache=cache, plan=plan), dict(k=None, v=x, cache=cache, plan=plan),
                dict(v=x, cache=cache, plan=nv.AttnPlan(1, 5, 2, 2, page_size=16, block_table=1)),
                dict(v=x, cache=cache, plan=nv.AttnPlan(1, 4, 2, 2, page_size=32, block_table=1)),
                dict(v=x, cache=cache, plan=nv.AttnPlan(1, 4, 2, 2))):
        args = dict(q=x, k=x, q_norm=w, k_norm=w, pos=pos, cos_t=cos, sin_t=cos)
        args.update(bad)
        with pytest.raises(ValueError):
            nv.nvfp4_qk_norm_rope(**args)
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_qk_norm_rope(x, x, w, w, pos, cos, cos, rope_dim=24, halves=True)
    one = cos[:1].expand(8, 32)                               # rows that are one: no table of 8
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_qk_norm_rope(x, x, w, w, pos, one, one)
    with pytest.raises(ValueError):
        nv.nvfp4_kv4_append(x, x[:3], plan, cache)
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_kv4_expand(cache, plan, nv.KVCache.empty(5, 2, 16, 64))


def test_cache_whose_offsets_pass_32_bits(nv):
    """Pages 1 GB apart: rows behind 4 GB are written, expanded, attended and copied as others."""
    Hkv, page, D, T, pages = 2, 16, 64, 75, 7
    gen = torch.Generator("cuda").manual_seed(9)
    far, stride = [], 10 ** 9
    for n in (D // 2, D // 2, D // 16, D // 16):
        flat = torch.empty((pages - 1) * stride + Hkv * page * n, dtype=torch.uint8, device="cuda")
        far.append(flat.as_strided((pages, Hkv, page, n), (stride, page * n, n, 1)))
    assert (pages - 2) * stride > 2 ** 32
    near = nv.KVCache4.empty(pages, Hkv, page, D)
    far = nv.KVCache4(*far, near.k_g, near.v_g)
    plan = plan_of(nv, [T], [0], 4, Hkv, page, pages)
    plan.block_table[0, :5] = i32([6, 1, 5, 0, 4])
    nv.nvfp4_attn_plan(plan, i32([T]), i32([0]))
    q = torch.randn(T, 4, D, device="cuda", generator=gen).bfloat16()
    k, v = (torch.randn(T, Hkv, D, device="cuda", generator=gen).bfloat16() for _ in range(2))
    ws, got = nv.workspace(nv.attn_workspace_bytes()), []
    for cache in (near, far):
        nv.nvfp4_kv4_append(k, v, plan, cache)
        nv.nvfp4_qk_norm_rope(None, k[:, :, :].clone(), v=v, plan=plan, cache=cache)
        nv.nvfp4_pages_copy(cache, i32([6, 5]), i32([3, 2]))
        out, rows = torch.empty_like(q), nv.KVCache(*(torch.zeros(pages, Hkv, page, D, device="cuda").bfloat16() for _ in range(2)))
        nv.nvfp4_attn_paged4(q, cache, plan, out, ws)
        nv.nvfp4_kv4_expand(cache, plan, rows)
        got.append((out, rows.k, rows.v, *(x[[6, 1, 5, 0, 3, 2]] for x in (cache.k, cache.v, cache.k_sf, cache.v_sf))))
    assert nv.device_status() == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert (got[0][0].float().abs().sum() > 0) and torch.equal(far.k[3], far.k[6])
