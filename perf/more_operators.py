"""Operators of a serving layer around its cache, measured: norms of query and
key heads with the rotation in the same pass (``qk``), new rows into a cache
held in 4 bits and the rows of a step out of it (``cache4``), attention over
that cache (``attn4``), forked requests (``fork``), and pages that come free,
with the others moved together (``free``).

``run`` computes each either in its plain form (elementary torch operations in
32 bits) or, where ``own`` is true, by the calls a user makes of this package.
Head layouts are the package's own QKV width of 7168 (40 query, 8 key and 8
value heads of 128 columns) and generic ones.

The 4-bit cache: E2M1 codes, two to a byte, the even column in the low half;
an E4M3 scale for each 16 columns of a row; one binary32 scale for all keys and
one for all values, powers of two here, so that no rounding depends on them.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6


# --------------------------------------------------------------------- cases
def listed():
    layer = {"heads": 40, "kv_heads": 8, "head_dim": 128}
    return [
        # the query and key heads of a small decode step: latency
        {"name": "qk_decode_8", "op": "qk", "requests": 8, "q_lo": 1, "q_hi": 1, "ctx_lo": 100, "ctx_hi": 5000,
         "page": 0, "rope_dim": 64, "halves": False, **layer},
        # five long prompts in one go, keys and values straight into the (bf16) cache
        {"name": "qk_prompt_16272", "op": "qk", "requests": 5, "q_lo": 1000, "q_hi": 6600, "ctx_lo": 0, "ctx_hi": 77,
         "page": 64, "rope_dim": 128, "halves": True, **layer},
        # a decode step's rows into the 4-bit cache, and its requests' rows out of it
        {"name": "cache4_17", "op": "cache4", "requests": 17, "q_lo": 1, "q_hi": 1, "ctx_lo": 10, "ctx_hi": 1000,
         "page": 16, "window": 0, **layer},
        # the same for five long prompts: what their attention is given
        {"name": "cache4_16272", "op": "cache4", "requests": 5, "q_lo": 1000, "q_hi": 6600, "ctx_lo": 0, "ctx_hi": 77,
         "page": 64, "window": 0, **layer},
        # a single user's next token
        {"name": "attn4_decode_1", "op": "attn4", "requests": 1, "q_lo": 1, "q_hi": 1, "ctx_lo": 333, "ctx_hi": 333,
         "page": 16, "window": 0, **layer},
        # a decode step of 64 users with uneven contexts
        {"name": "attn4_decode_64", "op": "attn4", "requests": 64, "q_lo": 1, "q_hi": 1, "ctx_lo": 200,
         "ctx_hi": 8192, "page": 16, "window": 0, **layer},
        # two users deep in long contexts: few rows, a long axis
        {"name": "attn4_long_2", "op": "attn4", "requests": 2, "q_lo": 1, "q_hi": 1, "ctx_lo": 65537,
         "ctx_hi": 131071, "page": 64, "window": 0, **layer},
        # the last 1024-token ubatch of a 16384-token prompt
        {"name": "attn4_chunk_1024", "op": "attn4", "requests": 1, "q_lo": 1024, "q_hi": 1024, "ctx_lo": 15360,
         "ctx_hi": 15360, "page": 64, "window": 0, **layer},
        # one prompt answered eight times over: its last page copied in each of four layers' caches
        {"name": "fork_8", "op": "fork", "requests": 1, "children": 8, "ctx_lo": 777, "ctx_hi": 777, "page": 16,
         "kv_heads": 8, "head_dim": 128, "layers": 4},
        # beams of 8 for each of 64 users
        {"name": "fork_512", "op": "fork", "requests": 64, "children": 8, "ctx_lo": 200, "ctx_hi": 8192, "page": 16,
         "kv_heads": 8, "head_dim": 128, "layers": 1},
        # the free list after some of a server's requests have ended
        {"name": "free_64", "op": "free", "requests": 64, "ended": 9, "ctx_lo": 100, "ctx_hi": 4096, "page": 16,
         "kv_heads": 8, "head_dim": 128, "compact": False},
        # a large server's cache moved together, to give its end back
        {"name": "compact_400", "op": "free", "requests": 400, "ended": 90, "ctx_lo": 20, "ctx_hi": 4096, "page": 16,
         "kv_heads": 8, "head_dim": 128, "compact": True},
    ]


def _log_int(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "cache4", "attn4", "attn4", "attn4", "fork", "free"])
    page = rng.choice([16, 32, 64, 128])
    heads, kv_heads = rng.choice([(40, 8), (20, 4), (64, 8), (20, 20), (8, 1), (28, 4)])
    dim = rng.choice([64, 128, 128, 96])
    window = rng.choice([0, 0, 0, _log_int(rng, 16, 4000)])
    if op in ("qk", "cache4"):
        requests = _log_int(rng, 1, 64)
        q = _log_int(rng, 1, 14000 // requests)
        case = {"op": op, "requests": requests, "q_lo": max(1, q // 3), "q_hi": q, "ctx_lo": rng.randint(0, 40),
                "ctx_hi": rng.randint(50, 700), "page": page, "heads": heads, "kv_heads": kv_heads, "head_dim": dim}
        if op == "cache4":
            return dict(case, window=window)
        if rng.random() < 0.5:
            case["page"] = 0                         # no cache: the rotated keys go out
        return dict(case, rope_dim=rng.choice([dim, dim // 2, 32]), halves=rng.choice([False, True]))
    if op == "fork":
        requests = _log_int(rng, 1, 64)
        return {"op": op, "requests": requests, "children": rng.randint(1, 8), "ctx_lo": rng.randint(0, 100),
                "ctx_hi": _log_int(rng, 120, 5000), "page": page, "kv_heads": rng.choice([1, 4, 8]),
                "head_dim": dim, "layers": rng.choice([1, 2]) if requests < 30 else 1}
    if op == "free":
        requests = _log_int(rng, 1, 2000)
        return {"op": op, "requests": requests, "ended": rng.randint(0, requests // 2),
                "ctx_lo": rng.randint(0, 100), "ctx_hi": _log_int(rng, 120, 600000 // requests if requests > 120 else 5000),
                "page": page, "kv_heads": rng.choice([1, 4, 8]), "head_dim": dim, "compact": rng.random() < 0.5}
    kind = rng.choice(["decode", "decode", "chunk", "mixed"])
    if kind == "decode":
        requests = _log_int(rng, 1, 128)
        hi = _log_int(rng, 40, min(100000, 1600000 // (requests * kv_heads)))
        lo, q_lo, q_hi = max(1, hi // rng.choice([1, 4, 30])), 1, rng.choice([1, 1, 1, 4])
    elif kind == "chunk":
        requests, q_lo = 1, _log_int(rng, 16, 1000)
        q_hi, lo = q_lo, _log_int(rng, 1, 14000)
        hi = lo
    else:
        requests, q_lo, q_hi = rng.randint(2, 24), 1, _log_int(rng, 20, 120)
        hi = _log_int(rng, 100, 4000)
        lo = max(1, hi // 10)
    return {"op": op, "requests": requests, "q_lo": q_lo, "q_hi": q_hi, "ctx_lo": lo, "ctx_hi": hi, "page": page,
            "window": window, "heads": heads, "kv_heads": kv_heads, "head_dim": dim}


def _spread(lo, hi, n, phase):
    """n whole numbers spread over lo..hi (over their logarithm), in a scattered order."""
    if lo == hi:
        return [lo] * n
    a, b = math.log(lo + 1), math.log(hi + 1)
    return [int(round(math.exp(a + (b - a) * ((i * 0.6180339887 + phase) % 1.0)) - 1)) for i in range(n)]


def _lengths(case):
    """(cached tokens, new tokens) of each request."""
    n = case["requests"]
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], n, 0.37)
    return ctx, _spread(case["q_lo"], case["q_hi"], n, 0.11) if "q_lo" in case else [0] * n


# -------------------------------------------------------------------- inputs
def _normal(gen, *shape, std=1.0):
    return (torch.randn(shape, device=DEV, dtype=torch.float32, generator=gen) * std).to(torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _cache(gen, pages, heads, page, dim):
    """A bf16 cache in use: keys or values of a few units."""
    return _normal(gen, pages, heads, page, dim, std=1.5)


def _cache4(gen, pages, heads, page, dim, g):
    """The same held in 4 bits: codes and scales."""
    codes = torch.empty(pages, heads, page, dim // 2, dtype=torch.uint8, device=DEV)
    sf = torch.empty(pages, heads, page, dim // 16, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (heads * page * dim))
    for i in range(0, pages, step):
        codes[i:i + step], sf[i:i + step] = _quantize(_cache(gen, min(step, pages - i), heads, page, dim), g)
    return codes, sf


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    op = case["op"]
    s = {"op": op, "case": case}
    if op in ("fork", "free"):
        (_prepare_fork if op == "fork" else _prepare_free)(s, case, gen, rng)
        if own:
            _own_pages(s)
        return s
    ctx, q = _lengths(case)
    R, T = len(ctx), sum(q)
    H, Hkv, D, P = case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    s.update({"R": R, "T": T, "H": H, "Hkv": Hkv, "D": D, "page": P, "window": case.get("window", 0),
              "ctx_len": _ints(ctx), "q_len": _ints(q), "cu_q": _ints(np.concatenate([[0], np.cumsum(q)])),
              "kv_len": _ints([c + n for c, n in zip(ctx, q)]), "q_max": max(q),
              "kv_max": max(c + n for c, n in zip(ctx, q))})
    # the projection's output: query, key and value heads side by side
    qkv = _normal(gen, T, H + 2 * Hkv, D, std=1.5)
    s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    if P:                                            # pages scattered over the cache, three of them free
        need = [-(-(c + n) // P) for c, n in zip(ctx, q)]
        pages = sum(need) + 3
        ids = rng.permutation(pages)
        table, at = np.full((R, max(need)), -1, np.int32), 0
        for r, n in enumerate(need):
            table[r, :n] = ids[at:at + n]
            at += n
        s["table"] = torch.from_numpy(table).to(DEV)
    s["pos"], s["slot"] = _positions(s)
    if op == "qk":
        half = case["rope_dim"] // 2
        angle = torch.arange(s["kv_max"], dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(half, dtype=torch.float64) / half)
        s["cos"], s["sin"] = angle.cos().float().to(DEV), angle.sin().float().to(DEV)
        s["q_norm"], s["k_norm"] = (1 + _normal(gen, D, std=0.2).float()).to(torch.bfloat16), _normal(gen, D)
        s["rope_dim"], s["halves"] = case["rope_dim"], case["halves"]
        s["q_out"] = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
        if P:
            s["kc"], s["vc"] = (_cache(gen, pages, Hkv, P, D) for _ in range(2))
        else:
            s["k_out"] = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV)
    else:
        s["k_g"], s["v_g"] = 2.0 ** -6, 2.0 ** -7
        s["k_codes"], s["k_sf"] = _cache4(gen, pages, Hkv, P, D, s["k_g"])
        s["v_codes"], s["v_sf"] = _cache4(gen, pages, Hkv, P, D, s["v_g"])
        if op == "cache4":
            s["kx"], s["vx"] = (torch.zeros(pages, Hkv, P, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        else:
            s["out"] = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
            s["lse"] = torch.empty(T, H, dtype=torch.float32, device=DEV)
    if own:
        _own_step(s)
    return s


def _positions(s):
    """Position and cache slot of each packed row."""
    request = torch.repeat_interleave(torch.arange(s["R"], device=DEV), s["q_len"], output_size=s["T"])
    pos = torch.arange(s["T"], device=DEV, dtype=torch.int32) - s["cu_q"][request] + s["ctx_len"][request]
    if not s["page"]:
        return pos, None
    return pos, s["table"][request, pos // s["page"]] * s["page"] + pos % s["page"]


def _prepare_fork(s, case, gen, rng):
    """Rows of a server's table: parents in use, room for their children."""
    ctx, _ = _lengths(case)
    P, n = case["page"], len(ctx) * case["children"]
    need = [-(-c // P) for c in ctx]
    pages = sum(need) + n + 3
    ids = rng.permutation(pages).astype(np.int32)
    order = rng.permutation(len(ctx) + n)            # parents and children lie in any rows
    table, at = np.full((len(ctx) + n, max(need) + 2), -1, np.int32), 0
    lens = np.zeros(len(ctx) + n, np.int32)
    for r, h in enumerate(need):
        table[order[r], :h] = ids[at:at + h]
        lens[order[r]] = ctx[r]
        at += h
    s["table"], s["ctx_len"] = torch.from_numpy(table).to(DEV), torch.from_numpy(lens).to(DEV)
    s["src"] = _ints(np.repeat(order[:len(ctx)], case["children"]))
    s["dst"] = _ints(order[len(ctx):])
    s["free"], s["cursor"], s["cursor_out"] = torch.from_numpy(ids[at:]).to(DEV), _ints([int(rng.integers(4))]), _ints([0])
    s["copy_src"], s["copy_dst"] = _ints([-1] * n), _ints([-1] * n)
    s["caches"] = [tuple(_cache(gen, pages, case["kv_heads"], P, case["head_dim"]) for _ in range(2))
                   for _ in range(case["layers"])]
    s["page"], s["pages"] = P, pages


def _prepare_free(s, case, gen, rng):
    """Rows of a server's table, every fourth request sharing the front half of
    the one before it; some have ended (length zero)."""
    ctx, _ = _lengths(case)
    R, P = len(ctx), case["page"]
    need = [-(-c // P) for c in ctx]
    pages = sum(need) + 5
    ids = rng.permutation(pages).astype(np.int32)
    table, at = np.full((R, max(need) + 1), -1, np.int32), 0
    for r, h in enumerate(need):
        table[r, :h] = ids[at:at + h]
        at += h
        if r % 4 == 3:
            both = min(h, need[r - 1]) // 2
            table[r, :both] = table[r - 1, :both]
    lens = np.array(ctx, np.int32)
    lens[rng.permutation(R)[:case["ended"]]] = 0
    s["table"], s["ctx_len"] = torch.from_numpy(table).to(DEV), torch.from_numpy(lens).to(DEV)
    s["free"], s["count"] = _ints([0] * pages), _ints([0])
    s["page"], s["pages"], s["compact"] = P, pages, case["compact"]
    if case["compact"]:
        s["table_out"] = torch.empty_like(s["table"])
        s["move_src"], s["move_dst"] = _ints([0] * (pages // 2)), _ints([0] * (pages // 2))
        s["caches"] = [tuple(_cache(gen, pages, case["kv_heads"], P, case["head_dim"]) for _ in range(2))]


def _own_step(s):
    """The buffers and the plan of a step, which a program keeps for all of its layers."""
    import nvfp4_block_scaled_device_gb300 as nv
    if s["page"]:
        s["step"] = nv.AttnPlan(s["R"], s["T"], s["H"], s["Hkv"], page_size=s["page"], block_table=s["table"],
                                window=s["window"])
        nv.nvfp4_attn_plan(s["step"], s["q_len"], s["ctx_len"])
    if s["op"] == "qk":
        if s["page"]:
            s["cache"] = nv.KVCache(s["kc"], s["vc"])
        return
    s["cache"] = nv.KVCache4(s["k_codes"], s["v_codes"], s["k_sf"], s["v_sf"], torch.full((1,), s["k_g"], device=DEV),
                             torch.full((1,), s["v_g"], device=DEV))
    if s["op"] == "cache4":
        s["expanded"] = nv.KVCache(s["kx"], s["vx"])
    else:
        # a layer's worth of bf16 pages, which all layers share: for prompts
        s["expanded"] = nv.KVCache.empty(s["cache"].pages, s["Hkv"], s["page"], s["D"])
        s["ws"] = nv.workspace(nv.attn_workspace_bytes())


def _own_pages(s):
    import nvfp4_block_scaled_device_gb300 as nv
    s["requests"] = nv.PageTable(s["table"], s["ctx_len"], s["page"], s["pages"])
    s["own_caches"] = [nv.KVCache(k, v) for k, v in s.get("caches", [])]


# ------------------------------------------------------------- the operators
def run(s):
    if own:
        return _run_own(s)
    return {"qk": _plain_qk, "cache4": _plain_cache4, "attn4": _plain_attn4, "fork": _plain_fork,
            "free": _plain_free}[s["op"]](s)


def _outputs(s, *names):
    out = {n: s[n] for n in names if n in s}
    for i, (k, v) in enumerate(s.get("caches", [])):
        out[f"k{i}"], out[f"v{i}"] = k, v
    return out


_NAMES = {"qk": ("q_out", "k_out", "kc", "vc"), "cache4": ("kx", "vx"), "attn4": ("out", "lse"),
          "fork": ("table", "ctx_len", "cursor_out", "copy_src", "copy_dst"),
          "free": ("free", "count", "table_out", "move_src", "move_dst")}


def _run_own(s):
    import nvfp4_block_scaled_device_gb300 as nv
    op = s["op"]
    if op == "qk":
        if s["page"]:
            nv.nvfp4_qk_norm_rope(s["q"], s["k"], s["q_norm"], s["k_norm"], s["pos"], s["cos"], s["sin"],
                                  q_out=s["q_out"], halves=s["halves"], eps=EPS, v=s["v"], plan=s["step"],
                                  cache=s["cache"])
        else:
            nv.nvfp4_qk_norm_rope(s["q"], s["k"], s["q_norm"], s["k_norm"], s["pos"], s["cos"], s["sin"],
                                  q_out=s["q_out"], k_out=s["k_out"], halves=s["halves"], eps=EPS)
    elif op == "cache4":
        nv.nvfp4_kv4_append(s["k"], s["v"], s["step"], s["cache"])
        nv.nvfp4_kv4_expand(s["cache"], s["step"], s["expanded"])
    elif op == "attn4":
        nv.nvfp4_attn_paged4(s["q"], s["cache"], s["step"], s["out"], s["ws"], lse=s["lse"], expanded=s["expanded"])
    elif op == "fork":
        nv.nvfp4_pages_fork(s["requests"], s["src"], s["dst"], s["free"], s["cursor"], s["cursor_out"], s["copy_src"],
                            s["copy_dst"])
        nv.nvfp4_pages_copy(s["own_caches"], s["copy_src"], s["copy_dst"])
    elif s["compact"]:
        nv.nvfp4_pages_free(s["requests"], s["free"], s["count"], s["table_out"], s["move_src"], s["move_dst"])
        nv.nvfp4_pages_copy(s["own_caches"], s["move_src"], s["move_dst"])
    else:
        nv.nvfp4_pages_free(s["requests"], s["free"], s["count"])
    return _outputs(s, *_NAMES[op])


def _plain_heads(x, w, s):
    """Norm and rotation of the heads of x [T, heads, D], in 32 bits."""
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    rd, D = s["rope_dim"], s["D"]
    c, sn = (t[s["pos"].long()][:, None] for t in (s["cos"], s["sin"]))
    r = x[..., D - rd:]
    a, b = (r[..., :rd // 2], r[..., rd // 2:]) if s["halves"] else (r[..., 0::2], r[..., 1::2])
    a, b = a * c - b * sn, a * sn + b * c
    r = torch.cat([a, b], -1) if s["halves"] else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([x[..., :D - rd], r], -1).to(torch.bfloat16)


def _plain_qk(s):
    s["q_out"].copy_(_plain_heads(s["q"], s["q_norm"], s))
    k = _plain_heads(s["k"], s["k_norm"], s)
    if s["page"]:
        slot = s["slot"].long()
        page, row = slot // s["page"], slot % s["page"]
        s["kc"][page, :, row] = k
        s["vc"][page, :, row] = s["v"]
    else:
        s["k_out"].copy_(k)
    return _outputs(s, *_NAMES["qk"])


def _quantize(x, g):
    """bf16 rows [..., D] to 4 bits: codes [..., D / 2] and scales [..., D / 16]."""
    x = x.float().unflatten(-1, (-1, 16))
    sf = (x.abs().amax(-1) / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    den = sf.float() * g
    y = x / torch.where(den == 0, 1.0, den)[..., None]
    m = y.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = torch.where(den[..., None] == 0, 0, code + 8 * torch.signbit(x).to(torch.uint8)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), sf.view(torch.uint8)


def _values(codes, sf, g):
    """What codes and scales stand for, in 32 bits."""
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], -1).flatten(-2).unflatten(-1, (-1, 16))
    return (v * (sf.view(torch.float8_e4m3fn).float() * g)[..., None]).flatten(-2)


def _plain_cache4(s):
    slot, P = s["slot"].long(), s["page"]
    page, row = slot // P, slot % P
    for x, t in (("k", s["k"]), ("v", s["v"])):
        codes, sf = _quantize(t, s[x + "_g"])
        s[x + "_codes"][page, :, row] = codes
        s[x + "_sf"][page, :, row] = sf
    # the rows that a new token sees
    at = torch.arange(s["table"].shape[1] * P, device=DEV)
    seen = at < s["kv_len"][:, None]
    if s["window"]:
        seen &= at > s["ctx_len"][:, None] - s["window"]
    request, at = seen.nonzero(as_tuple=True)
    page, row = s["table"][request, at // P].long(), at % P
    for x in "kv":
        s[x + "x"][page, :, row] = _values(s[x + "_codes"][page, :, row], s[x + "_sf"][page, :, row],
                                           s[x + "_g"]).to(torch.bfloat16)
    return _outputs(s, *_NAMES["cache4"])


def _softmax_v(scores, seen, v):
    """Softmax over the last axis of the keys that are seen, times v; the
    logarithm of the sum.  scores [..., rows, keys], v [..., keys, columns]."""
    scores = scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return out, (top + total.log()).squeeze(-1)


def _plain_attn4(s):
    R, T, H, Hkv, D, n = s["R"], s["T"], s["H"], s["Hkv"], s["D"], s["q_max"]
    L = s["kv_max"]
    table = s["table"].clamp(min=0).long()
    k, v = (_values(s[x + "_codes"][table], s[x + "_sf"][table], s[x + "_g"]).transpose(2, 3).flatten(1, 2)[:, :L]
            for x in "kv")                                                    # [R, L, Hkv, D]
    request = torch.repeat_interleave(torch.arange(R, device=DEV), s["q_len"], output_size=T)
    row = torch.arange(T, device=DEV) - s["cu_q"][request]
    q = torch.zeros(R, n, H, D, device=DEV)
    q[request, row] = s["q"].float()
    q = q.unflatten(2, (Hkv, H // Hkv)).permute(0, 2, 3, 1, 4)                # [R, Hkv, group, n, D]
    p = (s["ctx_len"][:, None] + torch.arange(n, device=DEV))[:, :, None]     # position of each row
    j = torch.arange(L, device=DEV)
    seen = (j <= p) & (j < s["kv_len"][:, None, None])
    if s["window"]:
        seen &= j > p - s["window"]
    out, lse = _softmax_v(torch.matmul(q * D ** -0.5, k.permute(0, 2, 3, 1)[:, :, None]), seen[:, None, None],
                          v.permute(0, 2, 1, 3)[:, :, None])
    out, lse = out.permute(0, 3, 1, 2, 4)[request, row], lse.permute(0, 3, 1, 2)[request, row]
    return {"out": out.reshape(T, H, D).to(torch.bfloat16), "lse": lse.reshape(T, H).contiguous()}


def _plain_fork(s):
    P, table = s["page"], s["table"]
    src, dst = s["src"].long(), s["dst"].long()
    ctx = s["ctx_len"][src]
    need = (ctx + P - 1) // P
    partial = ctx % P != 0
    page = s["free"][(s["cursor"] + torch.cumsum(partial, 0) - partial.int()).clamp(0, s["free"].numel() - 1)]
    j = torch.arange(table.shape[1], device=DEV)
    last = (j == need[:, None] - 1) & partial[:, None]
    rows = torch.where(j < need[:, None], table[src], -1)
    s["copy_src"].copy_(torch.where(last, rows, 0).sum(1) - (~partial).int())
    s["copy_dst"].copy_(torch.where(partial, page, -1))
    table[dst] = torch.where(last, page[:, None], rows)
    s["ctx_len"][dst] = ctx
    s["cursor_out"].copy_(s["cursor"] + partial.sum())
    _plain_copy(s, "copy_src", "copy_dst")
    return _outputs(s, *_NAMES["fork"])


def _plain_copy(s, src, dst):
    both = s[src] >= 0
    a, b = s[src][both].long(), s[dst][both].long()
    for cache in s["caches"]:
        for x in cache:
            x[b] = x[a]


def _plain_free(s):
    P, table, pages = s["page"], s["table"], s["pages"]
    held = torch.arange(table.shape[1], device=DEV) < (s["ctx_len"][:, None] + P - 1) // P
    used = torch.zeros(pages, dtype=torch.bool, device=DEV)
    used[table[held].long()] = True
    ids = torch.arange(pages, device=DEV, dtype=torch.int32)
    n = used.sum()
    s["count"].copy_(pages - n)
    if not s["compact"]:
        _fill(s["free"], ids[~used])
        return _outputs(s, *_NAMES["free"])
    _fill(s["free"], ids[ids >= n])
    src, dst = ids[used & (ids >= n)], ids[~used & (ids < n)]
    _fill(s["move_src"], src)
    _fill(s["move_dst"], dst)
    ids[src.long()] = dst
    s["table_out"].copy_(torch.where(held, ids[table.clamp(min=0).long()], -1))
    _plain_copy(s, "move_src", "move_dst")
    return _outputs(s, *_NAMES["free"])


def _fill(out, values):
    out.fill_(-1)
    out[:values.numel()] = values


# ---------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    ctx, q = _lengths(case)
    R, T = len(ctx), sum(q)
    Hkv, D, P = case["kv_heads"], case["head_dim"], case["page"]
    if op in ("fork", "free"):
        need = [-(-c // P) for c in ctx]
        page = 2 * 2 * Hkv * P * D                   # of K and V
        if op == "fork":
            n = case["children"]
            copies = n * sum(c % P != 0 for c in ctx) * case["layers"]
            # the parents' rows in, the children's out, pages copied
            return {"bytes": 4 * (sum(need) + n * R * (max(need) + 2) + 6 * n * R) + 2 * page * copies,
                    "flops": copies * page // 2}
        pages = sum(need) + 5
        # requests that ended hold no page: on average, so many of the entries and pages are left
        left = (R - case["ended"]) / R
        held = int(sum(need) * left)
        moved = int(pages * left * (1 - left)) if case["compact"] else 0
        table = R * (max(need) + 1) if case["compact"] else 0
        return {"bytes": 4 * (R + held + pages + table + 4 * moved) + 2 * page * moved, "flops": held + pages}
    H = case["heads"]
    if op == "qk":
        heads = H + Hkv + (Hkv if P else 0)
        return {"bytes": 2 * 2 * T * heads * D + 4 * T * case["rope_dim"] + 2 * 2 * D + 4 * T * (2 if P else 1),
                "flops": 7 * T * (H + Hkv) * D}
    row = Hkv * D * 9 // 16                          # of codes and scales, K or V
    W = case["window"]
    if op == "cache4":
        rows = sum(c + n - (max(0, c - W + 1) if W else 0) for c, n in zip(ctx, q))
        return {"bytes": 2 * T * (2 * Hkv * D + row) + 4 * T + 2 * rows * (row + 2 * Hkv * D),
                "flops": 2 * (T + rows) * Hkv * D}
    pairs = rows = 0
    for c, n in zip(ctx, q):
        p = np.arange(c, c + n, dtype=np.int64)
        pairs += int((np.minimum(p + 1, W) if W else p + 1).sum())
        rows += c + n - (max(0, c - W + 1) if W else 0)
    tables = 4 * (2 * R + 1) + 4 * sum(-(-(c + n) // P) for c, n in zip(ctx, q))
    return {"bytes": 2 * 2 * T * H * D + 4 * T * H + 2 * rows * row + tables, "flops": 4 * D * H * pairs}


# --------------------------------------------------------------------- exact
def exact(case, seed):
    """From the definitions, in 64 bits, request by request."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"qk": _exact_qk, "cache4": _exact_cache4, "attn4": _exact_attn4, "fork": _exact_fork,
            "free": _exact_free}[case["op"]](s)


def _exact_qk(s):
    D, rd = s["D"], s["rope_dim"]
    at = s["pos"].tolist()
    c, sn = s["cos"][at].double(), s["sin"][at].double()
    out = {}
    for name in "qk":
        x, w = s[name].double(), s[name + "_norm"].double()
        norm = torch.sqrt(torch.einsum("thd,thd->th", x, x) / D + EPS)
        y = x / norm[:, :, None] * w
        for i in range(rd // 2):
            a, b = (D - rd + i, D - rd // 2 + i) if s["halves"] else (D - rd + 2 * i, D - rd + 2 * i + 1)
            z = torch.complex(y[..., a], y[..., b]) * torch.complex(c[:, i], sn[:, i])[:, None]
            y[..., a], y[..., b] = z.real, z.imag
        out[name] = y
    if not s["page"]:
        return {"q_out": out["q"], "k_out": out["k"]}
    kc, vc = s["kc"].double(), s["vc"].double()
    page, row = (torch.tensor(t, device=DEV) for t in zip(*(divmod(i, s["page"]) for i in s["slot"].tolist())))
    kc[page, :, row], vc[page, :, row] = out["k"], s["v"].double()
    return {"q_out": out["q"], "kc": kc, "vc": vc}


def _nearest(x, values):
    """Index of the nearest of the ascending values, the even one of two as near."""
    hi = torch.searchsorted(values, x.contiguous()).clamp(1, values.numel() - 1)
    lo = hi - 1
    below, above = x - values[lo], values[hi] - x
    return torch.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_4bit(x, g):
    """The values that rows x [..., D] take in 4 bits."""
    scales = torch.tensor([(m if e == 0 else 8 + m) * 2.0 ** (max(e, 1) - 10) for e in range(16) for m in range(8)][:127],
                          dtype=torch.float64, device=DEV)
    x = x.double().reshape(*x.shape[:-1], -1, 16)
    unit = scales[_nearest(x.abs().max(-1).values / 6 / g, scales)][..., None] * g
    codes = torch.tensor(_E2M1, dtype=torch.float64, device=DEV)
    mag = codes[_nearest(x.abs() / torch.where(unit > 0, unit, 1.0), codes)]
    return (torch.copysign(mag, x) * unit).reshape(*x.shape[:-2], -1)


def _decoded(codes, sf, g):
    """What codes and scales stand for, digit by digit."""
    codes, sf = codes.long(), sf.long()
    e, m = (sf >> 3).double(), (sf & 7).double()
    unit = torch.where(sf < 8, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(e - 7)) * g
    nib = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.int64, device=DEV)
    nib[..., 0::2], nib[..., 1::2] = codes % 16, codes // 16
    v = torch.tensor(_E2M1 + [-x for x in _E2M1], dtype=torch.float64, device=DEV)[nib]
    return v * unit.repeat_interleave(16, -1)


def _exact_cache4(s):
    ctx, q, P = s["ctx_len"].tolist(), s["q_len"].tolist(), s["page"]
    out, first = {}, 0
    for name in "kv":
        out[name + "x"] = torch.zeros(s["kx"].shape, dtype=torch.float64, device=DEV)
    for r, (c, n) in enumerate(zip(ctx, q)):
        begin = max(0, c - s["window"] + 1) if s["window"] else 0
        at = torch.arange(begin, c + n, device=DEV)
        page, row = s["table"][r].long()[torch.div(at, P, rounding_mode="floor")], at % P
        for name in "kv":
            old = _decoded(s[name + "_codes"][page, :, row], s[name + "_sf"][page, :, row], s[name + "_g"])
            old[c - begin:] = _exact_4bit(s[name][first:first + n], s[name + "_g"])
            out[name + "x"][page, :, row] = old
        first += n
    return out


def _exact_attn4(s):
    ctx, q = s["ctx_len"].tolist(), s["q_len"].tolist()
    T, H, Hkv, D = s["T"], s["H"], s["Hkv"], s["D"]
    out = torch.zeros(T, H, D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    at = 0
    for r, (c, n) in enumerate(zip(ctx, q)):
        i = torch.arange(n, device=DEV)[:, None] + c
        j = torch.arange(c + n, device=DEV)[None, :]
        hidden = j > i
        if s["window"]:
            hidden = hidden | (i - j >= s["window"])
        pages = s["table"][r, :-(-(c + n) // s["page"])].long()
        for h in range(Hkv):
            k, v = (_decoded(s[x + "_codes"][pages, h], s[x + "_sf"][pages, h], s[x + "_g"]).reshape(-1, D)[:c + n]
                    for x in "kv")
            for g in range(h * H // Hkv, (h + 1) * H // Hkv):
                x = s["q"][at:at + n, g].double() @ k.T / math.sqrt(D)
                x[hidden] = -math.inf
                lse[at:at + n, g] = torch.logsumexp(x, 1)
                out[at:at + n, g] = torch.exp(x - lse[at:at + n, g, None]) @ v
        at += n
    return {"out": out, "lse": lse}


def _exact_copies(s, pairs):
    out = {}
    for i, cache in enumerate(s["caches"]):
        for name, x in zip("kv", cache):
            y = x.double()
            for a, b in pairs:
                y[b] = x[a].double()
            out[f"{name}{i}"] = y
    return out


def _exact_fork(s):
    P, table, ctx = s["page"], s["table"].cpu().numpy().copy(), s["ctx_len"].tolist()
    free, at = s["free"].tolist(), s["cursor"].item()
    copies = []
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        full, rest = divmod(ctx[a], P)
        table[b] = -1
        table[b, :full] = table[a, :full]
        copies.append((-1, -1))
        if rest:                                     # a page that the child will write behind its parent's rows
            copies[-1] = (int(table[a, full]), free[at])
            table[b, full] = free[at]
            at += 1
        ctx[b] = ctx[a]
    return {"table": torch.from_numpy(table).to(DEV), "ctx_len": _ints(ctx), "cursor_out": _ints([at]),
            "copy_src": _ints([a for a, _ in copies]), "copy_dst": _ints([b for _, b in copies]),
            **_exact_copies(s, [c for c in copies if c[0] >= 0])}


def _exact_free(s):
    P, pages, table = s["page"], s["pages"], s["table"].cpu().numpy()
    rows = [table[r, :-(-c // P)].tolist() for r, c in enumerate(s["ctx_len"].tolist())]
    used = {p for row in rows for p in row}
    pad = lambda x, n: _ints(list(x) + [-1] * (n - len(x)))
    out = {"count": _ints([pages - len(used)])}
    if not s["compact"]:
        return {"free": pad([p for p in range(pages) if p not in used], pages), **out}
    moves = list(zip(sorted(p for p in used if p >= len(used)), [p for p in range(len(used)) if p not in used]))
    to = dict(moves)
    new = np.full(table.shape, -1, np.int32)
    for r, row in enumerate(rows):
        new[r, :len(row)] = [to.get(p, p) for p in row]
    return {"free": pad(range(len(used), pages), pages), **out, "table_out": torch.from_numpy(new).to(DEV),
            "move_src": pad([a for a, _ in moves], pages // 2), "move_dst": pad([b for _, b in moves], pages // 2),
            **_exact_copies(s, moves)}
