"""Attention operators, measured: the step tables built on the device from
request lengths (``plan``), the write of new K/V rows into the paged cache
(``append``), causal attention over packed prompts (``prompt``) and attention
of new tokens over the paged cache (``paged``).

``run`` computes each either in its plain form (elementary torch operations
in 32 bits) or, where ``own`` is true, by the calls a user makes of this
package.  Head layouts are the package's own QKV width of 7168 (40 query, 8
key and 8 value heads of 128 columns) and generic ones.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------- cases
def listed():
    layer = {"heads": 40, "kv_heads": 8, "head_dim": 128}
    return [
        # one decode step's tables: 64 running requests, one new token each
        {"name": "plan_decode_64", "op": "plan", "requests": 64, "q_lo": 1, "q_hi": 1, "ctx_lo": 100, "ctx_hi": 4096,
         "page": 16, "heads": 40, "kv_heads": 8},
        # a large mixed batch: thousands of requests, some with a few new tokens (speculated or a short chunk)
        {"name": "plan_mixed_4096", "op": "plan", "requests": 4096, "q_lo": 1, "q_hi": 13, "ctx_lo": 1, "ctx_hi": 8192,
         "page": 64, "heads": 40, "kv_heads": 8},
        # the cache write of a small decode step
        {"name": "append_17", "op": "append", "requests": 17, "q_lo": 1, "q_hi": 1, "ctx_lo": 10, "ctx_hi": 1000,
         "page": 16, "kv_heads": 8, "head_dim": 128},
        # the cache write of a long prompt in one go
        {"name": "append_16384", "op": "append", "requests": 5, "q_lo": 1000, "q_hi": 6600, "ctx_lo": 0, "ctx_hi": 77,
         "page": 64, "kv_heads": 8, "head_dim": 128},
        # one short prompt: latency
        {"name": "prompt_17", "op": "prompt", "lens": "17", "window": 0, **layer},
        # a ubatch of 1024 tokens packed from prompts of uneven lengths
        {"name": "prompt_packed_1024", "op": "prompt", "lens": "1,17,130,300,77,499", "window": 0, **layer},
        # a sliding-window layer of a model with as many key heads as query heads, 64 columns each
        {"name": "prompt_window_4097", "op": "prompt", "lens": "1531,2566", "window": 512, "heads": 20, "kv_heads": 20,
         "head_dim": 64},
        # one long prompt: the arithmetic bound
        {"name": "prompt_8192", "op": "prompt", "lens": "8192", "window": 0, **layer},
        # a single user's next token
        {"name": "decode_1", "op": "paged", "requests": 1, "q_lo": 1, "q_hi": 1, "ctx_lo": 333, "ctx_hi": 333,
         "page": 16, "window": 0, **layer},
        # a decode step of 64 users with uneven contexts
        {"name": "decode_64", "op": "paged", "requests": 64, "q_lo": 1, "q_hi": 1, "ctx_lo": 200, "ctx_hi": 8192,
         "page": 16, "window": 0, **layer},
        # two users deep in long contexts: few rows, a long axis
        {"name": "decode_long_2", "op": "paged", "requests": 2, "q_lo": 1, "q_hi": 1, "ctx_lo": 65537,
         "ctx_hi": 131071, "page": 64, "window": 0, **layer},
        # the last 1024-token ubatch of a 16384-token prompt
        {"name": "chunk_1024_at_15360", "op": "paged", "requests": 1, "q_lo": 1024, "q_hi": 1024, "ctx_lo": 15360,
         "ctx_hi": 15360, "page": 64, "window": 0, **layer},
    ]


def _log_int(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "prompt", "prompt", "paged", "paged", "paged"])
    page = rng.choice([16, 32, 64, 128])
    heads, kv_heads = rng.choice([(40, 8), (20, 4), (64, 8), (20, 20), (8, 1), (28, 4)])
    dim = rng.choice([64, 128, 128, 96])
    window = rng.choice([0, 0, 0, _log_int(rng, 16, 4000)])
    if op == "plan":
        hi = _log_int(rng, 1, 40)
        return {"op": op, "requests": _log_int(rng, 1, 4096) if hi < 8 else _log_int(rng, 1, 600), "q_lo": 1,
                "q_hi": hi, "ctx_lo": rng.randint(0, 50), "ctx_hi": _log_int(rng, 60, 8192), "page": page,
                "heads": heads, "kv_heads": kv_heads}
    if op == "append":
        requests = _log_int(rng, 1, 64)
        q = _log_int(rng, 1, 14000 // requests)
        return {"op": op, "requests": requests, "q_lo": max(1, q // 3), "q_hi": q, "ctx_lo": rng.randint(0, 40),
                "ctx_hi": rng.randint(50, 700), "page": page, "kv_heads": kv_heads, "head_dim": dim}
    if op == "prompt":
        total = _log_int(rng, 3, 8000 if heads <= 40 else 5500)
        n = min(total, _log_int(rng, 1, 12))
        cuts = sorted(rng.sample(range(1, total), n - 1)) if n > 1 else []
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        return {"op": op, "lens": ",".join(map(str, lens)), "window": window, "heads": heads, "kv_heads": kv_heads,
                "head_dim": dim}
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
    if case["op"] == "prompt":
        q = [int(x) for x in case["lens"].split(",")]
        return [0] * len(q), q
    n = case["requests"]
    return _spread(case["ctx_lo"], case["ctx_hi"], n, 0.37), _spread(case["q_lo"], case["q_hi"], n, 0.11)


# -------------------------------------------------------------------- inputs
def _normal(gen, *shape, std=1.0):
    return (torch.randn(shape, device=DEV, dtype=torch.float32, generator=gen) * std).to(torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _new(case, ctx, q):
    """Pages that each request's new tokens open."""
    P = case["page"]
    return [-(-(c + n) // P) - -(-c // P) for c, n in zip(ctx, q)]


def _tables(case, ctx, q, rng):
    """Pages of a cache in use, scattered over it: the table with the cached
    tokens' pages in it, the pages that are free, in the order they are taken."""
    P = case["page"]
    have = [-(-c // P) for c in ctx]
    need = [-(-(c + n) // P) for c, n in zip(ctx, q)]
    spare = 1000 if case["op"] == "plan" else 3      # free pages that stay free
    pages = sum(need) + spare
    ids = rng.permutation(pages).astype(np.int32)
    width = max(need)
    table = np.full((len(ctx), width), -1, np.int32)
    at = 0
    for r, h in enumerate(have):
        table[r, :h] = ids[at:at + h]
        at += h
    return table, ids[at:], pages


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    op = case["op"]
    ctx, q = _lengths(case)
    if op == "plan":
        order = rng.permutation(len(ctx))            # the requests of a step come in any order
        ctx, q = [ctx[i] for i in order], [q[i] for i in order]
    R, T = len(ctx), sum(q)
    cu = np.concatenate([[0], np.cumsum(q)])
    s = {"op": op, "R": R, "T": T, "q_max": max(q), "ctx_len": _ints(ctx), "q_len": _ints(q), "cu_q": _ints(cu),
         "kv_len": _ints([c + n for c, n in zip(ctx, q)]), "kv_max": max(c + n for c, n in zip(ctx, q)),
         "window": case.get("window", 0)}
    Hkv = case["kv_heads"]
    if op != "prompt":
        table, free, pages = _tables(case, ctx, q, rng)
        s["page"] = P = case["page"]
        taken = int(rng.integers(free.size - sum(_new(case, ctx, q)) + 1))      # by earlier steps
        s["free"], s["cursor"] = torch.from_numpy(free).to(DEV), _ints([taken])
        s["table"] = torch.from_numpy(table).to(DEV)
    if op == "plan":
        s["pos"], s["slot"] = (torch.empty(T, dtype=torch.int32, device=DEV) for _ in range(2))
        s["cursor_out"] = _ints([0])
    else:
        D = case["head_dim"]
        H = case.get("heads", Hkv)
        s["D"], s["H"], s["Hkv"] = D, H, Hkv
        # the projection's output: query, key and value heads side by side
        width = (H + 2 * Hkv) * D
        s["qkv"] = _normal(gen, T, width, std=1.5)
        s["q"] = s["qkv"][:, :H * D].unflatten(1, (H, D))
        s["k"] = s["qkv"][:, H * D:(H + Hkv) * D].unflatten(1, (Hkv, D))
        s["v"] = s["qkv"][:, (H + Hkv) * D:].unflatten(1, (Hkv, D))
    if op in ("append", "paged"):
        s["kc"], s["vc"] = (_normal(gen, pages, Hkv, P, D) for _ in range(2))
    if op == "append":
        del s["qkv"], s["q"]
    if op in ("prompt", "paged"):
        s["out"] = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(T, H, dtype=torch.float32, device=DEV)
    if op in ("append", "paged"):                    # the step's tables as the plan leaves them
        full = s["table"].clone()
        _plain_pages(s, full)
        if op == "paged" or not own:
            s["table"] = full
        s["slot"] = _plain_slots(s, full)[1]
    if own:
        _prepare_own(s, case)
    return s


def _prepare_own(s, case):
    """The buffers and the plan of a step, which a program keeps for all of its layers."""
    import nvfp4_block_scaled_device_gb300 as nv
    op = s["op"]
    H, Hkv = case.get("heads", case["kv_heads"]), case["kv_heads"]
    if op == "prompt":
        s["step"] = nv.AttnPlan(s["R"], s["T"], H, Hkv, window=s["window"])
    else:
        s["step"] = nv.AttnPlan(s["R"], s["T"], H, Hkv, page_size=s["page"], block_table=s["table"],
                                window=s["window"])
    if op in ("append", "paged"):
        s["cache"] = nv.KVCache(s["kc"], s["vc"])
    if op in ("prompt", "paged"):
        s["ws"] = nv.workspace(nv.attn_workspace_bytes())
        nv.nvfp4_attn_plan(s["step"], s["q_len"], s["ctx_len"] if op == "paged" else None)
    elif op == "append":
        nv.nvfp4_attn_plan(s["step"], s["q_len"], s["ctx_len"], s["free"], s["cursor"])


# ------------------------------------------------------------- the operators
def run(s):
    if own:
        return _run_own(s)
    return {"plan": _plain_plan, "append": _plain_append, "prompt": _plain_prompt, "paged": _plain_paged}[s["op"]](s)


def _run_own(s):
    import nvfp4_block_scaled_device_gb300 as nv
    op, step = s["op"], s["step"]
    if op == "plan":
        nv.nvfp4_attn_plan(step, s["q_len"], s["ctx_len"], s["free"], s["cursor"])
        return {"cu_q": step.cu_q, "kv_len": step.kv_len, "pos": step.pos, "slot": step.slot,
                "table": step.block_table, "cursor": step.cursor}
    if op == "append":
        nv.nvfp4_kv_append(s["k"], s["v"], step, s["cache"])
        return {"k": s["kc"], "v": s["vc"]}
    if op == "prompt":
        nv.nvfp4_attn_prompt(s["q"], s["k"], s["v"], step, s["out"], s["ws"], lse=s["lse"])
    else:
        nv.nvfp4_attn_paged(s["q"], s["cache"], step, s["out"], s["ws"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_pages(s, table):
    """New pages into the table, in place; how many were taken."""
    P = s["page"]
    have, need = (s["ctx_len"] + P - 1) // P, (s["ctx_len"] + s["q_len"] + P - 1) // P
    taken = need - have
    first = torch.cumsum(taken, 0) - taken
    j = torch.arange(table.shape[1], device=DEV)
    at = s["cursor"] + first[:, None] + j - have[:, None]
    new = (j >= have[:, None]) & (j < need[:, None])
    table.copy_(torch.where(new, s["free"][at.clamp(0, s["free"].numel() - 1)], table))
    return taken.sum(dtype=torch.int32)


def _plain_slots(s, table):
    request = torch.repeat_interleave(torch.arange(s["R"], device=DEV), s["q_len"], output_size=s["T"])
    pos = torch.arange(s["T"], device=DEV, dtype=torch.int32) - s["cu_q"][request] + s["ctx_len"][request]
    return pos, table[request, pos // s["page"]] * s["page"] + pos % s["page"]


def _plain_plan(s):
    cu = torch.zeros(s["R"] + 1, dtype=torch.int32, device=DEV)
    cu[1:] = torch.cumsum(s["q_len"], 0)
    cursor = s["cursor"] + _plain_pages(s, s["table"])
    pos, slot = _plain_slots(dict(s, cu_q=cu), s["table"])
    return {"cu_q": cu, "kv_len": s["ctx_len"] + s["q_len"], "pos": pos, "slot": slot, "table": s["table"],
            "cursor": cursor}


def _plain_append(s):
    slot = s["slot"].long()
    page, row = slot // s["page"], slot % s["page"]
    s["kc"][page, :, row] = s["k"]
    s["vc"][page, :, row] = s["v"]
    return {"k": s["kc"], "v": s["vc"]}


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


def _plain_prompt(s):
    T, H, Hkv, D = s["T"], s["H"], s["Hkv"], s["D"]
    t = torch.arange(T, device=DEV)
    request = torch.repeat_interleave(torch.arange(s["R"], device=DEV), s["q_len"], output_size=T)
    seen = (request[:, None] == request) & (t <= t[:, None])
    if s["window"]:
        seen &= t > t[:, None] - s["window"]
    q = s["q"].float().unflatten(1, (Hkv, H // Hkv)).permute(1, 2, 0, 3)      # [kv head, group, token, column]
    k = s["k"].float().permute(1, 2, 0)[:, None]
    v = s["v"].float().permute(1, 0, 2)[:, None]
    out, lse = _softmax_v(torch.matmul(q * D ** -0.5, k), seen, v)
    return {"out": out.permute(2, 0, 1, 3).reshape(T, H, D).to(torch.bfloat16),
            "lse": lse.permute(2, 0, 1).reshape(T, H).contiguous()}


def _plain_paged(s):
    R, T, H, Hkv, D, n = s["R"], s["T"], s["H"], s["Hkv"], s["D"], s["q_max"]
    L = s["kv_max"]
    table = s["table"].clamp(min=0).long()
    k, v = (c[table].transpose(2, 3).flatten(1, 2)[:, :L].float() for c in (s["kc"], s["vc"]))   # [R, L, Hkv, D]
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


# ---------------------------------------------------------------------- work
def _seen_keys(case):
    """(row, key) pairs of one head, and the cached or packed key rows that any row reaches."""
    ctx, q = _lengths(case)
    W = case.get("window", 0)
    pairs = rows = 0
    for c, n in zip(ctx, q):
        p = np.arange(c, c + n, dtype=np.int64)
        pairs += int((np.minimum(p + 1, W) if W else p + 1).sum())
        rows += c + n - (max(0, c - W + 1) if W else 0)
    return pairs, rows


def work(case):
    ctx, q = _lengths(case)
    R, T = len(ctx), sum(q)
    if case["op"] == "plan":
        new = sum(_new(case, ctx, q))
        # lengths in; offsets, lengths, positions, slots out; a page id for each request's first token; new pages in and out
        return {"bytes": 4 * (2 * R + 2 * R + 1 + 2 * T + R + 2 * new + 2), "flops": T}
    Hkv, D = case["kv_heads"], case["head_dim"]
    if case["op"] == "append":
        return {"bytes": 4 * T + 2 * 2 * 2 * T * Hkv * D, "flops": T}
    pairs, rows = _seen_keys(case)
    H = case["heads"]
    tables = 4 * (R + 1) + (4 * R + 4 * sum(-(-(c + n) // case["page"]) for c, n in zip(ctx, q))
                            if case["op"] == "paged" else 0)
    return {"bytes": 2 * 2 * T * H * D + 4 * T * H + 2 * 2 * rows * Hkv * D + tables, "flops": 4 * D * H * pairs}


# --------------------------------------------------------------------- exact
def exact(case, seed):
    """From the definitions, in 64 bits, request by request."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "plan":
        return _exact_plan(s)
    ctx, q = s["ctx_len"].tolist(), s["q_len"].tolist()
    if case["op"] == "append":
        k, v = s["kc"].double(), s["vc"].double()
        for t, slot in enumerate(s["slot"].tolist()):
            page, row = divmod(slot, s["page"])
            k[page, :, row, :] = s["k"][t].double()
            v[page, :, row, :] = s["v"][t].double()
        return {"k": k, "v": v}
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
        for h in range(Hkv):
            if case["op"] == "prompt":
                k, v = s["k"][at:at + n, h].double(), s["v"][at:at + n, h].double()
            else:
                pages = s["table"][r, :-(-(c + n) // s["page"])].long()
                k, v = (x[pages, h].reshape(-1, D)[:c + n].double() for x in (s["kc"], s["vc"]))
            for g in range(h * H // Hkv, (h + 1) * H // Hkv):
                x = s["q"][at:at + n, g].double() @ k.T / math.sqrt(D)
                x[hidden] = -math.inf
                lse[at:at + n, g] = torch.logsumexp(x, 1)
                out[at:at + n, g] = torch.exp(x - lse[at:at + n, g, None]) @ v
        at += n
    return {"out": out, "lse": lse}


def _exact_plan(s):
    ctx, q, P = s["ctx_len"].tolist(), s["q_len"].tolist(), s["page"]
    free, at = s["free"].tolist(), s["cursor"].item()
    table = s["table"].cpu().numpy().copy()
    cu, pos, slot = [0], [], []
    for r, (c, n) in enumerate(zip(ctx, q)):
        cu.append(cu[-1] + n)
        for p in range(c, c + n):
            if p % P == 0:                           # a token that opens a page takes the next free one
                table[r, p // P] = free[at]
                at += 1
            pos.append(p)
            slot.append(int(table[r, p // P]) * P + p % P)
    return {"cu_q": _ints(cu), "kv_len": _ints([c + n for c, n in zip(ctx, q)]), "pos": _ints(pos),
            "slot": _ints(slot), "table": torch.from_numpy(table).to(DEV), "cursor": _ints([at])}
