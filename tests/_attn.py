"""Plain binary64 forms of the attention operators, request by request
(helpers of the attention tests, not a test module)."""
import math

import torch

# |out - ref| <= 2^-8 |ref| (the output's rounding to bf16: half a step)
#             + (2^-8 + 2^-11) sum_j p_j |v_j|
# where 2^-8 is the rounding of each probability to bf16 and 2^-11 covers the
# binary32 scores: a score's error is below 2^-15 for the sizes tested (|q|,
# |k| entries of a few units, head_dim <= 128: 128 products' accumulation
# errors of 2^-23 sum |q k| scale, sum |q k| scale <= 2^8), and a relative
# error of 2^-15 in each p, numerator and sum, stays far below 2^-11.
OUT_REL = 2.0 ** -8
OUT_P = 2.0 ** -8 + 2.0 ** -11
# lse: the same score error, plus the binary32 logarithm and sum
LSE_ABS = 2.0 ** -14
LSE_REL = 2.0 ** -20


def reference(q, keys, vals, ctx, scale, window=0):
    """One request: q [n, H, D], keys/vals [L, Hkv, D] float64 (the rows a
    request's tokens may see), its first row at position ctx.  Returns out,
    sum p|v|, lse."""
    n, H, D = q.shape
    L, Hkv, _ = keys.shape
    out, mag = (torch.zeros(n, H, D, dtype=torch.float64, device=q.device) for _ in range(2))
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device=q.device)
    i = torch.arange(n, device=q.device)[:, None] + ctx
    j = torch.arange(L, device=q.device)[None, :]
    seen = j <= i
    if window:
        seen &= j > i - window
    rows = seen.any(1)
    for h in range(H):
        k, v = keys[:, h * Hkv // H], vals[:, h * Hkv // H]
        s = (q[:, h] @ k.T) * scale
        s[~seen] = -math.inf
        top = s.amax(1, keepdim=True)
        p = torch.where(seen, torch.exp(s - torch.where(top == -math.inf, 0.0, top)), 0.0)
        tot = p.sum(1, keepdim=True)
        p = p / torch.where(tot == 0, 1.0, tot)
        out[:, h], mag[:, h] = p @ v, p @ v.abs()
        lse[rows, h] = (top + torch.log(tot))[rows, 0]
    return out, mag, lse


def check(out, lse, ref, mag, ref_lse, what=""):
    err = (out.double() - ref).abs()
    bound = OUT_REL * ref.abs() + OUT_P * mag + 1e-30
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first at "
                           f"{bad.nonzero()[0].tolist()}: {out[tuple(bad.nonzero()[0])].item()} for "
                           f"{ref[tuple(bad.nonzero()[0])].item()}")
    if lse is not None:
        same = (lse.double() == ref_lse) | ((lse.double() - ref_lse).abs() <= LSE_ABS + LSE_REL * ref_lse.abs())
        assert same.all(), f"{what}: lse off at {(~same).nonzero()[0].tolist()}"
