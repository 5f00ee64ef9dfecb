"""Plain forms of the 4-bit cache (helpers of its tests, not a test module)."""
import torch

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def decode(codes, sf):
    """Code times E4M3 scale of codes [..., D / 2] and scales [..., D / 16], float64."""
    lut = torch.tensor(_E2M1 + [-x for x in _E2M1], dtype=torch.float64, device=codes.device)
    v = torch.stack([lut[(codes & 15).long()], lut[(codes >> 4).long()]], -1).flatten(-2)
    return v * sf.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)


def random_cache4(nv, gen, pages, heads, page, dim, k_g=2.0 ** -6, v_g=2.0 ** -5, scale_bytes=(0x28, 0x58)):
    """A 4-bit cache of random codes, with scales between the two bytes' values."""
    u8 = lambda lo, hi, n: torch.randint(lo, hi, (pages, heads, page, n), device="cuda", generator=gen).to(torch.uint8)
    g = lambda x: torch.full((1,), x, device="cuda")
    return nv.KVCache4(u8(0, 256, dim // 2), u8(0, 256, dim // 2), u8(*scale_bytes, dim // 16),
                       u8(*scale_bytes, dim // 16), g(k_g), g(v_g))
