"""Plain forms of the 4-bit weights: random codes and scales, and their exact
values in float64."""
import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def pitch(H, group):
    return (H // group + 15) // 16 * 16


def scale64(code, group):
    if group == 16:
        return code.view(torch.float8_e4m3fn).double()
    return torch.where(code == 255, float("nan"), torch.exp2(code.double() - 127.0))


def code64(codes):
    """Values of packed E2M1 codes [..., H / 2] -> [..., H]."""
    both = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).long()
    v = E2M1.to(codes.device).double()[both & 7]
    return torch.where(both > 7, -v, v)


def value64(codes, scales, group):
    H = codes.shape[-1] * 2
    s = scale64(scales[..., :H // group].contiguous(), group)
    return code64(codes) * s.repeat_interleave(group, dim=-1)


def random_w4(lead, rows, H, group, g, pad=None):
    """Codes [*lead, rows, H / 2] of all sixteen kinds and scales [*lead, rows,
    pitch] of about H ** -0.5 (some negative, zero or subnormal among the E4M3
    ones); the padding holds NaN codes."""
    codes = torch.randint(0, 256, (*lead, rows, H // 2), generator=g, dtype=torch.uint8)
    n = H // group
    sc = torch.full((*lead, rows, pitch(H, group) if pad is None else pad),
                    0x7F if group == 16 else 0xFF, dtype=torch.uint8)
    if group == 16:
        s = (torch.rand(*lead, rows, n, generator=g) + 0.5) * H ** -0.5 * 0.5
        s = torch.where(torch.rand(s.shape, generator=g) < 0.1, -s, s)
        s = torch.where(torch.rand(s.shape, generator=g) < 0.05, 0.0, s)
        s = torch.where(torch.rand(s.shape, generator=g) < 0.05, 2.0 ** -8, s)
        sc[..., :n] = s.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        base = 127 - 2 - int(H).bit_length() // 2
        sc[..., :n] = torch.randint(base - 3, base + 2, (*lead, rows, n), generator=g,
                                    dtype=torch.uint8)
    return codes, sc
