"""Plain 64-bit forms of the 8-bit cache and of head norms, for the tests, and
the bounds that results are held to.

e4m3: code c = s eeee mmm stands for (-1)^s m 2^-9 where eeee is 0, else
(-1)^s (8 + m) 2^(eeee - 10); neighbours of x lie 2^(max(floor log2 |x|, -6) -
3) apart, and a rounding is off by at most half of that.  A row of codes with
the scale s stands for c 2^(s - 127).

A head's norm in fp32 steps: the sum of d squares is off by at most (d + 2)
2^-24 of itself, its root by half of that; mean, eps, root, quotient and the
products with the factor and the weight add at most 8 roundings.
"""
import torch

import paged_ref as R

U = 2.0 ** -24


def two_to(e):
    """2^e exactly (a library's power need not be)."""
    return (e.long() + 1023 << 52).view(torch.float64)


def code_values(device="cpu"):
    """What the 256 codes stand for; NaN for the two that are none."""
    c = torch.arange(256, device=device)
    e, m = c >> 3 & 15, (c & 7).double()
    x = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * two_to(e - 10))
    x = torch.where(c & 127 == 127, torch.full_like(x, float("nan")), x)
    return torch.where(c >= 128, -x, x)


def powers(device="cpu"):
    """2^(s - 127) for the scales 0 .. 254, NaN for 255."""
    return torch.tensor([2.0 ** (s - 127) for s in range(255)] + [float("nan")], dtype=torch.float64, device=device)


def numbers(pages, scales):
    """What pages [..., d] (e4m3) with scales [...] stand for, in 64 bits."""
    dev = pages.device
    return code_values(dev)[pages.view(torch.uint8).long()] * powers(dev)[scales.long()][..., None]


def scale_of(top):
    """The scale of a row with the largest magnitude `top` (64 bits): the smallest power with top <= 448 2^e."""
    steps = 448.0 * powers(top.device)[10:247]
    return 10 + torch.searchsorted(steps, top.contiguous()).clamp_max(236)


def half_step(x, scale):
    """Half the distance of the codes' numbers around x (64 bits) in a row of that scale."""
    power = powers(x.device)[scale.long()]
    _, e = torch.frexp(x.abs() / power)
    return two_to((e - 1).clamp_min(-6) - 4) * power


def quantize(x, dtype=torch.float8_e4m3fn):
    """Rows x [..., d] as (codes, scales): the nearest codes, of two the even one; rows that are not finite as NaN."""
    x = x.double()
    bad = ~torch.isfinite(x).all(dim=-1)
    x = torch.where(bad[..., None], torch.zeros_like(x), x)
    scale = scale_of(x.abs().amax(dim=-1))
    step = 2 * half_step(x, scale[..., None])
    power = powers(x.device)[scale][..., None]
    y = (torch.round(x / step) * step / power).clamp(-448.0, 448.0)  # (round: ties to even)
    scale = torch.where(bad, torch.full_like(scale, 255), scale)
    return y.float().to(dtype), scale.to(torch.uint8)


def norm_rotate(x, weight, eps, rope, pos, interleaved):
    """x [.., T, d] normed (weight None: not) and rotated (rope None: not), with the bound of fp32 steps."""
    x = x.double()
    t = torch.zeros_like(x)
    if weight is not None:
        d = x.shape[-1]
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + eps) * weight.double()
        t = x.abs() * ((d + 2) / 2 + 8) * U
    if rope is None:
        return x, t
    y, more = R.rotate(x, rope, pos, interleaved)
    # the pair's errors come through the rotation with factors of at most one each
    h = rope.shape[1] // 2
    i = torch.arange(h, device=x.device)
    a_at, b_at = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    both = t[..., a_at] + t[..., b_at]
    t = t.clone()
    t[..., a_at], t[..., b_at] = both, both
    return y, t + more


def paginate(x, lens, seed=0, extra=3):
    """Quantises [B, H, N, d] and scatters the rows into a shuffled pool:
    (codes, scales, table, the rows' numbers in 64 bits).  Positions behind a
    sequence's length and unused pages hold what is never written: NaN's codes
    and arbitrary scales, 255 among them."""
    B, H, N, d = x.shape
    codes, scale = quantize(x)
    lens = [max(0, min(int(n), N)) for n in lens]
    pages, table = R.paginate(codes.view(torch.uint8), lens, extra, seed, 0x7f, torch.uint8)
    scales, _ = R.paginate(scale[..., None], lens, extra, seed, 255, torch.uint8)
    rest, _ = R.paginate(torch.zeros(B, H, N, 1), lens, extra, seed, 1.0, torch.float32)
    g = torch.Generator().manual_seed(seed)
    odd = torch.randint(0, 256, scales.shape, generator=g).to(torch.uint8)
    scales = torch.where((rest == 1.0) & (odd < 128), odd, scales)[..., 0].contiguous()
    return pages.view(torch.float8_e4m3fn), scales, table, numbers(codes, scale)
