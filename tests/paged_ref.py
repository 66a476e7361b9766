"""Plain 64-bit forms of the paged serving operators, for the GPU tests, and
the bounds that their results are held to.

Bounds.  A rounding to bf16 is off by at most 2^-8 of the value, an fp32 step
by at most 2^-24 (2^-23 where a sum may truncate, as tensor cores do).  With
A = sum_j p_j |v_j| / sum_j p_j, an attention output is off by at most
  2^-8 A                 the weights p are rounded to bf16 before P V,
  2^-8 |o|               the output is rounded to bf16,
  2 ds A                 ds bounds the error of a score (numerator and sum),
  (S + 64) 2^-23 A       sums over S keys in fp32 and the exponentials,
and a score by
  (d + 2) 2^-23 scale sum_i |q_i k_i|      the dot and its scaling,
  cap 2^-20                                tanh's absolute error times the cap,
  4 |bias| 2^-24                           the distance bias.
"""
import numpy as np
import torch

PAGE = 64
NAN = float("nan")


def paginate(x, lens, extra=3, seed=0, fill=NAN, dtype=torch.bfloat16):
    """Scatter [B, H, N, d] into a shuffled pool: positions behind a
    sequence's length and unused pages hold `fill`; table entries behind the
    last used page hold -7."""
    B, H, N, d = x.shape
    nb = -(-N // PAGE)
    used = [-(-int(n) // PAGE) for n in lens]
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(sum(used) + extra, generator=g)
    pages = torch.full((sum(used) + extra, H, PAGE, d), fill, dtype=dtype)
    table = torch.full((B, nb), -7, dtype=torch.int32)
    at = 0
    for b in range(B):
        for j in range(used[b]):
            pg = int(perm[at]); at += 1
            table[b, j] = pg
            m = min(PAGE, int(lens[b]) - j * PAGE)
            pages[pg, :, :m] = x[b, :, j * PAGE:j * PAGE + m].to(dtype)
    return pages, table


def attend(q, k, v, keep, scale, softcap=0.0, bias=None):
    """One head: q [T, d], k and v [S, d], keep bool [T, S], bias [T, S] or
    None.  Returns (out, bound) in 64 bits."""
    q, k, v = q.double(), k.double(), v.double()
    d = q.shape[1]
    dead = ~keep.any(dim=0)  # keys that no row sees may hold anything
    k = torch.where(dead[:, None], torch.zeros((), dtype=torch.float64, device=k.device), k)
    v = torch.where(dead[:, None], torch.zeros((), dtype=torch.float64, device=k.device), v)
    x = scale * (q @ k.t())
    mag = scale * (q.abs() @ k.abs().t())
    ds = (d + 2) * 2.0 ** -23 * torch.where(keep, mag, torch.zeros_like(mag)).amax(dim=1, keepdim=True)
    if softcap:
        x = softcap * torch.tanh(x / softcap)
        ds = ds + softcap * 2.0 ** -20
    if bias is not None:
        x = x + bias
        ds = ds + 4 * 2.0 ** -24 * torch.where(keep, bias.abs(), torch.zeros_like(x)).amax(dim=1, keepdim=True)
    x = x.masked_fill(~keep, -float("inf"))
    mx = x.amax(dim=1, keepdim=True)
    e = torch.where(keep, torch.exp(x - torch.where(torch.isfinite(mx), mx, torch.zeros_like(mx))),
                    torch.zeros_like(x))
    total = e.sum(dim=1, keepdim=True)
    w = torch.where(total > 0, e / total.clamp_min(1e-300), torch.zeros_like(e))
    o, A = w @ v, w @ v.abs()
    S = keep.sum(dim=1, keepdim=True)
    return o, A * (2.0 ** -8 + 2 * ds + (S + 64) * 2.0 ** -23) + 2.0 ** -8 * o.abs() + 1e-30


def spans(pos, length, window=0, first=None, prefix=0):
    lo = torch.zeros_like(pos)
    if first is not None:
        lo = torch.maximum(lo, first.to(lo))
    if window:
        lo = torch.maximum(lo, pos - window + 1)
    return lo, torch.clamp(torch.clamp(pos, min=prefix - 1), max=length - 1)


def dense(q, k, v, length, pos, scale, softcap=0.0, window=0, slopes=None, first=None, prefix=0):
    """One sequence: q [Hq, T, d] at positions pos [T], k and v [Hkv, >= length, d]."""
    G = q.shape[0] // k.shape[0]
    lo, hi = spans(pos, length, window, first, prefix)
    key = torch.arange(length, device=q.device)
    keep = (key[None] >= lo[:, None]) & (key[None] <= hi[:, None])
    back = (key[None] - pos[:, None]).double()
    res = [attend(q[h], k[h // G, :length], v[h // G, :length], keep, scale, softcap,
                  None if slopes is None else slopes[h].double() * back) for h in range(q.shape[0])]
    return torch.stack([r[0] for r in res]), torch.stack([r[1] for r in res])


def selected(q, k, v, length, idx, scale):
    """One sequence: q [Hq, d], k and v [Hkv, >= length, d], idx [Hkv, W]."""
    G = q.shape[0] // k.shape[0]
    qb = (length - 1) // PAGE
    key = torch.arange(length, device=q.device)
    out, tol = [], []
    for h in range(q.shape[0]):
        blocks = [j for j in idx[h // G].tolist() if 0 <= j <= qb]
        keep = torch.isin(key // PAGE, torch.tensor(blocks, device=q.device, dtype=key.dtype))[None]
        o, t = attend(q[h:h + 1], k[h // G, :length], v[h // G, :length], keep, scale)
        out.append(o[0]); tol.append(t[0])
    return torch.stack(out), torch.stack(tol)


def rotate(x, rope, pos, interleaved):
    """x [.., T, d] rotated by the angles of pos [T]; rope [N, rot] cos, sin.
    Returns (rotated, bound) in 64 bits; the bound without the last rounding."""
    rot = rope.shape[1]
    h = rot // 2
    c, s = rope[pos, :h].double(), rope[pos, h:].double()
    x = x.double()
    y, mag = x.clone(), torch.zeros_like(x)
    i = torch.arange(h, device=x.device)
    a_at, b_at = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    a, b = x[..., a_at], x[..., b_at]
    y[..., a_at], y[..., b_at] = a * c - b * s, b * c + a * s
    m = a.abs() * c.abs() + b.abs() * s.abs()
    mag[..., a_at], mag[..., b_at] = m, b.abs() * c.abs() + a.abs() * s.abs()
    return y, 4 * 2.0 ** -24 * mag


def within(got, want, tol, what=""):
    got = got.double()
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, worst error "
                                 f"{float((got - want).abs().max()):.3e} where the bound is "
                                 f"{float(tol.flatten()[(got - want).abs().flatten().argmax()]):.3e}, "
                                 f"first at {np.argwhere(bad.cpu().numpy())[0].tolist()}")
