"""Timed calls of the quantised paged cache and of normed appending, and their plain forms.

The cache of the paged serving layer -- pages of 64 positions behind a page
table [B, ceil(N / 64)] -- in 8 bits: e4m3 elements [num_pages, H_kv, 64, d]
and, for each position and key head, one power of two (a biased exponent in a
byte, 2^(byte - 127)) for the keys and one for the values, scales uint8 [2,
num_pages, H_kv, 64].  A row's power is the smallest with which its largest
magnitude is at most 448, e4m3's largest number.  Five operators:

- append: new tokens' keys and queries are normed head by head (root mean
  square over the head, times a weight for each dim), rotated by their
  positions and put into pages of the model's own type;
- quantize: the same, or without norms, into 8-bit pages, which are then read
  back, new tokens first to last, as contiguous tensors;
- dense_decode, selected_decode: attention of one new token per sequence over
  8-bit pages, all of them or the 64-key blocks that the selector chose;
- dense_prefill: attention of a prompt, or of a chunk of one, over 8-bit pages.

`own` false: elementary torch operations.  `own` true: the calls of
pyramid_top_block_mean_gb300.pisa.  Lengths follow from the case's numbers,
the contents of every tensor from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 64
DEV = "cuda"
EPS = 1.0e-6


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of the 64-sequence decode workload with normed heads: one token each, positions up to 131072
        _append("append_norm_step_64", B=64, n=1, ctx=131072, Hq=32, Hkv=8, d=128),
        # the prompts of the pretrain shape, normed heads: two of up to 4096 tokens
        _append("append_norm_prompt_4k", B=2, n=4096, ctx=4096, Hq=16, Hkv=4, d=128),
        # the same decode step into 8-bit pages, its tokens read back
        _quantize("quantize_step_64", B=64, n=1, ctx=131072, Hq=32, Hkv=8, d=128),
        # the same prompts into 8-bit pages and back
        _quantize("quantize_prompt_4k", B=2, n=4096, ctx=4096, Hq=16, Hkv=4, d=128),
        # a few odd-length prompts behind a cached part, without norms, pairs of neighbours rotated, half of the dims
        _quantize("quantize_odd", B=3, n=197, ctx=2049, Hq=4, Hkv=2, d=64, rot=32, pairs=True, norm=False),
        # one short conversation: the smallest attention call, where latency counts
        _dense_decode("dense_decode_e4m3_197", B=1, L=197, Hq=16, Hkv=4, d=128),
        # a serving batch of 64 ragged sequences with capped scores
        _dense_decode("dense_decode_e4m3_64x8k", B=64, L=8192, Hq=32, Hkv=8, d=128, softcap=50.0),
        # two sequences of 131072 tokens: work split over the length
        _dense_decode("dense_decode_e4m3_2x128k", B=2, L=131072, Hq=32, Hkv=8, d=128),
        # one sequence, eleven blocks a head: latency
        _selected("selected_decode_e4m3_1", B=1, L=16384, Hq=16, Hkv=4, d=128, K=8),
        # the decode workload's batch, heads and K over caches of the continued-pretrain length
        _selected("selected_decode_e4m3_64", B=64, L=16384, Hq=32, Hkv=8, d=128, K=32),
        # a few tokens (a verified draft, a short turn) behind a long cache: few rows, a long axis
        _dense_prefill("dense_prefill_e4m3_61_after_64k", B=1, n=61, past=65536, Hq=16, Hkv=4, d=128),
        # the second half of a 16384-token prompt, appended in chunks of 8192: the largest
        _dense_prefill("dense_prefill_e4m3_8k_after_8k", B=1, n=8192, past=8192, Hq=16, Hkv=4, d=128),
    ]


def _append(name, B, n, ctx, Hq, Hkv, d, dtype="bf16", rot=None, pairs=False):
    return dict(name=name, op="append", B=B, n=n, ctx=ctx, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, rot=rot or d,
                pairs=pairs, norm=True)


def _quantize(name, B, n, ctx, Hq, Hkv, d, rot=None, pairs=False, norm=True):
    return dict(name=name, op="quantize", B=B, n=n, ctx=ctx, Hq=Hq, Hkv=Hkv, d=d, dtype="bf16", rot=rot or d,
                pairs=pairs, norm=norm)


def _dense_decode(name, B, L, Hq, Hkv, d, softcap=0.0, window=0, slopes=False):
    return dict(name=name, op="dense_decode", B=B, L=L, Hq=Hq, Hkv=Hkv, d=d, softcap=softcap, window=window,
                slopes=slopes)


def _selected(name, B, L, Hq, Hkv, d, K):
    return dict(name=name, op="selected_decode", B=B, L=L, Hq=Hq, Hkv=Hkv, d=d, K=K)


def _dense_prefill(name, B, n, past, Hq, Hkv, d, softcap=0.0, window=0, slopes=False, docs=0, prefix=0):
    return dict(name=name, op="dense_prefill", B=B, n=n, past=past, Hq=Hq, Hkv=Hkv, d=d, softcap=softcap,
                window=window, slopes=slopes, docs=docs, prefix=prefix)


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    """One more case: every operator, head layout, head size, option and length of the ranges above."""
    op = rng.choice(["append", "quantize", "dense_decode", "selected_decode", "dense_prefill"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 8])
    cap = rng.choice([0.0, 0.0, 30.0, 50.0])
    slopes = rng.random() < 0.25
    if op in ("append", "quantize"):
        n = 1 if rng.random() < 0.4 else _log(rng, 2, 4096)
        B = _log(rng, 1, max(1, min(64, 8192 // n)))
        ctx = n + _log(rng, 1, 131072 - n)
        rot, pairs = rng.choice([d, d // 2]), rng.random() < 0.3
        if op == "append":
            c = _append("", B, n, ctx, Hq, Hkv, d, rng.choice(["bf16", "bf16", "fp32"]), rot, pairs)
        else:
            c = _quantize("", B, n, ctx, Hq, Hkv, d, rot, pairs, rng.random() < 0.6)
    elif op == "dense_decode":
        B = _log(rng, 1, 64)
        L = _log(rng, 1, min(131072, 2 ** 28 // (B * Hkv * d)))
        window = _log(rng, 1, L) if rng.random() < 0.25 else 0
        c = _dense_decode("", B, L, Hq, Hkv, d, cap, window, slopes)
    elif op == "selected_decode":
        B = _log(rng, 1, 64)
        L = _log(rng, 1, min(65536, 2 ** 30 // (B * Hkv * d)))
        c = _selected("", B, L, Hq, Hkv, d, _log(rng, 1, 32))
    else:
        B = rng.choice([1, 1, 2, 4])
        n = _log(rng, 2, 8192)
        past = rng.choice([0, _log(rng, 1, 65536)])
        # pairs of a query and a key of all heads, kept under the largest listed case's
        room = 16 * 128 * 8192 * 12288 // (B * Hq * d)
        n = max(1, min(n, int(math.sqrt(room))))
        past = min(past, max(0, room // n - n))
        window = _log(rng, 1, n + past) if rng.random() < 0.25 else 0
        docs = rng.choice([0, 0, 2, 5])
        prefix = _log(rng, 1, n + past) if rng.random() < 0.25 else 0
        c = _dense_prefill("", B, n, past, Hq, Hkv, d, cap, window, slopes, docs, prefix)
    del c["name"]
    return c


# ------------------------------------------------- lengths that a case implies
def _lengths(case):
    """Per sequence: (length with the new tokens, new tokens)."""
    r = random.Random("%s %d" % (case["op"], case["B"]))
    out = []
    for b in range(case["B"]):
        if case["op"] in ("append", "quantize"):
            new = case["n"] if b == 0 else r.randint((case["n"] + 1) // 2, case["n"])
            past = case["ctx"] - case["n"]
            out.append((new + (past if b == 0 else r.randint(0, past)), new))
        elif case["op"] == "dense_prefill":
            new = case["n"] if b == 0 else r.randint((case["n"] + 1) // 2, case["n"])
            past = case["past"] if b == 0 else r.randint(case["past"] // 2, case["past"])
            out.append((new + past, new))
        else:
            L = case["L"]
            out.append((L if b == 0 else r.randint((L + 1) // 2, L), 1))
    return out


def _first_keys(case, length, new):
    """Document mask: the first position that each new token may read (documents of even length)."""
    pos = np.arange(length - new, length)
    if not case.get("docs"):
        return np.zeros(new, dtype=np.int64)
    step = -(-length // case["docs"])
    return pos // step * step


def _spans(case, b):
    """First and last visible key of each new token of sequence b (last < first: none)."""
    length, new = _lengths(case)[b]
    pos = np.arange(length - new, length)
    lo = _first_keys(case, length, new)
    if case.get("window"):
        lo = np.maximum(lo, pos - case["window"] + 1)
    hi = np.minimum(np.maximum(pos, case.get("prefix", 0) - 1), length - 1)
    return np.maximum(lo, 0), hi


def work(case):
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    lens = _lengths(case)
    if case["op"] in ("append", "quantize"):
        size = 4 if case["dtype"] == "fp32" else 2
        tokens = sum(new for _, new in lens)
        moved = tokens * (case["rot"] * 4 + 2 * Hq * d * size + 2 * Hkv * d * size)
        if case["op"] == "append":
            moved += tokens * 2 * Hkv * d * size
        else:  # written in 8 bits, read from there and written again
            moved += tokens * 2 * Hkv * (2 * (d + 1) + d * size)
        return {"bytes": moved, "flops": tokens * (Hq + Hkv) * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    if case["op"] == "selected_decode":
        keys = 0
        for length, _ in lens:
            qb = (length - 1) // PAGE
            blocks = min(case["K"], max(0, qb - 2)) + min(qb + 1, 3)
            keys += blocks * PAGE - (qb * PAGE + PAGE - length)
        return {"bytes": keys * Hkv * 2 * (d + 1) + 4 * B * Hq * d, "flops": 4 * keys * Hq * d}
    keys, pairs, tokens = 0, 0, 0
    for b in range(B):
        lo, hi = _spans(case, b)
        seen = np.maximum(hi - lo + 1, 0)
        pairs += int(seen.sum())
        keys += int(hi.max() - lo.min() + 1)
        tokens += lens[b][1]
    return {"bytes": keys * Hkv * 2 * (d + 1) + 4 * tokens * Hq * d, "flops": 4 * pairs * Hq * d}


# ------------------------------------------------------------------ inputs
def _rope_table(n, rot):
    """cos and sin of every position's angles, [n, rot]: angles in 64 bits, kept in 32."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    ang = torch.arange(n, device=DEV, dtype=torch.float64)[:, None] * freq[None]
    return torch.cat([ang.cos(), ang.sin()], dim=1).float().contiguous()


def _power(x):
    """Exponent of each row's power of two: the smallest e with max |x| <= 448 2^e."""
    m, e = torch.frexp(x.abs().amax(dim=-1))  # m in [1/2, 1): max = 2 m 2^(e - 1), and 448 = 1.75 2^8
    return (e - 9 + (m > 0.875).to(e.dtype)).clamp(-117, 119)


def _two_to(power, dtype):
    """2^power exactly, for whole powers."""
    if dtype == torch.float64:
        return ((power.long() + 1023) << 52).view(torch.float64)
    return ((power.int() + 127) << 23).view(torch.float32)


def _to_e4m3(x, power):
    """x over 2^power, rounded to the nearest number of e4m3 (ties to even): its values, times 2^power again."""
    scale = _two_to(power, x.dtype)[..., None]
    y = x / scale
    _, e = torch.frexp(y)
    step = _two_to((e - 1).clamp_min(-6) - 3, x.dtype)  # between neighbours
    return (torch.round(y / step) * step).clamp(-448.0, 448.0) * scale


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]
    dt = torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16
    lens = _lengths(case)
    n = case.get("n", 1)
    N = max(length for length, _ in lens)
    nb = -(-N // PAGE)

    def randn(*shape, amp=1.0):
        return (torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * amp).to(dt)

    s = {"case": case, "B": B, "Hq": Hq, "Hkv": Hkv, "d": d, "n": n, "N": N,
         "lens": torch.tensor([x for x, _ in lens], dtype=torch.int32, device=DEV),
         "new": torch.tensor([x for _, x in lens], dtype=torch.int32, device=DEV),
         "lens_host": lens}
    # the pages that the call reads or writes, scattered over a pool with some to spare
    appends = case["op"] in ("append", "quantize")
    first = [(length - new) // PAGE if appends else 0 for length, new in lens]
    last = [(length - 1) // PAGE for length, _ in lens]
    used = sum(hi - lo + 1 for lo, hi in zip(first, last))
    pool = used + used // 8 + 1
    order = torch.randperm(pool, generator=g, device=DEV)[:used].to(torch.int32)
    table = torch.zeros(B, nb, dtype=torch.int32, device=DEV)
    at = 0
    for b in range(B):
        count = last[b] - first[b] + 1
        table[b, first[b]:last[b] + 1] = order[at:at + count]
        at += count
    s["table"] = table
    s["scales"] = None
    if appends:
        in8 = case["op"] == "quantize"
        s["kp"] = torch.zeros(pool, Hkv, PAGE, d, device=DEV, dtype=torch.float8_e4m3fn if in8 else dt)
        s["vp"] = torch.zeros(pool, Hkv, PAGE, d, device=DEV, dtype=torch.float8_e4m3fn if in8 else dt)
        # queries, keys and values as the projection leaves them: one row of all heads for each token
        qkv = randn(B, n, Hq + 2 * Hkv, d)
        s["q"] = qkv[:, :, :Hq].transpose(1, 2)
        s["k"] = qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
        s["v"] = qkv[:, :, Hq + Hkv:].transpose(1, 2)
        s["rope"] = _rope_table(N, case["rot"])
        s["q_norm"] = s["k_norm"] = None
        if case["norm"]:
            s["q_norm"] = 1.0 + 0.25 * torch.randn(d, generator=g, device=DEV)
            s["k_norm"] = 1.0 + 0.25 * torch.randn(d, generator=g, device=DEV)
        if in8:
            s["scales"] = torch.full((2, pool, Hkv, PAGE), 127, dtype=torch.uint8, device=DEV)
            s["k_out"] = torch.zeros(B, Hkv, n, d, dtype=dt, device=DEV)
            s["k_read"], s["v_read"] = torch.zeros_like(s["k_out"]), torch.zeros_like(s["k_out"])
    else:
        # what the appending calls leave of keys and values
        k, v = randn(pool, Hkv, PAGE, d), randn(pool, Hkv, PAGE, d)
        kp, vp = _power(k.float()), _power(v.float())
        s["kp"] = (_to_e4m3(k.float(), kp) * _two_to(-kp, torch.float32)[..., None]).to(torch.float8_e4m3fn)
        s["vp"] = (_to_e4m3(v.float(), vp) * _two_to(-vp, torch.float32)[..., None]).to(torch.float8_e4m3fn)
        s["scales"] = torch.stack([kp, vp]).add(127).to(torch.uint8)
        s["q"] = randn(B, Hq, n, d, amp=2.0) if case["op"] == "dense_prefill" else randn(B, Hq, d, amp=2.0)
    s["slopes"] = None
    if case.get("slopes"):
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device=DEV, dtype=torch.float32) / Hq)
    s["first"] = None
    if case.get("docs"):
        first_key = torch.zeros(B, n, dtype=torch.int32)
        for b, (length, new) in enumerate(lens):
            first_key[b, :new] = torch.from_numpy(_first_keys(case, length, new))
        s["first"] = first_key.to(DEV)
    s["prefix"] = None
    if case.get("prefix"):
        s["prefix"] = torch.full((B,), case["prefix"], dtype=torch.int32, device=DEV)
    if case["op"] == "selected_decode":
        s["idx"] = _selection(case, lens, g)
    if own:
        from pyramid_top_block_mean_gb300 import pisa
        p = pisa.make_params(B, N, Hq, Hkv, d, K=case.get("K", 8), dtype="fp32" if dt == torch.float32 else "bf16")
        s["layer"] = pisa.PagedAttention(p, n=n, rope=s.get("rope"), interleaved=case.get("pairs", False),
                                         q_norm=s.get("q_norm"), k_norm=s.get("k_norm"), norm_eps=EPS)
        s["mask"] = None
        if case.get("softcap") or case.get("window") or s["slopes"] is not None or s["first"] is not None or \
                s["prefix"] is not None:
            s["mask"] = pisa.AttentionMask(softcap=case["softcap"], window=case["window"], slopes=s["slopes"],
                                           first_key=s["first"], prefix_lens=s["prefix"])
    return s


def _selection(case, lens, g):
    """Blocks as the selector returns them: K of the past ones and the first, previous and current, ascending, -1 behind."""
    B, Hkv, K = case["B"], case["Hkv"], case["K"]
    W = K + 3
    out = torch.full((B, Hkv, W), -1, dtype=torch.int32, device=DEV)
    for b, (length, _) in enumerate(lens):
        qb = (length - 1) // PAGE
        forced = sorted({0, max(qb - 1, 0), qb})
        free = max(0, qb - 2)
        take = min(K, free)
        row = torch.tensor(forced, dtype=torch.int64, device=DEV).expand(Hkv, -1)
        if take:
            pick = torch.rand(Hkv, free, generator=g, device=DEV).topk(take, dim=1).indices + 1
            row = torch.cat([row, pick], dim=1)
        out[b, :, :row.shape[1]] = row.sort(dim=1).values.to(torch.int32)
    return out


# --------------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    if own:
        layer = s["layer"]
        cache = (s["kp"], s["vp"], s["table"], s["lens"])
        if op == "append":
            q = layer.append(s["q"], s["k"], s["v"], *cache, new_lens=s["new"])
            return {"q": q, "k_pages": s["kp"], "v_pages": s["vp"]}
        if op == "quantize":
            q = layer.append(s["q"], s["k"], s["v"], *cache, new_lens=s["new"], k_out=s["k_out"], scales=s["scales"])
            layer.read(s["k_read"], s["v_read"], *cache, new_lens=s["new"], scales=s["scales"])
            return {"q": q, "k": s["k_out"], "k_read": s["k_read"], "v_read": s["v_read"]}
        if op == "dense_decode":
            return layer.dense_decode(s["q"], *cache, mask=s["mask"], scales=s["scales"])
        if op == "selected_decode":
            return layer.selected_decode(s["q"], *cache, s["idx"], scales=s["scales"])
        return layer.dense_prefill(s["q"], *cache, new_lens=s["new"], mask=s["mask"], scales=s["scales"])
    if op in ("append", "quantize"):
        return _plain_append(s)
    if op == "selected_decode":
        return _plain_selected_decode(s)
    return _plain_dense(s)


def _norm_rotate(x, weight, cos, sin, pairs):
    """x [B, H, n, d] normed head by head (weight: none, not) and rotated by cos, sin [B, n, rot / 2]."""
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * weight
    half = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    head, tail = x[..., :2 * half], x[..., 2 * half:]
    if pairs:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = head[..., :half], head[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, tail], dim=-1)


def _plain_append(s):
    case = s["case"]
    in8 = case["op"] == "quantize"
    half = case["rot"] // 2
    dt = s["q"].dtype
    i = torch.arange(s["n"], device=DEV)[None]
    live = i < s["new"][:, None]
    pos = (s["lens"][:, None] - s["new"][:, None] + i).clamp(0, s["N"] - 1).long()
    # keys in 64 bits where they are rounded to 8: a value next to a border
    wide = torch.float64 if in8 else torch.float32
    table = s["rope"][pos].to(wide)
    cos, sin = table[..., :half], table[..., half:]
    wq, wk = (w if w is None else w.to(wide) for w in (s["q_norm"], s["k_norm"]))
    q = _norm_rotate(s["q"].to(wide), wq, cos, sin, case["pairs"])
    k = _norm_rotate(s["k"].to(wide), wk, cos, sin, case["pairs"])
    q = torch.where(live[:, None, :, None], q, 0.0).to(dt)
    at = live.nonzero(as_tuple=True)
    page = torch.gather(s["table"].long(), 1, pos // PAGE)[at]
    slot = (pos % PAGE)[at]
    k, v = k.transpose(1, 2)[at], s["v"].transpose(1, 2)[at]  # [tokens, Hkv, d]
    if not in8:
        s["kp"][page, :, slot] = k.to(dt)
        s["vp"][page, :, slot] = v
        return {"q": q, "k_pages": s["kp"], "v_pages": s["vp"]}
    s["k_out"].transpose(1, 2)[at] = k.to(dt)
    for_v = v.to(wide)
    kp, vp = _power(k), _power(for_v)
    for x, power, pages, scales, out in ((k, kp, s["kp"], s["scales"][0], s["k_read"]),
                                         (for_v, vp, s["vp"], s["scales"][1], s["v_read"])):
        codes = (_to_e4m3(x, power) * _two_to(-power, wide)[..., None]).float().to(torch.float8_e4m3fn)
        pages.view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
        scales[page, :, slot] = (power + 127).to(torch.uint8)
        out.transpose(1, 2)[at] = _values(pages, scales, (page, slice(None), slot)).to(dt)
    return {"q": q, "k": s["k_out"], "k_read": s["k_read"], "v_read": s["v_read"]}


def _values(pages, scales, index):
    """What the rows pages[index] stand for, in 32 bits."""
    x = pages.view(torch.uint8)[index].view(torch.float8_e4m3fn).float()
    return x * _two_to(scales[index].int() - 127, torch.float32)[..., None]


def _plain_dense(s):
    """One new token, or n of them, over the whole cache: rows [B, Hkv, G, n], keys [B, Hkv, S]."""
    case, B, Hkv, n, d = s["case"], s["B"], s["Hkv"], s["n"], s["d"]
    G = s["Hq"] // Hkv
    S = s["table"].shape[1] * PAGE
    page = s["table"].long()
    k = _values(s["kp"], s["scales"][0], page).transpose(1, 2).reshape(B, Hkv, 1, S, d)
    v = _values(s["vp"], s["scales"][1], page).transpose(1, 2).reshape(B, Hkv, 1, S, d)
    q = s["q"].float().view(B, Hkv, G, n, d)
    x = torch.matmul(q, k.transpose(3, 4)).div_(math.sqrt(d))
    if case["softcap"]:
        x = x.div_(case["softcap"]).tanh_().mul_(case["softcap"])
    new, lens = s["new"].long()[:, None, None], s["lens"].long()[:, None, None]
    i = torch.arange(n, device=DEV)[None, :, None]
    pos = lens - new + i
    key = torch.arange(S, device=DEV)[None, None, :]
    if s["slopes"] is not None:
        x += s["slopes"].view(1, Hkv, G, 1, 1) * (key - pos).float()[:, None, None]
    hi = pos
    if s["prefix"] is not None:
        hi = torch.maximum(pos, torch.minimum(s["prefix"].long()[:, None, None], lens) - 1)
    keep = (key <= hi) & (i < new)
    if case["window"]:
        keep &= key > pos - case["window"]
    if s["first"] is not None:
        keep &= key >= s["first"].long()[:, :, None]
    x.masked_fill_(~keep[:, None, None], float("-inf"))
    x = x.sub_(x.amax(dim=-1, keepdim=True).clamp_min(-3.0e38)).exp_()
    o = torch.matmul(x, v) / x.sum(dim=-1, keepdim=True).clamp_min(1.0e-30)
    return o.view(s["q"].shape).to(s["q"].dtype)


def _plain_selected_decode(s):
    G, W = s["Hq"] // s["Hkv"], s["idx"].shape[2]
    blocks = s["idx"].long()
    page = torch.gather(s["table"].long()[:, None].expand(-1, s["Hkv"], -1), 2, blocks.clamp_min(0))
    head = torch.arange(s["Hkv"], device=DEV)[None, :, None]
    k = _values(s["kp"], s["scales"][0], (page, head)).flatten(2, 3)
    v = _values(s["vp"], s["scales"][1], (page, head)).flatten(2, 3)
    pos = blocks[..., None] * PAGE + torch.arange(PAGE, device=DEV)
    keep = ((blocks >= 0)[..., None] & (pos < s["lens"][:, None, None, None])).view(s["B"], s["Hkv"], 1, W * PAGE)
    q = s["q"].float().view(s["B"], s["Hkv"], G, s["d"])
    x = (q @ k.transpose(2, 3) / math.sqrt(s["d"])).masked_fill(~keep, float("-inf"))
    e = torch.exp(x - x.amax(dim=-1, keepdim=True))
    o = (e @ v) / e.sum(dim=-1, keepdim=True)
    return o.view(s["B"], s["Hq"], s["d"]).to(s["q"].dtype)


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] in ("append", "quantize"):
        return _exact_append(s, f64)
    if work(case)["flops"] > 6.0e12:
        return None
    B, Hq, Hkv, n, d = s["B"], s["Hq"], s["Hkv"], s["n"], s["d"]
    q = s["q"].view(B, Hq, n, d)
    out = torch.zeros(B, Hq, n, d, dtype=f64, device=DEV)
    table = s["table"].cpu().numpy()
    code = torch.arange(256, device=DEV, dtype=torch.uint8)
    numbers = code.view(torch.float8_e4m3fn).float().to(f64)  # what each of the 256 codes stands for
    bytes_k, bytes_v = (s[x].view(torch.uint8).view(-1, d) for x in ("kp", "vp"))
    powers = _powers_of_two()[s["scales"].view(2, -1).long()]  # 2^(byte - 127)
    for b in range(B):
        length, new = s["lens_host"][b]
        if case["op"] == "selected_decode":
            lo, hi = np.zeros(1, dtype=np.int64), np.array([length - 1])
        else:
            lo, hi = _spans(case, b)
        lo, hi = torch.from_numpy(lo).to(DEV), torch.from_numpy(hi).to(DEV)
        t = torch.arange(length - new, length, device=DEV)
        for h in range(Hkv):
            if case["op"] == "selected_decode":
                block = [j for j in s["idx"][b, h].tolist() if j >= 0]
                at = np.concatenate([np.arange(j * PAGE, min((j + 1) * PAGE, length)) for j in block])
            else:
                at = np.arange(int(lo.min()), length)
            row = torch.from_numpy((table[b, at // PAGE].astype(np.int64) * Hkv + h) * PAGE + at % PAGE).to(DEV)
            key = torch.from_numpy(at).to(DEV)
            k = numbers[bytes_k[row].long()] * powers[0][row][:, None]
            v = numbers[bytes_v[row].long()] * powers[1][row][:, None]
            for head in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                step = max(16, 2 ** 27 // max(1, len(at)))
                for i in range(0, new, step):
                    j = min(new, i + step)
                    # keys behind the last one that these rows see play no part
                    m = int(torch.searchsorted(key, hi[i:j].max(), right=True))
                    z = torch.einsum("td,sd->ts", q[b, head, i:j].to(f64), k[:m]) * d ** -0.5
                    if case.get("softcap"):
                        z = torch.tanh(z / case["softcap"]) * case["softcap"]
                    if s["slopes"] is not None:
                        z = z - s["slopes"][head].to(f64) * (t[i:j, None] - key[None, :m]).to(f64)
                    hidden = torch.logical_or(key[None, :m] < lo[i:j, None], key[None, :m] > hi[i:j, None])
                    weight = torch.softmax(z.masked_fill(hidden, -1.0e300), dim=1).masked_fill(hidden, 0.0)
                    out[b, head, i:j] = torch.einsum("ts,sd->td", weight, v[:m])
    return out if case["op"] == "dense_prefill" else out.view(B, Hq, d)


def _exact_append(s, f64):
    case = s["case"]
    B, Hkv, n, rot = s["B"], s["Hkv"], s["n"], case["rot"]
    half = rot // 2
    # where each rotated dim finds its partner, and with which sign the partner's sine comes in
    dim = torch.arange(rot, device=DEV)
    if case["pairs"]:
        partner, sign, angle = dim ^ 1, torch.where(dim % 2 == 0, -1.0, 1.0), dim // 2
    else:
        partner, sign, angle = (dim + half) % rot, torch.where(dim < half, -1.0, 1.0), dim % half
    length = s["lens"].long()[:, None]
    new = s["new"].long()[:, None]
    i = torch.arange(n, device=DEV)[None]
    pos = (length - new + i).clamp(0, s["N"] - 1)
    live = (i < new)
    cos = s["rope"].to(f64)[pos][..., :half][..., angle][:, None]
    sin = s["rope"].to(f64)[pos][..., half:][..., angle][:, None] * sign.to(f64)

    def turn(x, weight):
        x = x.to(f64)
        if weight is not None:
            mean_square = torch.einsum("bhnd,bhnd->bhn", x, x) / x.shape[-1]
            x = x / torch.sqrt(mean_square + EPS)[..., None] * weight.to(f64)
        y = x.clone()
        y[..., :rot] = x[..., :rot] * cos + x[..., :rot][..., partner] * sin
        return y

    mask = live[:, None, :, None]
    q = turn(s["q"], s["q_norm"]) * mask
    k, v = turn(s["k"], s["k_norm"]), s["v"].to(f64)
    if case["op"] == "quantize":
        # a value is rounded from 64 bits here and from 32 in a kernel: which side of a border a normed and rotated
        # key next to it comes to has no exact answer; values are rounded as they come
        return {"q": q, "k": k * mask, "k_read": None, "v_read": _nearest(v) * mask}
    kp = torch.zeros(s["kp"].shape, dtype=f64, device=DEV).view(-1, Hkv, PAGE, s["d"])
    vp = torch.zeros_like(kp)
    page = torch.gather(s["table"].long(), 1, pos // PAGE)
    b_at, i_at = live.nonzero(as_tuple=True)
    slot = (page[b_at, i_at], slice(None), (pos % PAGE)[b_at, i_at])
    kp[slot] = k[b_at, :, i_at]
    vp[slot] = v[b_at, :, i_at]
    return {"q": q, "k_pages": kp, "v_pages": vp}


def _powers_of_two():
    """2^-127 .. 2^128 in 64 bits."""
    return torch.tensor([2.0 ** e for e in range(-127, 129)], dtype=torch.float64, device=DEV)


def _nearest(x):
    """The nearest e4m3 number times the row's power of two, found among all of them (of two as near, the even code)."""
    codes = torch.arange(127, device=DEV)
    powers = _powers_of_two()
    numbers = torch.where(codes < 8, codes * 2.0 ** -9, (8 + codes % 8) * powers[codes // 8 - 10 + 127])
    # the first of the powers 2^-117 .. 2^119 that takes the row's largest magnitude to 448 or less
    top = x.abs().amax(dim=-1, keepdim=True).contiguous()
    power = powers[10:247][torch.searchsorted(448.0 * powers[10:247], top).clamp_max(236)]
    y = x.abs() / power
    above = torch.searchsorted(numbers, y.contiguous()).clamp(1, 126)
    lo, hi = numbers[above - 1], numbers[above]
    down = torch.where(y - lo == hi - y, (above - 1) % 2 == 0, y - lo < hi - y)
    return torch.sign(x) * torch.where(down, lo, hi) * power
