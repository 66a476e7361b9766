"""Timed calls of the paged serving operators and their plain forms.

Four operators over a key/value cache kept in pages of 64 positions
[num_pages, H_kv, 64, d] behind a page table [B, ceil(N / 64)]:

- append: new tokens' keys and values go to their places in the pages, keys
  (and the queries beside them) rotated by their positions on the way;
- dense_decode: attention of one new token per sequence over its whole cache,
  with an optional tanh cap, window and distance bias;
- selected_decode: attention of one new token per sequence over the 64-key
  blocks that the selector chose for each key head;
- dense_prefill: attention of a prompt, or of a chunk of one, over the cache,
  with an optional tanh cap, window, distance bias, document mask and prefix
  mask.

`own` false: elementary torch operations in 32 bits.  `own` true: the calls
of pyramid_top_block_mean_gb300.pisa.  Lengths follow from the case's numbers,
the contents of every tensor from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 64
DEV = "cuda"


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of the 64-sequence decode workload: one token each, positions up to 131072
        _append("append_step_64", B=64, n=1, ctx=131072, Hq=32, Hkv=8, d=128),
        # the prompts of the pretrain shape: two of up to 4096 tokens
        _append("append_prompt_4k", B=2, n=4096, ctx=4096, Hq=16, Hkv=4, d=128),
        # a few odd-length fp32 prompts behind a cached part, pairs of neighbours rotated, half of the dims
        _append("append_odd_fp32", B=3, n=197, ctx=2049, Hq=4, Hkv=2, d=64, dtype="fp32", rot=32, pairs=True),
        # one short conversation: the smallest call, where latency counts
        _dense_decode("dense_decode_197", B=1, L=197, Hq=16, Hkv=4, d=128),
        # a serving batch of 64 ragged sequences with capped scores
        _dense_decode("dense_decode_64x8k", B=64, L=8192, Hq=32, Hkv=8, d=128, softcap=50.0),
        # two sequences of 131072 tokens: work split over the length
        _dense_decode("dense_decode_2x128k", B=2, L=131072, Hq=32, Hkv=8, d=128),
        # one sequence, eleven blocks a head: latency
        _selected("selected_decode_1", B=1, L=16384, Hq=16, Hkv=4, d=128, K=8),
        # the decode workload's batch, heads and K over caches of the continued-pretrain length
        _selected("selected_decode_64", B=64, L=16384, Hq=32, Hkv=8, d=128, K=32),
        # four short prompts of single-head groups, whose first tokens see each other, with a distance bias
        _dense_prefill("dense_prefill_short", B=4, n=197, past=0, Hq=8, Hkv=8, d=64, slopes=True, prefix=50),
        # two packed prompts of the pretrain shape, documents kept apart
        _dense_prefill("dense_prefill_4k_docs", B=2, n=4096, past=0, Hq=16, Hkv=4, d=128, docs=3),
        # a few tokens (a verified draft, a short turn) behind a long cache: few rows, a long axis
        _dense_prefill("dense_prefill_61_after_64k", B=1, n=61, past=65536, Hq=16, Hkv=4, d=128),
        # a whole 16384-token prompt with capped scores: the largest
        _dense_prefill("dense_prefill_16k_cap", B=1, n=16384, past=0, Hq=16, Hkv=4, d=128, softcap=50.0),
    ]


def _append(name, B, n, ctx, Hq, Hkv, d, dtype="bf16", rot=None, pairs=False):
    return dict(name=name, op="append", B=B, n=n, ctx=ctx, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, rot=rot or d,
                pairs=pairs)


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
    op = rng.choice(["append", "dense_decode", "selected_decode", "dense_prefill"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 8])
    cap = rng.choice([0.0, 0.0, 30.0, 50.0])
    slopes = rng.random() < 0.25
    if op == "append":
        n = 1 if rng.random() < 0.4 else _log(rng, 2, 4096)
        B = _log(rng, 1, max(1, min(64, 8192 // n)))
        c = _append("", B, n, n + _log(rng, 1, 131072 - n), Hq, Hkv, d, rng.choice(["bf16", "bf16", "fp32"]),
                    rng.choice([d, d // 2]), rng.random() < 0.3)
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
        # pairs of one query head and one key, kept under the largest listed case's
        room = 16 * 128 * 16384 * 8192 // (B * Hq * d)
        n = max(1, min(n, int(math.sqrt(room))))
        past = min(past, room // n)
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
        if case["op"] == "append":
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
    if case["op"] == "append":
        size = 2 if case["dtype"] == "bf16" else 4
        tokens = sum(new for _, new in lens)
        moved = 2 * tokens * (Hq + 2 * Hkv) * d * size + tokens * case["rot"] * 4
        return {"bytes": moved, "flops": 3 * tokens * (Hq + Hkv) * case["rot"]}
    if case["op"] == "selected_decode":
        keys = 0
        for length, _ in lens:
            qb = (length - 1) // PAGE
            blocks = min(case["K"], max(0, qb - 2)) + min(qb + 1, 3)
            keys += blocks * PAGE - (qb * PAGE + PAGE - length)
        return {"bytes": keys * Hkv * d * 4 + 4 * B * Hq * d, "flops": 4 * keys * Hq * d}
    keys, pairs, tokens = 0, 0, 0
    for b in range(B):
        lo, hi = _spans(case, b)
        seen = np.maximum(hi - lo + 1, 0)
        pairs += int(seen.sum())
        keys += int(hi.max() - lo.min() + 1)
        tokens += lens[b][1]
    return {"bytes": keys * Hkv * d * 4 + 4 * tokens * Hq * d, "flops": 4 * pairs * Hq * d}


# ------------------------------------------------------------------ inputs
def _rope_table(n, rot):
    """cos and sin of every position's angles, [n, rot]: angles in 64 bits, kept in 32."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    ang = torch.arange(n, device=DEV, dtype=torch.float64)[:, None] * freq[None]
    return torch.cat([ang.cos(), ang.sin()], dim=1).float().contiguous()


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
    append = case["op"] == "append"
    first = [(length - new) // PAGE if append else 0 for length, new in lens]
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
    if append:
        s["kp"] = torch.zeros(pool, Hkv, PAGE, d, device=DEV, dtype=dt)
        s["vp"] = torch.zeros(pool, Hkv, PAGE, d, device=DEV, dtype=dt)
        # queries, keys and values as the projection leaves them: one row of all heads for each token
        qkv = randn(B, n, Hq + 2 * Hkv, d)
        s["q"] = qkv[:, :, :Hq].transpose(1, 2)
        s["k"] = qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
        s["v"] = qkv[:, :, Hq + Hkv:].transpose(1, 2)
        s["rope"] = _rope_table(N, case["rot"])
    else:
        s["kp"] = randn(pool, Hkv, PAGE, d)
        s["vp"] = randn(pool, Hkv, PAGE, d)
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
        s["layer"] = pisa.PagedAttention(p, n=n, rope=s.get("rope"), interleaved=case.get("pairs", False))
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
        if op == "append":
            q = layer.append(s["q"], s["k"], s["v"], s["kp"], s["vp"], s["table"], s["lens"], new_lens=s["new"])
            return {"q": q, "k_pages": s["kp"], "v_pages": s["vp"]}
        if op == "dense_decode":
            return layer.dense_decode(s["q"], s["kp"], s["vp"], s["table"], s["lens"], mask=s["mask"])
        if op == "selected_decode":
            return layer.selected_decode(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["idx"])
        return layer.dense_prefill(s["q"], s["kp"], s["vp"], s["table"], s["lens"], new_lens=s["new"],
                                   mask=s["mask"])
    if op == "append":
        return _plain_append(s)
    if op == "dense_decode":
        return _plain_dense_decode(s)
    if op == "selected_decode":
        return _plain_selected_decode(s)
    return _plain_dense_prefill(s)


def _rotate(x, cos, sin, pairs):
    """x [..., T, d] by its rows' angles (cos, sin [T, rot / 2]); dims from rot on stay."""
    half = cos.shape[1]
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
    half = case["rot"] // 2
    dt = s["q"].dtype
    q_out = torch.zeros(s["q"].shape, device=DEV, dtype=dt)
    for b, (length, new) in enumerate(s["lens_host"]):
        pos = torch.arange(length - new, length, device=DEV)
        cos, sin = s["rope"][pos, :half], s["rope"][pos, half:]
        q_out[b, :, :new] = _rotate(s["q"][b, :, :new].float(), cos, sin, case["pairs"]).to(dt)
        k = _rotate(s["k"][b, :, :new].float(), cos, sin, case["pairs"]).to(dt)
        page = s["table"][b, pos // PAGE].long()
        s["kp"][page, :, pos % PAGE] = k.transpose(0, 1)
        s["vp"][page, :, pos % PAGE] = s["v"][b, :, :new].transpose(0, 1)
    return {"q": q_out, "k_pages": s["kp"], "v_pages": s["vp"]}


def _gather(pages, table, b, lo, hi):
    """Rows lo..hi of sequence b from its pages, [Hkv, hi - lo + 1, d] in 32 bits."""
    j0, j1 = lo // PAGE, hi // PAGE
    x = pages[table[b, j0:j1 + 1].long()].transpose(0, 1).flatten(1, 2)
    return x[:, lo - j0 * PAGE:hi + 1 - j0 * PAGE].float()


def _plain_attend(s, q, k, v, key0, pos, lo, hi, heads):
    """q [H, T, d], k and v [S, d] of one key head; row t sees the keys lo[t]..hi[t]."""
    case = s["case"]
    x = q.float() @ k.t() / math.sqrt(s["d"])
    if case["softcap"]:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    key = torch.arange(key0, key0 + k.shape[0], device=DEV)
    if s["slopes"] is not None:
        x = x + s["slopes"][heads][:, None, None] * (key[None, :] - pos[:, None]).float()
    keep = (key[None, :] >= lo[:, None]) & (key[None, :] <= hi[:, None])
    x = x.masked_fill(~keep, float("-inf"))
    top = x.amax(dim=-1, keepdim=True).clamp_min(-3.0e38)
    e = torch.exp(x - top)
    total = e.sum(dim=-1, keepdim=True)
    return (e @ v) / total.clamp_min(1.0e-30)


def _plain_dense_decode(s):
    case = s["case"]
    G = s["Hq"] // s["Hkv"]
    out = torch.zeros_like(s["q"])
    for b, (length, _) in enumerate(s["lens_host"]):
        lo = max(0, length - case["window"]) if case["window"] else 0
        k = _gather(s["kp"], s["table"], b, lo, length - 1)
        v = _gather(s["vp"], s["table"], b, lo, length - 1)
        q = s["q"][b].float().view(s["Hkv"], G, s["d"])
        x = q @ k.transpose(1, 2) / math.sqrt(s["d"])
        if case["softcap"]:
            x = case["softcap"] * torch.tanh(x / case["softcap"])
        if s["slopes"] is not None:
            back = torch.arange(lo - length + 1, 1, device=DEV).float()
            x = x + s["slopes"].view(s["Hkv"], G, 1) * back
        e = torch.exp(x - x.amax(dim=-1, keepdim=True))
        o = (e @ v) / e.sum(dim=-1, keepdim=True)
        out[b] = o.view(s["Hq"], s["d"]).to(out.dtype)
    return out


def _plain_selected_decode(s):
    G, W = s["Hq"] // s["Hkv"], s["idx"].shape[2]
    blocks = s["idx"].long()
    page = torch.gather(s["table"].long()[:, None].expand(-1, s["Hkv"], -1), 2, blocks.clamp_min(0))
    head = torch.arange(s["Hkv"], device=DEV)[None, :, None]
    k = s["kp"][page, head].flatten(2, 3).float()
    v = s["vp"][page, head].flatten(2, 3).float()
    pos = blocks[..., None] * PAGE + torch.arange(PAGE, device=DEV)
    keep = ((blocks >= 0)[..., None] & (pos < s["lens"][:, None, None, None])).view(s["B"], s["Hkv"], 1, W * PAGE)
    q = s["q"].float().view(s["B"], s["Hkv"], G, s["d"])
    x = (q @ k.transpose(2, 3) / math.sqrt(s["d"])).masked_fill(~keep, float("-inf"))
    e = torch.exp(x - x.amax(dim=-1, keepdim=True))
    o = (e @ v) / e.sum(dim=-1, keepdim=True)
    return o.view(s["B"], s["Hq"], s["d"]).to(s["q"].dtype)


def _plain_dense_prefill(s):
    case = s["case"]
    G = s["Hq"] // s["Hkv"]
    out = torch.zeros_like(s["q"])
    for b, (length, new) in enumerate(s["lens_host"]):
        pos = torch.arange(length - new, length, device=DEV)
        lo = torch.zeros_like(pos)
        if s["first"] is not None:
            lo = torch.maximum(lo, s["first"][b, :new].long())
        if case["window"]:
            lo = torch.maximum(lo, pos - case["window"] + 1)
        hi = pos.clamp_min(case["prefix"] - 1).clamp_max(length - 1)
        k = _gather(s["kp"], s["table"], b, 0, length - 1)
        v = _gather(s["vp"], s["table"], b, 0, length - 1)
        rows = max(64, 2 ** 28 // (G * length))
        for t0 in range(0, new, rows):
            t1 = min(new, t0 + rows)
            # without a prefix the keys after the last row's are seen by none of them
            end = length if case["prefix"] else length - new + t1
            for h in range(s["Hkv"]):
                heads = slice(h * G, (h + 1) * G)
                o = _plain_attend(s, s["q"][b, heads, t0:t1], k[h, :end], v[h, :end], 0, pos[t0:t1], lo[t0:t1],
                                  hi[t0:t1], heads)
                out[b, heads, t0:t1] = o.to(out.dtype)
    return out


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "append":
        return _exact_append(s, f64)
    if work(case)["flops"] > 6.0e12:
        return None
    B, Hq, Hkv, n, d = s["B"], s["Hq"], s["Hkv"], s["n"], s["d"]
    q = s["q"].view(B, Hq, n, d)
    out = torch.zeros(B, Hq, n, d, dtype=f64, device=DEV)
    table = s["table"].cpu().numpy()
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
            k = s["kp"].view(-1, d)[row].to(f64)
            v = s["vp"].view(-1, d)[row].to(f64)
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
    B, Hq, Hkv, n, d, rot = s["B"], s["Hq"], s["Hkv"], s["n"], s["d"], case["rot"]
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

    def turn(x):
        x = x.to(f64)
        y = x.clone()
        y[..., :rot] = x[..., :rot] * cos + x[..., :rot][..., partner] * sin
        return y

    q = turn(s["q"]) * live[:, None, :, None]
    k, v = turn(s["k"]), s["v"].to(f64)
    kp = torch.zeros(s["kp"].shape, dtype=f64, device=DEV).view(-1, Hkv, PAGE, d)
    vp = torch.zeros_like(kp)
    page = torch.gather(s["table"].long(), 1, pos // PAGE)
    b_at, i_at = live.nonzero(as_tuple=True)
    slot = (page[b_at, i_at], slice(None), (pos % PAGE)[b_at, i_at])
    kp[slot] = k[b_at, :, i_at]
    vp[slot] = v[b_at, :, i_at]
    return {"q": q, "k_pages": kp, "v_pages": vp}
