"""Timed cases of the softmax-attention layers of a hybrid stack: appending
rotated keys and values to a paged cache, and the attention of new tokens --
single ones, drafts, chunks of prompts -- over that cache.

``run`` computes one pass through an operator, in elementary torch operations
in 32 bits (``own`` false) or through the library's entry points (``own``
true), on what ``prepare`` gives.  ``exact`` states the operators in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
SCORES = 1 << 29  # scores that the plain form holds at once


# ---------------------------------------------------------------------------
# The cases.  Each of ``nseq`` sequences has new tokens (``form``: "one" each,
# "drafts" of the same number each, "chunks" of uneven lengths, or "mixed": one
# token for three sequences in four, chunks for the rest) behind up to
# ``context`` tokens that are in the cache already.
# ---------------------------------------------------------------------------
def listed():
    return [
        # A handful of chats, one new token each: latency counts.
        dict(name="append_step", op="append", form="one", nseq=3, tokens=3, context=700, heads=24, kv_heads=8, size=80, page=16,
             io="f16", rotary=80, interleaved=False),
        # A prefill batch's keys and values; pages as long as a recurrent state's slot is large.
        dict(name="append_chunks", op="append", form="chunks", nseq=16, tokens=32768, context=1000, heads=32, kv_heads=8,
             size=128, page=272, io="bf16", rotary=128, interleaved=False),
        # A chunk far into a long document, half of each head rotated, in neighbouring pairs.
        dict(name="append_far", op="append", form="chunks", nseq=1, tokens=2001, context=900000, heads=20, kv_heads=4, size=64,
             page=64, io="bf16", rotary=32, interleaved=True),
        # The same handful of chats: latency counts.
        dict(name="decode_small", op="attend", form="one", nseq=3, tokens=3, context=700, heads=24, kv_heads=8, size=80, page=16,
             io="f16", window=0),
        # A full decode batch.
        dict(name="decode_batch", op="attend", form="one", nseq=256, tokens=256, context=4000, heads=32, kv_heads=8, size=128,
             page=64, io="bf16", window=0),
        # Two long documents, their heads alone too few to fill the GPU.
        dict(name="decode_long", op="attend", form="one", nseq=2, tokens=2, context=130000, heads=16, kv_heads=2, size=128,
             page=272, io="bf16", window=0),
        # The drafts of a speculative window.
        dict(name="drafts", op="attend", form="drafts", nseq=32, tokens=160, context=5000, heads=20, kv_heads=4, size=96,
             page=32, io="f16", window=0),
        # One short prompt.
        dict(name="prompt_short", op="attend", form="chunks", nseq=1, tokens=197, context=0, heads=16, kv_heads=16, size=64,
             page=16, io="bf16", window=0),
        # A running batch: single tokens and chunks of prompts in one call.
        dict(name="mixed", op="attend", form="mixed", nseq=43, tokens=4003, context=6000, heads=24, kv_heads=8, size=96, page=272,
             io="f16", window=0),
        # A full prefill batch.
        dict(name="prompt_batch", op="attend", form="chunks", nseq=16, tokens=32768, context=0, heads=32, kv_heads=8, size=128,
             page=64, io="bf16", window=0),
        # A chunk of a long document.
        dict(name="prompt_long", op="attend", form="chunks", nseq=1, tokens=2048, context=100000, heads=16, kv_heads=4, size=128,
             page=272, io="bf16", window=0),
        # A layer that sees the last 1024 tokens.
        dict(name="prompt_window", op="attend", form="chunks", nseq=4, tokens=16001, context=3000, heads=16, kv_heads=8, size=128,
             page=64, io="bf16", window=1024),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend"])
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    heads = kv_heads * rng.choice([r for r in (1, 2, 3, 4, 5, 8, 16) if kv_heads * r <= 64])
    size = rng.choice([64, 128, 8 * rng.randint(4, 16)])
    page = rng.choice([8, 16, 32, 64, 128, 256, 16 * rng.randint(1, 60)])
    case = dict(op=op, heads=heads, kv_heads=kv_heads, size=size, page=page, io=rng.choice(["f16", "bf16"]))
    form = rng.choice(["one", "drafts", "chunks", "mixed"])
    if form in ("one", "drafts"):
        nseq = _log_int(rng, 1, 256)
        case |= dict(form=form, nseq=nseq, tokens=nseq * (1 if form == "one" else rng.randint(2, 8)))
        most = 256 * 4000 * 8 * 128 // (nseq * kv_heads * size)
        context = _log_int(rng, 1, max(2, min(130000, most)))
    else:
        tokens = _log_int(rng, 2, min(32768, 32768 * 32 // heads))
        nseq = min(tokens // 2, _log_int(rng, 1, 64))
        case |= dict(form=form, nseq=nseq, tokens=tokens)
        # scores to hold and to work through: no more than the chunk of the long document has
        most = 2048 * 100000 * 16 // (tokens * heads)
        context = _log_int(rng, 1, max(2, min(100000, most, 1000000 // nseq)))
    if op == "append":
        rotary = 16 * rng.randint(1, size // 16)
        return case | dict(context=_log_int(rng, 1, min(900000, 1000000 // nseq)), rotary=rotary, interleaved=rng.random() < 0.5)
    return case | dict(context=context, window=rng.choice([0, 0, rng.randint(1, 4096)]))


def _lengths(case):
    """(new tokens, tokens in the cache with them) of every sequence, uneven as real ones are."""
    rng = random.Random(case["nseq"] * 1000003 + case["tokens"])
    n, total = case["nseq"], case["tokens"]
    if case["form"] in ("one", "drafts"):
        new = [total // n] * n
    else:
        share = [math.exp(2.0 * rng.random()) for _ in range(n)]
        if case["form"] == "mixed":
            share = [s if b % 4 == 3 or n < 4 else 0.0 for b, s in enumerate(share)]
        left, scale = total - n, sum(share)
        new = [1 + int(left * s / scale) for s in share]
        new[max(range(n), key=lambda b: new[b])] += total - sum(new)
    context = [0] * n
    if case["context"]:
        context = [int(case["context"] * (0.125 + 0.875 * rng.random())) for _ in range(n)]
    return [(q, c + q) for q, c in zip(new, context)]


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def prepare(case, seed):
    torch.cuda.init()
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    cpu = torch.Generator().manual_seed(int(seed))
    io = DTYPES[case["io"]]
    H, G, D, page, rows = case["heads"], case["kv_heads"], case["size"], case["page"], case["tokens"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(io)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=DEV)

    s = dict(case)
    lengths = _lengths(case)
    s["lengths"] = lengths
    s["max_seqlen"], s["max_kv_len"] = max(q for q, _ in lengths), max(k for _, k in lengths)
    s["kv_lens"] = ints([k for _, k in lengths])
    s["cu_seqlens"] = None
    if case["form"] != "one":
        s["cu_seqlens"] = torch.cat([ints([0]), ints([q for q, _ in lengths]).cumsum(0).int()])
    # pages handed out in no order; the table is as wide as the longest sequence needs, -1 behind a shorter one's pages
    held = [-(-k // page) for _, k in lengths]
    if case["op"] == "append" and sum(held) * page * G * D > 1 << 30:
        # the cache of a far chunk: only the pages that it touches are its own
        s["far"] = True
    first = [(k - q) // page if "far" in s else 0 for q, k in lengths]
    pages = sum(h - f for h, f in zip(held, first)) + 3
    order = torch.randperm(pages, generator=cpu)
    table = torch.full((len(lengths), max(held)), -1, dtype=torch.int32)
    at = 0
    for b, (h, f) in enumerate(zip(held, first)):
        table[b, f:h] = order[at:at + h - f].int()
        at += h - f
    s["block_table"] = table.to(DEV)
    s["k_cache"], s["v_cache"] = normal(pages, page, G, D), normal(pages, page, G, D)
    if case["op"] == "append":
        # queries, keys and values are slices of one projection's output
        qkv = normal(rows, (H + 2 * G) * D).view(rows, H + 2 * G, D)
        s["q"], s["k"], s["v"] = qkv.split([H, G, G], dim=1)
        s["inv_freq"] = torch.pow(10000.0, -torch.arange(0, case["rotary"], 2, device=DEV) / case["rotary"]).float()
    else:
        # heads that look at everything alike and heads that single tokens out
        sharp = torch.exp2(torch.linspace(-1.0, 2.0, H, device=DEV))
        s["q"] = (normal(rows, H, D).float() * sharp[:, None]).to(io)
    return s


# ---------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------
def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _positions(s):
    """(sequence, position) of every new token."""
    n = len(s["lengths"])
    if s["cu_seqlens"] is None:
        seq = torch.arange(n, device=DEV)
        return seq, s["kv_lens"].long() - 1
    cu = s["cu_seqlens"].long()
    new = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), new, output_size=s["tokens"])
    return seq, torch.arange(s["tokens"], device=DEV) - cu[seq] + (s["kv_lens"].long() - new)[seq]


def _plain_append(s):
    seq, pos = _positions(s)
    half = s["rotary"] // 2
    # far positions: the angle in 64 bits
    angle = pos[:, None].double() * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def rotated(t):
        y = t.float()
        if s["interleaved"]:
            a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        else:
            a, b = y[..., :half], y[..., half:2 * half]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        return torch.cat([turned, y[..., 2 * half:]], dim=-1).to(t.dtype)

    page = s["block_table"][seq, pos // s["page"]].long()
    s["k_cache"][page, pos % s["page"]] = rotated(s["k"])
    s["v_cache"][page, pos % s["page"]] = s["v"]
    return {"q": rotated(s["q"]), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _attend(q, k, v, pos, length, window, scale):
    """q [.., rows, share, D], k and v [.., keys, D] in 32 bits, pos [.., rows], length [..]: outputs and their lse."""
    share, rows = q.shape[-2], q.shape[-3]
    x = torch.matmul(q.flatten(-3, -2), k.transpose(-1, -2)).mul_(scale).unflatten(-2, (rows, share))
    key = torch.arange(k.shape[-2], device=DEV)
    seen = (key <= pos[..., None]) & (key < length[..., None, None])
    if window:
        seen &= key > pos[..., None] - window
    x.masked_fill_(~seen[..., None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(m).exp_()
    z = x.sum(-1, keepdim=True)
    out = torch.matmul(x.flatten(-3, -2), v).unflatten(-2, (rows, share)) / z
    return out, (m + torch.log(z))[..., 0]


def _plain_attend(s):
    H, G, D, page = s["heads"], s["kv_heads"], s["size"], s["page"]
    scale, share = D ** -0.5, H // G
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["tokens"], H, dtype=torch.float32, device=DEV)
    table = s["block_table"].long().clamp(min=0)
    if s["form"] in ("one", "drafts"):
        # all sequences at once, as many heads as fit: [nseq, heads, rows, share, D]
        n, rows, keys = s["nseq"], s["tokens"] // s["nseq"], s["max_kv_len"]
        pos = s["kv_lens"].long()[:, None, None] - rows + torch.arange(rows, device=DEV)
        length = s["kv_lens"].long()[:, None]
        step = max(1, SCORES // (n * keys * max(share * rows, 2 * D)))
        for g in range(0, G, step):
            e = min(g + step, G)
            k, v = (c[table, :, g:e].flatten(1, 2)[:, :keys].transpose(1, 2).float() for c in (s["k_cache"], s["v_cache"]))
            q = s["q"][:, g * share:e * share].float().view(n, rows, e - g, share, D).transpose(1, 2)
            o, z = _attend(q, k, v, pos, length, s["window"], scale)
            out[:, g * share:e * share] = o.transpose(1, 2).reshape(n * rows, -1, D).to(out.dtype)
            lse[:, g * share:e * share] = z.transpose(1, 2).reshape(n * rows, -1)
        return {"out": out, "lse": lse}
    t0 = 0
    for b, (rows, keys) in enumerate(s["lengths"]):
        # one sequence's heads at once, as many query rows as fit: [heads, rows, share, D]
        mine = table[b, :-(-keys // page)]
        k, v = (c[mine].flatten(0, 1)[:keys].transpose(0, 1).float() for c in (s["k_cache"], s["v_cache"]))
        step = max(1, SCORES // (H * keys))
        for i in range(0, rows, step):
            n = min(step, rows - i)
            at = slice(t0 + i, t0 + i + n)
            pos = keys - rows + i + torch.arange(n, device=DEV)
            end = keys - rows + i + n  # later keys are not visible to these rows
            lo = max(0, keys - rows + i + 1 - s["window"]) if s["window"] else 0
            q = s["q"][at].float().view(n, G, share, D).transpose(0, 1)
            o, z = _attend(q, k[:, lo:end], v[:, lo:end], pos - lo, torch.tensor(end - lo, device=DEV), s["window"], scale)
            out[at] = o.transpose(0, 1).reshape(n, H, D).to(out.dtype)
            lse[at] = z.transpose(0, 1).reshape(n, H)
        t0 += rows
    return {"out": out, "lse": lse}


_plain = {"append": _plain_append, "attend": _plain_attend}


def _own_append(s):
    import selective_state_update_gb300 as ssu
    q = ssu.ssu_paged_append(s["k_cache"], s["v_cache"], s["k"], s["v"], s["block_table"], s["kv_lens"],
                             cu_seqlens=s["cu_seqlens"], q=s["q"], inv_freq=s["inv_freq"], interleaved=s["interleaved"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attend(s):
    import selective_state_update_gb300 as ssu
    out, lse = ssu.ssu_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"],
                                       cu_seqlens=s["cu_seqlens"], window=s["window"], max_seqlen=s["max_seqlen"],
                                       max_kv_len=s["max_kv_len"], return_lse=True)
    return {"out": out, "lse": lse}


_own = {"append": _own_append, "attend": _own_attend}


# ---------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------
def work(case):
    H, G, D, rows = case["heads"], case["kv_heads"], case["size"], case["tokens"]
    if case["op"] == "append":
        return {"bytes": 2 * rows * (H + 2 * G) * D * 2, "flops": 3 * rows * (H + G) * case["rotary"]}
    keys = pairs = 0
    window = case["window"]
    for q, k in _lengths(case):
        first = max(0, k - q + 1 - window) if window else 0  # the first key that any row sees
        keys += k - first
        for p in (range(k - q, k) if window else ()):
            pairs += min(p + 1, window)
        if not window:
            pairs += q * (k - q) + q * (q + 1) // 2
    return {"bytes": 2 * keys * G * D * 2 + 2 * rows * H * D * 2 + rows * H * 4, "flops": 4 * pairs * H * D}


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_append if case["op"] == "append" else _exact_attend)(s)


def _exact_append(s):
    D, R, page = s["size"], s["rotary"], s["page"]
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    # a pair is one complex number, turned by its position's angle
    i = torch.arange(R // 2, device=DEV)
    left, right = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + R // 2)

    def turn(x, pos):
        y = x.double()
        z = torch.complex(y[..., left], y[..., right])
        z = z * torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos.double()[:, None, None] * s["inv_freq"].double())
        y[..., left], y[..., right] = z.real, z.imag
        return y

    q, t0 = [], 0
    for b, (n, length) in enumerate(s["lengths"]):
        pos = torch.arange(length - n, length, device=DEV)
        rows = slice(t0, t0 + n)
        q.append(turn(s["q"][rows], pos))
        flat = s["block_table"][b].long()[torch.div(pos, page, rounding_mode="floor")] * page + pos.remainder(page)
        k_cache.view(-1, *k_cache.shape[2:])[flat] = turn(s["k"][rows], pos)
        v_cache.view(-1, *v_cache.shape[2:])[flat] = s["v"][rows].double()
        t0 += n
    return {"q": torch.cat(q), "k_cache": k_cache, "v_cache": v_cache}


def _exact_attend(s):
    H, G, D, page, window = s["heads"], s["kv_heads"], s["size"], s["page"], s["window"]
    if sum(q * k for q, k in s["lengths"]) * H * D * 4 > 4e12:
        return None
    share = H // G
    out = torch.empty(s["tokens"], H, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["tokens"], H, dtype=torch.float64, device=DEV)
    t0 = 0
    for b, (n, length) in enumerate(s["lengths"]):
        where = torch.arange(length, device=DEV)
        flat = s["block_table"][b].long()[where // page] * page + where % page
        for g in range(G):
            k = s["k_cache"][:, :, g].reshape(-1, D)[flat].double()
            v = s["v_cache"][:, :, g].reshape(-1, D)[flat].double()
            step = max(1, (SCORES // 4) // (share * length))
            for i in range(0, n, step):
                m = min(step, n - i)
                q = s["q"][t0 + i:t0 + i + m, g * share:(g + 1) * share].double()
                score = torch.einsum("ird,jd->rij", q, k) / math.sqrt(D)
                gap = (length - n + i + torch.arange(m, device=DEV))[:, None] - where
                hidden = (gap < 0) | (gap >= window) if window else gap < 0
                score = score.masked_fill(hidden, -math.inf)
                z = torch.logsumexp(score, -1)
                out[t0 + i:t0 + i + m, g * share:(g + 1) * share] = torch.einsum("rij,jd->ird", torch.exp(score - z[..., None]), v)
                lse[t0 + i:t0 + i + m, g * share:(g + 1) * share] = z.t()
        t0 += n
    return {"out": out, "lse": lse}
