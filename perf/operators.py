"""Timed cases of the operators around the state update: linear attention with
a decay for each head (one-token step and chunked prompt prefill on the slot
pool), the residual-adding RMS norm with an 8-bit output, and the log
probabilities of given tokens.

``run`` computes one pass through an operator, in elementary torch operations
in 32 bits (``own`` false) or through the library's entry points (``own``
true), on what ``prepare`` gives.  ``exact`` states the operators in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
CHUNK = 128  # tokens of one chunk of the plain chunked form
BLOCK = 128  # columns of one scale of a block-scaled norm
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# The cases.
# ---------------------------------------------------------------------------
def listed():
    return [
        # A handful of chats decoding on a model with grouped key / value heads
        # and head sizes that are no powers of two: latency counts.
        dict(name="step_small", op="step", batch=3, heads=24, kv_heads=8, dstate=96, dim=80, io="f16", state="bf16"),
        # A full decode batch: the state pool's traffic is all there is.
        dict(name="step_batch", op="step", batch=256, heads=32, kv_heads=32, dstate=128, dim=128, io="bf16", state="f32"),
        # One short prompt.
        dict(name="prefill_short", op="prefill", tokens=197, nseq=1, heads=16, kv_heads=16, dstate=64, dim=64, io="bf16",
             state="f32", resumed=False),
        # A mixed batch of prompts of uneven lengths, some of them continued
        # from a cached state.
        dict(name="prefill_mixed", op="prefill", tokens=5003, nseq=11, heads=24, kv_heads=8, dstate=96, dim=80, io="f16",
             state="bf16", resumed=True),
        # A full prefill batch.
        dict(name="prefill_batch", op="prefill", tokens=32768, nseq=16, heads=32, kv_heads=32, dstate=128, dim=128,
             io="bf16", state="f32", resumed=True),
        # One long document, its heads alone too few to fill the GPU.
        dict(name="prefill_long", op="prefill", tokens=40001, nseq=1, heads=16, kv_heads=4, dstate=128, dim=128, io="bf16",
             state="f32", resumed=False),
        # The norm before a layer in one decode step, its projections in 8 bits.
        dict(name="norm_decode", op="norm", rows=8, hidden=4096, io="bf16", residual=True, quant="row"),
        # An odd width, 16-bit output.
        dict(name="norm_odd", op="norm", rows=1001, hidden=2565, io="f16", residual=False, quant="none"),
        # A prefill batch's norm with one scale per 128 columns.
        dict(name="norm_batch", op="norm", rows=16384, hidden=8192, io="bf16", residual=True, quant="block"),
        # The drafts of one speculative window.
        dict(name="logprobs_verify", op="logprobs", rows=5, vocab=50001, io="f32", top_k=5),
        # A decode batch's sampled tokens with the alternatives an API returns.
        dict(name="logprobs_decode", op="logprobs", rows=256, vocab=100352, io="f16", top_k=20),
        # Scoring a prompt: every token's logits.
        dict(name="logprobs_prompt", op="logprobs", rows=4096, vocab=131072, io="bf16", top_k=20),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    kv_heads = rng.choice([1, 2, 4, 8, 16, 32])
    heads = kv_heads * rng.choice([r for r in (1, 2, 3, 4, 8) if kv_heads * r <= 64])
    return heads, kv_heads


def draw(rng):
    op = rng.choice(["step", "prefill", "norm", "logprobs"])
    if op == "step":
        heads, kv_heads = _heads(rng)
        dstate, dim = 8 * rng.randint(4, 16), 8 * rng.randint(4, 16)
        state = rng.choice(["f32", "f16", "bf16"])
        most = 256 * 32 * 128 * 128 * 4 // (heads * dstate * dim * BYTES[state])
        return dict(op=op, batch=min(_log_int(rng, 1, 700), most), heads=heads, kv_heads=kv_heads, dstate=dstate, dim=dim,
                    io=rng.choice(["f32", "f16", "bf16"]), state=state)
    if op == "prefill":
        heads, kv_heads = _heads(rng)
        dstate, dim = 8 * rng.randint(4, 16), 8 * rng.randint(4, 16)
        most = min(40000, 32768 * 32 // heads)
        tokens = _log_int(rng, 1, most)
        return dict(op=op, tokens=tokens, nseq=min(tokens, _log_int(rng, 1, 32)), heads=heads, kv_heads=kv_heads,
                    dstate=dstate, dim=dim, io=rng.choice(["f16", "bf16"]), state=rng.choice(["f32", "f16", "bf16"]),
                    resumed=rng.random() < 0.5)
    if op == "norm":
        hidden = rng.choice([8 * rng.randint(32, 1024), rng.randint(200, 8192)])
        rows = _log_int(rng, 1, min(16384, 16384 * 8192 // (2 * hidden)))
        return dict(op=op, rows=rows, hidden=hidden, io=rng.choice(["f32", "f16", "bf16"]), residual=rng.random() < 0.5,
                    quant=rng.choice(["none", "row", "block"]))
    vocab = _log_int(rng, 1000, 262144)
    io = rng.choice(["f32", "f16", "bf16"])
    rows = _log_int(rng, 1, max(1, min(4096, 4096 * 131072 * 2 // (vocab * BYTES[io]))))
    return dict(op=op, rows=rows, vocab=vocab, io=io, top_k=rng.choice([0, 1, 5, 8, 20, 32]))


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _lengths(tokens, nseq, g):
    """``nseq`` lengths of at least one token that add up to ``tokens``, uneven as real prompts are."""
    share = torch.rand(nseq, generator=g).mul_(2.0).exp_()
    cut = torch.floor(share.cumsum(0) / share.sum() * (tokens - nseq)).long()
    cut[-1] = tokens - nseq
    return torch.diff(cut, prepend=torch.zeros(1, dtype=torch.long)).add_(1)


def _chunks(lengths):
    """The plan of the plain chunked form: the token row of every (chunk, place), the chunks' sequences, first tokens
    and lengths, and each sequence's last chunk."""
    per = (lengths + CHUNK - 1) // CHUNK
    n = int(per.sum())
    seq = torch.repeat_interleave(torch.arange(len(lengths)), per)
    first = torch.cumsum(per, 0) - per
    start = (torch.arange(n) - first[seq]) * CHUNK
    size = torch.minimum(lengths[seq] - start, torch.tensor(CHUNK))
    base = torch.cumsum(lengths, 0) - lengths
    place = torch.arange(CHUNK)
    rows = (base[seq] + start)[:, None] + place
    rows = torch.where(place < size[:, None], rows, int(lengths.sum()))  # one row past the end: none
    return dict(rows=rows.to(DEV), seq=seq.to(DEV), start=start.to(DEV), size=size.to(DEV), last=(first + per - 1).to(DEV))


def prepare(case, seed):
    torch.cuda.init()
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    cpu = torch.Generator().manual_seed(int(seed))
    io = DTYPES[case["io"]]

    def normal(*shape, dtype=io, std=1.0):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).mul_(std).to(dtype)

    s = dict(case)
    if case["op"] in ("step", "prefill"):
        H, G, N, P = case["heads"], case["kv_heads"], case["dstate"], case["dim"]
        rows = case["batch"] if case["op"] == "step" else case["tokens"]
        nseq = case["batch"] if case["op"] == "step" else case["nseq"]
        # queries, keys and values are slices of one projection's output
        qkv = normal(rows, H * N + G * N + G * P)
        s["q"] = qkv[:, :H * N].view(rows, H, N)
        s["k"] = qkv[:, H * N:H * N + G * N].view(rows, G, N)
        s["v"] = qkv[:, H * N + G * N:].view(rows, G, P)
        # the decay rates of the heads: a geometric series, from a few tokens' memory to a few thousand's
        s["log_decay"] = -torch.exp2(-torch.linspace(1.0, 10.0, H, device=DEV))
        # a pool with a few slots to spare, handed out in no order; its states as large as a stream of such inputs leaves
        slots = nseq + 3
        s["pool"] = normal(slots, H, P, N, dtype=DTYPES[case["state"]], std=4.0)
        order = torch.randperm(slots, generator=cpu)[:nseq]
        s["slots"] = order.to(device=DEV, dtype=torch.int32)
        if case["op"] == "prefill":
            lengths = _lengths(rows, nseq, cpu)
            s["max_seqlen"] = int(lengths.max())
            s["cu_seqlens"] = torch.cat([torch.zeros(1, dtype=torch.long), lengths.cumsum(0)]).to(device=DEV, dtype=torch.int32)
            # a prompt that resumes reads its slot; a new one starts from zeros (slot -1)
            resumed = (torch.arange(nseq) % 2 == 1) if case["resumed"] else torch.zeros(nseq, dtype=torch.bool)
            s["read"] = torch.where(resumed, order, -1).to(device=DEV, dtype=torch.int32)
            s["lengths"] = lengths.to(DEV)
            s["chunks"] = _chunks(lengths)
    elif case["op"] == "norm":
        R, D = case["rows"], case["hidden"]
        # a residual stream: rows of different sizes, a few columns far larger than the others
        loud = torch.where(torch.rand(D, generator=g, device=DEV) < 0.004, 20.0, 1.0)
        s["x"] = normal(R, D)
        if case["residual"]:
            level = torch.randn(R, 1, generator=g, device=DEV).mul_(0.5).exp_()
            s["residual"] = (torch.randn(R, D, generator=g, device=DEV) * loud * level).to(io)
        s["weight"] = normal(D, std=0.1).add_(1.0)
        s["eps"] = 1e-5
    else:
        R, V = case["rows"], case["vocab"]
        # logits of a trained model: a broad bulk and a few dozen tokens that stand out
        x = normal(R, V, dtype=torch.float32, std=2.0)
        at = torch.randint(V, (R, 48), generator=g, device=DEV)
        x.scatter_add_(1, at, torch.rand(R, 48, generator=g, device=DEV).mul_(14.0))
        s["logits"] = x.to(io)
        pick = torch.randint(48, (R, 1), generator=g, device=DEV)
        s["tokens"] = at.gather(1, pick)[:, 0].contiguous()
    return s


# ---------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------
def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _seed_states(pool, read):
    """The states of the slots ``read``, zeros where it is -1, in 32 bits."""
    states = pool[read.clamp(min=0).long()].float()
    return torch.where((read >= 0)[:, None, None, None], states, 0.0)


def _by_head(t, heads):
    """A per-kv-head tensor [rows, kv_heads, n] for every head, in 32 bits."""
    return t.float().repeat_interleave(heads // t.shape[1], dim=1)


def _plain_step(s):
    H = s["heads"]
    scale = s["dstate"] ** -0.5
    k, v = _by_head(s["k"], H), _by_head(s["v"], H)
    states = _seed_states(s["pool"], s["slots"]) * torch.exp(s["log_decay"])[:, None, None]
    states = states + v[..., :, None] * k[..., None, :]
    y = scale * (states * s["q"].float()[..., None, :]).sum(-1)
    s["pool"][s["slots"].long()] = states.to(s["pool"].dtype)
    return {"y": y.to(s["q"].dtype), "pool": s["pool"]}


def _plain_prefill(s):
    H, T, c = s["heads"], s["tokens"], s["chunks"]
    scale = s["dstate"] ** -0.5
    g = s["log_decay"]
    rows, size = c["rows"], c["size"]

    def chunked(t):  # [chunks, heads, places, n], zeros past a chunk's end
        t = torch.cat([t, t.new_zeros(1, *t.shape[1:])])
        return _by_head(t[rows].flatten(0, 1), H).unflatten(0, rows.shape).transpose(1, 2).contiguous()

    q, k, v = chunked(s["q"]), chunked(s["k"]), chunked(s["v"])
    place = torch.arange(CHUNK, device=DEV)
    gap = place[:, None] - place
    decay = torch.where(gap >= 0, torch.exp(g[:, None, None] * gap.clamp(min=0)), 0.0)
    inside = (q @ k.transpose(-1, -2) * decay) @ v
    # each chunk's own contribution to the state at its end
    left = (size[:, None] - 1 - place).clamp(min=0)
    weight = torch.exp(g[:, None] * left[:, None, :])  # [chunks, heads, places]
    own_state = (v * weight[..., None]).transpose(-1, -2) @ k  # [chunks, heads, dim, dstate]
    # the state that enters each chunk: what the earlier chunks of its sequence left, and the sequence's first state
    end = c["start"] + size
    earlier = (c["seq"][:, None] == c["seq"]) & (c["start"][:, None] >= end)
    reach = torch.where(earlier, torch.exp(g[:, None, None] * (c["start"][:, None] - end).clamp(min=0)), 0.0)
    first = _seed_states(s["pool"], s["read"])[c["seq"]] * torch.exp(g * c["start"][:, None])[:, :, None, None]
    enter = torch.einsum("hnm,mhx->nhx", reach, own_state.flatten(2)).view_as(first) + first
    before = (q @ enter.transpose(-1, -2)) * torch.exp(g[:, None] * (place + 1))[..., None]
    y = q.new_zeros(T + 1, H, s["dim"])
    y[rows.flatten()] = (scale * (inside + before)).transpose(1, 2).flatten(0, 1)
    last = c["last"]
    final = enter[last] * torch.exp(g * size[last][:, None])[:, :, None, None] + own_state[last]
    s["pool"][s["slots"].long()] = final.to(s["pool"].dtype)
    return {"y": y[:T].to(s["q"].dtype), "pool": s["pool"]}


def _plain_norm(s):
    x = s["x"].float()
    if s["residual"] is not False:
        x = x + s["residual"].float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * s["weight"].float()
    out = {"residual": x.to(s["x"].dtype)} if s["residual"] is not False else {}
    if s["quant"] == "none":
        return out | {"y": y.to(s["x"].dtype)}
    R, D = y.shape
    width = D if s["quant"] == "row" else BLOCK
    blocks = -(-D // width)
    yb = torch.nn.functional.pad(y, (0, blocks * width - D)).view(R, blocks, width)
    amax = yb.abs().amax(-1, keepdim=True)
    scales = torch.where(amax > 0, amax / 448.0, 1.0)
    factor = torch.where(amax > 0, (448.0 / amax).clamp(max=torch.finfo(torch.float32).max), 1.0)
    codes = (yb * factor).clamp(-448.0, 448.0).view(R, -1)[:, :D].to(torch.float8_e4m3fn)
    return out | {"codes": codes, "scales": scales.view(R, blocks) if s["quant"] == "block" else scales.view(R)}


def _plain_logprobs(s):
    x = s["logits"].float()
    m = x.amax(-1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    z = e.sum(-1, keepdim=True)
    lse = torch.log(z)
    entropy = (lse - (d * e).sum(-1, keepdim=True) / z)[:, 0]
    logprobs = (d.gather(1, s["tokens"][:, None]) - lse)[:, 0]
    out = {"logprobs": logprobs, "entropy": entropy}
    if s["top_k"]:
        # ties go to the lowest index: order by the value's bits, made monotone, and then by the index downwards
        bits = (x + 0.0).view(torch.int32)
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 32)
        key = key + (0xFFFFFFFF - torch.arange(x.shape[1], device=x.device))
        ids = 0xFFFFFFFF - (torch.topk(key, s["top_k"], dim=-1).values & 0xFFFFFFFF)
        out |= {"top_ids": ids, "top_logprobs": d.gather(1, ids) - lse}
    return out


_plain = {"step": _plain_step, "prefill": _plain_prefill, "norm": _plain_norm, "logprobs": _plain_logprobs}


def _own_step(s):
    import selective_state_update_gb300 as ssu
    y = ssu.ssu_linear_attention_step(s["pool"], s["q"], s["k"], s["v"], s["log_decay"], state_batch_indices=s["slots"])
    return {"y": y, "pool": s["pool"]}


def _own_prefill(s):
    import selective_state_update_gb300 as ssu
    y = ssu.ssu_linear_attention_prefill(s["pool"], s["q"], s["k"], s["v"], s["log_decay"], s["cu_seqlens"],
                                         state_batch_indices=s["read"], dst_state_batch_indices=s["slots"],
                                         max_seqlen=s["max_seqlen"])
    return {"y": y, "pool": s["pool"]}


def _own_norm(s):
    import selective_state_update_gb300 as ssu
    residual = s["residual"] if s["residual"] is not False else None
    y, scales, stream = ssu.ssu_add_rmsnorm(s["x"], s["weight"], eps=s["eps"], residual=residual, quant=s["quant"])
    out = {"residual": stream} if residual is not None else {}
    return out | ({"y": y} if scales is None else {"codes": y, "scales": scales})


def _own_logprobs(s):
    import selective_state_update_gb300 as ssu
    logprobs, entropy, ids, top = ssu.ssu_token_logprobs(s["logits"], s["tokens"], top_k=s["top_k"])
    out = {"logprobs": logprobs, "entropy": entropy}
    return out | ({"top_ids": ids, "top_logprobs": top} if s["top_k"] else {})


_own = {"step": _own_step, "prefill": _own_prefill, "norm": _own_norm, "logprobs": _own_logprobs}


# ---------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------
def work(case):
    io = BYTES[case["io"]]
    if case["op"] in ("step", "prefill"):
        H, G, N, P = case["heads"], case["kv_heads"], case["dstate"], case["dim"]
        rows = case["batch"] if case["op"] == "step" else case["tokens"]
        state = H * N * P * BYTES[case["state"]]
        if case["op"] == "step":
            states = 2 * case["batch"] * state
        else:  # every sequence's state is written, every second one read where prompts resume
            states = (case["nseq"] + (case["nseq"] // 2 if case["resumed"] else 0)) * state
        operands = rows * (H * N + G * N + G * P + H * P) * io
        # a token's rank-1 update, the decay and the read-out
        return {"bytes": states + operands, "flops": rows * H * 5 * N * P}
    if case["op"] == "norm":
        R, D = case["rows"], case["hidden"]
        out = {"none": io * R * D, "row": R * D + 4 * R, "block": R * D + 4 * R * -(-D // BLOCK)}[case["quant"]]
        return {"bytes": R * D * io * (3 if case["residual"] else 1) + D * io + out, "flops": 6 * R * D}
    R, V = case["rows"], case["vocab"]
    return {"bytes": R * V * io + R * (8 + 8 + 12 * case["top_k"]), "flops": 5 * R * V}


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"step": _exact_step, "prefill": _exact_prefill, "norm": _exact_norm, "logprobs": _exact_logprobs}[case["op"]](s)


def _exact_step(s):
    share = s["heads"] // s["kv_heads"]
    kv = torch.arange(s["heads"], device=DEV) // share
    where = s["slots"].long()
    pool = s["pool"].double()
    outer = torch.einsum("bhp,bhn->bhpn", s["v"].double()[:, kv], s["k"].double()[:, kv])
    new = torch.addcmul(outer, pool[where], s["log_decay"].double().exp()[:, None, None])
    y = torch.einsum("bhpn,bhn->bhp", new, s["q"].double()) / math.sqrt(s["dstate"])
    pool[where] = new
    return {"y": y, "pool": pool}


def _exact_prefill(s):
    """The recurrence itself, one token of every sequence after the other."""
    longest = s["max_seqlen"]
    if longest > 45000:
        return None
    H, nseq = s["heads"], s["nseq"]
    kv = torch.arange(H, device=DEV) // (H // s["kv_heads"])
    lam = s["log_decay"].double().exp()[:, None, None]
    base = s["cu_seqlens"][:-1].long()
    pool = s["pool"].double()
    fresh = s["read"] < 0
    state = pool[s["read"].clamp(min=0).long()]
    state[fresh] = 0.0
    y = torch.zeros(s["tokens"], H, s["dim"], dtype=torch.float64, device=DEV)
    lengths = s["lengths"].cpu()
    order = torch.argsort(lengths, descending=True)
    # sequences in order of length, so that those still running are the first ones
    state, base, sorted_lengths = state[order.to(DEV)], base[order.to(DEV)], lengths[order].tolist()
    live = nseq
    for t in range(longest):
        while sorted_lengths[live - 1] <= t:
            live -= 1
        at = base[:live] + t
        k, v, q = s["k"][at].double()[:, kv], s["v"][at].double()[:, kv], s["q"][at].double()
        now = state[:live]
        now.mul_(lam).addcmul_(v.unsqueeze(-1), k.unsqueeze(-2))
        y[at] = torch.matmul(now, q.unsqueeze(-1)).squeeze(-1) / math.sqrt(s["dstate"])
    pool[s["slots"].long()[order.to(DEV)]] = state
    return {"y": y, "pool": pool}


def _exact_norm(s):
    r = s["x"].double()
    out = {}
    if torch.is_tensor(s["residual"]):
        r = r + s["residual"].double()
        out["residual"] = r
    y = s["weight"].double() * r / torch.sqrt(r.pow(2).sum(-1, keepdim=True) / r.shape[1] + s["eps"])
    if s["quant"] == "none":
        return out | {"y": y}
    width = y.shape[1] if s["quant"] == "row" else BLOCK
    parts = [p / p.abs().amax(-1, keepdim=True) * 448 for p in y.split(width, 1)]
    scales = torch.stack([p.abs().amax(-1) / 448 for p in y.split(width, 1)], 1)
    return out | {"codes": torch.cat(parts, 1), "scales": scales if s["quant"] == "block" else scales[:, 0]}


def _exact_logprobs(s):
    logprobs, entropy, top = [], [], []
    for x, token in zip(s["logits"].split(256), s["tokens"].split(256)):
        lp = x.double()
        lp = lp - torch.logsumexp(lp, -1, keepdim=True)
        logprobs.append(lp.gather(1, token[:, None])[:, 0])
        entropy.append(-(lp.exp() * lp).sum(-1))
        top.append(torch.topk(lp, s["top_k"], -1).values if s["top_k"] else None)
    out = {"logprobs": torch.cat(logprobs), "entropy": torch.cat(entropy)}
    return out | ({"top_ids": None, "top_logprobs": torch.cat(top)} if s["top_k"] else {})
