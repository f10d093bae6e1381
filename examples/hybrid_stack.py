"""A small stack of linear-attention layers served on the library's slot pools:
prompts through the chunked prefill, single tokens through the step, every
layer's input normed to 8 bits, and every token's log probability.

    python examples/hybrid_stack.py [--layers 4] [--new 16] [--attention-every 2]

The weights are random; what the example shows is how the calls fit together.
Per layer and call:

    ssu_add_rmsnorm(..., quant="row")   residual += last output; the normed row as E4M3 codes and one scale
    projection                          q, k, v as slices of one tensor (no copies)
    ssu_linear_attention_prefill/_step  on the layer's pool, through the sequences' slots
    projection

With --attention-every n every n-th layer is softmax attention instead, over a paged
cache of its own whose pages the sequences share:

    ssu_paged_append                    keys and values into their pages, keys and queries turned by their position
    ssu_paged_attention                 of the new tokens over what the cache then holds

and at the end ssu_add_rmsnorm (16-bit), the vocabulary's projection and
ssu_token_logprobs.  It closes by scoring the generated text in one prefill: the
chunked and the recurrent form have to agree.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_update_gb300 as ssu  # noqa: E402

PAD = -1


class HybridStack:
    def __init__(self, vocab=2048, hidden=512, layers=4, heads=8, kv_heads=2, head_size=64, slots=16, quant="row", seed=0,
                 device="cuda", attention_every=0, page=16, pages=128):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=g, device=device) * cols ** -0.5).bfloat16()

        self.heads, self.kv_heads, self.head_size, self.quant = heads, kv_heads, head_size, quant
        self.embed, self.unembed = weight(vocab, hidden) * hidden ** 0.5, weight(vocab, hidden)
        self.wqkv = [weight((heads + 2 * kv_heads) * head_size, hidden) for _ in range(layers)]
        self.wout = [weight(hidden, heads * head_size) for _ in range(layers)]
        self.norms = [torch.ones(hidden, device=device, dtype=torch.bfloat16) for _ in range(layers + 1)]
        # one decay rate per head, from a memory of two tokens to one of a thousand
        self.log_decay = -torch.exp2(-torch.linspace(1.0, 10.0, heads, device=device))
        # one pool per layer; a sequence has the same slot in all of them
        # (an attention layer has pages of keys and values instead)
        attends = [attention_every > 0 and i % attention_every == attention_every - 1 for i in range(layers)]
        self.pools = [tuple(torch.zeros(pages, page, kv_heads, head_size, device=device, dtype=torch.bfloat16) for _ in range(2)) if a
                      else torch.zeros(slots, heads, head_size, head_size, device=device) for a in attends]
        self.page, self.free = page, list(range(pages)) if any(attends) else None  # (None: no layer has pages)
        self.inv_freq = 10000.0 ** -(torch.arange(0, head_size, 2, device=device) / head_size)
        self.held = {}  # slot -> its pages and its number of tokens
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def _project(self, x, scales, w):
        """x w^T, x in 16 bits or as codes with one scale a row (the scale is applied to the product)."""
        if scales is None:
            return x @ w.t()
        return ((x.to(w.dtype) @ w.t()).float() * scales[:, None]).to(w.dtype)

    def forward(self, tokens, mix):
        """Logits of ``tokens``; ``mix(pool, q, k, v)`` is the attention of one layer."""
        delta, stream = self.embed[tokens], None
        for w_in, w_out, norm, pool in zip(self.wqkv, self.wout, self.norms, self.pools):
            x, scales, summed = ssu.ssu_add_rmsnorm(delta, norm, residual=stream, residual_out=stream, quant=self.quant)
            stream = delta if stream is None else summed
            qkv = self._project(x, scales, w_in).unflatten(1, (-1, self.head_size))
            q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], dim=1)
            delta = mix(pool, q, k, v).flatten(1) @ w_out.t()
        x, _, _ = ssu.ssu_add_rmsnorm(delta, self.norms[-1], residual=stream, residual_out=stream)
        return x @ self.unembed.t()

    def _grow(self, slots, new, fresh=False):
        """Room for ``new`` more tokens in each slot's pages, all of them where it is ``fresh``: (block table, lengths
        with them).  Padding has neither."""
        if self.free is None:
            return None, None
        slots = slots.tolist()
        held = {s: ([], 0) if fresh else self.held.get(s, ([], 0)) for s in slots if s != PAD}
        free = self.free + [p for s in held if fresh for p in self.held.get(s, ([], 0))[0]]
        more = {s: (held[s][1] + n + self.page - 1) // self.page - len(held[s][0]) for s, n in zip(slots, new) if s != PAD}
        if sum(more.values()) > len(free):
            raise RuntimeError(f"{sum(more.values())} more pages are needed and {len(free)} are free")
        for s, n in zip(slots, new):
            if s != PAD:
                self.held[s] = held[s][0] + [free.pop() for _ in range(more[s])], held[s][1] + n
        self.free = free
        rows = [self.held[s] if s != PAD else ([], 0) for s in slots]
        wide = max((len(pages) for pages, _ in rows), default=0)
        table = torch.tensor([pages + [PAD] * (wide - len(pages)) for pages, _ in rows], dtype=torch.int32, device=self.embed.device)
        return table.view(len(rows), wide), torch.tensor([n for _, n in rows], dtype=torch.int32, device=self.embed.device)

    def _attend(self, cache, q, k, v, table, lengths, **kw):
        q = ssu.ssu_paged_append(*cache, k, v, table, lengths, q=q, inv_freq=self.inv_freq, cu_seqlens=kw.get("cu_seqlens"),
                                 status=self.status)
        return ssu.ssu_paged_attention(q, *cache, table, lengths, status=self.status, **kw)

    def prefill(self, tokens, lengths, slots):
        """New prompts, packed: their states go to ``slots``."""
        cu = torch.tensor([0, *lengths], device=tokens.device).cumsum(0).int()
        fresh = torch.full_like(slots, PAD)  # every prompt starts from a zero state
        table, kv_lens = self._grow(slots, lengths, fresh=True)  # ... and with no pages

        def mix(pool, q, k, v):
            if isinstance(pool, tuple):
                return self._attend(pool, q, k, v, table, kv_lens, cu_seqlens=cu, max_seqlen=max(lengths), max_kv_len=max(lengths))
            return ssu.ssu_linear_attention_prefill(
                pool, q, k, v, self.log_decay, cu, state_batch_indices=fresh, dst_state_batch_indices=slots, pad_slot_id=PAD,
                max_seqlen=max(lengths), status=self.status)

        return self.forward(tokens, mix)

    def step(self, tokens, slots):
        """One token for the sequence in each slot."""
        table, kv_lens = self._grow(slots, [1] * len(slots))

        def mix(pool, q, k, v):
            if isinstance(pool, tuple):
                return self._attend(pool, q, k, v, table, kv_lens)
            return ssu.ssu_linear_attention_step(
                pool, q, k, v, self.log_decay, state_batch_indices=slots, pad_slot_id=PAD, status=self.status)

        return self.forward(tokens, mix)


def run(layers=4, new=16, lengths=(37, 200, 5), quant="row", top_k=5, seed=0, attention_every=0):
    """Generates ``new`` tokens for prompts of the given lengths.  Returns the generated tokens' log probabilities as
    the steps saw them and as one prefill over the whole texts sees them, [sequences, new] each."""
    model = HybridStack(layers=layers, quant=quant, seed=seed, attention_every=attention_every)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    prompts = [torch.randint(2048, (n,), generator=g, device="cuda") for n in lengths]
    slots = torch.arange(len(lengths), device="cuda", dtype=torch.int32) * 2 + 1

    logits = model.prefill(torch.cat(prompts), lengths, slots)
    last = torch.tensor(lengths, device="cuda").cumsum(0) - 1
    nobody = torch.full((len(lengths),), -1, device="cuda", dtype=torch.int64)
    _, entropy, alternatives, _ = ssu.ssu_token_logprobs(logits[last], nobody, top_k=top_k)
    made, seen = [], []
    for _ in range(new):
        token = alternatives[:, 0].contiguous()  # greedy
        made.append(token)
        seen.append(ssu.ssu_token_logprobs(logits[last] if len(made) == 1 else logits, token)[0])
        logits = model.step(token, slots)
        _, entropy, alternatives, _ = ssu.ssu_token_logprobs(logits, nobody, top_k=top_k)
    made, seen = torch.stack(made, 1), torch.stack(seen, 1)

    # the same texts in one go: token t is predicted by the logits at t - 1
    texts = [torch.cat([p, m]) for p, m in zip(prompts, made)]
    whole = [len(t) for t in texts]
    logits = model.prefill(torch.cat(texts), whole, slots)
    target = torch.cat([torch.cat([t[1:], t.new_full((1,), -1)]) for t in texts])
    scored = ssu.ssu_token_logprobs(logits, target)[0].split(whole)
    again = torch.stack([s[n - 1:n - 1 + new] for s, n in zip(scored, lengths)])
    if int(model.status.item()) != 0:
        raise RuntimeError(f"device status {int(model.status.item())}")
    return seen, again, made, entropy


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--new", type=int, default=16)
    ap.add_argument("--quant", default="row", choices=["none", "row"])
    ap.add_argument("--attention-every", type=int, default=0)
    a = ap.parse_args()
    seen, again, made, entropy = run(layers=a.layers, new=a.new, quant=a.quant, attention_every=a.attention_every)
    for i, (t, s) in enumerate(zip(made.tolist(), seen.tolist())):
        print(f"sequence {i}: " + " ".join(f"{x}({lp:.2f})" for x, lp in zip(t, s)))
    print("entropy of the next token:", [round(x, 3) for x in entropy.tolist()])
    print(f"largest difference between stepping and prefilling: {(seen - again).abs().max().item():.4f} nats")
