"""Inputs and 64-bit definitions of the paged cache's calls, for their tests."""
import math

import torch

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
NAN = float("nan")


class Batch:
    """Sequences of (new tokens, tokens in the cache) on a cache whose every row that holds no token of theirs is NaN;
    table entries behind a sequence's pages, and rows of q behind the last sequence, are no numbers either."""

    def __init__(self, lens, heads, kv_heads, dim, page, io="bf16", seed=0, layout="plain", behind=0, table_dtype=torch.int32,
                 meta_dtype=torch.int32, single=False, sharp=1.0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.lens, self.heads, self.kv_heads, self.dim, self.page = lens, heads, kv_heads, dim, page
        self.io, self.single = DTYPES[io], single
        held = [-(-k // page) for _, k in lens]
        pages = sum(held) + 2
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
        width = max(max(held), 1)
        table = torch.full((len(lens), width), -7, dtype=table_dtype)
        at = 0
        for b, h in enumerate(held):
            table[b, :h] = torch.tensor(order[at:at + h], dtype=table_dtype)
            at += h
        self.table = table.to(DEV)
        self.rows = sum(n for n, _ in lens)
        self.k_cache, self.v_cache = self.caches(pages, layout)
        self.k_cache.fill_(NAN)
        self.v_cache.fill_(NAN)
        for b, (n, kv) in enumerate(lens):
            if kv == 0:
                continue
            i = torch.arange(kv, device=DEV)
            where = (self.table[b].long()[i // page], i % page)
            self.k_cache[where] = torch.randn(kv, kv_heads, dim, generator=g, device=DEV).to(self.io)
            self.v_cache[where] = torch.randn(kv, kv_heads, dim, generator=g, device=DEV).to(self.io)
        self.q = torch.full((self.rows + behind, heads, dim), NAN, dtype=self.io, device=DEV)
        self.q[:self.rows] = (sharp * torch.randn(self.rows, heads, dim, generator=g, device=DEV)).to(self.io)
        self.kv_lens = torch.tensor([k for _, k in lens], dtype=meta_dtype, device=DEV)
        cu = [0]
        for n, _ in lens:
            cu.append(cu[-1] + n)
        self.cu = None if single else torch.tensor(cu, dtype=meta_dtype, device=DEV)
        self.starts = cu

    def caches(self, pages, layout):
        G, D, P = self.kv_heads, self.dim, self.page
        new = lambda *shape: torch.empty(shape, dtype=self.io, device=DEV)
        if layout == "plain":
            return new(pages, P, G, D), new(pages, P, G, D)
        if layout == "interleaved":  # a page's keys and values side by side
            both = new(pages, 2, P, G, D)
            return both[:, 0], both[:, 1]
        if layout == "heads first":
            return new(pages, G, P, D).transpose(1, 2), new(pages, G, P, D).transpose(1, 2)
        if layout == "padded":
            both = new(pages, P + 8, G, 2 * D + 8)
            return both[:, :P, :, :D], both[:, :P, :, D + 8:]
        raise ValueError(layout)

    def tokens(self, cache, b):
        i = torch.arange(self.lens[b][1], device=DEV)
        return cache[self.table[b].long()[i // self.page], i % self.page]


def attention(batch, scale=None, window=0):
    """(out, lse, tolerance of out, tolerance of lse), [rows, heads, ...] in 64 bits.

    With u half a step of the io type, and A = scale sum |q_d k_d| of a score: a score in fp32 is off by dim 2^-24 A at
    most (its products are exact, its sums are of dim terms), and by 4 2^-24 |score| for the scaling and the difference
    to the maximum; 2^x adds 2^-22.  So a weight p is off by r = dim 2^-24 A + 2^-22 (|score| + 1) relative, twice that
    with the sum that it is divided by.  The weight meets v rounded, u (fp16: below 2^-14 by 2^-25 absolutely, beside a sum
    that is at least 1), the products' sum of n terms adds n 2^-24, and the output's rounding u |out| (fp16: or 2^-25)."""
    D = batch.dim
    scale = D ** -0.5 if scale is None else scale
    share = batch.heads // batch.kv_heads
    u = torch.finfo(batch.io).eps / 2
    tiny = 2.0 ** -25 if batch.io == torch.float16 else 0.0
    shape = (batch.rows, batch.heads)
    out = torch.zeros(*shape, D, dtype=torch.float64, device=DEV)
    lse = torch.full(shape, -math.inf, dtype=torch.float64, device=DEV)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b, (n, kv) in enumerate(batch.lens):
        if n == 0 or kv == 0:
            continue
        rows = slice(batch.starts[b], batch.starts[b] + n)
        q = batch.q[rows].double()
        k = batch.tokens(batch.k_cache, b).double().repeat_interleave(share, 1)
        v = batch.tokens(batch.v_cache, b).double().repeat_interleave(share, 1)
        x = scale * torch.einsum("ihd,jhd->ihj", q, k)
        size = scale * torch.einsum("ihd,jhd->ihj", q.abs(), k.abs())
        pos = torch.arange(kv - n, kv, device=DEV)[:, None]
        j = torch.arange(kv, device=DEV)
        seen = (j <= pos) & ((j > pos - window) if window else True)
        x = x.masked_fill(~seen[:, None], -math.inf)
        size = size.masked_fill(~seen[:, None], 0.0)
        some = seen.any(-1)[:, None]
        z = torch.logsumexp(x, -1)
        p = torch.where(some[..., None], torch.exp(x - z[..., None]), 0.0)
        out[rows] = torch.einsum("ihj,jhd->ihd", p, v)
        lse[rows] = z
        score = x.masked_fill(~seen[:, None], 0.0).abs().amax(-1)
        r = D * 2.0 ** -24 * size.amax(-1) + 2.0 ** -22 * (score + 1)
        weight = torch.einsum("ihj,jhd->ihd", p, v.abs())
        visible = torch.einsum("ij,jhd->ihd", seen.double(), v.abs())
        tol[rows] = u * out[rows].abs() + tiny + (u + 2 * r[..., None] + kv * 2.0 ** -24) * weight + tiny * visible
        tol_lse[rows] = r + kv * 2.0 ** -24 + 2.0 ** -22 * z.abs().nan_to_num(0, 0, 0)
    return out, lse, tol, tol_lse


def check(batch, out, lse, want):
    ref, ref_lse, tol, tol_lse = want
    n = batch.rows
    wrong = ~((out[:n].double() - ref).abs() <= tol)
    assert not wrong.any(), f"{int(wrong.sum())} outputs off, first at {wrong.nonzero()[0].tolist()}: " \
        f"{out[:n][wrong][:4].tolist()} for {ref[wrong][:4].tolist()}, allowed {tol[wrong][:4].tolist()}"
    none = torch.isinf(ref_lse)
    assert torch.equal(none, torch.isneginf(lse[:n]))
    assert ((lse[:n].double() - ref_lse).abs() <= tol_lse)[~none].all()
