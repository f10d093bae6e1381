"""Attention over the paged cache where scores are far apart or far from zero:
what a row's weights come to then has to be the softmax all the same."""
import math

import pytest
import torch

import selective_state_update_gb300 as ssu
from paged_testlib import DEV, Batch

pytestmark = pytest.mark.gpu

# by kernel: single tokens, drafts, rows of tiles, units whose keys are cut, a window that ends inside tiles
FORMS = {
    "single tokens": dict(lens=[(1, 1), (1, 65), (1, 700), (1, 9000)], single=True),
    "drafts": dict(lens=[(3, 70), (3, 3), (3, 900)]),
    "more drafts": dict(lens=[(9, 70), (9, 9), (9, 900)]),
    "chunks": dict(lens=[(90, 700), (300, 300), (40, 1200)]),
    "cut": dict(lens=[(70, 9000)]),
}


def call(b, **kw):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = ssu.ssu_paged_attention(b.q, b.k_cache, b.v_cache, b.table, b.kv_lens, cu_seqlens=b.cu, max_seqlen=max(n for n, _ in b.lens),
                                  return_lse=True, status=status, **kw)
    assert int(status.item()) == 0
    return got


def one_largest(b, size_q, size_k):
    """Queries of positive numbers; in every sequence one key that all of its new tokens see is the largest by far, its
    position another one for each: (the values of it, row by row; its scores in 64 bits; both [rows, heads, ...])."""
    b.q[:b.rows] = (size_q * (b.q[:b.rows].float().abs().clamp(0.0, 2.0) * 0.25 + 0.5)).to(b.io)
    share = b.heads // b.kv_heads
    values, scores = [], []
    for s, (n, kv) in enumerate(b.lens):
        at = (kv - n) * (2 * s + 1) // (2 * len(b.lens))
        i = torch.arange(kv, device=DEV)
        where = (b.table[s].long()[i // b.page], i % b.page)
        k = b.tokens(b.k_cache, s).float().abs().clamp(0.0, 2.0) * -0.25 - 0.25  # every score below zero but one
        k[at] = 1.0
        b.k_cache[where] = (size_k * k).to(b.io)
        page = b.table[s, at // b.page].long()
        key, value = (c[page, at % b.page].double().repeat_interleave(share, 0) for c in (b.k_cache, b.v_cache))
        values.append(value.expand(n, -1, -1))
        scores.append(torch.einsum("ihd,hd->ih", b.q[b.starts[s]:b.starts[s] + n].double(), key))
    return torch.cat(values), torch.cat(scores)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("io,size_q,size_k,scale", [
    ("bf16", 1.0, 1.0, 1e4), ("f16", 1.0, 1.0, 1e6), ("f16", 1.0, 1.0, 1e8), ("bf16", 1.0, 1.0, 1e8), ("bf16", 1.0, 1.0, 1e10),
    ("f16", 1.0, 1.0, 1e30), ("bf16", 1.0, 1.0, 1e30), ("f16", 3e4, 3e4, 1.0), ("bf16", 1e15, 1e15, 1.0), ("bf16", 1e15, 1e15, 1e-3),
])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 128), (6, 2, 40)])
def test_one_key_far_above_the_others(libssu, form, io, size_q, size_k, scale, heads, kv_heads, dim):
    """The largest score is ahead of the others by 0.5 x 1.25 x 40 x 1e4 = 2.5e5 at least, so that every other weight is
    nothing in fp32.  So out is that key's value: the weight, rounded to the io type, over itself, and out's own rounding,
    half a step u each, 2^-20 for the fp32 between.  lse is the score: its
    products have one sign, so dim + 8 roundings of 2^-24 bound what it is off by."""
    b = Batch(heads=heads, kv_heads=kv_heads, dim=dim, page=48, io=io, **FORMS[form])
    value, score = one_largest(b, size_q, size_k)
    score = score * scale
    assert score.max() < 2e38  # (in units of log2 it stays finite)
    out, lse = call(b, scale=scale)
    u = torch.finfo(b.io).eps / 2
    tiny = 2.0 ** -25 if b.io == torch.float16 else 0.0
    wrong = ~((out.double() - value).abs() <= (2 * u + 2.0 ** -20) * value.abs() + tiny)
    assert not wrong.any(), (int(wrong.sum()), wrong.nonzero()[0].tolist(), out[wrong][:4].tolist(), value[wrong][:4].tolist())
    off = ((lse.double() - score).abs() / score).max()
    assert math.isfinite(float(off)) and off <= (dim + 8) * 2.0 ** -24


@pytest.mark.parametrize("lens,single", [([(1, 20000), (1, 3000)], True), ([(3, 20000), (3, 3000)], False), ([(9, 20000), (9, 3000)], False),
                                         ([(40, 20000), (300, 3000)], False), ([(2000, 2600)], False)])
@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("gap", [20.0, 25.0, 27.5])
def test_many_small_weights_beside_a_large_one(libssu, lens, single, io, gap):
    """A sequence's first token, whose value is zero, is ahead of the others by about 2^gap.  What is left is their
    part of the weight, right to the roundings of the weights, which for fp16 are half a step u of each and, of those
    below 2^-21 of the largest one, 2^-32 of it (the largest is held as 2^7 or more, and below 2^-14 fp16 rounds by
    2^-25); the other terms are those of ``paged_testlib.attention``."""
    b = Batch(lens, 4, 2, 64, 48, io, single=single)
    u = torch.finfo(b.io).eps / 2
    g = torch.Generator(device=DEV).manual_seed(3)
    b.q[:b.rows] = 0.0
    b.q[:b.rows, :, 0] = 1.0
    b.q[:b.rows, :, 1] = (torch.randn(b.rows, 4, generator=g, device=DEV) * 0.5).to(b.io)
    for s, (n, kv) in enumerate(lens):
        i = torch.arange(kv, device=DEV)
        where = (b.table[s].long()[i // 48], i % 48)
        k = b.tokens(b.k_cache, s).float() * 0.5
        k[:, :, 0] = 0.0
        k[0, :, 0], k[0, :, 1] = gap, 0.0
        v = b.tokens(b.v_cache, s).float().abs() + 0.5
        v[0] = 0.0
        b.k_cache[where], b.v_cache[where] = k.to(b.io), v.to(b.io)
    scale = math.log(2.0)
    out, lse = call(b, scale=scale)
    for s, (n, kv) in enumerate(lens):
        q = b.q[b.starts[s]:b.starts[s] + n].double()
        k, v = (b.tokens(c, s).double().repeat_interleave(2, 1) for c in (b.k_cache, b.v_cache))
        x = scale * torch.einsum("ihd,jhd->ihj", q, k)
        size = scale * torch.einsum("ihd,jhd->ihj", q.abs(), k.abs()).amax(-1)
        seen = torch.arange(kv, device=DEV) <= torch.arange(kv - n, kv, device=DEV)[:, None]
        x = x.masked_fill(~seen[:, None], -math.inf)
        p = torch.softmax(x, -1)
        want = torch.einsum("ihj,jhd->ihd", p, v)
        r = 64 * 2.0 ** -24 * size + 2.0 ** -22 * (scale * gap + 1)
        tol = (2 * u + 2 * r[..., None] + kv * 2.0 ** -24) * want + (2.0 ** -25 if io == "f16" else 0.0)
        tol += p.amax(-1)[..., None] * 2.0 ** -32 * torch.einsum("ij,jhd->ihd", seen.double(), v)
        got = out[b.starts[s]:b.starts[s] + n].double()
        wrong = ~((got - want).abs() <= tol)
        assert not wrong.any(), (s, int(wrong.sum()), got[wrong][:4].tolist(), want[wrong][:4].tolist(), tol[wrong][:4].tolist())
        z = torch.logsumexp(x, -1)
        assert ((lse[b.starts[s]:b.starts[s] + n].double() - z).abs() <= r + kv * 2.0 ** -24 + 2.0 ** -22 * z.abs()).all()
