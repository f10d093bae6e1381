"""Appending to the paged cache against its definition in 64 bits, and the
cache's calls together.

Tolerance: a turned element is x c - y s in fp32, rounded once: the angle is off by
2^-23 at most (its rounding to fp32 below pi), c and s by as much again, the sum by
2^-23 (|x| + |y|); with u half a step of the type that is 2^-21 (|x| + |y|) +
u |result| (fp16: or 2^-25)."""
import pytest
import torch

import selective_state_update_gb300 as ssu
from paged_testlib import DEV, NAN, Batch, attention, check

pytestmark = pytest.mark.gpu


def frequencies(rotary):
    return torch.pow(10000.0, -torch.arange(0, rotary, 2, device=DEV) / rotary).float() if rotary else None


def turned(x, pos, inv_freq, interleaved):
    """x [rows, heads, dim] turned, and the tolerance."""
    y, u = x.double(), torch.finfo(x.dtype).eps / 2
    slack = torch.zeros_like(y)
    if inv_freq is not None:
        half = inv_freq.numel()
        j = torch.arange(half, device=DEV)
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        angle = pos.double()[:, None, None] * inv_freq.double()
        p, q = y[..., a], y[..., b]
        slack[..., a] = slack[..., b] = 2.0 ** -21 * (p.abs() + q.abs())
        y[..., a], y[..., b] = p * angle.cos() - q * angle.sin(), q * angle.cos() + p * angle.sin()
        slack[..., a] += u * y[..., a].abs() + (2.0 ** -25 if x.dtype == torch.float16 else 0.0)
        slack[..., b] += u * y[..., b].abs() + (2.0 ** -25 if x.dtype == torch.float16 else 0.0)
    return y, slack


def new_rows(batch, seed=9, behind=0):
    """q, k, v of the new tokens as slices of one projection."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = batch.rows + behind
    qkv = torch.randn(n, batch.heads + 2 * batch.kv_heads, batch.dim, generator=g, device=DEV).to(batch.io)
    return qkv.split([batch.heads, batch.kv_heads, batch.kv_heads], dim=1)


LENS = {
    "single": [(1, 1), (1, 16), (1, 17), (1, 1000), (1, 0)],
    "chunks": [(5, 5), (0, 7), (40, 300), (1, 1), (17, 33), (3, 0), (6, 2)],
    "one": [(700, 1700)],
    "many": [(i % 3, 40 + i) for i in range(600)],
}


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("io,heads,kv_heads,dim,page,rotary,interleaved,layout", [
    ("bf16", 8, 2, 128, 64, 128, False, "plain"), ("f16", 6, 2, 80, 16, 80, True, "plain"),
    ("bf16", 4, 4, 64, 272, 32, False, "interleaved"), ("f16", 5, 1, 40, 8, 16, True, "heads first"),
    ("bf16", 20, 4, 72, 48, 64, False, "padded"), ("f16", 3, 3, 8, 16, 0, False, "plain"),
])
def test_append(libssu, lens, io, heads, kv_heads, dim, page, rotary, interleaved, layout):
    single = lens == "single"
    wide = torch.int64 if lens == "chunks" else torch.int32
    b = Batch(LENS[lens], heads, kv_heads, dim, page, io, layout=layout, single=single, table_dtype=wide, meta_dtype=wide)
    q, k, v = new_rows(b)
    freq = frequencies(rotary)
    want_k, want_v = b.k_cache.double(), b.v_cache.double()
    slack = torch.zeros_like(want_k)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = ssu.ssu_paged_append(b.k_cache, b.v_cache, k, v, b.table, b.kv_lens, cu_seqlens=b.cu, q=q, inv_freq=freq,
                               interleaved=interleaved, status=status)
    assert int(status.item()) == 0
    for s, (n, kv) in enumerate(b.lens):
        rows = slice(b.starts[s], b.starts[s] + n)
        pos = torch.arange(kv - n, kv, device=DEV)
        y, tol = turned(q[rows], pos, freq, interleaved)
        assert ((out[rows].double() - y).abs() <= tol).all()
        keep = pos >= 0
        y, tol = turned(k[rows], pos, freq, interleaved)
        where = (b.table[s].long()[pos[keep] // page], pos[keep] % page)
        want_k[where], slack[where] = y[keep], tol[keep]
        want_v[where] = v[rows][keep].double()
    # every other place of the caches, NaN or not, is as it was
    assert torch.equal(torch.isnan(b.k_cache), torch.isnan(want_k)) and torch.equal(torch.isnan(b.v_cache), torch.isnan(want_v))
    assert ((b.k_cache.double() - want_k).nan_to_num(0.0).abs() <= slack).all()
    assert torch.equal(b.v_cache.double().nan_to_num(0.5), want_v.nan_to_num(0.5))


@pytest.mark.parametrize("position", [4095, 1 << 17, (1 << 24) + 1, (1 << 27) + 12345])
def test_far_positions(libssu, position):
    # only the last page exists
    page, heads, dim = 4096, 2, 64
    cache = [torch.zeros(1, page, heads, dim, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    table = torch.full((1, position // page + 1), -1, dtype=torch.int32, device=DEV)
    table[0, -1] = 0
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v = (torch.randn(1, heads, dim, generator=g, device=DEV).bfloat16() for _ in range(3))
    freq = frequencies(dim)
    out = ssu.ssu_paged_append(*cache, k, v, table, torch.tensor([position + 1], dtype=torch.int32, device=DEV), q=q, inv_freq=freq)
    pos = torch.tensor([position], device=DEV)
    y, tol = turned(q, pos, freq, False)
    assert ((out.double() - y).abs() <= tol).all()
    y, tol = turned(k, pos, freq, False)
    assert ((cache[0][0, position % page].double() - y[0]).abs() <= tol[0]).all()
    assert torch.equal(cache[1][0, position % page], v[0])


def test_in_place_without_queries_and_rows_of_no_sequence(libssu):
    b = Batch([(5, 9), (30, 40)], 8, 2, 64, 16)
    q, k, v = new_rows(b, behind=3)
    freq = frequencies(64)
    keep = q.clone()
    out = ssu.ssu_paged_append(b.k_cache, b.v_cache, k, v, b.table, b.kv_lens, cu_seqlens=b.cu, q=q, inv_freq=freq)
    got_k, got_v = b.k_cache.clone(), b.v_cache.clone()
    b.k_cache.fill_(0.0)
    b.v_cache.fill_(0.0)
    assert ssu.ssu_paged_append(b.k_cache, b.v_cache, k, v, b.table, b.kv_lens, cu_seqlens=b.cu, inv_freq=freq) is None
    for s in range(2):
        n, kv = b.lens[s]
        assert torch.equal(b.tokens(b.k_cache, s)[kv - n:], b.tokens(got_k, s)[kv - n:])
        assert torch.equal(b.tokens(b.v_cache, s)[kv - n:], b.tokens(got_v, s)[kv - n:])
    assert ssu.ssu_paged_append(b.k_cache, b.v_cache, k, v, b.table, b.kv_lens, cu_seqlens=b.cu, q=q, q_out=q, inv_freq=freq) is q
    assert torch.equal(q[:b.rows], out[:b.rows])
    assert torch.equal(q[b.rows:], keep[b.rows:])


def test_bad_pages_and_lengths(libssu):
    for kv_lens, cu, entry, bit, stored in (([70, 5], [0, 3, 6], 10 ** 6, ssu.DEV_BAD_SLOT, True),
                                            ([70, 5], [0, 3, 6], -1, ssu.DEV_BAD_SLOT, True),
                                            ([70, 500], [0, 3, 6], None, ssu.DEV_BAD_SEQLEN, False),
                                            ([70, -2], [0, 3, 6], None, ssu.DEV_BAD_SEQLEN, False),
                                            ([70, 5], [0, 3, 7], None, ssu.DEV_BAD_SEQLEN, False)):
        b = Batch([(3, 70), (3, 5)], 8, 2, 64, 16)
        q, k, v = new_rows(b)
        b.kv_lens = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
        b.cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        if entry is not None:
            b.table[1, 0] = entry
        b.k_cache.fill_(0.0)
        b.v_cache.fill_(0.0)
        out = torch.full((6, 8, 64), 3.0, dtype=b.io, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        ssu.ssu_paged_append(b.k_cache, b.v_cache, k, v, b.table, b.kv_lens, cu_seqlens=b.cu, q=q, q_out=out,
                             inv_freq=frequencies(64), status=status)
        assert int(status.item()) == bit
        assert torch.equal(b.tokens(b.v_cache, 0)[67:], v[:3])
        assert int((b.v_cache != 0).any(-1).sum()) == 6  # three tokens, two heads
        assert bool((out[3:] == 3.0).all()) != stored


def test_captured(libssu):
    b = Batch([(1, 30), (1, 31)], 8, 2, 64, 16, single=True)
    q, k, v = new_rows(b)
    freq = frequencies(64)
    out = ssu.ssu_paged_append(b.k_cache, b.v_cache, k, v, b.table, b.kv_lens, q=q, inv_freq=freq).clone()
    want = b.k_cache.clone(), b.v_cache.clone()
    b.k_cache.fill_(NAN)
    b.v_cache.fill_(NAN)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ssu.ssu_paged_append(b.k_cache, b.v_cache, k, v, b.table, b.kv_lens, q=q, inv_freq=freq)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, out)
    for s, (n, kv) in enumerate(b.lens):
        for cache, w in zip((b.k_cache, b.v_cache), want):
            assert torch.equal(b.tokens(cache, s)[kv - 1], b.tokens(w, s)[kv - 1])


@pytest.mark.parametrize("io,heads,kv_heads,dim,page,window", [("bf16", 8, 2, 128, 64, 0), ("f16", 6, 2, 80, 48, 40)])
def test_a_run_of_both(libssu, io, heads, kv_heads, dim, page, window):
    """Prompts in chunks, drafts and single tokens, as a server would run them: every call's outputs are the attention of
    what the cache then holds."""
    steps = [[70, 5, 0], [33, 1, 90], [1, 1, 1], [4, 4, 4], [1, 130, 1], [1, 1, 1]]
    total = [sum(s[i] for s in steps) for i in range(3)]
    b = Batch([(0, t) for t in total], heads, kv_heads, dim, page, io)
    b.k_cache.fill_(NAN)
    b.v_cache.fill_(NAN)
    freq = frequencies(16 * (dim // 16))
    held = [0, 0, 0]
    for i, step in enumerate(steps):
        held = [h + s for h, s in zip(held, step)]
        b.lens = list(zip(step, held))
        b.starts = [0, step[0], step[0] + step[1]]
        b.rows = sum(step)
        b.kv_lens = torch.tensor(held, dtype=torch.int32, device=DEV)
        b.cu = None if step == [1, 1, 1] else torch.tensor([*b.starts, b.rows], dtype=torch.int32, device=DEV)
        q, k, v = new_rows(b, seed=i)
        b.q = ssu.ssu_paged_append(b.k_cache, b.v_cache, k, v, b.table, b.kv_lens, cu_seqlens=b.cu, q=q, inv_freq=freq)
        out, lse = ssu.ssu_paged_attention(b.q, b.k_cache, b.v_cache, b.table, b.kv_lens, cu_seqlens=b.cu, window=window,
                                           return_lse=True)
        check(b, out, lse, attention(b, window=window))
        for s in range(3):
            pos = torch.arange(held[s] - step[s], held[s], device=DEV)
            rows = slice(b.starts[s], b.starts[s] + step[s])
            y, tol = turned(k[rows], pos, freq, False)
            assert ((b.tokens(b.k_cache, s)[pos].double() - y).abs() <= tol).all()
            assert torch.equal(b.tokens(b.v_cache, s)[pos], v[rows])
