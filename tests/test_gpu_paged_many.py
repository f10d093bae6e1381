"""The paged cache's calls on many rows: appends whose CTAs take one, two and four
rows, and attention with many pieces of work a CTA.  Tolerances are those of
``test_gpu_paged_append`` and ``paged_testlib``."""
import pytest
import torch

import selective_state_update_gb300 as ssu
from paged_testlib import DEV, NAN, Batch, attention, check
from test_gpu_paged_append import frequencies, new_rows, turned

pytestmark = pytest.mark.gpu


def drawn(count, new, context, seed):
    g = torch.Generator().manual_seed(seed)
    n, c = (torch.randint(lo, hi + 1, (count,), generator=g).tolist() for lo, hi in (new, context))
    return list(zip(n, (a + b for a, b in zip(n, c))))


APPENDS = {
    "single": dict(lens=[(1, k) for _, k in drawn(1300, (0, 0), (0, 150), 1)], single=True),
    "short ones": dict(lens=drawn(1500, (0, 5), (0, 60), 2)),
    "chunks": dict(lens=[(700, 900), (0, 3), (1301, 1301), (1, 40), (2, 1), (333, 4000)]),
}


# heads + 2 kv_heads by 16 elements of a head: the pieces of a row, which say how many rows a CTA takes
@pytest.mark.parametrize("lens", APPENDS, ids=lambda s: s.replace(" ", "_"))
@pytest.mark.parametrize("io,heads,kv_heads,dim,page,rotary,interleaved,layout", [
    ("bf16", 32, 8, 128, 16, 128, False, "plain"), ("f16", 32, 8, 128, 48, 64, True, "plain"),         # one row: 384
    ("bf16", 16, 4, 128, 16, 32, True, "interleaved"), ("f16", 17, 1, 104, 24, 96, False, "padded"),   # two: 192, 133
    ("bf16", 8, 2, 64, 16, 64, False, "heads first"), ("f16", 5, 1, 40, 8, 16, True, "plain"),         # four: 48, 21
    ("bf16", 1, 1, 8, 16, 0, False, "plain"),                                                          # four: 3
])
@pytest.mark.parametrize("queries", ["out", "in place", "none"])
def test_append_of_many_rows(libssu, lens, io, heads, kv_heads, dim, page, rotary, interleaved, layout, queries):
    b = Batch(heads=heads, kv_heads=kv_heads, dim=dim, page=page, io=io, layout=layout, **APPENDS[lens])
    assert b.rows > 8 * torch.cuda.get_device_properties(0).multi_processor_count
    q, k, v = new_rows(b)
    freq = frequencies(rotary)
    seq = torch.repeat_interleave(torch.arange(len(b.lens), device=DEV), torch.tensor([n for n, _ in b.lens], device=DEV))
    pos = torch.arange(b.rows, device=DEV) + torch.tensor([kv - n - s for (n, kv), s in zip(b.lens, b.starts)], device=DEV)[seq]
    want_q, slack_q = turned(q, pos, freq, interleaved)
    y, tol = turned(k, pos, freq, interleaved)
    want_k, want_v = b.k_cache.double(), b.v_cache.double()
    slack = torch.zeros_like(want_k)
    keep = pos >= 0
    where = (b.table[seq[keep], pos[keep] // page].long(), pos[keep] % page)
    want_k[where], slack[where], want_v[where] = y[keep], tol[keep], v[keep].double()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw = dict(out=dict(q=q), none={}).get(queries) if queries != "in place" else dict(q=q, q_out=q)
    out = ssu.ssu_paged_append(b.k_cache, b.v_cache, k, v, b.table, b.kv_lens, cu_seqlens=b.cu, inv_freq=freq, interleaved=interleaved,
                               status=status, **kw)
    assert int(status) == 0
    if queries != "none":
        assert ((out.double() - want_q).abs() <= slack_q).all()
    assert torch.equal(torch.isnan(b.k_cache), torch.isnan(want_k)) and torch.equal(torch.isnan(b.v_cache), torch.isnan(want_v))
    assert ((b.k_cache.double() - want_k).nan_to_num(0.0).abs() <= slack).all()
    assert torch.equal(b.v_cache.double().nan_to_num(0.5), want_v.nan_to_num(0.5))


@pytest.mark.parametrize("heads,kv_heads,dim", [(32, 8, 128), (16, 4, 128), (8, 2, 64)])
def test_append_of_many_rows_with_bad_ones_among_them(libssu, heads, kv_heads, dim):
    """Every seventh sequence has a length that its table has no room for, every eleventh no page: neither is stored, their
    neighbours in a CTA are."""
    lens = drawn(900, (1, 3), (0, 30), 4)
    b = Batch(lens, heads, kv_heads, dim, 16)
    q, k, v = new_rows(b, behind=9)
    held = [k if s % 7 else 10 ** 6 for s, (_, k) in enumerate(lens)]
    b.kv_lens = torch.tensor(held, dtype=torch.int32, device=DEV)
    b.table[::11] = -1
    b.k_cache.fill_(NAN)
    b.v_cache.fill_(NAN)
    out = torch.full((b.rows + 9, heads, dim), 3.0, dtype=b.io, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ssu.ssu_paged_append(b.k_cache, b.v_cache, k, v, b.table, b.kv_lens, cu_seqlens=b.cu, q=q, q_out=out, inv_freq=frequencies(dim),
                         status=status)
    assert int(status) == ssu.DEV_BAD_SEQLEN | ssu.DEV_BAD_SLOT
    stored = 0
    for s, (n, kv) in enumerate(lens):
        rows = slice(b.starts[s], b.starts[s] + n)
        if s % 7 == 0:
            assert (out[rows] == 3.0).all()
            continue
        assert not (out[rows] == 3.0).all()
        if s % 11 == 0:
            continue
        assert torch.equal(b.tokens(b.v_cache, s)[kv - n:], v[rows])
        stored += n
    assert (out[b.rows:] == 3.0).all()
    assert int((~torch.isnan(b.v_cache)).all(-1).sum()) == stored * kv_heads


@pytest.mark.parametrize("lens,heads,kv_heads", [
    (drawn(40, (300, 700), (0, 0), 5), 32, 16),      # prompts: 19 pieces a CTA
    (drawn(250, (0, 90), (0, 400), 6), 32, 16),      # short chunks behind a context, some of one tile of rows
    (drawn(500, (0, 9), (0, 300), 7), 64, 8),        # mostly tile A alone, some with less in the cache than is new
], ids=["prompts", "chunks", "short"])
@pytest.mark.parametrize("io,dim,page", [("bf16", 64, 64), ("f16", 128, 48)])
@pytest.mark.parametrize("window", [0, 100])
def test_attention_of_many_pieces_a_cta(libssu, lens, heads, kv_heads, io, dim, page, window):
    lens = [(n, max(k - 40, 0)) if i % 50 == 9 else (n, k) for i, (n, k) in enumerate(lens)]
    b = Batch(lens, heads, kv_heads, dim, page, io)
    pair = 2 * (128 // (heads // kv_heads))
    pieces = sum(-(-n // pair) for n, _ in lens) * kv_heads / torch.cuda.get_device_properties(0).multi_processor_count
    assert pieces > 12
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = attention(b, window=window)
    for _ in range(2):
        out, lse = ssu.ssu_paged_attention(b.q, b.k_cache, b.v_cache, b.table, b.kv_lens, cu_seqlens=b.cu, window=window,
                                           max_seqlen=max(max(n for n, _ in lens), 65), return_lse=True, status=status)
        assert int(status) == 0
        check(b, out, lse, want)
