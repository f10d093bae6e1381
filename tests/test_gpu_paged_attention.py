"""Attention over the paged cache against its definition in 64 bits; the
tolerance's derivation stands at ``paged_testlib.attention``."""
import pytest
import torch

import selective_state_update_gb300 as ssu
from paged_testlib import DEV, NAN, Batch, attention, check

pytestmark = pytest.mark.gpu


def call(b, window=0, scale=None, hints=True, **kw):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    if hints:
        kw |= dict(max_seqlen=max(n for n, _ in b.lens), max_kv_len=max(k for _, k in b.lens))
    got = ssu.ssu_paged_attention(b.q, b.k_cache, b.v_cache, b.table, b.kv_lens, cu_seqlens=b.cu, window=window, scale=scale,
                                  return_lse=True, status=status, **kw)
    assert int(status.item()) == 0
    return got


SINGLE = [(1, 1), (1, 2), (1, 63), (1, 64), (1, 65), (1, 127), (1, 128), (1, 129), (1, 1000)]


@pytest.mark.parametrize("io,heads,kv_heads,dim,page", [
    ("bf16", 8, 2, 128, 64), ("f16", 6, 2, 80, 16), ("bf16", 4, 4, 64, 272), ("f16", 5, 1, 8, 8), ("bf16", 16, 1, 96, 48),
    ("bf16", 128, 1, 128, 32), ("f16", 40, 2, 72, 528), ("bf16", 3, 1, 40, 1024),
])
@pytest.mark.parametrize("window", [0, 1, 70])
def test_single_tokens(libssu, io, heads, kv_heads, dim, page, window):
    b = Batch(SINGLE, heads, kv_heads, dim, page, io, single=True)
    check(b, *call(b, window), attention(b, window=window))


CHUNKS = {
    "drafts": [(4, 4), (4, 7), (4, 66), (4, 500)],
    "empty ones": [(0, 0), (3, 3), (0, 9), (1, 0), (5, 2), (2, 64), (0, 0)],
    "prompts": [(1, 1), (17, 17), (128, 128), (129, 129), (200, 200), (63, 63)],
    "behind a context": [(100, 400), (1, 700), (33, 129), (256, 513), (2, 1000)],
    "one": [(300, 300)],
    "one far": [(5, 3001)],
}


@pytest.mark.parametrize("lens", CHUNKS, ids=lambda s: s.replace(" ", "_"))
@pytest.mark.parametrize("io,heads,kv_heads,dim,page", [
    ("bf16", 8, 2, 128, 64), ("f16", 6, 2, 80, 16), ("bf16", 4, 4, 64, 272), ("f16", 5, 1, 40, 8), ("f16", 20, 4, 96, 48),
    ("bf16", 128, 1, 128, 32),
])
@pytest.mark.parametrize("window", [0, 1, 130])
def test_chunks(libssu, lens, io, heads, kv_heads, dim, page, window):
    b = Batch(CHUNKS[lens], heads, kv_heads, dim, page, io)
    check(b, *call(b, window), attention(b, window=window))


@pytest.mark.parametrize("hints", [dict(max_seqlen=1, max_kv_len=1), dict(max_seqlen=10000, max_kv_len=1 << 20), dict()])
@pytest.mark.parametrize("lens", ["drafts", "behind a context", "empty ones"])
def test_hints_never_change_validity(libssu, lens, hints):
    b = Batch(CHUNKS[lens], 8, 2, 128, 64)
    check(b, *call(b, hints=False, **hints), attention(b))


@pytest.mark.parametrize("layout", ["interleaved", "heads first", "padded"])
@pytest.mark.parametrize("single", [True, False])
def test_layouts_and_strides(libssu, layout, single):
    lens = SINGLE if single else CHUNKS["behind a context"]
    b = Batch(lens, 6, 2, 72, 48, "f16", layout=layout, single=single, table_dtype=torch.int64, meta_dtype=torch.int64)
    want = attention(b)
    # q a slice of a projection, out one of a wider tensor, the table one of a larger one
    wide = torch.full((b.rows, 10, 88), NAN, dtype=b.io, device=DEV)
    wide[:, 2:8, :72] = b.q
    b.q = wide[:, 2:8, :72]
    table = torch.full((len(lens), b.table.shape[1] + 3), -9, dtype=torch.int64, device=DEV)
    table[:, :b.table.shape[1]] = b.table
    b.table = table[:, :b.table.shape[1]]
    target = torch.full((b.rows, 8, 80), 7.0, dtype=b.io, device=DEV)
    out, lse = call(b, out=target[:, 1:7, :72])
    check(b, out, lse, want)
    target[:, 1:7, :72] = 7.0
    assert (target == 7.0).all()


@pytest.mark.parametrize("lens,single", [(SINGLE, True), (CHUNKS["behind a context"], False)])
def test_rows_behind_the_last_sequence_stay(libssu, lens, single):
    b = Batch(lens, 8, 2, 128, 64, behind=0 if single else 9, single=single)
    out = torch.full_like(b.q, 3.0)
    got, lse = call(b, out=out)
    check(b, got, lse, attention(b))
    assert (out[b.rows:] == 3.0).all()


@pytest.mark.parametrize("scale,sharp", [(1.0, 1.0), (0.01, 1.0), (0.125, 40.0)])
@pytest.mark.parametrize("lens", ["drafts", "behind a context", "prompts"])
@pytest.mark.parametrize("io", ["f16", "bf16"])
def test_scales(libssu, io, lens, scale, sharp):
    b = Batch(CHUNKS[lens], 8, 2, 64, 16, io, sharp=sharp)
    check(b, *call(b, scale=scale), attention(b, scale=scale))


@pytest.mark.parametrize("lens,heads", [([(4, 300), (3, 70)], 8), ([(90, 300), (40, 40), (150, 600)], 8), ([(260, 300)], 4)])
@pytest.mark.parametrize("window", [0, 33])
@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("bad", [NAN, float("inf"), -float("inf")])
def test_no_numbers_reach_those_that_see_them_and_no_other(libssu, lens, heads, window, io, bad):
    b = Batch(lens, heads, 4, 64, 16, io)
    before, _ = call(b, window)
    before = before.clone()
    at = []  # one of the new tokens, not the first, of each sequence
    for s, (n, kv) in enumerate(lens):
        key = kv - n + n // 2
        at.append(key)
        b.v_cache[b.table[s, key // 16].long(), key % 16, 1, 5] = bad
    out, _ = call(b, window)
    hit = torch.zeros(b.rows, heads, 64, dtype=torch.bool, device=DEV)
    share = heads // 4
    for s, (n, kv) in enumerate(lens):
        pos = torch.arange(kv - n, kv, device=DEV)
        sees = (pos >= at[s]) & ((pos < at[s] + window) if window else True)
        hit[b.starts[s]:b.starts[s] + n, share:2 * share, 5] = sees[:, None]
    assert torch.equal(out[~hit], before[~hit])
    assert not torch.isfinite(out[hit]).any()
    if bad == bad:  # an infinity keeps its sign where its weight is not zero
        assert ((out[hit] == bad) | torch.isnan(out[hit])).all()


@pytest.mark.parametrize("lens,single", [([(1, 300), (1, 70)], True), ([(90, 300), (40, 40)], False)])
def test_no_numbers_in_keys_and_queries(libssu, lens, single):
    b = Batch(lens, 8, 4, 64, 16, single=single)
    before = call(b)[0].clone()
    n, kv = lens[0]
    key = kv - n + n // 2
    b.k_cache[b.table[0, key // 16].long(), key % 16, 2, 3] = NAN
    b.q[b.rows - 1, 7, 0] = NAN
    out, lse = call(b)
    hit = torch.zeros(b.rows, 8, dtype=torch.bool, device=DEV)
    hit[n // 2:n, 4:6] = True
    hit[b.rows - 1, 7] = True
    assert torch.equal(out[~hit], before[~hit])
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()


def test_bad_metadata_is_flagged_and_skipped(libssu):
    for kv_lens, cu, entry, bit in (([70, 5, 64], [0, 6, 4, 9], None, ssu.DEV_BAD_SEQLEN),
                                    ([70, -1, 64], [0, 3, 6, 9], None, ssu.DEV_BAD_SEQLEN),
                                    ([70, 4000, 64], [0, 3, 6, 9], None, ssu.DEV_BAD_SEQLEN),
                                    ([70, 5, 64], [0, 3, 6, 99], None, ssu.DEV_BAD_SEQLEN),
                                    ([70, 5, 64], [0, 3, 6, 9], 10 ** 6, ssu.DEV_BAD_SLOT),
                                    ([70, 5, 64], [0, 3, 6, 9], -1, ssu.DEV_BAD_SLOT)):
        b = Batch([(3, 70), (3, 5), (3, 64)], 8, 2, 64, 16)
        want = attention(b)
        b.kv_lens = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
        b.cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        if entry is not None:
            b.table[1, 0] = entry
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = torch.full_like(b.q, 3.0)
        ssu.ssu_paged_attention(b.q, b.k_cache, b.v_cache, b.table, b.kv_lens, cu_seqlens=b.cu, out=out, status=status)
        assert int(status.item()) == bit
        assert ((out[:3].double() - want[0][:3]).abs() <= want[2][:3]).all() or cu[1] != 3
        if entry is None and cu == [0, 3, 6, 9]:
            assert (out[3:6] == 3.0).all()
            assert ((out[6:].double() - want[0][6:]).abs() <= want[2][6:]).all()


@pytest.mark.parametrize("lens,heads,single", [([(1, 9000)] * 3, 8, True), ([(7, 5000), (1, 9000)], 8, False),
                                               ([(64, 20000), (300, 2500)], 8, False)])
def test_long_ones_are_split_and_repeat_bit_for_bit(libssu, lens, heads, single):
    b = Batch(lens, heads, 2, 128, 64, single=single)
    out, lse = call(b)
    check(b, out, lse, attention(b))
    for _ in range(3):
        again, lse2 = call(b)
        assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("single", [True, False])
def test_captured_on_another_stream_and_replayed(libssu, single):
    one, two = (Batch([(1, 5), (1, 3000)] if single else [(40, 50), (9, 3000)], 8, 2, 128, 64, seed=s, single=single) for s in (1, 2))
    want = [attention(one), attention(two)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    kept, graphs = [], []
    for b in (one, two):  # two graphs, alive at once, each with a workspace of its own
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            kept.append(ssu.ssu_paged_attention(b.q, b.k_cache, b.v_cache, b.table, b.kv_lens, cu_seqlens=b.cu, return_lse=True))
        graphs.append(graph)
    for _ in range(2):
        for out, lse in kept:
            out.fill_(NAN)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for b, (out, lse), w in zip((one, two), kept, want):
            check(b, out, lse, w)
    # lengths are read at every replay
    one.lens = [(n, k - 2) if n > 1 or k > 100 else (n, k) for n, k in one.lens]
    one.kv_lens.copy_(torch.tensor([k for _, k in one.lens], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    check(one, *kept[0], attention(one))


def test_given_stream(libssu):
    b = Batch(CHUNKS["behind a context"], 8, 2, 128, 64)
    want = attention(b)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for s in (stream, stream.cuda_stream):
        out, lse = call(b, stream=s)
        stream.synchronize()
        check(b, out, lse, want)


@pytest.mark.parametrize("lens,single", [([(1, 900), (1, 77)], True), ([(70, 900), (150, 300)], False)])
def test_offsets_past_32_bits(libssu, lens, single):
    b = Batch(lens, 8, 2, 128, 64, single=single)
    want = attention(b)
    # the same pages at the far end of a cache of 2^32 elements and more
    pages = (1 << 32) // (64 * 2 * 128) + 100
    far_k, far_v = (torch.empty(pages, 64, 2, 128, dtype=b.io, device=DEV) for _ in range(2))
    n = b.k_cache.shape[0]
    far_k[-n:], far_v[-n:] = b.k_cache, b.v_cache
    b.k_cache, b.v_cache = far_k, far_v
    b.table = torch.where(b.table >= 0, b.table + (pages - n), b.table)
    check(b, *call(b), want)


def test_many_sequences(libssu):
    g = torch.Generator().manual_seed(5)
    lens = [(int(n), int(n) + int(c)) for n, c in zip(torch.randint(0, 4, (700,), generator=g), torch.randint(0, 90, (700,), generator=g))]
    b = Batch(lens, 4, 2, 64, 16, "f16")
    check(b, *call(b), attention(b))


def test_nothing_to_do(libssu):
    b = Batch([(1, 5)], 4, 2, 64, 16, single=True)
    out, lse = ssu.ssu_paged_attention(b.q[:0], b.k_cache, b.v_cache, b.table[:0], b.kv_lens[:0], return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    b = Batch([(0, 5), (0, 0)], 4, 2, 64, 16, behind=4)
    out = torch.full_like(b.q, 3.0)
    ssu.ssu_paged_attention(b.q, b.k_cache, b.v_cache, b.table, b.kv_lens, cu_seqlens=b.cu, out=out)
    assert (out == 3.0).all()


@pytest.mark.parametrize("lens,heads,kv_heads", [
    ([(2400, 5000)], 8, 2),                    # one unit a CTA and a little more
    ([(1, 6000)] * 5 + [(130, 400)] * 3, 24, 8),  # long and short ones in one call
    ([(3, 30000)], 128, 1),                    # a single row of units, cut many times
    ([(700, 700), (900, 4000), (60, 9000)], 12, 4),
])
@pytest.mark.parametrize("io,dim,page", [("bf16", 128, 272), ("f16", 72, 24)])
def test_units_cut_or_not(libssu, lens, heads, kv_heads, io, dim, page):
    b = Batch(lens, heads, kv_heads, dim, page, io)
    out, lse = call(b)
    check(b, out, lse, attention(b))
    again, lse2 = call(b, hints=False)
    check(b, again, lse2, attention(b))


@pytest.mark.parametrize("page", [8, 24, 40, 56, 104, 120, 136, 248, 264, 400])
@pytest.mark.parametrize("lens", [[(1, 1), (1, 513), (1, 299)], [(200, 513), (70, 130)]], ids=["single", "chunks"])
def test_pages_that_end_inside_a_tile(libssu, page, lens):
    b = Batch(lens, 8, 2, 128 if page % 16 else 80, page, single=lens[0][0] == 1)
    check(b, *call(b, window=0), attention(b))
    check(b, *call(b, window=150), attention(b, window=150))


@pytest.mark.parametrize("rows,heads,kv_heads", [(16, 16, 1), (17, 17, 1), (32, 8, 1), (33, 33, 1), (64, 16, 1), (65, 65, 1), (24, 12, 2)])
@pytest.mark.parametrize("window", [0, 90])
def test_each_number_of_rows(libssu, rows, heads, kv_heads, window):
    n = rows // (heads // kv_heads)
    b = Batch([(n, n), (n, n + 63), (n, 1500), (max(n - 1, 0), 200)], heads, kv_heads, 128, 32)
    check(b, *call(b, window), attention(b, window=window))
