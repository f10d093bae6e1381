"""The attention's workspace over a paged cache: what it may come to, and that a
smaller one never changes more than how the work is split."""
import ctypes

import pytest
import torch

import selective_state_update_gb300 as ssu
from selective_state_update_gb300 import build as ssu_build
from selective_state_update_gb300 import paged


@pytest.fixture(scope="module")
def library():
    ssu_build.build()
    return ssu.lib()


def size(L, rows, nseq, width, page=64, heads=16, kv_heads=4, dim=128, kv_len=0, seqlen=None):
    a = paged.PagedArgs(pages=1000, page_size=page, heads=heads, kv_heads=kv_heads, dim=dim, rows=rows, nseq=nseq, io_dtype=2, k_cache=4096,
                        v_cache=8192, block_table=256, table_stride=width, table_width=width, kv_lens=512, cu_seqlens=768, q=1024, out=2048)
    a.k_cache_stride[:] = a.v_cache_stride[:] = (page * kv_heads * dim, kv_heads * dim, dim)
    a.q_stride[:] = a.out_stride[:] = (heads * dim, dim)
    n = ctypes.c_uint64(0)
    assert L.ssu_paged_attention_workspace_size(ctypes.byref(a), rows if seqlen is None else seqlen, kv_len, ctypes.byref(n)) == ssu.OK
    return n.value


PART = 4 * 2 * 128 * (128 + 2) * 4  # a part of a unit: four heads, two tiles of rows


def test_a_short_chunk_takes_little(library):
    # 300 tokens are 5 units of 64; 2000 keys 16 tiles, which are cut into 5 parts at most
    assert size(library, 300, 1, 2048 // 64) <= 25 * PART + 4096
    assert size(library, 300, 1, 1000, kv_len=2000) <= 25 * PART + 4096
    assert size(library, 300, 1, 1000, kv_len=1024) <= 4096
    # the hint counts where it is below the table's room, and the other way round
    assert size(library, 300, 1, 2048 // 64, kv_len=100000) == size(library, 300, 1, 2048 // 64)


def test_the_most_it_takes(library):
    for rows, nseq, width in ((300, 1, 1 << 20), (2048, 1, 4096), (32768, 16, 4096), (65536, 3000, 100)):
        n = size(library, rows, nseq, width)
        assert n <= 137 * 10 ** 6 + 48 * rows + 96 * nseq, (rows, n)
        # a hint never asks for more
        for kv_len in (1, 1025, 5000, 1 << 30, (1 << 63) - 1):
            assert size(library, rows, nseq, width, kv_len=kv_len) <= n
    assert size(library, 2048, 1, 1 << 40, page=1 << 20) <= 137 * 10 ** 6 + 48 * 2048 + 96


@pytest.mark.gpu
@pytest.mark.parametrize("kv_len", [1100, 3000, 9000, 20000])
@pytest.mark.parametrize("lens", [[(70, 20000)], [(300, 9000), (33, 20000), (1, 5)]])
def test_less_room_for_parts_than_the_lengths_want(libssu, lens, kv_len):
    from paged_testlib import DEV, Batch, attention, check
    b = Batch(lens, 8, 2, 128, 64)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = ssu.ssu_paged_attention(b.q, b.k_cache, b.v_cache, b.table, b.kv_lens, cu_seqlens=b.cu, max_seqlen=max(n for n, _ in lens),
                                       max_kv_len=kv_len, return_lse=True, status=status)
    assert int(status) == 0
    check(b, out, lse, attention(b))
