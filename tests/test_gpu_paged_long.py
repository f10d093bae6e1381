"""Attention over the paged cache for lengths that take a CTA longer than a wait of its
warps may take without any tile being copied."""
import torch

import pytest

import selective_state_update_gb300 as ssu
from paged_testlib import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,share", [(40, 2), (70, 4)])
def test_a_piece_that_takes_seconds(libssu, rows, share):
    """200 million keys, all of them rows of one page, with a hint that has them in one piece: 1.6 million key tiles, 2
    seconds.  Queries are zero: every weight is one, and a sum of those, multiples of 16 but for the last tiles' up to
    256, stays exact in fp32 up to 2^28 or is off by 2^-23.  The products' sums are the tensor cores': what of a
    product lies below 2^-25 of the sum that it is added to is cut off.  So the sums of the first columns, one to a key
    or to every second one, lose what the derived bound (keys x 2^-24 of them) allows, all: they are positive and none
    too large.  Those of the last columns are of 192 or 384 products of 2^20, all of them multiples of 2^20: exact."""
    page, heads, dim, pages = 1 << 20, share, 8, 192
    keys = page * pages
    k_cache = torch.randn(1, page, 1, dim, device=DEV).bfloat16()
    v_cache = torch.zeros(1, page, 1, dim, device=DEV, dtype=torch.bfloat16)
    at = torch.arange(page, device=DEV)
    v_cache[0, :, 0, 0] = 1.0
    v_cache[0, :, 0, 1] = (1 - 2 * (at % 2)).bfloat16()
    v_cache[0, :, 0, 2] = (at < page // 2).bfloat16()
    v_cache[0, :, 0, 3] = (at // 128 % 4 == 1).bfloat16()
    v_cache[0, 5, 0, 4] = 2.0 ** 20
    v_cache[0, 7, 0, 5], v_cache[0, 9, 0, 5] = 2.0 ** 20, -(2.0 ** 20)
    v_cache[0, [11, 13], 0, 6] = 2.0 ** 20
    v_cache[0, -1, 0, 7] = 2.0 ** 20
    q = torch.zeros(rows, heads, dim, device=DEV, dtype=torch.bfloat16)
    table = torch.zeros(1, pages, dtype=torch.int32, device=DEV)
    kv_lens = torch.tensor([keys], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = ssu.ssu_paged_attention(q, k_cache, v_cache, table, kv_lens, cu_seqlens=cu, max_seqlen=rows, max_kv_len=1,
                                       return_lse=True, status=status)
    assert int(status) == 0
    # (the keys that the first rows do not see are `rows` of 2^27 at most: 2^-20)
    want = torch.tensor([1.0, 0.0, 0.5, 0.25, 1.0, 0.0, 2.0, 0.0], device=DEV, dtype=torch.float64).repeat(rows, heads, 1)
    want[:, :, 7] = 191 / 192
    want[-1, :, 7] = 1.0  # the last row alone sees the last key
    tol = (2.0 ** -9 + 2.0 ** -20) * want + 2.0 ** -20
    assert ((out.double() - want).abs() <= tol)[:, :, 4:].all()
    assert (out.double() >= -tol)[:, :, :4].all() and (out.double() <= want + tol)[:, :, :4].all()
    seen = torch.arange(keys - rows + 1, keys + 1, device=DEV).double()
    assert ((lse.double() - seen.log()[:, None]).abs() <= 2.0 ** -20).all()
