"""Linear attention where one value's reach is the question.  What must not reach an
output must not change one bit of it; values are held to the tolerances of
test_gpu_linear_attention."""
import pytest
import torch

import selective_state_update_gb300 as ssu
from test_gpu_linear_attention import DEV, check_prefill, problem

pytestmark = pytest.mark.gpu


def fill_tensor_memory(dstate, heads=320):
    """Leaves finite growths near 1e32 in the tensor memory of every SM (more heads than SMs)."""
    big = torch.full((1, heads, 128, dstate), 0.0, device=DEV)
    x = torch.full((128, heads, 128), 2.0 ** 50, dtype=torch.bfloat16, device=DEV)
    cu = torch.tensor([0, 128], dtype=torch.int32, device=DEV)
    ssu.ssu_linear_attention_prefill(big, x[..., :dstate], x[..., :dstate], x, torch.zeros(heads, device=DEV), cu)
    assert 1e31 < float(big.max()) < 1e33


@pytest.mark.parametrize("before,dstate", [(128, 96), (128, 72), (128, 112), (64, 32), (64, 8), (128, 48)])
def test_prefill_fp16_after_large_growths(libssu, before, dstate):
    """Nothing of an earlier call is left in what the state's rows are scaled by."""
    fill_tensor_memory(before)
    check_prefill(200 + dstate, [300, 131], 80, 80, 64, dstate, torch.float16, torch.float32)


@pytest.mark.parametrize("poison", [6e4, float("inf"), float("nan")])
@pytest.mark.parametrize("lengths", [[70, 200, 61], [1, 140, 33], [128, 3, 97]])
def test_prefill_fp16_keeps_sequences_apart(libssu, lengths, poison):
    """Values beside a sequence in the packed tokens change no bit of its outputs and states."""
    pool, q, k, v, g = problem(210, sum(lengths), 2, 1, 64, 64, torch.float16, torch.float32, 3, std=1e-3)
    a, b = lengths[0], lengths[0] + lengths[1]
    cu = torch.tensor([0, a, b, sum(lengths)], dtype=torch.int32, device=DEV)
    for t in (q, k, v):
        t[a:b] = 0
    clean_pool, dirty_pool = pool.clone(), pool.clone()
    want = ssu.ssu_linear_attention_prefill(clean_pool, q, k, v, g, cu)
    for t in (q, k, v):
        t[a:b] = poison
    got = ssu.ssu_linear_attention_prefill(dirty_pool, q, k, v, g, cu)
    keep = [*range(a), *range(b, sum(lengths))]
    assert torch.equal(got[keep], want[keep])
    assert torch.equal(dirty_pool[[0, 2]], clean_pool[[0, 2]])


def test_prefill_fp16_rows_past_the_end(libssu):
    """The same for rows that belong to no sequence."""
    pool, q, k, v, g = problem(215, 200, 2, 1, 64, 64, torch.float16, torch.float32, 1, std=1e-3)
    cu = torch.tensor([0, 133], dtype=torch.int32, device=DEV)
    first = pool.clone()
    v[133:] = 0
    want = ssu.ssu_linear_attention_prefill(pool, q, k, v, g, cu)
    v[133:] = 6e4
    got = ssu.ssu_linear_attention_prefill(first, q, k, v, g, cu)
    assert torch.equal(got[:133], want[:133]) and torch.equal(first, pool)


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("rows,at,heads", [(100, 0, 4), (100, 99, 4), (300, 140, 4), (300, 127, 4), (300, 128, 4),
                                           (2600, 1333, 2)])
def test_prefill_values_that_are_no_numbers(libssu, rows, at, heads, poison, io):
    """A NaN or an infinity in v at token t, value dim p: the outputs of dim p are NaN from t on, and so is row p of the
    state; no bit of anything else changes."""
    dim = 13
    pool, q, k, v, _ = problem(220 + at, rows, heads, 1, 64, 96, io, torch.float32, 1)
    g = torch.full((heads,), -1e-4, device=DEV)
    cu = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    v[at, 0, dim] = 0
    dirty_pool = pool.clone()
    want = ssu.ssu_linear_attention_prefill(pool, q, k, v, g, cu)
    v[at, 0, dim] = poison
    got = ssu.ssu_linear_attention_prefill(dirty_pool, q, k, v, g, cu)
    assert torch.equal(got[:at], want[:at])
    others = [p for p in range(64) if p != dim]
    assert torch.equal(got[:, :, others], want[:, :, others])
    assert torch.equal(dirty_pool[:, :, others], pool[:, :, others])
    assert torch.isnan(got[at:, :, dim].float()).all()
    assert torch.isnan(dirty_pool[0, :, dim]).all()


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
def test_prefill_many_values_that_are_no_numbers(libssu, io):
    """Several of them in one chunk: each dim from its first one on."""
    pool, q, k, v, _ = problem(230, 250, 2, 1, 80, 64, io, torch.float32, 1)
    g = torch.full((2,), -1e-3, device=DEV)
    cu = torch.tensor([0, 250], dtype=torch.int32, device=DEV)
    where = [(5, 3), (9, 3), (40, 70), (127, 0), (128, 1), (249, 79), (200, 33), (131, 33)]
    for t, p in where:
        v[t, 0, p] = 0
    dirty_pool = pool.clone()
    want = ssu.ssu_linear_attention_prefill(pool, q, k, v, g, cu)
    for n, (t, p) in enumerate(where):
        v[t, 0, p] = (float("nan"), float("inf"), -float("inf"))[n % 3]
    got = ssu.ssu_linear_attention_prefill(dirty_pool, q, k, v, g, cu)
    first = {}
    for t, p in where:
        first[p] = min(t, first.get(p, 250))
    for p in range(80):
        t = first.get(p, 250)
        assert torch.equal(got[:t, :, p], want[:t, :, p]), p
        assert torch.isnan(got[t:, :, p].float()).all(), p
        if t == 250:
            assert torch.equal(dirty_pool[:, :, p], pool[:, :, p])


@pytest.mark.parametrize("late", [6e4, float("inf"), float("nan")])
def test_prefill_fp16_later_keys_leave_earlier_outputs(libssu, late):
    """A key however large or bad changes no bit of the outputs of tokens before it."""
    pool, q, k, v, g = problem(240, 128, 4, 1, 64, 64, torch.float16, torch.float32, 1)
    k.copy_(torch.sign(k.float()) * 2.0 ** -18)  # far below it: 2^33 of the products
    v.mul_(1000)
    pool.zero_()
    cu = torch.tensor([0, 128], dtype=torch.int32, device=DEV)
    for at in (20, 33, 95):
        kk = k.clone()
        kk[at] = 0
        want = ssu.ssu_linear_attention_prefill(pool.clone(), q, kk, v, g, cu, scale=1.0)
        kk[at] = late
        got = ssu.ssu_linear_attention_prefill(pool.clone(), q, kk, v, g, cu, scale=1.0)
        assert torch.equal(got[:at], want[:at])


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [0, 63, 128, 249])
def test_prefill_queries_and_keys_that_are_no_numbers(libssu, at, poison, io):
    """In q they stay in their token's outputs of that head, in k they reach no earlier token."""
    pool, q, k, v, g = problem(250 + at, 250, 4, 2, 72, 40, io, torch.float32, 1)
    cu = torch.tensor([0, 250], dtype=torch.int32, device=DEV)
    first = pool.clone()
    want = ssu.ssu_linear_attention_prefill(pool, q, k, v, g, cu)
    bad_q, bad_k = q.clone(), k.clone()
    bad_q[at, 1, 7] = poison
    bad_k[at, 1, 7] = poison
    state = first.clone()
    got = ssu.ssu_linear_attention_prefill(state, bad_q, k, v, g, cu)
    assert not torch.isfinite(got[at, 1].float()).any()
    got[at, 1] = want[at, 1]
    assert torch.equal(got, want) and torch.equal(state, pool)
    state = first.clone()
    got = ssu.ssu_linear_attention_prefill(state, q, bad_k, v, g, cu)
    assert torch.equal(got[:at], want[:at]) and torch.equal(got[:, :2], want[:, :2])
    assert not torch.isfinite(got[at:, 2:].float()).any()
    assert torch.equal(state[:, :2], pool[:, :2])
    columns = [n for n in range(40) if n != 7]
    assert torch.equal(state[..., columns], pool[..., columns]) and not torch.isfinite(state[:, 2:, :, 7]).any()
