"""Log probabilities of given tokens, entropy and top alternatives against the
definition in 64 bits.

x - m is one fp32 difference (2^-24 of it).  Every exponential is within 2^-21
plus 2^-23 |x - m| of its value relatively, and e^-d d is below 1, so the sum is
within 2^-20; it is added up over at most a few hundred terms a thread and a
tree (2^-15 covers 512).  Hence |d logprob| <= 2^-15 + 2^-22 |logprob|; the
entropy's second sum has terms (x - m) e^(x - m) of the same accuracy, divided by
s: |d entropy| <= 2^-15 (2 + entropy).  The alternatives' ids are exact."""
import pytest
import torch

import selective_state_update_gb300 as ssu

pytestmark = pytest.mark.gpu
DEV = "cuda"


def order(x, k):
    """The k largest by (value, lowest index): a stable sort downwards."""
    return torch.sort(x.double() + 0.0, dim=-1, descending=True, stable=True).indices[:, :k]


def check(x, tokens, k):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lp, ent, ids, top = ssu.ssu_token_logprobs(x, tokens, top_k=k, status=status)
    assert int(status.item()) == 0
    d = x.double()
    d = d - d.amax(-1, keepdim=True)  # first: a maximum of -3e38 would swallow the sum's logarithm in 64 bits too
    ref = d - d.exp().sum(-1, keepdim=True).log()
    want = ref.gather(1, tokens.long()[:, None])[:, 0]
    p = ref.exp()
    entropy = -torch.where(p > 0, p * ref, 0.0).sum(-1)

    def near(got, want):
        same = (got.double() == want) | ((got.double() - want).abs() <= 2.0 ** -15 + 2.0 ** -22 * want.abs())
        assert same.all(), (got, want)

    near(lp, want)
    assert ((ent.double() - entropy).abs() <= 2.0 ** -15 * (2 + entropy)).all()
    if k == 0:
        assert ids is None and top is None
        return
    assert ids.dtype == tokens.dtype and torch.equal(ids.long(), order(x, k))
    near(top, ref.gather(1, ids.long()))


def logits(seed, rows, vocab, dtype, pad=0, std=3.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = (torch.randn(rows, vocab + pad, generator=g, device=DEV) * std).to(dtype)[:, :vocab]
    return x, torch.randint(vocab, (rows,), generator=g, device=DEV)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (2, 5), (1, 31), (3, 33), (1, 4096), (5, 50001), (40, 8192), (160, 4099),
                                        (400, 1000), (2, 200003), (310, 20000)])
def test_shapes(libssu, rows, vocab, dtype):
    x, tok = logits(rows + vocab, rows, vocab, dtype)
    for k in sorted({0, 1, min(5, vocab), min(20, vocab), min(32, vocab)}):
        check(x, tok, k)


@pytest.mark.parametrize("pad", [1, 3, 8])
def test_strides_and_alignment(libssu, pad):
    x, tok = logits(20 + pad, 7, 5000, torch.bfloat16, pad=pad)
    check(x, tok.int(), 20)
    check(x[:, 1:], tok.clamp(max=4998), 20)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [3, 200])
def test_ties_go_to_the_lowest_index(libssu, rows, dtype):
    g = torch.Generator(device=DEV).manual_seed(31)
    x = torch.randint(-3, 4, (rows, 30000), generator=g, device=DEV).to(dtype)
    x[0] = 1.5
    x[1] = 0.0
    x[1, 7::2] = -0.0
    check(x, torch.arange(rows, device=DEV), 32)


@pytest.mark.parametrize("rows", [4, 200])
def test_orders_that_crowd_a_thread(libssu, rows):
    """Sorted rows, and all large logits at one stride, where one thread holds every candidate."""
    v = 65536
    up = torch.arange(v, device=DEV, dtype=torch.float32) / v * 10
    x = up.repeat(rows, 1)
    x[1] = up.flip(0)
    for i, stride in enumerate((2048, 4096)):
        x[2 + i] = -up
        x[2 + i, 3::stride] = 5 + torch.arange(len(x[0, 3::stride]), device=DEV, dtype=torch.float32) / 64
    tok = torch.full((rows,), v - 1, device=DEV)
    check(x, tok, 32)
    check(x.bfloat16(), tok, 32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows", [8, 400])
def test_masks(libssu, rows, dtype):
    """Masked by -inf and by the type's lowest value; one logit left; none left."""
    x, _ = logits(40, rows, 3000, dtype)
    low = torch.finfo(dtype).min
    x[0, 1000:] = -float("inf")
    x[1, :2500] = low
    x[2] = -float("inf")
    x[2, 17] = 2.0
    x[3] = low
    x[3, 17] = 2.0
    x[4] = low
    x[5] = -float("inf")
    x[6] = -float("inf")
    x[6, 5] = low
    tok = torch.full((rows,), 17, device=DEV)
    keep = torch.ones(rows, dtype=torch.bool)
    keep[5] = False
    check(x[keep], tok[keep], 20)
    tok[0] = 2000  # a masked token
    check(x[:1], tok[:1], 5)
    lp, ent, ids, top = ssu.ssu_token_logprobs(x, tok, top_k=4)
    assert lp[5] == -float("inf") and ent[5] == 0 and (top[5] == -float("inf")).all() and ids[5].tolist() == [0, 1, 2, 3]


@pytest.mark.parametrize("rows", [3, 400])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_rows_stay_alone(libssu, rows, bad):
    x, tok = logits(50, rows, 10000, torch.float32)
    clean = ssu.ssu_token_logprobs(x, tok, top_k=8)
    x[1, 1234] = bad
    got = ssu.ssu_token_logprobs(x, tok, top_k=8)
    assert torch.isnan(got[0][1]) and torch.isnan(got[1][1])
    assert ((got[2][1] >= 0) & (got[2][1] < 10000)).all()
    rest = [i for i in range(rows) if i != 1]
    for a, b in zip(clean, got):
        assert torch.equal(a[rest], b[rest])
    x[1] = float("nan")
    ids = ssu.ssu_token_logprobs(x, tok, top_k=8)[2]
    assert ids[1].tolist() == list(range(8))


def test_no_token_and_bad_tokens(libssu):
    x, tok = logits(60, 5, 100, torch.float32)
    tok[1], tok[2], tok[3] = -1, 100, -7
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lp, ent, ids, top = ssu.ssu_token_logprobs(x, tok, top_k=3, status=status)
    assert int(status.item()) == ssu.DEV_BAD_ENTRY
    assert lp[1] == 0 and torch.isnan(lp[2]) and torch.isnan(lp[3]) and torch.isfinite(lp[[0, 4]]).all()
    assert torch.isfinite(ent).all() and torch.isfinite(top).all()
    status.zero_()
    ssu.ssu_token_logprobs(x[:2], tok[:2], status=status)
    assert int(status.item()) == 0


def test_large_and_small_values(libssu):
    x, tok = logits(70, 4, 9000, torch.float32, std=1.0)
    x[0] *= 1e4
    x[1] += 3e4
    x[2] *= 1e30
    x[3] = 0
    check(x, tok, 20)


def test_no_rows(libssu):
    x, tok = logits(80, 0, 100, torch.bfloat16)
    lp, ent, ids, top = ssu.ssu_token_logprobs(x, tok, top_k=3)
    assert lp.shape == (0,) and ent.shape == (0,) and ids.shape == (0, 3) and top.shape == (0, 3)


def test_offsets_past_32_bits(libssu):
    far = torch.zeros(2 ** 31 + 2 ** 17, dtype=torch.bfloat16, device=DEV)
    rows = far.as_strided((3, 70000), (2 ** 30, 1))
    x, tok = logits(90, 3, 70000, torch.bfloat16)
    rows.copy_(x)
    for a, b in zip(ssu.ssu_token_logprobs(x, tok, top_k=20), ssu.ssu_token_logprobs(rows, tok, top_k=20)):
        assert torch.equal(a, b)


def test_refusals_on_device(libssu):
    x, tok = logits(95, 3, 100, torch.float32)
    with pytest.raises(ValueError, match="top_k"):
        ssu.ssu_token_logprobs(x, tok, top_k=33)
    with pytest.raises(ValueError, match="tokens"):
        ssu.ssu_token_logprobs(x, tok[:2])
    with pytest.raises(ValueError, match="tokens"):
        ssu.ssu_token_logprobs(x, tok.float())
    with pytest.raises(ValueError, match="logits"):
        ssu.ssu_token_logprobs(x.t(), tok)
    with pytest.raises(ValueError, match="logits"):
        ssu.ssu_token_logprobs(x.double(), tok)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("vocab", [31, 257, 2049, 32003])
def test_many_rows(libssu, vocab, dtype):
    """Enough rows for small CTAs; among them masked ones, with fewer left than are asked for, just as many, and ties."""
    x, tok = logits(60 + vocab, 1301, vocab, dtype)
    k = min(32, vocab)
    g = torch.Generator(device=DEV).manual_seed(61)
    for row, left in enumerate((1, k // 2, k, k + 3)):
        hidden = torch.randperm(vocab, generator=g, device=DEV)[left:]
        x[row, hidden] = -float("inf")
        tok[row] = x[row].argmax()
        x[row + 4, hidden] = torch.finfo(dtype).min
        tok[row + 4] = x[row + 4].argmax()
    x[8] = 0.25
    x[9] = x[9].round()
    check(x, tok, k)
    check(x, tok.int(), 0)


def test_more_steps_than_groups(libssu):
    """A row in one part, longer than the noted groups hold one by one; sorted rows crowd the last of them."""
    x, tok = logits(70, 160, 110003, torch.float32)
    x[0] = torch.arange(110003, device=DEV) / 1e4
    x[1] = x[0].flip(0)
    check(x, tok, 32)
