"""Linear attention with a decay for each head, against its definition in 64
bits.

With u the largest relative rounding error of the io type (2^-8 bf16, 2^-11
fp16, 2^-24 fp32) and us that of the pool's type:

Step.  The new state is one exponential, two products and a sum of each element
in fp32, so |dS| <= 2^-20 (|e^g S| + |v k|) + us |S|; the output sums at most 128
products of it: |dy| <= 2^-16 scale sum |S q| + u |y|.

Prefill.  The scores q . k and every sum are fp32 (2^-15 of the sum of the
magnitudes, covering sums over a few thousand terms).  Two operands are rounded
once to the io type: a score times its decay before it meets v, u of the
magnitudes |q . k| e^.. |v|; and the state S_c that enters a chunk of 128 tokens
before it meets q, u of |S_c| |q|.  The decayed v enters the state in parts that
hold 22 bits and more.  So, with A = scale sum_j e^{g(i-j)} |q_i . k_j| |v_j| over the
tokens of the prompt, E = scale e^{g(i-c+1)} |S_c| |q_i| and B the magnitudes of all
(A with |q_i| . |k_j| and the first state's part): |dy| <= u (|y| + A + E) + 2^-15 B,
and |dS| <= 2^-15 (sum of magnitudes) + us |S|.
Values below the types' normal ranges add 2^-24 (fp16) absolutely."""
import pytest
import torch

import selective_state_update_gb300 as ssu

pytestmark = pytest.mark.gpu
DEV = "cuda"
CHUNK = 128  # tokens of the prefill's chunks
HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -24, torch.bfloat16: 0.0}


def problem(seed, rows, heads, kv_heads, dim, dstate, io, state, slots, decays=None, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device=DEV)
    qkv = (normal(rows, (heads + kv_heads) * dstate + kv_heads * dim) * std).to(io)
    q = qkv[:, :heads * dstate].unflatten(1, (heads, dstate))
    k = qkv[:, heads * dstate:(heads + kv_heads) * dstate].unflatten(1, (kv_heads, dstate))
    v = qkv[:, (heads + kv_heads) * dstate:].unflatten(1, (kv_heads, dim))
    pool = (normal(slots, heads, dim, dstate) * 2).to(state)
    if decays is None:
        decays = -torch.exp2(-torch.linspace(0.0, 9.0, heads))
    return pool, q, k, v, torch.as_tensor(decays, dtype=torch.float32).to(DEV)


def reference(q, k, v, log_decay, lengths, first, scale):
    """(y, A + E, B, states, their magnitudes) in 64 bits by the quadratic form; first: [nseq, heads, dim, dstate]."""
    heads = q.shape[1]
    kv = torch.arange(heads, device=q.device) // (heads // k.shape[1])
    q, k, v = q.double().transpose(0, 1), k.double()[:, kv].transpose(0, 1), v.double()[:, kv].transpose(0, 1)
    g = log_decay.double()
    power = lambda n: torch.where(n == 0, 1.0, torch.exp(g.view(-1, *[1] * n.dim()) * n.clamp(min=1)))  # e^(g n), also for g = -inf
    ys, As, Bs, finals, mags = [], [], [], [], []
    t = 0
    for b, n in enumerate(lengths):
        s0 = first[b].double()
        qb, kb, vb = q[:, t:t + n], k[:, t:t + n], v[:, t:t + n]
        i = torch.arange(n, device=q.device)
        w = torch.where(i[:, None] >= i, power((i[:, None] - i).clamp(min=0)), 0.0)
        score = (qb @ kb.transpose(1, 2)) * w
        reach = power(i + 1)[..., None]
        ys.append(scale * (score @ vb + reach * (qb @ s0.transpose(1, 2))))
        E = torch.zeros_like(ys[-1])
        for c in range(0, n, CHUNK):
            left = power(c - 1 - i[:c])[..., None]
            s_c = power(torch.tensor(c, device=q.device))[:, None, None] * s0 + (vb[:, :c] * left).transpose(1, 2) @ kb[:, :c]
            e = slice(c, c + CHUNK)
            E[:, e] = scale * power(i[e] - c + 1)[..., None] * (qb[:, e].abs() @ s_c.abs().transpose(1, 2))
        As.append(scale * (score.abs() @ vb.abs()) + E)
        Bs.append(scale * (((qb.abs() @ kb.abs().transpose(1, 2)) * w) @ vb.abs() + reach * (qb.abs() @ s0.abs().transpose(1, 2))))
        left = power(n - 1 - i)[..., None]
        lam = power(torch.tensor(n, device=q.device))[:, None, None]
        finals.append(lam * s0 + (vb * left).transpose(1, 2) @ kb)
        mags.append(lam * s0.abs() + (vb.abs() * left).transpose(1, 2) @ kb.abs())
        t += n
    cat = lambda ts: torch.cat(ts, 1).transpose(0, 1)
    return cat(ys), cat(As), cat(Bs), torch.stack(finals), torch.stack(mags)


def close(got, want, tol, what):
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off; worst {(d / tol).nan_to_num(nan=1e9).max():.3g} times"


def check_prefill(seed, lengths, heads, kv_heads, dim, dstate, io, state, decays=None, fresh=(), std=1.0, index=torch.int32,
                  max_seqlen=None, scale=None):
    nseq = len(lengths)
    pool, q, k, v, g = problem(seed, sum(lengths), heads, kv_heads, dim, dstate, io, state, 2 * nseq + 2, decays, std)
    order = torch.randperm(2 * nseq + 2, generator=torch.Generator().manual_seed(seed))
    read, dst = order[:nseq].clone(), order[nseq:2 * nseq].clone()
    read[list(fresh)] = -1
    first = torch.where((read >= 0)[:, None, None, None].to(DEV), pool[read.clamp(min=0).to(DEV)].double(), 0.0)
    before = pool.clone()
    cu = torch.tensor([0, *lengths]).cumsum(0).to(device=DEV, dtype=index)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = ssu.ssu_linear_attention_prefill(pool, q, k, v, g, cu, scale=scale, state_batch_indices=read.to(DEV, index),
                                         dst_state_batch_indices=dst.to(DEV, index), status=status, max_seqlen=max_seqlen)
    assert int(status.item()) == 0
    sc = dstate ** -0.5 if scale is None else scale
    yr, A, B, sr, mag = reference(q, k, v, g, lengths, first, sc)
    assert y.dtype == io and y.shape == yr.shape
    u, us = HALF_ULP[io], HALF_ULP[state]
    close(y, yr, u * yr.abs() + u * A + 2.0 ** -15 * B + TINY[io] + 1e-30, "y")
    close(pool[dst.to(DEV)], sr, 2.0 ** -15 * mag + us * sr.abs() + TINY[state] + 1e-30, "states")
    rest = torch.ones(len(pool), dtype=torch.bool)
    rest[dst] = False
    assert torch.equal(pool[rest.to(DEV)], before[rest.to(DEV)])
    return y, pool


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lengths", [[1], [2, 1, 3], [127], [128], [129], [0, 5, 0, 300, 1, 256, 0], [600, 31]])
def test_prefill_lengths(libssu, lengths, io):
    check_prefill(10 + len(lengths) + lengths[0], lengths, 4, 2, 64, 64, io, torch.float32, fresh=[0])


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim,dstate", [(8, 8), (8, 128), (128, 8), (64, 128), (128, 64), (80, 96), (120, 72), (128, 128)])
def test_prefill_head_sizes(libssu, dim, dstate, io):
    check_prefill(30 + dim + dstate, [200, 1, 77], 6, 2, dim, dstate, io, torch.float32)


@pytest.mark.parametrize("state", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (5, 5), (8, 1), (12, 4)])
def test_prefill_head_layouts_and_pool_types(libssu, heads, kv_heads, state):
    check_prefill(50 + heads, [150, 260], heads, kv_heads, 64, 96, torch.bfloat16, state, index=torch.int64)


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
def test_prefill_decays(libssu, io):
    """From no memory at all to none lost, in one call."""
    check_prefill(60, [300, 140], 6, 6, 32, 64, io, torch.float32, decays=[float("-inf"), -60.0, -3.0, -0.1, -1e-4, 0.0])


@pytest.mark.parametrize("std", [1e-3, 30.0])
def test_prefill_fp16_magnitudes(libssu, std):
    """Inputs far from one: states and scores leave fp16's range (scale keeps y inside it)."""
    check_prefill(65, [300, 9], 2, 2, 64, 64, torch.float16, torch.float32, std=std, scale=1.0 if std < 1 else 2.0 ** -16)


@pytest.mark.parametrize("max_seqlen", [None, 2500])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float16])
def test_prefill_long_sequences_on_few_heads(libssu, io, max_seqlen):
    """Too few heads to fill the GPU: long sequences are worked on in pieces."""
    check_prefill(70, [2500, 1, 1300], 2, 1, 128, 128, io, torch.float32, max_seqlen=max_seqlen, fresh=[2])


def test_prefill_result_does_not_hang_on_max_seqlen(libssu):
    """A wrong hint changes the split, not the answer."""
    for hint in (1, 100000):
        check_prefill(75, [900, 1, 700], 2, 1, 64, 64, torch.bfloat16, torch.float32, max_seqlen=hint)


def test_prefill_is_the_same_from_call_to_call(libssu):
    a = check_prefill(80, [700, 33, 400], 4, 2, 128, 128, torch.bfloat16, torch.float32)
    b = check_prefill(80, [700, 33, 400], 4, 2, 128, 128, torch.bfloat16, torch.float32)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_prefill_keeps_sequences_apart(libssu, poison):
    """NaN and infinities in one sequence and its state reach no other one."""
    lengths = [70, 200, 61]
    pool, q, k, v, g = problem(90, sum(lengths), 2, 1, 64, 64, torch.bfloat16, torch.float32, 3)
    cu = torch.tensor([0, 70, 270, 331], dtype=torch.int32, device=DEV)
    clean, clean_pool = q.clone(), pool.clone()
    y0 = ssu.ssu_linear_attention_prefill(clean_pool, q, k, v, g, cu)
    for t in (q, k, v):
        t[70:270] = poison
    pool[1] = poison
    y1 = ssu.ssu_linear_attention_prefill(pool, q, k, v, g, cu)
    keep = [*range(70), *range(270, 331)]
    assert torch.equal(y0[keep], y1[keep])
    assert torch.equal(clean_pool[[0, 2]], pool[[0, 2]])
    assert not torch.isfinite(y1[70:270].float()).any()
    del clean


def test_prefill_bad_metadata_is_flagged_and_skipped(libssu):
    """Malformed bounds, a bad slot and an entry outside the table: flagged, nothing of the sequence written, the
    others right."""
    pool, q, k, v, g = problem(95, 300, 2, 2, 64, 64, torch.bfloat16, torch.float32, 6)
    cu = torch.tensor([0, 100, 200, 300], dtype=torch.int32, device=DEV)
    good, good_pool = None, pool.clone()
    good = ssu.ssu_linear_attention_prefill(good_pool, q, k, v, g, cu)

    def run(cu=cu, read=None, rows=[0, 1, 2]):
        p = pool.clone()
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = torch.full_like(good, 7.0)
        idx = torch.tensor(rows if read is None else read, dtype=torch.int32, device=DEV)
        ssu.ssu_linear_attention_prefill(p, q, k, v, g, cu, state_batch_indices=idx, out=out, status=status)
        return p, out, int(status.item())

    p, out, st = run(read=[0, 6, 2])
    assert st == ssu.DEV_BAD_SLOT and torch.equal(out[:100], good[:100]) and torch.equal(out[200:], good[200:])
    assert (out[100:200] == 7).all() and torch.equal(p[[1, 3, 4, 5]], pool[[1, 3, 4, 5]])
    p, out, st = run(read=[0, 1])
    assert st == ssu.DEV_BAD_ENTRY and torch.equal(out[:200], good[:200]) and (out[200:] == 7).all()
    p, out, st = run(cu=torch.tensor([0, 100, 200, 301], dtype=torch.int32, device=DEV))
    assert st == ssu.DEV_BAD_SEQLEN and torch.equal(out[:200], good[:200]) and (out[200:] == 7).all()
    assert torch.equal(p[2:], pool[2:])
    p, out, st = run(cu=torch.tensor([0, 100, 60, 300], dtype=torch.int32, device=DEV))
    assert st == ssu.DEV_BAD_SEQLEN and torch.equal(out[:60], good[:60])
    p, out, st = run(cu=torch.tensor([-5, 100, 200, 300], dtype=torch.int32, device=DEV))
    assert st == ssu.DEV_BAD_SEQLEN and torch.equal(out[100:], good[100:]) and (out[:100] == 7).all()


@pytest.mark.parametrize("heads,times", [(1, 40), (2, 200)])
def test_prefill_bounds_that_go_back(libssu, heads, times):
    """Bounds that name the same rows again and again, more tokens than the call has: flagged, each rising pair computed
    (here all of the same rows, to the same outputs), nothing out of bounds."""
    pool, q, k, v, g = problem(96, 2500, heads, 1, 64, 64, torch.bfloat16, torch.float32, times * 2)
    cu = torch.tensor([0, 2500] * times, dtype=torch.int32, device=DEV)
    none = torch.full((2 * times - 1,), -1, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = ssu.ssu_linear_attention_prefill(pool, q, k, v, g, cu, state_batch_indices=none, max_seqlen=2500, status=status)
    assert int(status.item()) == ssu.DEV_BAD_SEQLEN
    one = ssu.ssu_linear_attention_prefill(pool, q, k, v, g, cu[:2].contiguous(), state_batch_indices=none[:1])
    yr, A, B, _, _ = reference(q, k, v, g, [2500], torch.zeros(1, heads, 64, 64, device=DEV), 64 ** -0.5)
    for out in (y, one):
        close(out, yr, 2.0 ** -8 * (yr.abs() + A) + 2.0 ** -15 * B, "y")


def test_prefill_then_step_is_one_sequence(libssu):
    """A prompt's state goes on token by token: the same as the longer prompt, within the tolerance of each."""
    pool, q, k, v, g = problem(97, 140, 4, 2, 64, 64, torch.bfloat16, torch.float32, 2)
    cu = torch.tensor([0, 137], dtype=torch.int32, device=DEV)
    slot = torch.tensor([1], dtype=torch.int32, device=DEV)
    first = pool[1:].double().clone()
    y = [ssu.ssu_linear_attention_prefill(pool, q[:137], k[:137], v[:137], g, cu, state_batch_indices=slot)]
    for t in range(137, 140):
        y.append(ssu.ssu_linear_attention_step(pool, q[t:t + 1], k[t:t + 1], v[t:t + 1], g, state_batch_indices=slot))
    yr, A, B, sr, mag = reference(q, k, v, g, [140], first, 64 ** -0.5)
    close(torch.cat(y), yr, 2.0 ** -8 * (yr.abs() + A) + 2.0 ** -15 * B, "y")
    close(pool[1:], sr, 2.0 ** -15 * mag, "state")


@pytest.mark.parametrize("state", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("io", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads,kv_heads,dim,dstate", [(1, 1, 8, 8), (4, 4, 64, 64), (6, 2, 80, 96), (3, 1, 120, 72),
                                                       (2, 2, 128, 128), (2, 1, 72, 120), (2, 2, 8, 16)])
def test_step(libssu, heads, kv_heads, dim, dstate, io, state):
    batch = 5
    pool, q, k, v, g = problem(100 + dim + heads, batch, heads, kv_heads, dim, dstate, io, state, 12)
    read = torch.tensor([3, -1, 7, 0, 5], device=DEV)
    dst = torch.tensor([3, 9, 1, -1, 11], device=DEV)  # in place, from nothing, elsewhere, nowhere
    before = pool.clone()
    first = torch.where((read >= 0)[:, None, None, None], pool[read.clamp(min=0)].double(), 0.0)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = ssu.ssu_linear_attention_step(pool, q, k, v, g, state_batch_indices=read, dst_state_batch_indices=dst.int(),
                                      status=status)
    assert int(status.item()) == 0
    scale = dstate ** -0.5
    kv = torch.arange(heads, device=DEV) // (heads // kv_heads)
    outer = v.double()[:, kv].unsqueeze(-1) * k.double()[:, kv].unsqueeze(-2)
    old = first * g.double().exp()[:, None, None]
    s = old + outer
    sq = s * q.double().unsqueeze(-2)
    yr = scale * sq.sum(-1)
    u, us = HALF_ULP[io], HALF_ULP[state]
    close(y, yr, 2.0 ** -16 * scale * sq.abs().sum(-1) + u * yr.abs() + TINY[io], "y")
    live = dst >= 0
    close(pool[dst[live]], s[live], 2.0 ** -20 * (old.abs() + outer.abs())[live] + us * s[live].abs() + TINY[state], "states")
    untouched = [i for i in range(12) if i not in dst.tolist()]
    assert torch.equal(pool[untouched], before[untouched])


def test_step_flags_and_skips(libssu):
    pool, q, k, v, g = problem(130, 3, 2, 1, 64, 64, torch.bfloat16, torch.float32, 3)
    before, out = pool.clone(), torch.full((3, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ssu.ssu_linear_attention_step(pool, q, k, v, g, state_batch_indices=torch.tensor([0, 3, -2], dtype=torch.int32, device=DEV),
                                  out=out, status=status)
    assert int(status.item()) == ssu.DEV_BAD_SLOT
    assert (out[1:] == 7).all() and (out[0] != 7).any() and torch.equal(pool[1:], before[1:])
    status.zero_()
    ssu.ssu_linear_attention_step(pool, q, k, v, g, state_batch_indices=torch.tensor([1, 2], dtype=torch.int32, device=DEV),
                                  out=out, status=status)
    assert int(status.item()) == ssu.DEV_BAD_ENTRY and (out[2] == 7).all()


def test_no_sequences(libssu):
    pool, q, k, v, g = problem(140, 0, 2, 1, 64, 64, torch.bfloat16, torch.float32, 3)
    before = pool.clone()
    assert ssu.ssu_linear_attention_step(pool, q, k, v, g).shape == (0, 2, 64)
    cu = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert ssu.ssu_linear_attention_prefill(pool, q, k, v, g, cu).shape == (0, 2, 64)
    cu = torch.zeros(4, dtype=torch.int32, device=DEV)  # three empty sequences
    assert ssu.ssu_linear_attention_prefill(pool, q, k, v, g, cu).shape == (0, 2, 64)
    assert torch.equal(pool, before)


def test_offsets_past_32_bits(libssu):
    """A pool slot, and rows of q, k and v, more than 2^31 elements in."""
    heads, dim, dstate = 16, 128, 128
    slots = 2 ** 31 // (heads * dim * dstate) + 2
    pool = torch.zeros(slots, heads, dim, dstate, dtype=torch.bfloat16, device=DEV)
    small, _, _, _, g = problem(150, 3, heads, heads, dim, dstate, torch.bfloat16, torch.bfloat16, 1)
    pool[-1] = small[0]
    far = torch.zeros(2 ** 31 + 2 ** 16, dtype=torch.bfloat16, device=DEV)
    rows = far.as_strided((3, heads, dstate), (2 ** 30, dstate, 1))
    rows.copy_(torch.randn(3, heads, dstate, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV))
    near = rows.clone()
    last = torch.tensor([slots - 1], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    ref_pool = small.clone()
    want = ssu.ssu_linear_attention_prefill(ref_pool, near, near, near, g, cu)
    got = ssu.ssu_linear_attention_prefill(pool, rows, rows, rows, g, cu, state_batch_indices=last)
    assert torch.equal(got, want) and torch.equal(pool[-1], ref_pool[0])
    want = ssu.ssu_linear_attention_step(ref_pool, near[2:], near[2:], near[2:], g)
    got = ssu.ssu_linear_attention_step(pool, rows[2:], rows[2:], rows[2:], g, state_batch_indices=last)
    assert torch.equal(got, want) and torch.equal(pool[-1], ref_pool[0])


def test_runs_on_the_stream_it_is_given(libssu):
    pool, q, k, v, g = problem(160, 300, 4, 2, 64, 64, torch.bfloat16, torch.float32, 2)
    cu = torch.tensor([0, 100, 300], dtype=torch.int32, device=DEV)
    ref_pool = pool.clone()
    want = ssu.ssu_linear_attention_prefill(ref_pool, q, k, v, g, cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    ssu.ssu_linear_attention_prefill(pool, q, k, v, g, cu, out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want) and torch.equal(pool, ref_pool)


def test_capture(libssu):
    """Both forms run inside a CUDA graph and again on its replay."""
    pool, q, k, v, g = problem(170, 300, 4, 2, 64, 64, torch.bfloat16, torch.float32, 3)
    cu = torch.tensor([0, 100, 300], dtype=torch.int32, device=DEV)
    start = pool.clone()

    def both():
        a = ssu.ssu_linear_attention_prefill(pool, q, k, v, g, cu)
        b = ssu.ssu_linear_attention_step(pool, q[:2], k[:2], v[:2], g)
        return a, b

    want = [t.clone() for t in both()]
    after = pool.clone()
    pool.copy_(start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    pool.copy_(start)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(pool, after)


@pytest.mark.parametrize("lengths,heads", [([40] * 60 + [300], 4), ([3000, 5, 700], 2)])
def test_planned_calls_on_streams_and_in_graphs(libssu, lengths, heads):
    """Calls with a workspace (many sequences; a cut one): on another stream, and on a graph's replays, as on this one."""
    pool, q, k, v, g = problem(180, sum(lengths), heads, 1, 64, 64, torch.bfloat16, torch.float32, len(lengths))
    cu = torch.tensor([0, *lengths]).cumsum(0).to(DEV, torch.int32)
    start, kw = pool.clone(), dict(max_seqlen=max(lengths))
    want = ssu.ssu_linear_attention_prefill(pool, q, k, v, g, cu, **kw)
    after = pool.clone()
    pool.copy_(start)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    ssu.ssu_linear_attention_prefill(pool, q, k, v, g, cu, out=out, stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want) and torch.equal(pool, after)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ssu.ssu_linear_attention_prefill(pool, q, k, v, g, cu, **kw)
    for _ in range(2):
        pool.copy_(start)
        graph.replay()
        assert torch.equal(got, want) and torch.equal(pool, after)
