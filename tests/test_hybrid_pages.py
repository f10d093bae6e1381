"""The example stack's pages: only layers of softmax attention need them, and a
stack without such layers is bounded by its slots alone."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def stack(device="cpu", **kw):
    import hybrid_stack
    return hybrid_stack.HybridStack(vocab=64, hidden=128, layers=2, heads=2, kv_heads=1, slots=4, device=device, **kw)


def seen(model, call):
    """What the call gives an attention layer for its cache (None: nothing)."""
    got = []
    model._attend = lambda cache, q, k, v, table, lengths, **kw: got.append((table, lengths))
    model.forward = lambda tokens, mix: [mix(pool, None, None, None) for pool in model.pools if isinstance(pool, tuple)]
    call(model)
    return got[0] if got else None


def slots(*ids):
    return torch.tensor(ids, dtype=torch.int32)


def test_without_attention_layers_pages_are_not_counted():
    model = stack()
    tokens = torch.zeros(2100, dtype=torch.int64)
    for _ in range(3):
        assert seen(model, lambda m: m.prefill(tokens, [2000, 100], slots(1, 3))) is None
        assert seen(model, lambda m: m.step(tokens[:2], slots(1, 3))) is None
    assert not model.held


def test_without_attention_layers_a_step_reads_no_slot_on_the_host():
    model = stack()

    class Slots:
        def __getattr__(self, name):
            raise AssertionError(f"slots.{name}")

        def __len__(self):
            return 2

    seen(model, lambda m: m.step(torch.zeros(2, dtype=torch.int64), Slots()))


def test_padded_slots_have_no_pages():
    model = stack(attention_every=2, pages=8)
    tokens = torch.zeros(40, dtype=torch.int64)
    table, lengths = seen(model, lambda m: m.prefill(tokens, [17, 3, 20], slots(2, -1, 0)))
    assert lengths.tolist() == [17, 0, 20] and table.shape == (3, 2) and (table[1] == -1).all()
    for n in range(1, 15):
        table, lengths = seen(model, lambda m: m.step(tokens[:4], slots(-1, 2, -1, 0)))
        assert lengths.tolist() == [0, 17 + n, 0, 20 + n]
    assert len(model.free) == 8 - 2 - 3 and len(set(model.free)) == len(model.free)
    # a step of padding alone, and one of no sequence
    table, lengths = seen(model, lambda m: m.step(tokens[:2], slots(-1, -1)))
    assert table.shape == (2, 0) and lengths.tolist() == [0, 0]
    table, lengths = seen(model, lambda m: m.step(tokens[:0], slots()))
    assert table.shape == (0, 0) and lengths.tolist() == []


def test_a_prompt_without_room_is_refused_and_changes_nothing():
    model = stack(attention_every=2, pages=8)
    tokens = torch.zeros(200, dtype=torch.int64)
    seen(model, lambda m: m.prefill(tokens[:60], [40, 20], slots(0, 1)))
    free, held = list(model.free), {s: (list(p), n) for s, (p, n) in model.held.items()}
    with pytest.raises(RuntimeError, match="pages"):
        seen(model, lambda m: m.prefill(tokens, [70, 130], slots(2, 0)))
    assert sorted(model.free) == sorted(free) and model.held == held
    # the pages of a slot that starts anew are free for it
    table, lengths = seen(model, lambda m: m.prefill(tokens[:90], [90], slots(0)))
    assert lengths.tolist() == [90] and len(set(table[0].tolist())) == 6


@pytest.mark.gpu
def test_without_attention_layers_more_tokens_than_pages_and_a_captured_step(libssu):
    g = torch.Generator(device="cuda").manual_seed(0)
    lengths, where = [2000, 100], slots(1, 3).cuda()
    tokens = torch.randint(64, (sum(lengths),), generator=g, device="cuda")
    token = torch.zeros(2, dtype=torch.int64, device="cuda")
    model, again = stack("cuda"), stack("cuda")
    for m in (model, again):
        m.prefill(tokens, lengths, where)
    want = [model.step(token, where).clone() for _ in range(3)]
    again.step(token, where)  # (the projections' library makes its own set-up at its first call)
    again.prefill(tokens, lengths, where)
    torch.cuda.synchronize()
    pools = [p.clone() for p in again.pools]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = again.step(token, where)
    for p, kept in zip(again.pools, pools):
        p.copy_(kept)
    for w in want:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    assert int(again.status) == 0
