"""Calls that need device scratch, made by two host threads on one stream: the
launches of one call may come between the other's, so each has scratch of its own
or keeps its launches together."""
import threading

import pytest
import torch

import selective_state_update_gb300 as ssu
from test_gpu_linear_attention import DEV, problem

pytestmark = pytest.mark.gpu


def both(calls, times):
    """Each call in a thread of its own, `times` times over, at once; what they return."""
    results, errors = [[] for _ in calls], []
    start = threading.Barrier(len(calls))

    def work(i):
        try:
            start.wait()
            for _ in range(times):
                results[i].append(calls[i]())
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    return results


def prefill(seed, lengths, heads, stream):
    """(call, its outputs by itself): sequences that start from zeros and leave their states."""
    pool, q, k, v, g = problem(seed, sum(lengths), heads, 1, 64, 64, torch.bfloat16, torch.float32, len(lengths))
    cu = torch.tensor([0, *lengths]).cumsum(0).to(DEV, torch.int32)
    fresh = torch.full((len(lengths),), -1, dtype=torch.int32, device=DEV)
    slots = torch.arange(len(lengths), dtype=torch.int32, device=DEV)

    def call(stream=stream):
        return ssu.ssu_linear_attention_prefill(pool, q, k, v, g, cu, state_batch_indices=fresh, dst_state_batch_indices=slots,
                                                max_seqlen=max(lengths), out=torch.empty_like(q), stream=stream)

    return call, call(None).clone()


@pytest.mark.parametrize("raw", [False, True])
def test_linear_attention_prefill(libssu, raw):
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    calls, wants = zip(*[prefill(400 + i, lengths, heads, stream) for i, (lengths, heads) in
                         enumerate([([40] * 60 + [300], 4), ([3000, 5, 700], 2)])])
    torch.cuda.synchronize()
    kept = set(ssu._SSD_WORKSPACE)
    for outs, want in zip(both(calls, 20), wants):
        side.synchronize()
        for out in outs:
            assert torch.equal(out, want)
    assert set(ssu._SSD_WORKSPACE) == kept  # nothing is held for the stream
