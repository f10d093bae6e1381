"""Calls that need device scratch, made by two host threads on one stream: the
launches of one call may come between the other's, so each has scratch of its own
or keeps its launches together."""
import threading

import pytest
import torch

import selective_state_update_gb300 as ssu
import workloads
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


def test_ssd_prefill(libssu):
    """On the workspace kept for the stream."""
    side = torch.cuda.Stream()
    calls, wants = [], []
    for seed, lengths in ((300, [130, 257, 1, 312]), (301, [900, 33])):
        g = workloads.ssd_problem(seed, lengths, heads=16, dim=64, dstate=128, groups=2, chunk_size=128).to(DEV)

        def call(stream=side, g=g):
            return ssu.ssu_ssd_prefill(g.x, g.dt, g.A, g.B, g.C, g.chunk_size, g.cu_chunk_seqlens, g.seq_idx, g.last_chunk_indices,
                                       D=g.D, z=g.z, dt_bias=g.dt_bias, dt_softplus=g.dt_softplus, dt_limit=g.dt_limit,
                                       initial_states=g.initial_states, state_dtype=g.state_dtype, nseq=g.nseq,
                                       out=torch.empty_like(g.x), stream=stream)

        calls.append(call)
        wants.append([t.clone() for t in call(None)])
    torch.cuda.synchronize()
    for outs, want in zip(both(calls, 20), wants):
        side.synchronize()
        for out in outs:
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_ssd_launches_stay_together(libssu, monkeypatch):
    """No other thread gets at the kept workspace between a call's look at it and its launches."""
    g = workloads.ssd_problem(302, [130], heads=16, dim=64, dstate=128, groups=2, chunk_size=128).to(DEV)
    kept, held = ssu._ssd_workspace, []

    def watched(*args):
        held.append(ssu._SSD_LAUNCHES.locked())
        return kept(*args)

    monkeypatch.setattr(ssu, "_ssd_workspace", watched)
    ssu.ssu_ssd_prefill(g.x, g.dt, g.A, g.B, g.C, g.chunk_size, g.cu_chunk_seqlens, g.seq_idx, g.last_chunk_indices, nseq=g.nseq)
    assert held == [True]
