"""The paged cache's calls where others are under way: the first call of a host
thread, the first of a process inside a capture, two host threads on one stream,
and the example stack with attention layers."""
import ctypes
import os
import subprocess
import sys
import threading

import pytest
import torch

import selective_state_update_gb300 as ssu
from paged_testlib import DEV, Batch, attention, check
from selective_state_update_gb300 import paged

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))

BATCHES = {
    "single tokens": dict(lens=[(1, 700), (1, 3)], single=True),
    "drafts": dict(lens=[(5, 700), (5, 90)]),
    "chunks": dict(lens=[(90, 700), (300, 2300), (1, 40)]),
    "a long context": dict(lens=[(70, 9000)]),
}


def batch(name, seed=1):
    return Batch(heads=8, kv_heads=2, dim=64, page=48, seed=seed, **BATCHES[name])


def call(b, **kw):
    return ssu.ssu_paged_attention(b.q, b.k_cache, b.v_cache, b.table, b.kv_lens, cu_seqlens=b.cu, max_seqlen=max(n for n, _ in b.lens), **kw)


@pytest.mark.parametrize("name", BATCHES)
def test_first_call_of_a_host_thread(libssu, name):
    b, got = batch(name), []
    want = call(b)

    def work():
        try:
            got.append(call(b))
        except Exception as e:  # noqa: BLE001
            got.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert isinstance(got[0], torch.Tensor), got[0]
    assert torch.equal(got[0], want)


CAPTURE = """
import sys
sys.path[:0] = [{root!r}, {here!r}]
import torch
import test_gpu_paged_calls as t
import selective_state_update_gb300 as ssu
b = t.batch({name!r})
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    q = ssu.ssu_paged_append(b.k_cache, b.v_cache, b.q[:, :2] * 0 + 1, b.q[:, :2], b.table, b.kv_lens, cu_seqlens=b.cu, q=b.q)
    out = t.call(b)
graph.replay()
torch.cuda.synchronize()
got = out.clone()
assert torch.equal(q, b.q)
assert torch.equal(got, t.call(b)) and torch.isfinite(got).all()
"""


@pytest.mark.parametrize("name", BATCHES)
def test_first_call_of_a_process_in_a_capture(libssu, name):
    code = CAPTURE.format(root=os.path.dirname(HERE), here=HERE, name=name)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("n,kv", [(600, 900), (600, 5000), (5, 900)])
@pytest.mark.parametrize("copies", [3, 300])
def test_bounds_that_overlap(libssu, n, kv, copies):
    """Bounds that go back and forth: every other sequence is the same rows again, those between them are bad.  What
    the call would list then passes what its workspace holds; nothing behind that is touched, and the rows hold what
    one of their sequences gives them."""
    b = Batch([(n, kv)], heads=8, kv_heads=2, dim=64, page=48, seed=5)
    want = attention(b)
    nseq = 2 * copies - 1
    table = b.table.expand(nseq, -1).contiguous()
    kv_lens = torch.full((nseq,), kv, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, n] * copies, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = torch.empty_like(b.q), torch.empty(n, 8, device=DEV)
    a = paged._paged_args(b.k_cache, b.v_cache, table, kv_lens, cu, n, 8, b.q, out, status)
    size = ctypes.c_uint64(0)
    assert libssu.ssu_paged_attention_workspace_size(a, n, 0, ctypes.byref(size)) == ssu.OK
    ws = torch.full((size.value + 4096,), 0x5a, dtype=torch.uint8, device=DEV)
    stream = torch.cuda.current_stream().cuda_stream
    assert libssu.ssu_paged_attention(a, 64 ** -0.5, 0, n, 0, lse.data_ptr(), ws.data_ptr(), size.value, stream) == ssu.OK
    torch.cuda.synchronize()
    assert int(status) == ssu.DEV_BAD_SEQLEN
    assert (ws[size.value:] == 0x5a).all()
    check(b, out, lse, want)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("one,two", [("single tokens", "chunks"), ("a long context", "chunks"), ("drafts", "single tokens")])
def test_two_host_threads_on_one_stream(libssu, one, two, raw):
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    batches = [batch(one, 1), batch(two, 2)]
    wants = [call(b).clone() for b in batches]
    torch.cuda.synchronize()
    results, errors, start = [[], []], [], threading.Barrier(2)

    def work(i):
        try:
            start.wait()
            for _ in range(20):
                results[i].append(call(batches[i], stream=stream))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    side.synchronize()
    for outs, want in zip(results, wants):
        for out in outs:
            assert torch.equal(out, want)


@pytest.mark.parametrize("name", ["chunks", "single tokens"])
def test_two_calls_at_once_on_two_streams(libssu, name):
    batches, streams = [batch(name, s) for s in (1, 2)], [torch.cuda.Stream(), torch.cuda.Stream()]
    wants = [call(b).clone() for b in batches]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(call(batches[i]))
    torch.cuda.synchronize()
    for outs, want in zip(got, wants):
        assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("quant,tol", [("none", 0.1), ("row", 0.3)])
def test_the_example_with_attention_layers(libssu, quant, tol):
    """Steps and one prefill over the same text agree; the tolerance is that of the stack without attention layers, whose
    roundings these have too (one of the weights in place of one of the decayed scores)."""
    sys.path.insert(0, os.path.join(os.path.dirname(HERE), "examples"))
    import hybrid_stack
    seen, again, made, entropy = hybrid_stack.run(layers=2, new=12, lengths=(37, 140, 5), quant=quant, attention_every=2)
    assert seen.shape == again.shape == made.shape == (3, 12)
    assert torch.isfinite(seen).all() and (seen <= 0).all() and (entropy > 0).all()
    assert (seen - again).abs().max() < tol
