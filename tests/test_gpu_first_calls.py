"""Calls where nothing was done before: the first of a host thread, the first of a
process inside a graph capture."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import selective_state_update_gb300 as ssu
from test_gpu_linear_attention import DEV, problem

pytestmark = pytest.mark.gpu


NAMES = ["step", "prefill", "planned prefill", "norm", "norm to 8 bits", "logprobs"]


def calls():
    """Calls of the operators around the update on small inputs, by name; each leaves its inputs as they are."""
    pool, q, k, v, g = problem(500, 300, 4, 2, 64, 64, torch.bfloat16, torch.float32, 60)
    fresh = torch.full((60,), -1, dtype=torch.int32, device=DEV)
    two, many = (torch.tensor(b, dtype=torch.int32, device=DEV) for b in ([0, 100, 300], list(range(0, 301, 5))))
    x, w = q.flatten(1).contiguous(), torch.ones(256, dtype=torch.bfloat16, device=DEV)
    tokens = torch.zeros(300, dtype=torch.int64, device=DEV)

    def prefill(cu, **kw):
        n = len(cu) - 1
        return ssu.ssu_linear_attention_prefill(pool, q, k, v, g, cu, state_batch_indices=fresh[:n], **kw)

    return {
        "step": lambda: ssu.ssu_linear_attention_step(pool, q[:2], k[:2], v[:2], g, state_batch_indices=fresh[:2]),
        "prefill": lambda: prefill(two),
        "planned prefill": lambda: prefill(many),
        "norm": lambda: ssu.ssu_add_rmsnorm(x, w)[0],
        "norm to 8 bits": lambda: ssu.ssu_add_rmsnorm(x, w, residual=x, quant="block")[0].view(torch.uint8),
        "logprobs": lambda: ssu.ssu_token_logprobs(x, tokens, top_k=5)[0],
    }


@pytest.mark.parametrize("name", NAMES)
def test_first_call_of_a_host_thread(libssu, name):
    call, got = calls()[name], []
    want = call()

    def work():
        try:
            got.append(call())
        except Exception as e:  # noqa: BLE001
            got.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert isinstance(got[0], torch.Tensor), got[0]
    assert torch.equal(got[0], want)


CAPTURE = """
import torch
from test_gpu_first_calls import calls

for name, call in calls().items():
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, call()), name
print("captured")
"""


def test_first_calls_inside_a_capture(libssu):
    """No kernel of these has been loaded before its capture: they need no ssu_prewarm."""
    here = os.path.dirname(os.path.abspath(__file__))
    paths = os.pathsep.join([here, os.path.dirname(here)])
    r = subprocess.run([sys.executable, "-c", CAPTURE], env=dict(os.environ, PYTHONPATH=paths), capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "captured", r.stderr[-2000:]
