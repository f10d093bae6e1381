"""The C entry points of the operators around the state update refuse pointers
that their element type does not allow (the device would fault on them); nothing
is launched, no GPU needed."""
import ctypes

import pytest

import selective_state_update_gb300 as ssu
from test_hybrid_abi import libssu, linattn, logprob, norm  # noqa: F401  (the fixture)


def refused(L, rc):
    assert rc == ssu.ERR_INVALID
    assert "aligned" in L.ssu_last_error().decode()


@pytest.mark.parametrize("kw", [dict(q=513), dict(k=769), dict(v=1025), dict(out=1537), dict(io_dtype=0, q=514),
                                dict(io_dtype=0, out=1538), dict(log_decay=1282), dict(d_status=2050)])
def test_linear_attention(libssu, kw):
    a = ctypes.byref(linattn(**kw))
    refused(libssu, libssu.ssu_linear_attention_step(a, None, None, None))
    refused(libssu, libssu.ssu_linear_attention_prefill(a, 2, 4096, 0, 0, None, None, None, 0, None))


@pytest.mark.parametrize("cu,kind", [(4098, 0), (4100, 1)])
def test_prefill_bounds(libssu, cu, kind):
    a = ctypes.byref(linattn())
    refused(libssu, libssu.ssu_linear_attention_prefill(a, 2, cu, kind, 0, None, None, None, 0, None))


@pytest.mark.parametrize("entries,kind", [(130, 0), (132, 1)])
def test_tables(libssu, entries, kind):
    a = ctypes.byref(linattn())
    t = ctypes.byref(ssu.SlotTable(entries=entries, type=kind, mode=0, s0=1, s1=1, extent=10))
    refused(libssu, libssu.ssu_linear_attention_step(a, t, None, None))
    refused(libssu, libssu.ssu_linear_attention_step(a, None, t, None))
    refused(libssu, libssu.ssu_linear_attention_prefill(a, 2, 4096, 0, 0, t, None, None, 0, None))


@pytest.mark.parametrize("kw", [dict(y=1025), dict(weight=513), dict(weight_dtype=0, weight=514), dict(dtype=0, weight_dtype=0, y=1026),
                                dict(format=1, scales=4098), dict(format=2, scales=4097)])
def test_norm(libssu, kw):
    refused(libssu, libssu.ssu_add_rmsnorm(ctypes.byref(norm(**kw)), None))


@pytest.mark.parametrize("kw", [dict(tokens=516), dict(token_type=0, tokens=514), dict(logprobs=1026), dict(entropy=1281),
                                dict(top_k=4, top_ids=4100, top_logprobs=8192), dict(top_k=4, top_ids=4096, top_logprobs=8193),
                                dict(d_status=2)])
def test_logprobs(libssu, kw):
    refused(libssu, libssu.ssu_token_logprobs(ctypes.byref(logprob(**kw)), None))
