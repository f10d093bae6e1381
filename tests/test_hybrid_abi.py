"""Host side of the operators around the state update: struct layouts, the
refusals of the C entry points (nothing is launched, no GPU needed) and of
their Python bindings."""
import ctypes
import os
import subprocess

import pytest
import torch

import selective_state_update_gb300 as ssu
from selective_state_update_gb300 import build as ssu_build
from selective_state_update_gb300 import hybrid

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def libssu():
    ssu_build.build()
    return ssu.lib()


def test_struct_layouts_match_the_header(tmp_path):
    names = {"ssu_linattn_args": hybrid.LinattnArgs, "ssu_norm_args": hybrid.NormArgs,
             "ssu_logprob_args": hybrid.LogprobArgs}
    lines = []
    for c, py in names.items():
        lines.append(f'printf("%zu\\n", sizeof({c}));')
        lines += [f'printf("%zu\\n", offsetof({c}, {f[0]}));' for f in py._fields_]
    probe = '#include <stddef.h>\n#include <stdio.h>\n#include "ssu.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0; }\n"
    exe = str(tmp_path / "probe")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), "-x", "c", "-", "-o", exe], input=probe,
                   text=True, check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for py in names.values():
        want.append(ctypes.sizeof(py))
        want += [getattr(py, f[0]).offset for f in py._fields_]
    assert got == want


def linattn(**kw):
    a = hybrid.LinattnArgs(slots=4, heads=4, kv_heads=2, dim=64, dstate=128, rows=10, io_dtype=2, state_dtype=0, scale=1.0,
                           state=256, q=512, k=768, v=1024, log_decay=1280, out=1536)
    a.q_stride[:] = a.k_stride[:] = (512, 128)
    a.v_stride[:] = a.out_stride[:] = (256, 64)
    for key, v in kw.items():
        if key.endswith("stride"):
            getattr(a, key)[:] = v
        else:
            setattr(a, key, v)
    return a


@pytest.mark.parametrize("kw,code,needle", [
    (dict(reserved0=1), ssu.ERR_INVALID, "reserved0"),
    (dict(io_dtype=5), ssu.ERR_INVALID, "io_dtype"),
    (dict(state_dtype=-1), ssu.ERR_INVALID, "state_dtype"),
    (dict(rows=-1), ssu.ERR_INVALID, "rows"),
    (dict(slots=0), ssu.ERR_INVALID, "slots"),
    (dict(kv_heads=3), ssu.ERR_INVALID, "multiple of kv_heads"),
    (dict(kv_heads=0), ssu.ERR_INVALID, "multiple of kv_heads"),
    (dict(dim=60), ssu.ERR_UNSUPPORTED, "multiples of 8"),
    (dict(dim=136), ssu.ERR_UNSUPPORTED, "multiples of 8"),
    (dict(dstate=0), ssu.ERR_UNSUPPORTED, "multiples of 8"),
    (dict(scale=float("nan")), ssu.ERR_INVALID, "scale"),
    (dict(state=None), ssu.ERR_INVALID, "NULL"),
    (dict(log_decay=None), ssu.ERR_INVALID, "NULL"),
    (dict(state=264), ssu.ERR_INVALID, "aligned"),
    (dict(k=None), ssu.ERR_INVALID, "NULL"),
    (dict(out=512), ssu.ERR_INVALID, "alias"),
    (dict(v_stride=(-8, 64)), ssu.ERR_INVALID, "stride"),
])
def test_linear_attention_refusals(libssu, kw, code, needle):
    a = linattn(**kw)
    assert libssu.ssu_linear_attention_step(ctypes.byref(a), None, None, None) == code
    assert needle in libssu.ssu_last_error().decode()
    assert libssu.ssu_linear_attention_prefill(ctypes.byref(a), 2, 4096, 0, 0, None, None, None, 0, None) == code
    assert needle in libssu.ssu_last_error().decode()


@pytest.mark.parametrize("kw,call,code,needle", [
    ({}, dict(nseq=-1), ssu.ERR_INVALID, "nseq"),
    ({}, dict(longest=-1), ssu.ERR_INVALID, "max_seqlen"),
    ({}, dict(meta=7), ssu.ERR_INVALID, "meta_type"),
    ({}, dict(cu=None), ssu.ERR_INVALID, "cu_seqlens"),
    (dict(io_dtype=0), {}, ssu.ERR_UNSUPPORTED, "fp16 or bf16"),
    (dict(q=520), {}, ssu.ERR_INVALID, "aligned"),
    (dict(k_stride=(132, 128)), {}, ssu.ERR_INVALID, "multiples of 8"),
    (dict(out_stride=(256, 4)), {}, ssu.ERR_INVALID, "multiples of 8"),
    (dict(rows=1 << 31), {}, ssu.ERR_INVALID, "tokens"),
])
def test_prefill_refusals(libssu, kw, call, code, needle):
    a = linattn(**kw)
    c = dict(nseq=2, cu=4096, meta=0, longest=0) | call
    assert libssu.ssu_linear_attention_prefill(ctypes.byref(a), c["nseq"], c["cu"], c["meta"], c["longest"], None, None,
                                               None, 0, None) == code
    assert needle in libssu.ssu_last_error().decode()


def test_prefill_workspace(libssu):
    """None for a call that gives every (sequence, head) a CTA; a plan for more of them; states as well where sequences
    are long for the heads there are.  A call checks what it is given."""
    n = ctypes.c_uint64(0)

    def size(nseq, longest, **kw):
        a = linattn(**kw)
        assert libssu.ssu_linear_attention_workspace_size(ctypes.byref(a), nseq, longest, ctypes.byref(n)) == ssu.OK
        return n.value

    assert size(2, 0, rows=300) == 0
    assert 0 < size(100, 0, rows=30000) < 1 << 20
    long = size(1, 0, rows=100000)
    assert long >= 2 * 4 * 64 * 128 * 4
    assert size(2, 300, rows=300) == 0
    a = linattn(rows=100000)
    for ws, have in ((None, 1 << 40), (512, long - 1), (520, 1 << 40)):
        assert libssu.ssu_linear_attention_prefill(ctypes.byref(a), 1, 4096, 0, 0, None, None, ws, have, None) == ssu.ERR_INVALID
        assert "workspace" in libssu.ssu_last_error().decode()
    assert libssu.ssu_linear_attention_workspace_size(ctypes.byref(a), -1, 0, ctypes.byref(n)) == ssu.ERR_INVALID
    assert libssu.ssu_linear_attention_workspace_size(ctypes.byref(a), 1, 0, None) == ssu.ERR_INVALID


def test_tables_are_checked(libssu):
    a = linattn()
    t = ssu.SlotTable(entries=128, type=5, mode=0, s0=1, s1=1, extent=2)
    assert libssu.ssu_linear_attention_step(ctypes.byref(a), ctypes.byref(t), None, None) == ssu.ERR_INVALID
    t = ssu.SlotTable(entries=128, type=0, mode=0, s0=1, s1=1, extent=-2)
    assert libssu.ssu_linear_attention_prefill(ctypes.byref(a), 2, 4096, 0, 0, None, ctypes.byref(t), None, 0,
                                               None) == ssu.ERR_INVALID


def test_empty_calls_launch_nothing(libssu):
    a = linattn(rows=0, q=None, k=None, v=None, out=None)
    assert libssu.ssu_linear_attention_step(ctypes.byref(a), None, None, None) == ssu.OK
    assert libssu.ssu_linear_attention_prefill(ctypes.byref(a), 0, None, 0, 0, None, None, None, 0, None) == ssu.OK
    n = norm(rows=0, x=None, y=None)
    assert libssu.ssu_add_rmsnorm(ctypes.byref(n), None) == ssu.OK
    lp = logprob(rows=0, logits=None, tokens=None)
    assert libssu.ssu_token_logprobs(ctypes.byref(lp), None) == ssu.OK


def norm(**kw):
    a = hybrid.NormArgs(rows=4, hidden=512, dtype=2, weight_dtype=2, format=0, eps=1e-5, x=256, residual=None, weight=512,
                        residual_out=None, y=1024, scales=None, x_stride=512, y_stride=512)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code,needle", [
    (dict(dtype=4), ssu.ERR_INVALID, "dtype"),
    (dict(weight_dtype=1), ssu.ERR_INVALID, "weight"),
    (dict(format=3), ssu.ERR_INVALID, "format"),
    (dict(rows=-1), ssu.ERR_INVALID, "rows"),
    (dict(hidden=0), ssu.ERR_INVALID, "hidden"),
    (dict(hidden=32769), ssu.ERR_UNSUPPORTED, "hidden"),
    (dict(eps=0.0), ssu.ERR_INVALID, "eps"),
    (dict(eps=float("nan")), ssu.ERR_INVALID, "eps"),
    (dict(x_stride=-1), ssu.ERR_INVALID, "stride"),
    (dict(residual=2048), ssu.ERR_INVALID, "go together"),
    (dict(residual_out=2048), ssu.ERR_INVALID, "go together"),
    (dict(format=1), ssu.ERR_INVALID, "scales"),
    (dict(scales=4096), ssu.ERR_INVALID, "scales"),
    (dict(x=None), ssu.ERR_INVALID, "NULL"),
    (dict(x=257), ssu.ERR_INVALID, "aligned"),
    (dict(y=256), ssu.ERR_INVALID, "alias"),
    (dict(residual=2048, residual_out=256), ssu.ERR_INVALID, "alias"),
    (dict(rows=1 << 31), ssu.ERR_INVALID, "rows"),
])
def test_norm_refusals(libssu, kw, code, needle):
    a = norm(**kw)
    assert libssu.ssu_add_rmsnorm(ctypes.byref(a), None) == code
    assert needle in libssu.ssu_last_error().decode()


def logprob(**kw):
    a = hybrid.LogprobArgs(rows=4, vocab=1000, row_stride=1000, dtype=2, token_type=1, top_k=0, reserved0=0, logits=256,
                           tokens=512, logprobs=1024, entropy=1280)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code,needle", [
    (dict(reserved0=2), ssu.ERR_INVALID, "reserved0"),
    (dict(dtype=3), ssu.ERR_INVALID, "dtype"),
    (dict(token_type=2), ssu.ERR_INVALID, "token_type"),
    (dict(rows=-4), ssu.ERR_INVALID, "rows"),
    (dict(vocab=0), ssu.ERR_INVALID, "vocab"),
    (dict(vocab=(1 << 30) + 1), ssu.ERR_INVALID, "vocab"),
    (dict(row_stride=-1), ssu.ERR_INVALID, "row_stride"),
    (dict(top_k=33, top_ids=4096, top_logprobs=8192), ssu.ERR_INVALID, "top_k"),
    (dict(top_k=-1), ssu.ERR_INVALID, "top_k"),
    (dict(top_k=9, vocab=8), ssu.ERR_INVALID, "top_k"),
    (dict(top_k=4), ssu.ERR_INVALID, "top_ids"),
    (dict(tokens=None), ssu.ERR_INVALID, "NULL"),
    (dict(logits=257), ssu.ERR_INVALID, "aligned"),
    (dict(rows=1 << 30), ssu.ERR_INVALID, "rows"),
])
def test_logprob_refusals(libssu, kw, code, needle):
    a = logprob(**kw)
    assert libssu.ssu_token_logprobs(ctypes.byref(a), None) == code
    assert needle in libssu.ssu_last_error().decode()


def test_python_bindings_refuse_cpu_tensors_and_shapes():
    pool, q, kv = torch.zeros(2, 4, 64, 128), torch.zeros(3, 4, 128), torch.zeros(3, 2, 128)
    v, g = torch.zeros(3, 2, 64), torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        ssu.ssu_linear_attention_step(pool, q, kv, v, g)
    with pytest.raises(ValueError, match="q must be"):
        ssu.ssu_linear_attention_step(pool, q[:, :2], kv, v, g)
    with pytest.raises(ValueError, match="v must be"):
        ssu.ssu_linear_attention_step(pool, q, kv, v[..., :32], g)
    with pytest.raises(ValueError, match="dtype of q"):
        ssu.ssu_linear_attention_step(pool, q, kv.half(), v, g)
    with pytest.raises(ValueError, match="log_decay"):
        ssu.ssu_linear_attention_step(pool, q, kv, v, g[:3])
    with pytest.raises(ValueError, match="unit stride"):
        ssu.ssu_linear_attention_step(pool, torch.zeros(3, 128, 4).transpose(1, 2), kv, v, g)
    with pytest.raises(ValueError, match="cu_seqlens"):
        ssu.ssu_linear_attention_prefill(pool, q, kv, v, g, torch.zeros(2))
    with pytest.raises(ValueError, match="x must be"):
        ssu.ssu_add_rmsnorm(torch.zeros(2, 8), torch.zeros(8))
    with pytest.raises(ValueError, match="logits must be"):
        ssu.ssu_token_logprobs(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64))
