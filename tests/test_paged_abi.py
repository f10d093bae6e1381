"""Host side of the paged cache's calls: the struct's layout, the refusals of the
C entry points (nothing is launched, no GPU needed) and of their bindings."""
import ctypes
import os
import subprocess

import pytest
import torch

import selective_state_update_gb300 as ssu
from selective_state_update_gb300 import build as ssu_build
from selective_state_update_gb300 import paged

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def libssu():
    ssu_build.build()
    return ssu.lib()


def test_struct_layout_matches_the_header(tmp_path):
    lines = ['printf("%zu\\n", sizeof(ssu_paged_args));']
    lines += [f'printf("%zu\\n", offsetof(ssu_paged_args, {f[0]}));' for f in paged.PagedArgs._fields_]
    probe = '#include <stddef.h>\n#include <stdio.h>\n#include "ssu.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0; }\n"
    exe = str(tmp_path / "probe")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), "-x", "c", "-", "-o", exe], input=probe,
                   text=True, check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(paged.PagedArgs)] + [getattr(paged.PagedArgs, f[0]).offset for f in paged.PagedArgs._fields_]
    assert paged._PAGED.size == got[0]


def args(**kw):
    a = paged.PagedArgs(pages=10, page_size=16, heads=4, kv_heads=2, dim=64, rows=6, nseq=3, io_dtype=2, k_cache=4096, v_cache=8192,
                        block_table=256, table_stride=5, table_width=5, kv_lens=512, cu_seqlens=768, q=1024, out=2048)
    a.k_cache_stride[:] = a.v_cache_stride[:] = (2048, 128, 64)
    a.q_stride[:] = a.out_stride[:] = (256, 64)
    for key, v in kw.items():
        if key.endswith("stride") and key != "table_stride":
            getattr(a, key)[:] = v
        else:
            setattr(a, key, v)
    return a


STRIDE = (ctypes.c_int64 * 2)(128, 64)


def append(L, a, k=16384, v=32768, ks=STRIDE, vs=STRIDE, freq=64, rotary=64):
    return L.ssu_paged_append(ctypes.byref(a) if a is not None else None, k, ks, v, vs, freq, rotary, 0, None)


def attend(L, a, scale=0.125, window=0, seqlen=0, kv_len=0, lse=None, ws=1 << 20, size=1 << 40):
    return L.ssu_paged_attention(ctypes.byref(a) if a is not None else None, scale, window, seqlen, kv_len, lse, ws, size, None)


@pytest.mark.parametrize("kw,code,needle", [
    (dict(reserved0=1), ssu.ERR_INVALID, "reserved0"),
    (dict(io_dtype=7), ssu.ERR_INVALID, "io_dtype"),
    (dict(io_dtype=0), ssu.ERR_UNSUPPORTED, "fp16 or bf16"),
    (dict(table_type=2), ssu.ERR_INVALID, "table_type"),
    (dict(meta_type=-1), ssu.ERR_INVALID, "meta_type"),
    (dict(rows=-1), ssu.ERR_INVALID, "negative"),
    (dict(nseq=-1), ssu.ERR_INVALID, "negative"),
    (dict(pages=0), ssu.ERR_INVALID, "pages"),
    (dict(pages=1 << 31), ssu.ERR_INVALID, "pages"),
    (dict(page_size=0), ssu.ERR_INVALID, "page_size"),
    (dict(page_size=12), ssu.ERR_UNSUPPORTED, "page_size"),
    (dict(page_size=1), ssu.ERR_UNSUPPORTED, "page_size"),
    (dict(heads=5), ssu.ERR_INVALID, "multiple of kv_heads"),
    (dict(kv_heads=0), ssu.ERR_INVALID, "multiple of kv_heads"),
    (dict(heads=258), ssu.ERR_UNSUPPORTED, "share"),
    (dict(dim=60), ssu.ERR_UNSUPPORTED, "dim"),
    (dict(dim=136), ssu.ERR_UNSUPPORTED, "dim"),
    (dict(rows=1 << 31), ssu.ERR_INVALID, "2^31"),
    (dict(cu_seqlens=None), ssu.ERR_INVALID, "one row"),
    (dict(table_width=-1), ssu.ERR_INVALID, "table_width"),
    (dict(k_cache=None), ssu.ERR_INVALID, "NULL"),
    (dict(v_cache=4096), ssu.ERR_INVALID, "the same"),
    (dict(v_cache=8200), ssu.ERR_INVALID, "aligned"),
    (dict(q=1032), ssu.ERR_INVALID, "aligned"),
    (dict(out=2050), ssu.ERR_INVALID, "aligned"),
    (dict(k_cache_stride=(2048, 128, 60)), ssu.ERR_INVALID, "strides"),
    (dict(v_cache_stride=(2048, 0, 64)), ssu.ERR_INVALID, "strides"),
    (dict(k_cache_stride=(1 << 40, 128, 64)), ssu.ERR_INVALID, "too large"),
    (dict(q_stride=(-256, 64)), ssu.ERR_INVALID, "strides"),
    (dict(out_stride=(256, 36)), ssu.ERR_INVALID, "strides"),
    (dict(kv_lens=None), ssu.ERR_INVALID, "kv_lens"),
    (dict(block_table=None), ssu.ERR_INVALID, "block_table"),
    (dict(kv_lens=514), ssu.ERR_INVALID, "aligned"),
    (dict(meta_type=1, cu_seqlens=772), ssu.ERR_INVALID, "aligned"),
    (dict(table_type=1, block_table=260), ssu.ERR_INVALID, "aligned"),
    (dict(d_status=2), ssu.ERR_INVALID, "aligned"),
])
def test_refusals_of_both(libssu, kw, code, needle):
    a = args(**kw)
    size = ctypes.c_uint64(0)
    for rc in (append(libssu, a), attend(libssu, a),
               libssu.ssu_paged_attention_workspace_size(ctypes.byref(a), 0, 0, ctypes.byref(size))):
        assert rc == code
        assert needle in libssu.ssu_last_error().decode()


@pytest.mark.parametrize("kw,call,code,needle", [
    (dict(), dict(rotary=72, freq=64), ssu.ERR_INVALID, "rotary"),
    (dict(), dict(rotary=-16), ssu.ERR_INVALID, "rotary"),
    (dict(), dict(rotary=24), ssu.ERR_UNSUPPORTED, "rotary"),
    (dict(), dict(rotary=0), ssu.ERR_INVALID, "inv_freq"),
    (dict(), dict(freq=None), ssu.ERR_INVALID, "inv_freq"),
    (dict(), dict(freq=66), ssu.ERR_INVALID, "aligned"),
    (dict(q=None), dict(), ssu.ERR_INVALID, "go together"),
    (dict(out=None), dict(), ssu.ERR_INVALID, "go together"),
    (dict(out=1024, out_stride=(512, 64)), dict(), ssu.ERR_INVALID, "in place"),
    (dict(), dict(k=None), ssu.ERR_INVALID, "NULL"),
    (dict(), dict(vs=None), ssu.ERR_INVALID, "NULL"),
    (dict(), dict(v=32776), ssu.ERR_INVALID, "aligned"),
    (dict(), dict(ks=(ctypes.c_int64 * 2)(128, 60)), ssu.ERR_INVALID, "strides"),
    (dict(), dict(k=4096), ssu.ERR_INVALID, "alias"),
    (dict(out=16384), dict(), ssu.ERR_INVALID, "alias"),
])
def test_refusals_of_append(libssu, kw, call, code, needle):
    assert append(libssu, args(**kw), **call) == code
    assert needle in libssu.ssu_last_error().decode()


@pytest.mark.parametrize("kw,call,code,needle", [
    (dict(), dict(scale=0.0), ssu.ERR_INVALID, "scale"),
    (dict(), dict(scale=-1.0), ssu.ERR_INVALID, "scale"),
    (dict(), dict(scale=float("nan")), ssu.ERR_INVALID, "scale"),
    (dict(), dict(scale=float("inf")), ssu.ERR_INVALID, "scale"),
    (dict(), dict(window=-1), ssu.ERR_INVALID, "window"),
    (dict(), dict(seqlen=-1), ssu.ERR_INVALID, "max_seqlen"),
    (dict(), dict(kv_len=-1), ssu.ERR_INVALID, "max_kv_len"),
    (dict(q=None), dict(), ssu.ERR_INVALID, "NULL"),
    (dict(out=None), dict(), ssu.ERR_INVALID, "NULL"),
    (dict(out=1024), dict(), ssu.ERR_INVALID, "alias"),
    (dict(out=8192), dict(), ssu.ERR_INVALID, "alias"),
    (dict(), dict(lse=1026), ssu.ERR_INVALID, "aligned"),
    (dict(), dict(ws=None), ssu.ERR_INVALID, "workspace"),
    (dict(), dict(ws=(1 << 20) + 16), ssu.ERR_INVALID, "workspace"),
    (dict(), dict(size=16), ssu.ERR_INVALID, "smaller"),
])
def test_refusals_of_attention(libssu, kw, call, code, needle):
    assert attend(libssu, args(**kw), **call) == code
    assert needle in libssu.ssu_last_error().decode()


def test_scales_that_leave_fp32_in_units_of_log2(libssu):
    assert attend(libssu, args(), scale=3e38) == ssu.ERR_INVALID  # 3e38 log2 e is infinite
    assert "scale" in libssu.ssu_last_error().decode()
    assert attend(libssu, args(rows=0), scale=2e38) == ssu.OK  # 2e38 log2 e is 2.89e38


def test_a_hint_past_the_call_is_the_call(libssu):
    # every max_seqlen of `rows` or more asks for the same workspace, those too whose rows 64 bits do not hold
    sizes = []
    for seqlen in (6, 7, 1 << 40, (1 << 63) - 1):
        size = ctypes.c_uint64(0)
        a = args(heads=256, q_stride=(16384, 64), out_stride=(16384, 64))
        assert libssu.ssu_paged_attention_workspace_size(ctypes.byref(a), seqlen, 0, ctypes.byref(size)) == ssu.OK
        sizes.append(size.value)
    assert len(set(sizes)) == 1


def test_null_and_nothing(libssu):
    assert append(libssu, None) == ssu.ERR_INVALID and attend(libssu, None) == ssu.ERR_INVALID
    for kw in (dict(rows=0), dict(nseq=0, kv_lens=None, block_table=None)):
        assert append(libssu, args(**kw), k=None, v=None) == ssu.OK
        assert attend(libssu, args(**kw), ws=None, size=0) == ssu.OK
        size = ctypes.c_uint64(7)
        assert libssu.ssu_paged_attention_workspace_size(ctypes.byref(args(**kw)), 0, 0, ctypes.byref(size)) == ssu.OK
        assert size.value == 0
    assert libssu.ssu_paged_attention_workspace_size(ctypes.byref(args()), 0, 0, None) == ssu.ERR_INVALID


def tensors(rows=6, nseq=3):
    cache = torch.zeros(10, 16, 2, 64, dtype=torch.bfloat16)
    return dict(q=torch.zeros(rows, 4, 64, dtype=torch.bfloat16), k_cache=cache, v_cache=cache.clone(),
                block_table=torch.zeros(nseq, 5, dtype=torch.int32), kv_lens=torch.ones(nseq, dtype=torch.int32))


def test_the_bindings_refuse_host_tensors(libssu):
    t = tensors()
    with pytest.raises(ValueError):
        ssu.ssu_paged_attention(**t)
    q = t.pop("q")
    with pytest.raises(ValueError):
        ssu.ssu_paged_append(t["k_cache"], t["v_cache"], q[:, :2], q[:, :2], t["block_table"], t["kv_lens"])


@pytest.mark.parametrize("change", [dict(q=torch.zeros(6, 4 * 64)), dict(k_cache=torch.zeros(10, 16, 128)),
                                    dict(q=torch.zeros(6, 4, 64, dtype=torch.float16)), dict(q=torch.zeros(6, 4, 72, dtype=torch.bfloat16))])
def test_the_bindings_refuse_shapes(libssu, change):
    with pytest.raises(ValueError):
        ssu.ssu_paged_attention(**(tensors() | change))
