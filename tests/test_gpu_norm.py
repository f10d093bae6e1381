"""The residual-adding RMS norm against its definition in 64 bits.

x + residual is one fp32 sum (exact for 16-bit inputs unless they differ by more
than 2^16 in size, so residual_out is held to the rounding of the fp32 sum, bit
for bit).  The norm is a sum of up to 32768 squares (a tree over the threads
above at most 32 in a row: under 2^-17 of the sum, half of it in the root), a
root and three products: |dy| <= 2^-17 |y| + half an ulp of the output (2^-8 of
the value covers bf16, 2^-11 fp16 above its subnormals).  An E4M3 code is the
nearest to y 448 / amax, whose relative error is as small, so it lies within half
a step of its place, a step being 2^-3 of the value's power of two (2^-9 below
2^-6), 2^-12 of the value more for the error of y and of the factor."""
import pytest
import torch

import selective_state_update_gb300 as ssu

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-38, torch.float16: 2.0 ** -24, torch.bfloat16: 1e-38}


def problem(seed, rows, hidden, dtype, wdtype=None, residual=True, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    make = lambda: (torch.randn(rows, hidden + pad, generator=g, device=DEV) *
                    torch.randn(rows, 1, generator=g, device=DEV).exp()).to(dtype)[:, :hidden]
    w = (1 + 0.2 * torch.randn(hidden, generator=g, device=DEV)).to(wdtype or dtype)
    return make(), w, make() if residual else None


def reference(x, w, residual, eps):
    r = x.float() + (residual.float() if residual is not None else 0.0)
    d = r.double()
    return r, d / torch.sqrt((d * d).mean(-1, keepdim=True) + eps) * w.double()


def check(x, w, residual, quant, eps=1e-5, **kw):
    r, y = reference(x, w, residual, eps)
    keep = residual.clone() if residual is not None else None
    out, scales, stream = ssu.ssu_add_rmsnorm(x, w, eps=eps, residual=residual, quant=quant, **kw)
    if residual is None:
        assert stream is None
    else:
        assert torch.equal(stream, r.to(x.dtype))
        if stream.data_ptr() != residual.data_ptr():
            assert torch.equal(residual, keep)
    if quant == "none":
        assert scales is None and out.dtype == x.dtype
        assert ((out.double() - y).abs() <= (2.0 ** -17 + HALF_ULP[x.dtype]) * y.abs() + TINY[x.dtype]).all()
        return out
    rows, hidden = x.shape
    width = hidden if quant == "row" else 128
    blocks = -(-hidden // width)
    amax = torch.nn.functional.pad(y.abs(), (0, blocks * width - hidden)).view(rows, blocks, width).amax(-1)
    want = torch.where(amax > 0, amax / 448, 1.0)
    assert out.dtype == torch.float8_e4m3fn and scales.dtype == torch.float32
    assert ((scales.double().view(rows, blocks) - want).abs() <= 2.0 ** -16 * want).all()
    place = y / torch.repeat_interleave(want, width, dim=1)[:, :hidden]
    step = torch.exp2(torch.floor(torch.log2(place.abs().clamp(min=2.0 ** -6))) - 3)
    assert ((out.double() - place).abs() <= step / 2 + 2.0 ** -12 * place.abs()).all()
    return out


@pytest.mark.parametrize("quant", ["none", "row", "block"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hidden", [1, 7, 8, 127, 128, 129, 1000, 2048, 2056, 2565, 4096, 8192, 8200, 16384, 20001, 32768])
def test_norm(libssu, hidden, dtype, quant):
    x, w, res = problem(hidden, 5, hidden, dtype)
    check(x, w, res, quant)
    check(x, w, None, quant)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows", [1, 3, 1000])
def test_norm_fp32_weight(libssu, rows, dtype):
    x, w, res = problem(rows, rows, 1536, dtype, wdtype=torch.float32)
    for quant in ("none", "row", "block"):
        check(x, w, res, quant)


@pytest.mark.parametrize("pad", [1, 8])
@pytest.mark.parametrize("quant", ["none", "row", "block"])
def test_norm_strided_rows(libssu, quant, pad):
    """Rows of wider tensors, and outputs into them."""
    x, w, res = problem(40 + pad, 9, 1024, torch.bfloat16, pad=pad)
    y_dtype = torch.bfloat16 if quant == "none" else torch.float8_e4m3fn
    out = torch.zeros(9, 1024 + 2 * pad, dtype=torch.uint8 if quant != "none" else y_dtype, device=DEV)
    view = (out if quant == "none" else out.view(torch.float8_e4m3fn))[:, pad:pad + 1024]
    keep = torch.zeros(9, 1024 + pad, dtype=torch.bfloat16, device=DEV)
    check(x, w, res, quant, out=view, residual_out=keep[:, :1024])
    assert (out[:, :pad] == 0).all() and (out[:, pad + 1024:] == 0).all() and (keep[:, 1024:] == 0).all()


def test_norm_in_place_residual(libssu):
    x, w, res = problem(50, 17, 4096, torch.bfloat16)
    r, _ = reference(x, w, res, 1e-5)
    want = ssu.ssu_add_rmsnorm(x, w, residual=res)
    got = ssu.ssu_add_rmsnorm(x, w, residual=res, residual_out=res)
    assert torch.equal(got[0], want[0]) and torch.equal(res, r.to(torch.bfloat16))


@pytest.mark.parametrize("hidden", [1024, 1001])
def test_norm_zero_and_tiny_rows(libssu, hidden):
    """A row of zeros has scale 1 and zero codes; a row far below eps is not blown up."""
    x, w, _ = problem(60, 4, hidden, torch.float32, residual=False)
    x[0] = 0
    x[1] *= 1e-30
    x[2, 128:256] = 0
    for quant in ("none", "row", "block"):
        out, scales, _ = ssu.ssu_add_rmsnorm(x, w, quant=quant)
        assert (out[0].float() == 0).all()
        if quant != "none":
            assert (scales[0] == 1).all()
        if quant == "block":
            assert scales[2, 1] == 1 and (out[2, 128:256].float() == 0).all()
    check(x, w, None, "none")


@pytest.mark.parametrize("hidden", [1024, 1001])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_norm_bad_row_stays_alone(libssu, hidden, bad):
    x, w, res = problem(70, 3, hidden, torch.bfloat16)
    clean = {q: ssu.ssu_add_rmsnorm(x, w, residual=res, quant=q) for q in ("none", "row", "block")}
    x[1, 5] = bad
    for q, (y, s, r) in clean.items():
        y2, s2, r2 = ssu.ssu_add_rmsnorm(x, w, residual=res, quant=q)
        assert torch.isnan(y2[1].float()[5])
        for row in (0, 2):
            assert torch.equal(y[row].float(), y2[row].float()) and torch.equal(r[row], r2[row])
            assert s is None or torch.equal(s[row], s2[row])


def test_norm_no_rows(libssu):
    x, w, res = problem(80, 0, 512, torch.bfloat16)
    y, s, r = ssu.ssu_add_rmsnorm(x, w, residual=res, quant="block")
    assert y.shape == (0, 512) and s.shape == (0, 4) and r.shape == (0, 512)


def test_norm_offsets_past_32_bits(libssu):
    far = torch.zeros(2 ** 31 + 2 ** 16, dtype=torch.bfloat16, device=DEV)
    rows = far.as_strided((3, 2048), (2 ** 30, 1))
    x, w, res = problem(90, 3, 2048, torch.bfloat16)
    rows.copy_(x)
    a = ssu.ssu_add_rmsnorm(x, w, residual=res, quant="row")
    b = ssu.ssu_add_rmsnorm(rows, w, residual=res, quant="row")
    assert torch.equal(a[0].float(), b[0].float()) and torch.equal(a[2], b[2])


def test_norm_refusals_on_device(libssu):
    x, w, res = problem(95, 3, 512, torch.bfloat16)
    with pytest.raises(ValueError, match="quant"):
        ssu.ssu_add_rmsnorm(x, w, quant="int8")
    with pytest.raises(ValueError, match="weight"):
        ssu.ssu_add_rmsnorm(x, w[:256])
    with pytest.raises(ValueError, match="weight"):
        ssu.ssu_add_rmsnorm(x, w.half())
    with pytest.raises(ValueError, match="residual"):
        ssu.ssu_add_rmsnorm(x, w, residual=res[:2])
    with pytest.raises(ValueError, match="needs a residual"):
        ssu.ssu_add_rmsnorm(x, w, residual_out=res)
    with pytest.raises(ValueError, match="unit column stride"):
        ssu.ssu_add_rmsnorm(x.t(), w)
    with pytest.raises(ValueError, match="scales"):
        ssu.ssu_add_rmsnorm(x, w, quant="row", scales=torch.zeros(4, device=DEV))
    with pytest.raises(ValueError, match="alias"):
        ssu.ssu_add_rmsnorm(x, w, out=x)
    with pytest.raises(ValueError, match="eps"):
        ssu.ssu_add_rmsnorm(x, w, eps=0.0)
    with pytest.raises(NotImplementedError, match="hidden"):
        ssu.ssu_add_rmsnorm(torch.zeros(1, 40000, device=DEV), torch.zeros(40000, device=DEV))
