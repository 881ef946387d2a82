"""GPU tests of eq_rmsnorm on rows whose sum of squares passes the fp32 range:
their normalised values are ordinary numbers, and have to come out as such.

Tolerances.  Such a row is computed from h 2^-80, an exact scaling but for
values below 2^-46, whose error of at most 2^-150 there is 2^-70 in h and, times
gamma / rms with an rms above 2^55, far below 2^-120 in the output.  Else the steps
are those of any row: the relative error of 1 / rms is below REL = 2^-18 (at
most 32 terms per thread, two butterflies of 5 levels, a few roundings), and
bf16 rounds by 2^-8 of the value.  The 8-bit codes are compared bit for bit with
the same fp32 steps in numpy on the scaled row.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

REL = 2.0 ** -18
TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
TYPES = [torch.bfloat16, torch.int8, torch.float8_e4m3fn]


@pytest.fixture(scope="module")
def eqw():
    from entropy_coded_weight_b200 import build
    build.build()
    import entropy_coded_weight_b200 as E
    E.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return E


LARGE = [1, 2, 4, 5, 6]  # rows of _rows() whose squares' sum passes 2^128


def _rows(tokens, cols, xt):
    g = torch.Generator().manual_seed(31 * tokens + cols)
    x = torch.randn(tokens, cols, generator=g, dtype=torch.float64)
    x[1] = x[1] * 1e30
    x[2] = 3e38                      # every square overflows by itself
    x[4] *= 1e-3                     # one large value among ordinary ones
    x[4, cols // 3] = -2e38
    x[5] = x[5].sign() * 1.5e19      # no thread's own sum need overflow
    x[5, 0] = 2e19
    x[6] = x[6].clamp(-3, 3) * 1e38
    return x.float().to(xt)


def _call(E, x, res, gamma, out_type, eps=1e-5):
    d = [None if t is None else t.cuda() for t in (x, res, gamma)]
    out = torch.zeros(x.shape, dtype=out_type, device="cuda")
    scale = None if out_type == torch.bfloat16 else torch.full((x.shape[0],), float("nan"), device="cuda")
    E.rmsnorm(d[0], out, gamma=d[2], eps=eps, residual=d[1], out_scale=scale)  # the residual in place
    torch.cuda.synchronize()
    return out.cpu(), None if scale is None else scale.cpu(), None if res is None else d[1].cpu()


def _check_large(x, res, gamma, eps, out, scale, res_out, rows):
    h32 = x.float() if res is None else x.float() + res.float()
    if res is not None:
        assert torch.equal(res_out, h32.to(res.dtype))
    h = h32.double()[rows]
    gm = torch.ones(x.shape[1]) if gamma is None else gamma.float()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + eps) * gm.double()
    assert torch.isfinite(y).all() and (y.abs().amax(1) > 0.1).all()
    if out.dtype == torch.bfloat16:
        assert ((out[rows].double() - y).abs() <= y.abs() * (2.0 ** -8 + 2 * REL) + 2.0 ** -120).all()
        return
    top = np.float32(TOP[out.dtype])
    p32 = ((h32[rows] * 2.0 ** -80) * gm).numpy()
    inv = top / np.abs(p32).max(1)
    v32 = torch.from_numpy(p32 * inv[:, None])
    code = v32.round().to(torch.int8) if out.dtype == torch.int8 else v32.clamp(-448, 448).to(out.dtype)
    assert torch.equal(out[rows].view(torch.uint8), code.view(torch.uint8))
    want = y.abs().amax(1) / float(top)
    assert ((scale[rows].double() - want).abs() <= want * 2 * REL).all()


@pytest.mark.parametrize("out_type", TYPES)
@pytest.mark.parametrize("xt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,cols", [(7, 5), (9, 100), (9, 256), (11, 512), (8, 1000), (7, 4096), (8, 5121),
                                         (7, 8192), (700, 640), (620, 2056), (7, 16384), (7, 32761), (7, 32768)])
def test_rows_beyond_the_range_of_their_squares(eqw, tokens, cols, xt, out_type):
    """Every access mode and thread shape; several rows per block, some large and some not."""
    x = _rows(tokens, cols, xt)
    gamma = (1 + 0.2 * torch.randn(cols, generator=torch.Generator().manual_seed(2))).clamp(0.5, 2).to(torch.bfloat16)
    out, scale, _ = _call(eqw, x, None, gamma, out_type)
    large = [r for r in LARGE if cols > 1]
    _check_large(x, None, gamma, 1e-5, out, scale, None, large)
    # the other rows are what they are without large ones beside them
    tame = x.clone()
    tame[large] = 1.0
    out1, scale1, _ = _call(eqw, tame, None, gamma, out_type)
    rest = [r for r in range(tokens) if r not in large]
    assert torch.equal(out[rest].view(torch.uint8), out1[rest].view(torch.uint8))
    assert scale is None or torch.equal(scale[rest], scale1[rest])


@pytest.mark.parametrize("out_type", TYPES)
@pytest.mark.parametrize("rt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [96, 1001, 4096])
def test_large_sums_with_a_residual_in_place(eqw, cols, rt, out_type):
    x = (_rows(8, cols, torch.float32) * 0.25).float()
    res = torch.randn(8, cols, generator=torch.Generator().manual_seed(3)).to(rt)
    res[1] = res[1] * 1e29
    out, scale, ro = _call(eqw, x, res, None, out_type)
    _check_large(x, res, None, 1e-5, out, scale, ro, [1, 2, 4, 6])


@pytest.mark.parametrize("out_type", TYPES)
def test_gamma_that_would_overflow_the_product(eqw, out_type):
    """h gamma passes the fp32 range, h gamma / rms does not."""
    x = torch.full((3, 264), 3e38)
    x[1] *= torch.linspace(-1, 1, 264)
    gamma = torch.linspace(4, 16, 264).to(torch.bfloat16)
    out, scale, _ = _call(eqw, x, None, gamma, out_type)
    _check_large(x, None, gamma, 1e-5, out, scale, None, [0, 1, 2])


def test_a_large_eps_still_counts(eqw):
    x = torch.full((2, 128), 1.2e19)
    out, _, _ = _call(eqw, x, None, None, torch.bfloat16, eps=3e38)
    h = x.double()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + 3e38)
    assert ((out.double() - y).abs() <= y.abs() * (2.0 ** -8 + 2 * REL)).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("cols", [96, 4096])
def test_a_bad_value_in_a_large_row(eqw, bad, cols):
    """Infinities and NaN stay what they were: the value NaN, the 8-bit row's scale NaN."""
    x = _rows(8, cols, torch.float32)
    x[1, 7] = bad
    out, _, _ = _call(eqw, x, None, None, torch.bfloat16)
    assert torch.isnan(out[1, 7])
    _check_large(x, None, None, 1e-5, out, None, None, [2, 4, 5, 6])
    for ot in (torch.int8, torch.float8_e4m3fn):
        out, scale, _ = _call(eqw, x, None, None, ot)
        assert torch.isnan(scale[1]) and torch.isfinite(scale[[0, 2, 3, 4, 5, 6, 7]]).all()
        _check_large(x, None, None, 1e-5, out, scale, None, [2, 4, 5, 6])
