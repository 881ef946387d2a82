"""GPU test of how exact eq_gemm_a8's E4M3 sums are.

The tensor core rounds its fp32 accumulator towards zero, a bias that grows with
the number of products that go through one accumulator: of the result's norm,
2.3e-7 at 32 slabs of 128 columns, 5e-7 at 64, 8.3e-7 at 96.  No accumulator takes
more than 32, the accumulators are added in fp32, rounded to nearest, and the two
scales add a rounding of at most 2^-24 each.  So the error stays at that of 32 slabs,
whatever the width and the launch shape: a quarter above it is the limit, and
every output keeps the proven bound (32-term instructions, one step per
instruction at 2^-22, see the depth below).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def eqw():
    from entropy_coded_weight_b200 import build
    build.build()
    import entropy_coded_weight_b200 as E
    E.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return E


@pytest.mark.parametrize("cols", [4096, 8192, 12288, 24576, 28672, 57344])
@pytest.mark.parametrize("tokens,rows", [(1, 512), (16, 4096), (64, 512), (100, 512), (256, 300), (300, 4096), (2048, 2048)])
def test_e4m3_sums_are_as_exact_at_any_width(eqw, tokens, rows, cols):
    g = torch.Generator(device="cuda").manual_seed(tokens + rows + cols)
    sym = (60 * torch.randn(rows, cols, generator=g, device="cuda")).clamp(-448, 448).to(torch.float8_e4m3fn)
    x8 = (100 * torch.randn(tokens, cols, generator=g, device="cuda")).clamp(-448, 448).to(torch.float8_e4m3fn)
    ws = torch.rand(rows, generator=g, device="cuda") + 0.5
    xs = torch.rand(tokens, generator=g, device="cuda") + 0.5
    y = torch.empty(tokens, rows, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    eqw.gemm_a8(sym, ws, x8, xs, y, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    x, w, sc = x8.double(), sym.double(), xs.double().unsqueeze(1) * ws.double()
    ref = (x @ w.t()) * sc
    err = (y.double() - ref).abs()
    # depth: an accumulator's 128 instructions, 32 terms in each, the accumulators
    depth = 128 + 32 + cols / 2048 + 8
    assert (err <= depth * 2.0 ** -22 * (x.abs() @ w.abs().t()) * sc + ref.abs() * 2.0 ** -22).all()
    assert float(err.norm() / ref.norm()) < 1.25 * 2.3e-7
