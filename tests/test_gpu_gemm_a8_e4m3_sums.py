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


@pytest.mark.parametrize("cols", [(1 << 24) + 16, 90_000_000])
def test_very_wide_matrices(eqw, cols):
    """More chains than 32-bit products of slabs and chains could number.  Few nonzero whole numbers: exact."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rows, tokens, n = 3, 2, 4096
    at = torch.randint(0, cols, (n,), generator=g, device="cuda").unique()
    at = torch.cat((at, torch.tensor([0, 1, cols - 17, cols - 1], device="cuda"))).unique()
    w = torch.randint(1, 5, (rows, at.numel()), generator=g, device="cuda")
    x = torch.randint(-4, 5, (tokens, at.numel()), generator=g, device="cuda")
    sym, x8 = (torch.zeros(k, cols, dtype=torch.uint8, device="cuda") for k in (rows, tokens))
    sym[:, at] = w.to(torch.int8).to(torch.float8_e4m3fn).view(torch.uint8)
    x8[:, at] = x.to(torch.int8).to(torch.float8_e4m3fn).view(torch.uint8)
    y = torch.empty(tokens, rows, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    eqw.gemm_a8(sym, torch.ones(rows, device="cuda"), x8.view(torch.float8_e4m3fn), torch.ones(tokens, device="cuda"),
                y, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(y.double(), x.double() @ w.double().t())
