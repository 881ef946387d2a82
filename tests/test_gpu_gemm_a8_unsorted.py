"""GPU test of eq_gemm_a8's super weights that are not sorted by row.

Such a list is reported (EQ_DEV_BAD_OUTLIER) and entries of it may be missed, but
nothing else may change: every output is the product, plus the terms of some of
its row's entries.  Whole numbers, so each of these sums is exact.
"""
import itertools

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


@pytest.mark.parametrize("kind", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("tokens,rows,cols", [(3, 700, 2048), (40, 2050, 512), (300, 700, 1024), (4096, 8192, 512)])
@pytest.mark.parametrize("order", [[600, 5, 300], [130, 128, 5, 699, 131, 2, 500, 4], [5, 699, 5, 130, 129, 5]])
def test_rows_out_of_order(eqw, tokens, rows, cols, kind, order):
    g = torch.Generator(device="cuda").manual_seed(tokens + rows + len(order))

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda")

    sym, x8 = ints(-3, 4, rows, cols).to(torch.int8).to(kind), ints(1, 4, tokens, cols).to(torch.int8).to(kind)
    col = ints(0, cols, len(order)).int()
    val = (2.0 ** torch.arange(len(order), device="cuda"))  # exact in bf16; every subset has its own sum
    y = torch.full((tokens, rows), 1e30, device="cuda")  # what a read before the product's store would find
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    eqw.gemm_a8(sym.view(torch.uint8), torch.ones(rows, device="cuda"), x8, torch.ones(tokens, device="cuda"), y, status,
                outliers=(torch.tensor(order, dtype=torch.int32, device="cuda"), col, val))
    torch.cuda.synchronize()
    assert int(status.item()) == eqw.EQ_DEV_BAD_OUTLIER
    base = x8.double() @ sym.double().t()
    plain = [r for r in range(rows) if r not in order]
    assert torch.equal(y[:, plain].double(), base[:, plain])
    for r in set(order):
        terms = [x8[:, col[i]].double() * val[i].double() for i, q in enumerate(order) if q == r]
        fits = torch.zeros(tokens, dtype=torch.bool, device="cuda")
        for n in range(len(terms) + 1):
            for some in itertools.combinations(terms, n):
                fits |= y[:, r].double() == base[:, r] + sum(some)
        assert fits.all(), r
