"""GPU tests of eq_gemv_w4's zero points beyond the codes' own range: whole
numbers up to 127 count in full (formats that store zero + 1 have 16), a byte
above 127 marks its row's outputs NaN.

Integer scales and tokens, sums below 2^24: the results are exact.
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


def _inputs(tokens, rows, cols, group, top):
    g = torch.Generator().manual_seed(tokens + rows + cols + group + top)
    n = -(-cols // group)
    q = torch.randint(0, 256, (rows, cols // 2), generator=g, dtype=torch.uint8)
    s = torch.randint(1, 4, (rows, n), generator=g).float()
    z = torch.randint(0, top + 1, (rows, n), generator=g, dtype=torch.uint8)
    z[0, 0], z[-1, -1] = top, top
    x = torch.randint(-3, 4, (tokens, cols), generator=g).to(torch.bfloat16)
    return q, s, z, x


def _exact(q, s, z, x, group):
    code = torch.stack((q & 15, q >> 4), 2).flatten(1).long()
    grp = torch.arange(code.shape[1]) // group
    return x.double() @ ((code - z.long()[:, grp]).double() * s.double()[:, grp]).t()


# |w| <= 127 with |s x| <= 9: sums stay below 2^24 up to 14000 columns
@pytest.mark.parametrize("top", [16, 17, 127])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("tokens,rows,cols", [(1, 200, 1280), (8, 130, 2080), (16, 64, 4128), (32, 257, 544)])
def test_zero_points_above_15(eqw, tokens, rows, cols, group, top):
    q, s, z, x = _inputs(tokens, rows, cols, group, top)
    y = torch.empty(tokens, rows, device="cuda")
    eqw.gemv_w4(q.cuda(), s.cuda(), x.cuda(), y, group=group, zeros=z.cuda())
    torch.cuda.synchronize()
    assert torch.equal(y.cpu().double(), _exact(q, s, z, x, group))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("bad", [128, 200, 255])
@pytest.mark.parametrize("tokens", [1, 20])
def test_zero_points_above_127_mark_their_row(eqw, tokens, bad, group):
    rows, cols = 150, 1056
    q, s, z, x = _inputs(tokens, rows, cols, group, 15)
    z[9, 1], z[77, -1] = bad, bad
    y = torch.empty(tokens, rows, device="cuda")
    eqw.gemv_w4(q.cuda(), s.cuda(), x.cuda(), y, group=group, zeros=z.cuda())
    torch.cuda.synchronize()
    y, keep = y.cpu(), [r for r in range(rows) if r not in (9, 77)]
    assert torch.isnan(y[:, [9, 77]]).all()
    assert torch.equal(y[:, keep].double(), _exact(q, s, z, x, group)[:, keep])
