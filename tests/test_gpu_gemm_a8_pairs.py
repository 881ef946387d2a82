"""GPU tests of the 8-bit GEMM's pair kernel (256 x 256 tiles on pairs of SMs).

A limit on a model's SMs always takes that kernel, at any size, and few SMs mean
many tiles per pair: both accumulators in turn, sums of E4M3 products in an
even and an odd number of parts, super weights on top of them, row and token
tiles that are cut short.

Small whole numbers with scales of one: every product, part and sum is below
2^24 and so exact whatever its order, and any slip of a tile, part or buffer shows.
"""
import numpy as np
import pytest
import torch

import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def eqw():
    from entropy_coded_weight_b200 import build
    build.build()
    import entropy_coded_weight_b200 as E
    E.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return E


DTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def _matrix(E, kind, rows, cols, n_out, seed, index=0):
    """Whole numbers in [-3, 3] as symbols, super weights in [-8, 8], scales of one."""
    rng = np.random.default_rng(seed)
    v = rng.integers(-3, 4, (rows, cols), dtype=np.int8)
    sym = v.copy() if kind == "int8" else torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.int8).numpy()
    m = W.random_int8_matrix(seed, rows, cols, layer=0, index=index) if kind == "int8" else \
        W.random_e4m3_matrix(seed, rows, cols, layer=0, index=index)
    m.symbols = sym.view(m.symbols.dtype).reshape(m.symbols.shape)
    m.scales = np.ones_like(m.scales)
    if n_out:
        at = np.unique(np.concatenate([rng.choice(rows * cols, n_out, replace=False),
                                       np.arange(3) + (rows - 1) * cols, [0, cols - 1]]))
        m.out_row, m.out_col = (at // cols).astype(np.uint32), (at % cols).astype(np.uint32)
        m.out_val = rng.integers(1, 9, at.size).astype(np.float32) * rng.choice([-1, 1], at.size).astype(np.float32)
    return m


def _want(orc, m, kind, x8):
    sym = torch.from_numpy(orc.stream_symbols(m)).view(DTYPE[kind]).double().reshape(m.rows, m.cols).cuda()
    x = x8.double()
    y = x @ sym.t()
    if len(m.out_row):
        r, c = (torch.from_numpy(a.astype(np.int64)).cuda() for a in (m.out_row, m.out_col))
        y.index_add_(1, r, x[:, c] * torch.from_numpy(m.out_val).double().cuda())
    return y


def _tokens(kind, tokens, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-3, 4, (tokens, cols), generator=g, device="cuda").to(torch.int8).to(DTYPE[kind])


# |sum| <= 9 cols + 24 per super weight: below 2^24 up to 10^6 columns
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("n_out", [0, 60])
@pytest.mark.parametrize("rows,cols", [(300, 24592), (700, 12304), (1100, 1040), (256, 16), (8, 12288), (513, 28672)])
def test_whole_numbers_are_exact(eqw, orc, rows, cols, n_out, kind):
    m = _matrix(eqw, kind, rows, cols, n_out, seed=rows + cols)
    blob = eqw.encode_host([m])
    model = eqw.Model(eqw.upload(blob), blob)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sym = torch.empty(m.n, dtype=torch.uint8, device="cuda")
    model.decode_symbols(0, sym, status)
    for limit in (2, 4, 10):
        model.set_sm_limit(limit)
        for tokens in (1, 255, 600, 1300):
            x8 = _tokens(kind, tokens, cols, tokens + limit)
            buf = torch.full((tokens * rows + 64,), float("nan"), device="cuda")
            y = buf[:tokens * rows].view(tokens, rows)
            model.gemm_symbols_a8(0, sym, x8, torch.ones(tokens, device="cuda"), y, status)
            torch.cuda.synchronize()
            assert int(status.item()) == 0
            assert torch.isnan(buf[tokens * rows:]).all()
            assert torch.equal(y.double(), _want(orc, m, kind, x8)), (limit, tokens)
    model.close()


@pytest.mark.parametrize("limit", [2, 6])
def test_a_layer_of_both_types(eqw, orc, limit):
    """Matrices of several widths and both types, with super weights, walked by few pairs; replayed from a graph."""
    shapes = [("int8", 300, 2048, 20), ("e4m3", 520, 24592, 30), ("e4m3", 90, 12304, 9), ("int8", 1000, 272, 0),
              ("e4m3", 257, 528, 0)]
    mats = [_matrix(eqw, k, r, c, n, seed=50 + i, index=i) for i, (k, r, c, n) in enumerate(shapes)]
    blob = eqw.encode_host(mats)
    model = eqw.Model(eqw.upload(blob), blob)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    syms = [torch.empty(m.n, dtype=torch.uint8, device="cuda") for m in mats]
    model.decode_symbols_block(0, syms, status)
    model.set_sm_limit(limit)
    tokens = 530
    x8s = [_tokens(k, tokens, c, 9 + i) for i, (k, _, c, _) in enumerate(shapes)]
    xss = [torch.ones(tokens, device="cuda") for _ in shapes]
    ys = [torch.full((tokens, r), float("nan"), device="cuda") for _, r, _, _ in shapes]
    model.gemm_symbols_a8_block(0, syms, x8s, xss, ys, status)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    want = [_want(orc, m, s[0], x) for m, s, x in zip(mats, shapes, x8s)]
    with torch.cuda.graph(graph):
        model.gemm_symbols_a8_block(0, syms, x8s, xss, ys, status)
    for again in range(3):
        for y, w in zip(ys, want):
            assert torch.equal(y.double(), w), again
            y.fill_(float("nan"))
        graph.replay()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    model.close()


@pytest.mark.parametrize("n_out", [0, 40])
@pytest.mark.parametrize("rows,cols", [(520, 24592), (300, 12288)])
def test_e4m3_values_within_the_bound(eqw, orc, rows, cols, n_out):
    """Ordinary values.  Products are exact; a sum's depth is at most cols / 32 instructions, 32 terms in each and
    the parts, taken at 2^-22 per step; two fp32 roundings for the scales, n + 3 for the super weights."""
    m = W.random_e4m3_matrix(rows, rows, cols, alpha=1.0)
    if n_out:
        m.out_row, m.out_col, m.out_val = W.outliers_for(np.random.default_rng(1), m.symbols, m.scales, n_out, m.dtype)
    blob = eqw.encode_host([m])
    model = eqw.Model(eqw.upload(blob), blob)
    model.set_sm_limit(4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sym = torch.empty(m.n, dtype=torch.uint8, device="cuda")
    model.decode_symbols(0, sym, status)
    tokens = 700
    g = torch.Generator(device="cuda").manual_seed(3)
    x8 = (100 * torch.randn(tokens, cols, generator=g, device="cuda")).clamp(-448, 448).to(torch.float8_e4m3fn)
    xs = torch.rand(tokens, generator=g, device="cuda") + 0.1
    y = torch.empty(tokens, rows, device="cuda")
    model.gemm_symbols_a8(0, sym, x8, xs, y, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    w = torch.from_numpy(orc.stream_symbols(m)).view(torch.float8_e4m3fn).double().reshape(rows, cols).cuda()
    x = x8.double()
    sc = xs.double().unsqueeze(1) * torch.from_numpy(m.scales).double().cuda()
    ref = (x @ w.t()) * sc
    tol = (cols / 32 + 40) * 2.0 ** -22 * (x.abs() @ w.abs().t()) * sc + ref.abs() * 2.0 ** -22
    if n_out:
        r, c = (torch.from_numpy(a.astype(np.int64)).cuda() for a in (m.out_row, m.out_col))
        v = torch.from_numpy(m.out_val).cuda().to(torch.bfloat16).double()
        term = x[:, c] * v * xs.double().unsqueeze(1)
        ref = ref.index_add(1, r, term)
        tol = tol.index_add(1, r, term.abs() * (len(v) + 3) * 2.0 ** -24) + ref.abs() * 2.0 ** -23
    assert ((y.double() - ref).abs() <= tol).all()
    model.close()
