"""GPU tests of eq_gemv_w4 where a CTA walks several row tiles: the code ring
wraps, the groups of decoders carry their barriers' phases from tile to tile,
the token tiles are rewritten, and a CTA that moves to another job takes that
job's table, columns and scales.

Integer scales, tokens, tables and zero points with sums below 2^24: every
result is exact, so a slab, tile or job taken for another shows.
"""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

TABLE = torch.arange(-5, 11)


@pytest.fixture(scope="module")
def eqw():
    from entropy_coded_weight_b200 import build
    build.build()
    import entropy_coded_weight_b200 as E
    E.load()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return E


def _inputs(tokens, rows, cols, group, codes, seed=0, st=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed + tokens + rows + cols + group)
    n = -(-cols // group)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda")

    q = ints(0, 256, rows, cols // 2).to(torch.uint8)
    s = ints(1, 4, rows, n).to(st)
    z = ints(0, 16, rows, n).to(torch.uint8) if codes == "zero" else None
    x = ints(-3, 4, tokens, cols).to(torch.bfloat16)
    return q, s, z, x


def _exact(q, s, z, table, x, group):
    code = torch.stack((q & 15, q >> 4), 2).flatten(1).long()
    grp = torch.arange(code.shape[1], device="cuda") // group
    if table is not None:
        w = table.cuda().double()[code]
    else:
        w = code.double() - (8.0 if z is None else z.double()[:, grp])
    return x.double() @ (w * s.double()[:, grp]).t()


# at most |w| = 15, |s x| = 9: sums stay below 2^24 up to 124000 columns
@pytest.mark.parametrize("codes", ["int", "zero", "table"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("tokens", [1, 8, 16, 32])
@pytest.mark.parametrize("rows,cols", [(40000, 1056), (70001, 544), (19000, 4128)])
def test_several_tiles_per_cta(eqw, rows, cols, tokens, group, codes):
    q, s, z, x = _inputs(tokens, rows, cols, group, codes)
    table = TABLE.to(torch.bfloat16) if codes == "table" else None
    buf = torch.full((tokens * rows + 64,), float("nan"), device="cuda")
    y = buf[:tokens * rows].view(tokens, rows)
    eqw.gemv_w4(q, s, x, y, group=group, zeros=z, table=table)
    torch.cuda.synchronize()
    assert torch.isnan(buf[tokens * rows:]).all()
    assert torch.equal(y.double(), _exact(q, s, z, table, x, group))


def _job(lib, q, s, z, table, x, y, group):
    j = lib.eq_w4_job()
    j.q, j.scales, j.x, j.y = q.data_ptr(), s.data_ptr(), x.data_ptr(), y.data_ptr()
    j.zeros = z.data_ptr() if z is not None else None
    j.x_stride, j.rows, j.cols, j.group = x.stride(0), q.shape[0], x.shape[1], group
    j.scale_type = {torch.float32: lib.EQ_F32, torch.bfloat16: lib.EQ_BF16, torch.float16: lib.EQ_F16}[s.dtype]
    if table is not None:
        j.use_table = 1
        j.table = (ctypes.c_uint16 * 16)(*(v & 0xFFFF for v in table.view(torch.int16).tolist()))
    return j


@pytest.mark.parametrize("codes", ["int", "zero", "table"])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("tokens", [1, 5, 16, 32])
def test_jobs_that_share_ctas(eqw, tokens, group, codes):
    """Five jobs of different tables, widths and scale types, more than three tiles per CTA in all."""
    from entropy_coded_weight_b200 import _lib
    shapes = [(9000, 1056, torch.float32), (20001, 544, torch.bfloat16), (130, 4128, torch.float16),
              (15000, 2080, torch.bfloat16), (12345, 32, torch.float32)]
    sets, jobs = [], []
    for i, (rows, cols, st) in enumerate(shapes):
        q, s, z, x = _inputs(tokens, rows, cols, group, codes, seed=i, st=st)
        table = (TABLE.roll(3 * i) - i).to(torch.bfloat16) if codes == "table" else None
        y = torch.full((tokens, rows), float("nan"), device="cuda")
        sets.append((q, s, z, table, x, y))
        jobs.append(_job(_lib, q, s, z, table, x, y, group))
    arr = (_lib.eq_w4_job * len(jobs))(*jobs)
    torch.cuda.synchronize()
    assert eqw.load().eq_gemv_w4(arr, len(jobs), tokens, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    for q, s, z, table, x, y in sets:
        assert torch.equal(y.double(), _exact(q, s, z, table, x, group))


def test_repeated_and_captured_calls_on_shared_ctas(eqw):
    """The same bits every time, eagerly and replayed, with scales that round."""
    q, s, z, x = _inputs(8, 40000, 1056, 128, "zero")
    s = torch.rand(s.shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    y, first = torch.empty(8, 40000, device="cuda"), torch.empty(8, 40000, device="cuda")
    eqw.gemv_w4(q, s, x, first, group=128, zeros=z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        eqw.gemv_w4(q, s, x, y, group=128, zeros=z)
    for _ in range(10):
        y.fill_(float("nan"))
        graph.replay()
        assert torch.equal(y, first)
    # a group's sum is an exact integer; one fused rounding per group, at most 34 where the totals meet
    ref, mag = _exact(q, s, z, None, x, 128), 0.0
    for grp in range(-(-1056 // 128)):
        c = slice(grp * 128, min(1056, (grp + 1) * 128))
        mag = mag + _exact(q[:, c.start // 2:c.stop // 2], s[:, grp:grp + 1], z[:, grp:grp + 1], None, x[:, c], 128).abs()
    assert ((first.double() - ref).abs() <= (1056 / 128 + 34) * 2.0 ** -24 * mag).all()
