"""Limits of the 8-bit GEMM's arguments: no GPU and no launch (every call is refused or empty)."""
import pytest

FAKE = 0x7F0000000000  # 256-byte aligned device-looking address; never dereferenced
OK, INVALID, UNSUPPORTED = 0, 1, 3
INT8, E4M3 = 1, 2


@pytest.fixture(scope="module")
def lib():
    from entropy_coded_weight_b200 import build
    build.build()
    from entropy_coded_weight_b200 import _lib
    return _lib


def _call(lib, tokens, **kw):
    a = dict(sym=FAKE, scale=FAKE, x8=FAKE, x_scale=FAKE, y=FAKE, out_row=None, out_col=None, out_val=None, rows=128,
             cols=64, dtype=E4M3, n_out=0, out_stride=0)
    a.update(kw)
    return lib.load().eq_gemm_a8((lib.eq_a8_job * 1)(lib.eq_a8_job(**a)), 1, tokens, FAKE, None)


@pytest.mark.parametrize("cols,code", [(1 << 26, OK), (642000 * 128, OK), (0x7FFFFF00, OK),
                                       (0x7FFFFF10, UNSUPPORTED), (1 << 31, UNSUPPORTED), ((1 << 32) - 16, UNSUPPORTED)])
def test_e4m3_columns(lib, cols, code):
    """Coordinates of the copies are signed 32-bit numbers: beyond 2^31 they would skip products."""
    assert _call(lib, 0, cols=cols) == code
    assert _call(lib, 0, cols=cols, dtype=INT8) == UNSUPPORTED


def test_parts_of_k():
    """The kernel's split of the slabs into chains, at the widest accepted matrix and around multiples of a chain:
    every product and sum below 2^32."""
    for cols in (0x7FFFFF00, 642000 * 128, 16, 2048, 2064, 12288, 12304, 28672):
        slabs = (cols + 127) // 128
        segs = (slabs + 15) // 16
        n, more = slabs // segs, slabs % segs
        assert n + (more > 0) <= 16 and n > 0 and n * segs + more == slabs
        assert cols + 127 < 2 ** 32 and slabs * 128 <= 2 ** 31
