"""A wait that gives up in the 8-bit GEMM's pair kernel ends the kernel.

eq_selftest_a8_wait_timeout runs the kernel's own epilogue on a tile with super
weights: seven warps reach the tile's barrier, the eighth gives up a wait on a
barrier that nothing arrives on and learns only then that the launch has failed.
It has to reach the barrier all the same, or the block never ends.
"""
import time

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


def test_an_epilogue_warp_that_gives_up_reaches_the_barrier(eqw, orc):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    eqw.selftest_a8_wait_timeout(status)
    torch.cuda.synchronize()
    dt = time.perf_counter() - t0
    assert int(status.item()) == eqw.EQ_DEV_TIMEOUT
    assert 0.5 < dt < 10.0, dt  # 2e9 cycles

    # the context is usable and the tensor memory free: the pair kernel (a limit on the SMs picks it), Int8, exact
    m = W.random_int8_matrix(8, 256, 1024, layer=0, index=0)
    blob = eqw.encode_host([m])
    model = eqw.Model(eqw.upload(blob), blob)
    model.set_sm_limit(4)
    status.zero_()
    sym = torch.empty(m.n, dtype=torch.uint8, device="cuda")
    model.decode_symbols(0, sym, status)
    x8 = torch.randint(-128, 128, (64, m.cols), generator=torch.Generator().manual_seed(1), dtype=torch.int8)
    y = torch.empty(64, m.rows, device="cuda")
    model.gemm_symbols_a8(0, sym, x8.cuda(), torch.ones(64, device="cuda"), y, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    s = x8.double() @ torch.from_numpy(orc.stream_symbols(m)).view(torch.int8).double().t()
    assert torch.equal(y.cpu(), s.float() * torch.from_numpy(m.scales))
    model.close()
