"""GPU test of 8-bit and 4-bit products on several streams at once.

Their CTAs share SMs and, up to 64 tokens, an SM's tensor memory, of which an
E4M3 product takes several accumulators' columns; clusters of different
launches must not wait for each other's.  Whole numbers with scales of one: every
result is exact.
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


def _ints(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device="cuda").to(torch.int8)


class _A8:
    def __init__(self, E, kind, tokens, rows, cols, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.E, self.sym, self.x8 = E, _ints(g, -3, 4, rows, cols).to(kind), _ints(g, -3, 4, tokens, cols).to(kind)
        self.ws, self.xs = torch.ones(rows, device="cuda"), torch.ones(tokens, device="cuda")
        self.y, self.status = torch.empty(tokens, rows, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        self.want = self.x8.double() @ self.sym.double().t()

    def call(self):
        self.E.gemm_a8(self.sym, self.ws, self.x8, self.xs, self.y, self.status)

    def good(self):
        return int(self.status.item()) == 0 and torch.equal(self.y.double(), self.want)


class _W4:
    def __init__(self, E, tokens, rows, cols, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.E, self.q = E, torch.randint(0, 256, (rows, cols // 2), generator=g, device="cuda", dtype=torch.uint8)
        self.s, self.x = torch.ones(rows, cols // 128, device="cuda"), _ints(g, -3, 4, tokens, cols).to(torch.bfloat16)
        self.y = torch.empty(tokens, rows, device="cuda")
        code = torch.stack((self.q & 15, self.q >> 4), 2).flatten(1).double() - 8
        self.want = self.x.double() @ code.t()

    def call(self):
        self.E.gemv_w4(self.q, self.s, self.x, self.y, group=128)

    def good(self):
        return torch.equal(self.y.double(), self.want)


@pytest.mark.parametrize("captured", [False, True])
def test_products_on_several_streams(eqw, captured):
    f8, i8 = torch.float8_e4m3fn, torch.int8
    work = [_A8(eqw, f8, 16, 4096, 28672, 1), _A8(eqw, f8, 64, 2000, 12288, 2), _A8(eqw, f8, 48, 900, 24576, 3),
            _A8(eqw, f8, 100, 1500, 8192, 4), _A8(eqw, i8, 9, 3000, 4096, 5), _A8(eqw, f8, 600, 1100, 4112, 6),
            _W4(eqw, 1, 5000, 4096, 7), _W4(eqw, 20, 700, 8192, 8)]
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    run = [w.call for w in work]
    if captured:
        for i, w in enumerate(work):
            w.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(w.graph):
                for _ in range(4):
                    w.call()
            run[i] = w.graph.replay
    for _ in range(10):
        for w in work:
            w.y.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(4):
            for go, st in zip(run, streams):
                with torch.cuda.stream(st):
                    go()
        torch.cuda.synchronize()
        assert all(w.good() for w in work)
