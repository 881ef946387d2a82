"""What the Python entry points of the activation and 4-bit operators refuse: no GPU, no launch."""
import pytest
import torch

import entropy_coded_weight_b200 as E


@pytest.fixture
def reach(monkeypatch):
    """CPU tensors get as far as the library call, which is recorded instead of made."""
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or 0

    monkeypatch.setattr(E, "_launch_stream", lambda *a: 0)
    monkeypatch.setattr(E, "load", lambda: Lib())
    return calls


def _a8(sym_dtype, x_dtype):
    return dict(sym=torch.zeros(8, 32, dtype=sym_dtype), scale=torch.ones(8), x8=torch.zeros(2, 32, dtype=x_dtype),
                x_scale=torch.ones(2), y=torch.zeros(2, 8), status=torch.zeros(1, dtype=torch.int32))


@pytest.mark.parametrize("x_dtype", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("sym_dtype", [torch.uint8, torch.int8, torch.float8_e4m3fn, torch.bool, torch.float8_e5m2])
def test_symbols_are_bytes_or_typed_like_the_tokens(reach, sym_dtype, x_dtype):
    a = _a8(sym_dtype, x_dtype)
    lists = [[a[k]] for k in ("sym", "scale", "x8", "x_scale", "y")]
    if sym_dtype in (torch.uint8, x_dtype):
        E.gemm_a8(**a)
        E.gemm_a8_block(*lists, a["status"])
        assert reach == ["eq_gemm_a8"] * 2
        return
    with pytest.raises(ValueError):
        E.gemm_a8(**a)
    with pytest.raises(ValueError):
        E.gemm_a8_block(*lists, a["status"])
    assert not reach


@pytest.mark.parametrize("status", [torch.zeros(0, dtype=torch.int32), torch.zeros(1, dtype=torch.int8),
                                    torch.zeros(1, dtype=torch.int64), torch.zeros(1), torch.zeros(2, dtype=torch.int16)])
def test_status_is_a_word(reach, status):
    """On an error the kernels OR four bytes into it."""
    a = {**_a8(torch.uint8, torch.int8), "status": status}
    lists = [[a[k]] for k in ("sym", "scale", "x8", "x_scale", "y")]

    class Info:
        rows, cols, dtype = 8, 32, E.EQ_INT8

    class Fake:
        _L, _m, d_blob = E.load(), None, None

        def info(self, matrix):
            return Info

        def layer_matrices(self, layer):
            return [0]

    m = [[a[k]] for k in ("sym", "x8", "x_scale", "y")]
    for call in (lambda st: E.gemm_a8(**{**a, "status": st}), lambda st: E.gemm_a8_block(*lists, st),
                 lambda st: E.Model.gemm_symbols_a8(Fake(), 0, *(v[0] for v in m), st),
                 lambda st: E.Model.gemm_symbols_a8_block(Fake(), 0, *m, st)):
        n = len(reach)
        with pytest.raises(ValueError):
            call(status)
        assert len(reach) == n
        call(torch.zeros(1, dtype=torch.int32))
        assert len(reach) == n + 1


BIG = 2 ** 32 + 1


def test_sizes_beyond_32_bits(reach):
    """2^32 + 1 tokens would arrive as one (every tensor here is empty or one row seen many times)."""
    none = torch.empty(0, 0, dtype=torch.uint8)
    meta = {k: torch.empty(BIG, device="meta") for k in ("x_scale", "out_scale")}
    a8 = dict(sym=none, scale=torch.empty(0), x8=torch.empty(BIG, 0, dtype=torch.int8), x_scale=meta["x_scale"],
              y=torch.empty(BIG, 0), status=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        E.gemm_a8(**a8)
    with pytest.raises(ValueError):
        E.gemm_a8_block(*([a8[k]] for k in ("sym", "scale", "x8", "x_scale", "y")), a8["status"])
    q, s = torch.empty(0, 16, dtype=torch.uint8), torch.empty(0, 1)
    x = torch.zeros(1, 32, dtype=torch.bfloat16).expand(BIG, 32)
    y = torch.empty(BIG, 0)
    with pytest.raises(ValueError):
        E.gemv_w4(q, s, x, y, group=32)
    with pytest.raises(ValueError):
        E.gemv_w4_block([q], [s], [x], [y], group=32)
    with pytest.raises(ValueError):
        E.rmsnorm(torch.empty(BIG, 0), torch.empty(BIG, 0, dtype=torch.int8), out_scale=meta["out_scale"])
    with pytest.raises(ValueError):
        E.rmsnorm(torch.empty(0, BIG), torch.empty(0, BIG, dtype=torch.bfloat16))
    assert not reach


def test_the_model_is_on_the_current_device(monkeypatch):
    """The kernels read scales and super weights from the model's own bytes: a model on another device than the
    current one is refused like any other tensor there."""
    class On:
        """A tensor on device `dev`, as far as the check of devices looks."""
        def __init__(self, t, dev):
            self.t, self.dev, self.device = t, dev, f"cuda:{dev}"

        def get_device(self):
            return self.dev

        def __getattr__(self, name):
            return getattr(self.t, name)

    class Info:
        rows, cols, dtype = 8, 32, E.EQ_INT8

    class Fake:
        _m = None

        def __init__(self, dev):
            self.d_blob, self.called = On(torch.zeros(1), dev), []
            self._L = self

        def info(self, matrix):
            return Info

        def layer_matrices(self, layer):
            return [0]

        def eq_gemm_symbols_a8(self, *a):
            return self.called.append(1) or 0

        eq_gemm_symbols_a8_block = eq_gemm_symbols_a8

    E._type(torch.zeros(1))  # sets the dtype table up before the device query is replaced
    monkeypatch.setattr(E, "_device", lambda: 1)
    monkeypatch.setattr(E, "_raw_stream", lambda dev: 0)
    a = {k: On(v, 1) for k, v in _a8(torch.uint8, torch.int8).items()}
    m = [a[k] for k in ("sym", "x8", "x_scale", "y")]
    for call in (lambda f: E.Model.gemm_symbols_a8(f, 0, *m, a["status"]),
                 lambda f: E.Model.gemm_symbols_a8_block(f, 0, *([v] for v in m), a["status"])):
        f = Fake(1)
        call(f)
        assert f.called
        f = Fake(0)
        with pytest.raises(ValueError):
            call(f)
        assert not f.called
