"""entropy_coded_weight_b200 -- B200 decoder for entropy-coded LLM weights.

Thin Python layer over libeqw.so (C ABI in include/eqw.h).  Every function
marshals arguments and calls the C entry point of the same name; all decoding
runs in the library's CUDA kernels.  PyTorch provides device memory, streams
and events.

Typical use (EntQuant technical summary, gist.science 2601.22787, section 2:
weights stored as a compressed bitstream in GPU memory and expanded block by
block just before each block's forward pass)::

    blob = encode_host(matrices)                 # host, threads over chunks
    d_blob = upload(blob)                        # one copy into HBM
    model = Model(d_blob, blob)                  # parse + validate
    out = torch.empty(model.block_bytes(layer), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    model.decode_block(layer, out, status)       # rANS decode + dequant + scatter
"""
from __future__ import annotations

import ctypes

import numpy as np

from . import _lib
from ._lib import (EQ_BF16, EQ_DEV_BAD_END, EQ_DEV_BAD_HEADER, EQ_DEV_BAD_OUTLIER, EQ_DEV_BAD_STATE,
                   EQ_DEV_BAD_TABLE, EQ_CODEC_HUFFMAN, EQ_DEV_TIMEOUT, EQ_E4M3, EQ_F16, EQ_F32, EQ_INT8,
                   EQ_TABLE_PER_CHUNK, PACK_A8, PACK_RMSNORM, PACK_W4, EqError, check, eq_matrix_in, eq_matrix_info,
                   load)

__all__ = [
    "EQ_INT8", "EQ_E4M3", "EqError", "Model", "encode_host", "upload", "gemv_bf16", "eq_status_string",
    "eq_format_version", "EQ_DEV_BAD_HEADER", "EQ_DEV_BAD_TABLE", "EQ_DEV_BAD_STATE", "EQ_DEV_BAD_END",
    "EQ_DEV_TIMEOUT", "EQ_DEV_BAD_OUTLIER", "EQ_BF16", "EQ_F32", "EQ_F16", "rmsnorm", "gemm_a8",
    "gemm_a8_block", "gemv_w4", "gemv_w4_block",
]


def _ptr(a) -> int | None:
    if a is None:
        return None
    if isinstance(a, np.ndarray):
        return a.ctypes.data
    return a.data_ptr()


def _stream_handle(stream) -> int | None:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def eq_status_string(code: int) -> str:
    return load().eq_status_string(code).decode()


def eq_format_version() -> int:
    return load().eq_format_version()


def _matrix_in_array(matrices, table_scope: str = "matrix", codec: str = "rans"):
    """eq_matrix_in[] for objects with layer, dtype, symbols, scales, out_row/out_col/out_val."""
    keep = []
    arr = (eq_matrix_in * max(1, len(matrices)))()
    for i, m in enumerate(matrices):
        sym = np.ascontiguousarray(m.symbols, dtype=np.uint8)
        if sym.ndim != 2:
            raise ValueError("symbols must be [rows, cols]")
        sc = np.ascontiguousarray(m.scales, dtype=np.float32)
        orow = np.ascontiguousarray(getattr(m, "out_row", np.zeros(0)), dtype=np.uint32)
        ocol = np.ascontiguousarray(getattr(m, "out_col", np.zeros(0)), dtype=np.uint32)
        oval = np.ascontiguousarray(getattr(m, "out_val", np.zeros(0)), dtype=np.float32)
        keep += [sym, sc, orow, ocol, oval]
        e = arr[i]
        e.layer = int(m.layer)
        e.dtype = int(m.dtype)
        e.rows, e.cols = sym.shape
        e.symbols = sym.ctypes.data if sym.size else None
        e.scales = sc.ctypes.data if sc.size else None
        e.n_out = orow.size
        e.out_row = orow.ctypes.data if orow.size else None
        e.out_col = ocol.ctypes.data if ocol.size else None
        e.out_val = oval.ctypes.data if oval.size else None
        e.flags = _flags(m, table_scope, codec)
    return arr, keep


def _flags(m, table_scope: str, codec: str) -> int:
    if table_scope not in ("matrix", "chunk") or codec not in ("rans", "huffman"):
        raise ValueError("table_scope must be 'matrix' or 'chunk', codec 'rans' or 'huffman'")
    return (int(getattr(m, "flags", 0)) | (EQ_TABLE_PER_CHUNK if table_scope == "chunk" else 0)
            | (EQ_CODEC_HUFFMAN if getattr(m, "codec", codec) == "huffman" else 0))


def encode_host(matrices, n_threads: int = 0, table_scope: str = "matrix", codec: str = "rans") -> np.ndarray:
    """Encode matrices into a container v1 blob (uint8 numpy array) with eq_encoder_run.

    ``table_scope``: "matrix" (one table from the whole matrix's histogram,
    written into every chunk) or "chunk" (each chunk's own histogram).
    ``codec``: "rans" (12-bit rANS) or "huffman" (canonical Huffman codes of
    at most 12 bits); a matrix's own ``codec`` attribute wins.
    """
    L = load()
    arr, keep = _matrix_in_array(matrices, table_scope, codec)
    h = ctypes.c_void_p()
    size = ctypes.c_size_t()
    check(L.eq_encoder_run(arr, len(matrices), n_threads, ctypes.byref(h), ctypes.byref(size)), "eq_encoder_run")
    try:
        out = np.empty(size.value, np.uint8)
        check(L.eq_encoded_write(h, out.ctypes.data, out.size), "eq_encoded_write")
    finally:
        L.eq_encoded_free(h)
    del keep
    return out


def _device_matrix_in_array(matrices, table_scope: str, codec: str = "rans"):
    """eq_matrix_in[] whose pointers are device addresses (CUDA tensors on one device)."""
    import torch
    keep = []
    arr = (eq_matrix_in * max(1, len(matrices)))()
    for i, m in enumerate(matrices):
        sym = m.symbols
        if not (isinstance(sym, torch.Tensor) and sym.is_cuda and sym.dtype == torch.uint8 and sym.dim() == 2):
            raise ValueError("symbols must be a uint8 CUDA tensor [rows, cols]")
        sym = sym.contiguous()
        sc = m.scales.to(torch.float32).contiguous()
        n_out = 0 if getattr(m, "out_row", None) is None else int(m.out_row.numel())
        orow = ocol = oval = None
        if n_out:
            orow = m.out_row.to(torch.int32).contiguous()  # the library reads them as uint32
            ocol = m.out_col.to(torch.int32).contiguous()
            oval = m.out_val.to(torch.float32).contiguous()
        keep += [sym, sc, orow, ocol, oval]
        e = arr[i]
        e.layer = int(m.layer)
        e.dtype = int(m.dtype)
        e.rows, e.cols = sym.shape
        e.symbols = sym.data_ptr() if sym.numel() else None
        e.scales = sc.data_ptr() if sc.numel() else None
        e.n_out = n_out
        e.out_row = orow.data_ptr() if n_out else None
        e.out_col = ocol.data_ptr() if n_out else None
        e.out_val = oval.data_ptr() if n_out else None
        e.flags = _flags(m, table_scope, codec)
    return arr, keep


def encode_device(matrices, table_scope: str = "matrix", stream=None, codec: str = "rans"):
    """eq_encode_device: encode matrices whose symbols, scales and super weights
    are CUDA tensors; returns the container as a uint8 CUDA tensor (the same
    bytes eq_encode_host writes).  Each matrix needs ``layer``, ``dtype``,
    ``symbols`` (uint8 [rows, cols]), ``scales`` (float32 [rows]) and optionally
    ``out_row``, ``out_col`` (integer), ``out_val`` (float32).  ``table_scope``
    and ``codec`` as for encode_host.  Synchronises the stream."""
    import torch
    arr, keep = _device_matrix_in_array(matrices, table_scope, codec)
    n = len(matrices)
    L = load()
    wb, ob, ln = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    check(L.eq_encode_device_workspace(arr, n, ctypes.byref(wb)), "eq_encode_device_workspace")
    check(L.eq_encode_bound(arr, n, ctypes.byref(ob)), "eq_encode_bound")
    dev = keep[0].device if keep else torch.device("cuda")
    work = torch.empty(max(1, wb.value), dtype=torch.uint8, device=dev)
    out = torch.empty(max(1, ob.value), dtype=torch.uint8, device=dev)
    check(L.eq_encode_device(arr, n, out.data_ptr(), ob.value, ctypes.byref(ln), work.data_ptr(), wb.value,
                             _stream_handle(stream)), "eq_encode_device")
    return out[:ln.value]


def upload(blob: np.ndarray, device=None):
    """Copy a host container into a fresh device tensor (uint8; the allocator aligns it to >= 256 B)."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(blob, dtype=np.uint8))
    return t.to(device or "cuda", non_blocking=False)


class Model:
    """A container resident in device memory (eq_model_open / eq_model_close)."""

    def __init__(self, d_blob, h_blob):
        self._L = load()
        self.d_blob = d_blob  # keep the device bytes alive
        self._h = np.ascontiguousarray(h_blob, dtype=np.uint8)
        if d_blob.numel() != self._h.size:
            raise ValueError("device and host copies differ in length")
        handle = ctypes.c_void_p()
        check(self._L.eq_model_open(d_blob.data_ptr(), self._h.size, self._h.ctypes.data, ctypes.byref(handle)),
              "eq_model_open")
        self._m = handle
        nl, nm = ctypes.c_uint32(), ctypes.c_uint32()
        check(self._L.eq_model_counts(self._m, ctypes.byref(nl), ctypes.byref(nm)), "eq_model_counts")
        self.n_layers, self.n_matrices = nl.value, nm.value
        self._h = None  # only needed while opening

    def close(self) -> None:
        if getattr(self, "_m", None):
            self._L.eq_model_close(self._m)
            self._m = None

    def set_sm_limit(self, max_sms: int) -> None:
        """eq_model_set_sm_limit: decode launches of this model use at most
        ``max_sms`` SMs (0: all), leaving the rest to a kernel that runs beside
        them, e.g. the consumer of the previous block."""
        check(self._L.eq_model_set_sm_limit(self._m, int(max_sms)), "eq_model_set_sm_limit")

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self) -> int:
        return self._m.value

    def info(self, matrix: int) -> eq_matrix_info:
        inf = eq_matrix_info()
        check(self._L.eq_matrix_get_info(self._m, matrix, ctypes.byref(inf)), "eq_matrix_get_info")
        return inf

    def layer_matrices(self, layer: int) -> range:
        f, c = ctypes.c_uint32(), ctypes.c_uint32()
        check(self._L.eq_layer_matrices(self._m, layer, ctypes.byref(f), ctypes.byref(c)), "eq_layer_matrices")
        return range(f.value, f.value + c.value)

    def block_layout(self, layer: int) -> tuple[list[int], int]:
        n = len(self.layer_matrices(layer))
        offs = (ctypes.c_size_t * max(1, n))()
        total = ctypes.c_size_t()
        check(self._L.eq_block_layout(self._m, layer, offs, n, ctypes.byref(total)), "eq_block_layout")
        return [offs[i] for i in range(n)], total.value

    def block_bytes(self, layer: int) -> int:
        return self.block_layout(layer)[1]

    def decode_plan(self, layer: int, sms: int) -> list[int]:
        """eq_decode_plan: per matrix of ``layer``, the leading chunks the
        two-chunks-per-warp kernel decodes on a GPU with ``sms`` SMs."""
        n = len(self.layer_matrices(layer))
        out = (ctypes.c_uint32 * max(1, n))()
        check(self._L.eq_decode_plan(self._m, layer, sms, out, n), "eq_decode_plan")
        return [out[i] for i in range(n)]

    def decode_matrix(self, matrix: int, out, status, stream=None) -> None:
        """eq_decode_matrix into ``out`` (device tensor, >= 2*rows*cols bytes)."""
        nbytes = out.numel() * out.element_size()
        check(self._L.eq_decode_matrix(self._m, matrix, out.data_ptr(), nbytes, status.data_ptr(),
                                       _stream_handle(stream)), "eq_decode_matrix")

    def decode_block(self, layer: int, out, status, stream=None) -> None:
        """eq_decode_block into ``out`` (device tensor, >= block_bytes(layer) bytes)."""
        nbytes = out.numel() * out.element_size()
        check(self._L.eq_decode_block(self._m, layer, out.data_ptr(), nbytes, status.data_ptr(),
                                      _stream_handle(stream)), "eq_decode_block")

    def decode_model_stream(self, layer: int, bufs, status, decode_stream, ev_free, ev_ready) -> None:
        """eq_decode_model_stream: wait ev_free[b], decode into bufs[b], record ev_ready[b] (b = layer & 1)."""
        nbytes = min(b.numel() * b.element_size() for b in bufs)
        pbuf = (ctypes.c_void_p * 2)(bufs[0].data_ptr(), bufs[1].data_ptr())
        pfree = (ctypes.c_void_p * 2)(*(e.cuda_event if e is not None else None for e in ev_free))
        pready = (ctypes.c_void_p * 2)(*(e.cuda_event for e in ev_ready))
        check(self._L.eq_decode_model_stream(self._m, layer, pbuf, nbytes, status.data_ptr(),
                                             _stream_handle(decode_stream), pfree, pready),
              "eq_decode_model_stream")

    def decode_symbols(self, matrix: int, out, status, stream=None) -> None:
        """eq_decode_symbols: the matrix's raw symbol bytes into ``out`` (uint8 CUDA tensor, >= rows*cols)."""
        nbytes = out.numel() * out.element_size()
        check(self._L.eq_decode_symbols(self._m, matrix, out.data_ptr(), nbytes, status.data_ptr(),
                                        _stream_handle(stream)), "eq_decode_symbols")

    def decode_symbols_block(self, layer: int, outs, status, stream=None) -> None:
        """eq_decode_symbols_block: raw symbol bytes of every matrix of ``layer`` into ``outs[i]``."""
        n = len(outs)
        po = (ctypes.c_void_p * max(1, n))(*(o.data_ptr() for o in outs))
        check(self._L.eq_decode_symbols_block(self._m, layer, po, n, status.data_ptr(), _stream_handle(stream)),
              "eq_decode_symbols_block")

    def gemm_symbols(self, matrix: int, sym, x, y, status, stream=None) -> None:
        """eq_gemm_symbols: y[t, r] = scale[r] * sum_c x[t, c] * value(sym[r, c]) (+ super weights), on the
        tensor cores; x bf16 [tokens, cols], y fp32 [tokens, rows] (CUDA tensors)."""
        check(self._L.eq_gemm_symbols(self._m, matrix, sym.data_ptr(), x.data_ptr(), x.shape[0], y.data_ptr(),
                                      status.data_ptr(), _stream_handle(stream)), "eq_gemm_symbols")

    def gemm_symbols_block(self, layer: int, syms, xs, ys, status, stream=None) -> None:
        """eq_gemm_symbols_block: ``gemm_symbols`` for every matrix of ``layer`` (``syms[i]``, ``xs[i]``,
        ``ys[i]`` belong to matrix i of the layer), one persistent tensor-core launch per weight type."""
        n = len(syms)
        if len(xs) != n or len(ys) != n:
            raise ValueError("syms, xs and ys must have one entry per matrix of the layer")
        tokens = xs[0].shape[0] if n else 0
        if any(x.shape[0] != tokens for x in xs):
            raise ValueError("every input of a block GEMM takes the same number of tokens")
        ps = (ctypes.c_void_p * max(1, n))(*(t.data_ptr() for t in syms))
        px = (ctypes.c_void_p * max(1, n))(*(t.data_ptr() for t in xs))
        py = (ctypes.c_void_p * max(1, n))(*(t.data_ptr() for t in ys))
        check(self._L.eq_gemm_symbols_block(self._m, layer, ps, px, tokens, py, n, status.data_ptr(),
                                            _stream_handle(stream)), "eq_gemm_symbols_block")

    def gemm_symbols_a8(self, matrix: int, sym, x8, x_scale, y, status, stream=None) -> None:
        """eq_gemm_symbols_a8: y[t, r] = scale[r] * x_scale[t] * sum_c x8[t, c] * value(sym[r, c]) (+ super
        weights) on the 8-bit tensor cores; x8 int8 or float8_e4m3fn [tokens, cols] like the matrix, x_scale
        fp32 [tokens], y fp32 [tokens, rows]."""
        info = self.info(matrix)
        tokens = _check_a8(info.rows, info.cols, info.dtype, sym, x8, x_scale, y)
        _check_status(status)
        st = _launch_stream(stream, sym, x8, x_scale, y, status, self.d_blob)
        check(self._L.eq_gemm_symbols_a8(self._m, matrix, sym.data_ptr(), x8.data_ptr(), x_scale.data_ptr(),
                                         tokens, y.data_ptr(), status.data_ptr(), st), "eq_gemm_symbols_a8")

    def gemm_symbols_a8_block(self, layer: int, syms, x8s, x_scales, ys, status, stream=None) -> None:
        """eq_gemm_symbols_a8_block: ``gemm_symbols_a8`` for every matrix of ``layer`` in directory order, one
        launch per weight type (of up to 8 matrices)."""
        mats = self.layer_matrices(layer)
        n = len(mats)
        if not len(syms) == len(x8s) == len(x_scales) == len(ys) == n:
            raise ValueError("syms, x8s, x_scales and ys must have one entry per matrix of the layer")
        tokens = x8s[0].shape[0] if n else 0
        for i, mi in enumerate(mats):
            info = self.info(mi)
            if x8s[i].shape[0] != tokens:
                raise ValueError("every input of a block GEMM takes the same number of tokens")
            _check_a8(info.rows, info.cols, info.dtype, syms[i], x8s[i], x_scales[i], ys[i])
        _check_status(status)
        st = _launch_stream(stream, status, self.d_blob, *syms, *x8s, *x_scales, *ys)

        def ptrs(ts):
            return (ctypes.c_void_p * max(1, n))(*(t.data_ptr() for t in ts))

        check(self._L.eq_gemm_symbols_a8_block(self._m, layer, ptrs(syms), ptrs(x8s), ptrs(x_scales), tokens,
                                               ptrs(ys), n, status.data_ptr(), st), "eq_gemm_symbols_a8_block")

    def decode_gemv_matrix(self, matrix: int, x, y, status, stream=None) -> None:
        """eq_decode_gemv_matrix: y = W x without materialising W (x bf16 [cols], y fp32 [rows], device)."""
        check(self._L.eq_decode_gemv_matrix(self._m, matrix, x.data_ptr(), y.data_ptr(), status.data_ptr(),
                                            _stream_handle(stream)), "eq_decode_gemv_matrix")

    def decode_gemv_block(self, layer: int, xs, ys, status, stream=None) -> None:
        """eq_decode_gemv_block: ys[i] = W_i xs[i] for matrix i of ``layer`` (directory order)."""
        n = len(xs)
        px = (ctypes.c_void_p * max(1, n))(*(x.data_ptr() for x in xs))
        py = (ctypes.c_void_p * max(1, n))(*(y.data_ptr() for y in ys))
        check(self._L.eq_decode_gemv_block(self._m, layer, px, py, n, status.data_ptr(), _stream_handle(stream)),
              "eq_decode_gemv_block")


def gemv_bf16(w, x, y, stream=None) -> None:
    """eq_gemv_bf16: y[r] = sum_c w[r, c] * x[c] (w bf16 [rows, cols], x bf16 [cols], y fp32 [rows])."""
    rows, cols = w.shape
    check(load().eq_gemv_bf16(w.data_ptr(), x.data_ptr(), y.data_ptr(), rows, cols, _stream_handle(stream)),
          "eq_gemv_bf16")


# ---- activation and 4-bit operators ------------------------------------------------------
# These run once per layer and decoded token, so their checks are written for few Python steps.
_TYPES: dict = {}  # torch dtype -> EQ_* element type
_device = _raw_stream = _bytes = None


def _setup() -> None:
    global _device, _raw_stream, _bytes
    import torch
    _bytes = torch.uint8
    _TYPES.update({torch.bfloat16: EQ_BF16, torch.float32: EQ_F32, torch.float16: EQ_F16, torch.int8: EQ_INT8,
                   torch.float8_e4m3fn: EQ_E4M3})
    _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _type(t) -> int:
    """EQ_* element type of a tensor (0, which every entry point refuses, for any other dtype)."""
    if _device is None:
        _setup()
    return _TYPES.get(t.dtype, 0)


def _launch_stream(stream, *tensors) -> int:
    """The stream handle to launch on, once every tensor is known to be on the current CUDA device."""
    if tensors[0].get_device() < 0:
        raise ValueError("every tensor must be on the GPU")
    dev = _device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensor on {t.device}, but the current CUDA device is cuda:{dev}")
    if stream is None:
        return _raw_stream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_MAX_U32 = 0xFFFFFFFF  # what the library takes sizes in; ctypes would cut a larger one without a word


def _rows(t, what: str, shape) -> int:
    """Row stride in elements of a [tokens, cols] tensor whose columns are adjacent."""
    if t.shape == shape:
        if t.is_contiguous():
            return shape[1]
        st = t.stride()
        if st[1] == 1 or shape[1] <= 1 or not shape[0]:
            return st[0] if shape[0] > 1 else shape[1]
    raise ValueError(f"{what} must be {tuple(shape)} with adjacent columns")


def rmsnorm(x, out, gamma=None, eps: float = 1e-6, residual=None, residual_out=None, out_scale=None,
            stream=None) -> None:
    """eq_rmsnorm: h = x + residual, residual_out = h, out = h / sqrt(mean h^2 + eps) * gamma, row by row.

    x and residual [tokens, cols] are bf16 or fp32, gamma bf16 [cols].  The
    dtype of ``out`` picks the output: bf16, or int8 / float8_e4m3fn codes
    with one fp32 scale per token in ``out_scale`` [tokens].  ``residual_out``
    defaults to ``residual`` itself (updated in place).  Rows may be strided.
    """
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must be [tokens, cols]")
    tokens, cols = shape
    if tokens > _MAX_U32 or cols > _MAX_U32:
        raise ValueError("x has more than 2^32 - 1 tokens or columns")
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs residual")
        rs = ros = rt = rp = rop = 0
    else:
        rs, rt, rp = _rows(residual, "residual", shape), _type(residual), residual.data_ptr()
        if residual_out is None:
            ros, rop = rs, rp
        else:
            ros, rop = _rows(residual_out, "residual_out", shape), residual_out.data_ptr()
            if residual_out.dtype != residual.dtype:
                raise ValueError("residual_out must have residual's dtype")
    gp = 0
    if gamma is not None:
        if _type(gamma) != EQ_BF16 or gamma.shape != (cols,) or not gamma.is_contiguous():
            raise ValueError("gamma must be bf16 [cols], contiguous")
        gp = gamma.data_ptr()
    xs, os, ot, sp = _rows(x, "x", shape), _rows(out, "out", shape), _type(out), 0
    if ot != EQ_BF16:
        if out_scale is None or _type(out_scale) != EQ_F32 or out_scale.numel() != tokens or \
                not out_scale.is_contiguous():
            raise ValueError("8-bit outputs need out_scale, fp32 [tokens], contiguous")
        sp = out_scale.data_ptr()
    st = _launch_stream(stream, x, out, gamma, residual, residual_out, out_scale)
    check(load().eq_rmsnorm(PACK_RMSNORM.pack(x.data_ptr(), rp, rop, gp, out.data_ptr(), sp, xs, rs, ros, os, tokens,
                                              cols, _type(x), rt, ot, eps), st), "eq_rmsnorm")


def _check_status(status) -> None:
    if status.element_size() != 4 or status.is_floating_point() or not status.numel():
        raise ValueError("status must be an int32 tensor of at least one element")


def _check_a8(rows: int, cols: int, dtype: int, sym, x8, x_scale, y) -> int:
    """Shapes and types of an 8-bit product's tensors; the number of tokens."""
    shape = x8.shape
    if len(shape) != 2 or shape[1] != cols or not x8.is_contiguous() or _type(x8) != dtype:
        raise ValueError("x8 must be [tokens, cols], contiguous, int8 or float8_e4m3fn like the symbols")
    tokens = shape[0]
    if tokens > _MAX_U32 or rows > _MAX_U32 or cols > _MAX_U32:
        raise ValueError("more than 2^32 - 1 tokens, rows or columns")
    if sym.element_size() != 1 or sym.numel() < rows * cols or not sym.is_contiguous():
        raise ValueError("sym must hold rows * cols bytes, contiguous")
    if _type(x_scale) != EQ_F32 or x_scale.numel() != tokens or not x_scale.is_contiguous():
        raise ValueError("x_scale must be fp32 [tokens], contiguous")
    if _type(y) != EQ_F32 or y.numel() != tokens * rows or not y.is_contiguous():
        raise ValueError("y must be fp32 [tokens, rows], contiguous")
    return tokens


def _a8_job(sym, scale, x8, x_scale, y, outliers) -> bytes:
    if sym.dim() != 2:
        raise ValueError("sym must be [rows, cols]")
    rows, cols = sym.shape
    dtype = _type(x8)
    _check_a8(rows, cols, dtype, sym, x8, x_scale, y)
    if sym.dtype != x8.dtype and sym.dtype != _bytes:
        raise ValueError("sym must be uint8 (the decoder's bytes) or of x8's dtype")
    if _type(scale) != EQ_F32 or scale.numel() != rows or not scale.is_contiguous():
        raise ValueError("scale must be fp32 [rows], contiguous")
    rp = cp = vp = n_out = 0
    if outliers is not None and outliers[0].numel():
        r, c, v = outliers
        if r.element_size() != 4 or c.element_size() != 4 or _type(v) != EQ_F32 or r.is_floating_point() or \
                c.is_floating_point() or not r.numel() == c.numel() == v.numel() or \
                not (r.is_contiguous() and c.is_contiguous() and v.is_contiguous()):
            raise ValueError("outliers are (row int32, col int32, value fp32), contiguous, of one length")
        _launch_stream(0, r, c, v)
        rp, cp, vp, n_out = r.data_ptr(), c.data_ptr(), v.data_ptr(), r.numel()
    return PACK_A8.pack(sym.data_ptr(), scale.data_ptr(), x8.data_ptr(), x_scale.data_ptr(), y.data_ptr(), rp, cp, vp,
                        rows, cols, dtype, n_out, 1)


def gemm_a8(sym, scale, x8, x_scale, y, status, outliers=None, stream=None) -> None:
    """eq_gemm_a8 for one matrix given by its decoded symbols: y[t, r] = scale[r] * x_scale[t] * sum_c x8[t, c] *
    sym[r, c] (+ super weights).

    ``sym`` [rows, cols] holds Int8 or E4M3 symbols, as bytes (uint8, ``Model.decode_symbols``) or typed like
    ``x8`` [tokens, cols], whose dtype, int8 or float8_e4m3fn, is taken for both (``rmsnorm``); ``scale`` fp32
    [rows], ``x_scale`` fp32 [tokens], ``y`` fp32 [tokens, rows].  ``outliers``: (row, col, value) tensors (int32, int32, fp32) sorted by row.
    """
    job = _a8_job(sym, scale, x8, x_scale, y, outliers)
    _check_status(status)
    st = _launch_stream(stream, sym, scale, x8, x_scale, y, status)
    check(load().eq_gemm_a8(job, 1, x8.shape[0], status.data_ptr(), st), "eq_gemm_a8")


def gemm_a8_block(syms, scales, x8s, x_scales, ys, status, outliers=None, stream=None) -> None:
    """eq_gemm_a8 for several matrices in one launch per type (of up to 8): ``gemm_a8`` on the i-th entry of every
    list.  All take the same number of tokens and may share inputs."""
    n = len(syms)
    if not len(scales) == len(x8s) == len(x_scales) == len(ys) == n or (outliers is not None and len(outliers) != n):
        raise ValueError("every list must have one entry per matrix")
    if not n:
        return
    tokens = x8s[0].shape[0]
    if any(x.shape[0] != tokens for x in x8s):
        raise ValueError("every input of a block GEMM takes the same number of tokens")
    jobs = b"".join(_a8_job(syms[i], scales[i], x8s[i], x_scales[i], ys[i], None if outliers is None else outliers[i])
                    for i in range(n))
    _check_status(status)
    st = _launch_stream(stream, status, *syms, *scales, *x8s, *x_scales, *ys)
    check(load().eq_gemm_a8(jobs, n, tokens, status.data_ptr(), st), "eq_gemm_a8")


_NO_TABLE = bytes(32)


def _w4_job(q, scales, x, y, group: int, zeros, table) -> bytes:
    qs = q.shape
    if len(qs) != 2 or q.element_size() != 1 or q.is_floating_point() or not q.is_contiguous():
        raise ValueError("q must be uint8 [rows, cols / 2], contiguous")
    rows, cols = qs[0], 2 * qs[1]
    if x.dim() != 2 or _type(x) != EQ_BF16:
        raise ValueError("x must be bf16 [tokens, cols]")
    if x.shape[0] > _MAX_U32 or rows > _MAX_U32 or cols > _MAX_U32:
        raise ValueError("more than 2^32 - 1 tokens, rows or columns")
    xs = _rows(x, "x", (x.shape[0], cols))
    n = rows * -(-cols // group) if group > 0 else -1
    if scales.numel() != n or not scales.is_contiguous():
        raise ValueError("scales must be [rows, ceil(cols / group)], contiguous")
    zp = 0
    if zeros is not None:
        if zeros.element_size() != 1 or zeros.is_floating_point() or zeros.numel() != n or not zeros.is_contiguous():
            raise ValueError("zeros must be uint8 [rows, ceil(cols / group)], contiguous")
        zp = zeros.data_ptr()
    if _type(y) != EQ_F32 or y.numel() != x.shape[0] * rows or not y.is_contiguous():
        raise ValueError("y must be fp32 [tokens, rows], contiguous")
    values = _NO_TABLE
    if table is not None:
        if table.is_cuda or table.numel() != 16 or _type(table) != EQ_BF16 or not table.is_contiguous():
            raise ValueError("table must be a CPU tensor of 16 bf16 values")
        values = ctypes.string_at(table.data_ptr(), 32)
    return PACK_W4.pack(q.data_ptr(), scales.data_ptr(), zp, x.data_ptr(), y.data_ptr(), xs, rows, cols, group,
                        _type(scales), table is not None, values)


def gemv_w4(q, scales, x, y, group: int = 128, zeros=None, table=None, stream=None) -> None:
    """eq_gemv_w4: y[t, r] = sum_g scales[r, g] * sum_{c in g} w(q[r, c]) * x[t, c] for 1 to 32 tokens.

    ``q`` uint8 [rows, cols / 2] holds two 4-bit codes per byte (the even column in the low half), ``scales``
    [rows, ceil(cols / group)] fp32, bf16 or fp16, ``x`` bf16 [tokens, cols] (rows may be strided), ``y`` fp32
    [tokens, rows].  A code q stands for q - 8, for q - zeros[r, g] (``zeros`` uint8, like ``scales``, 0 to
    127: a byte above makes its row's outputs NaN), or for ``table[q]`` (a CPU tensor of 16 bf16 values, read during
    the call).
    """
    job = _w4_job(q, scales, x, y, group, zeros, table)
    st = _launch_stream(stream, q, scales, x, y, zeros)
    check(load().eq_gemv_w4(job, 1, x.shape[0], st), "eq_gemv_w4")


def gemv_w4_block(qs, scales, xs, ys, group: int = 128, zeros=None, table=None, stream=None) -> None:
    """eq_gemv_w4 for several matrices of one group size: ``gemv_w4`` on the i-th entry of every list (``zeros`` a
    list or None), in one launch per code form (of up to 8).  All take the same tokens and may share inputs."""
    n = len(qs)
    if not len(scales) == len(xs) == len(ys) == n or (zeros is not None and len(zeros) != n):
        raise ValueError("every list must have one entry per matrix")
    if not n:
        return
    tokens = xs[0].shape[0]
    if any(x.shape[0] != tokens for x in xs):
        raise ValueError("every input of a block product takes the same number of tokens")
    jobs = b"".join(_w4_job(qs[i], scales[i], xs[i], ys[i], group, None if zeros is None else zeros[i], table)
                    for i in range(n))
    st = _launch_stream(stream, *qs, *scales, *xs, *ys, *(zeros or ()))
    check(load().eq_gemv_w4(jobs, n, tokens, st), "eq_gemv_w4")


def selftest_wait_timeout(status, stream=None) -> None:
    """eq_selftest_wait_timeout: make one bounded staging wait run out (about a
    second); the kernel ORs EQ_DEV_TIMEOUT into ``status`` (device int32)."""
    check(load().eq_selftest_wait_timeout(status.data_ptr(), _stream_handle(stream)), "eq_selftest_wait_timeout")


def selftest_gemm_wait_timeout(status, stream=None) -> None:
    """eq_selftest_gemm_wait_timeout: the prefill GEMM's MMA lane waits on a
    "full" barrier nothing arrives on until its bounded wait runs out (about a
    second); the block ORs EQ_DEV_TIMEOUT into ``status`` and frees its TMEM."""
    check(load().eq_selftest_gemm_wait_timeout(status.data_ptr(), _stream_handle(stream)),
          "eq_selftest_gemm_wait_timeout")


def selftest_a8_wait_timeout(status, stream=None) -> None:
    """eq_selftest_a8_wait_timeout: one epilogue warp of the 8-bit GEMM's pair kernel gives up (about a second) while
    the other seven wait for it; the block ORs EQ_DEV_TIMEOUT into ``status``, frees its TMEM and ends."""
    check(load().eq_selftest_a8_wait_timeout(status.data_ptr(), _stream_handle(stream)), "eq_selftest_a8_wait_timeout")
