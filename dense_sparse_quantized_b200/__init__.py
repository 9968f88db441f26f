"""Python binding of libdsq (the dense-and-sparse quantized GEMV for B200).

Argument marshalling only: every step of the product runs in the library's
CUDA kernels.  PyTorch supplies device memory and streams.  The binding
refuses to work without the compiled library (``python -m
dense_sparse_quantized_b200.build``); there is no fallback path.

    blob = pack(rows, cols, bits, mode, codes, table, zeros, row_ptr, col_idx, values)
    h = Handle(blob, device=0)
    y = h.gemv(x)              # x: cuda fp16 [batch, cols] -> y: cuda fp16 [batch, rows]
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(HERE, "libdsq.so")

DSQ_OK = 0
DSQ_ERR_INVALID_ARG = -1
DSQ_ERR_UNSUPPORTED = -2
DSQ_ERR_CUDA = -3
DSQ_ERR_OOM = -4
DSQ_ERR_BUFFER_TOO_SMALL = -5
DSQ_ERR_DEVICE = -6
DSQ_ERR_SCRATCH_LIMIT = -7
MODE_LUT_ROW = 0
MODE_AFFINE_G16 = 1
MODE_BITPLANE = 2
MODE_INTGRID = 3
DTYPE_F16 = 0
DTYPE_BF16 = 1
DTYPE_F32 = 2

EXPORTS = ("dsq_pack", "dsq_pack_two_axis", "dsq_pack_intgrid", "dsq_blob_desc", "dsq_create", "dsq_gemv", "dsq_gemv_launches", "dsq_decode",
           "dsq_handle_desc", "dsq_device_bytes", "dsq_check", "dsq_destroy", "dsq_status_string",
           "dsq_gemv_noalloc", "dsq_selftest_wait_timeout", "dsq_decompose",
           "dsq_kv_bytes", "dsq_kv_append", "dsq_kv_read", "dsq_kv_attend", "dsq_kv_attend_kernel",
           "dsq_kv_check", "dsq_kv_selftest_wait_timeout")


class DSQError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class Desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("bits", ctypes.c_int32),
                ("mode", ctypes.c_int32), ("nnz", ctypes.c_int64)]


class KVDesc(ctypes.Structure):
    _fields_ = [("device", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("pages", ctypes.c_int32)]


def _kv_numbers(bits, **sizes):
    """The sizes as ints; refused past ``bits``, whose low part ctypes would take."""
    for name, v in sizes.items():
        if not -1 << bits - 1 <= int(v) < 1 << bits - 1:
            raise ValueError(f"{name} must fit {bits} bits, is {v}")
    return [int(v) for v in sizes.values()]


def _kv_desc(device, kv_heads, head_dim, page_tokens, pages) -> KVDesc:
    return KVDesc(*_kv_numbers(32, device=device, kv_heads=kv_heads, head_dim=head_dim, page_tokens=page_tokens, pages=pages))


def _kv_window(window):
    """A window past every position is none."""
    return window if 0 <= window < 1 << 31 else -1 if window < 0 else (1 << 31) - 1


class KVRows(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_token", ctypes.c_int64),
                ("k_head", ctypes.c_int64), ("v_token", ctypes.c_int64), ("v_head", ctypes.c_int64),
                ("dtype", ctypes.c_int32)]


class KVQueries(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("q_token", ctypes.c_int64), ("q_head", ctypes.c_int64), ("out_token", ctypes.c_int64),
                ("out_head", ctypes.c_int64), ("q_tokens", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("q_heads", ctypes.c_int32), ("batch", ctypes.c_int32), ("table_pages", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("window", ctypes.c_int32), ("scale", ctypes.c_float),
                ("page_table", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("q_start", ctypes.c_void_p)]


_lib = None


def library() -> ctypes.CDLL:
    """The loaded libdsq.so; raises when it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIBRARY):
            raise RuntimeError(f"{LIBRARY} is missing: build it with "
                               "`python -m dense_sparse_quantized_b200.build`")
        lib = ctypes.CDLL(LIBRARY)
        P, I, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        lib.dsq_pack.argtypes = [ctypes.POINTER(Desc), P, P, P, P, P, P, P, ctypes.POINTER(SZ)]
        lib.dsq_pack_two_axis.argtypes = [ctypes.POINTER(Desc), P, P, P, P, P, P, P, P, P,
                                          ctypes.POINTER(SZ)]
        lib.dsq_pack_intgrid.argtypes = [ctypes.POINTER(Desc), P, P, P, P, P, P, ctypes.POINTER(SZ)]
        lib.dsq_blob_desc.argtypes = [P, SZ, ctypes.POINTER(Desc)]
        lib.dsq_create.argtypes = [P, SZ, I, ctypes.POINTER(P)]
        lib.dsq_gemv.argtypes = [P, P, P, I, P]
        lib.dsq_gemv_launches.argtypes = [P, I]
        lib.dsq_decode.argtypes = [P, P, P]
        lib.dsq_handle_desc.argtypes = [P, ctypes.POINTER(Desc)]
        lib.dsq_device_bytes.argtypes = [P]
        lib.dsq_device_bytes.restype = SZ
        lib.dsq_check.argtypes = [P]
        lib.dsq_destroy.argtypes = [P]
        lib.dsq_gemv_noalloc.argtypes = [ctypes.POINTER(Desc), P, SZ, P, P, I, P]
        lib.dsq_selftest_wait_timeout.argtypes = [P, P]
        lib.dsq_decompose.argtypes = [ctypes.POINTER(Desc), P, P, P, P, P, P, P, P, ctypes.POINTER(SZ), P]
        lib.dsq_kv_bytes.argtypes = [ctypes.POINTER(KVDesc), ctypes.POINTER(SZ)]
        lib.dsq_kv_append.argtypes = [ctypes.POINTER(KVDesc), P, ctypes.POINTER(KVRows), P, ctypes.c_int64, P]
        lib.dsq_kv_read.argtypes = [ctypes.POINTER(KVDesc), P, ctypes.POINTER(KVRows), P, ctypes.c_int64, P]
        lib.dsq_kv_attend.argtypes = [ctypes.POINTER(KVDesc), P, ctypes.POINTER(KVQueries), P,
                                      ctypes.POINTER(SZ), P]
        lib.dsq_kv_attend_kernel.argtypes = [ctypes.POINTER(KVDesc), ctypes.POINTER(KVQueries)]
        lib.dsq_kv_check.argtypes = [ctypes.POINTER(KVDesc)]
        lib.dsq_kv_selftest_wait_timeout.argtypes = [ctypes.POINTER(KVDesc), P]
        lib.dsq_status_string.argtypes = [I]
        lib.dsq_status_string.restype = ctypes.c_char_p
        for name in EXPORTS:
            if name != "dsq_status_string" and name != "dsq_device_bytes":
                getattr(lib, name).restype = I
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return library().dsq_status_string(int(status)).decode()


def _check(rc: int, what: str):
    if rc != DSQ_OK:
        raise DSQError(rc, what)


def _arr(a, dtype):
    if a is None:
        return None, None
    a = np.ascontiguousarray(a, dtype=dtype)
    return a, a.ctypes.data


def pack(rows: int, cols: int, bits: int, mode, codes, table, zeros, row_ptr, col_idx,
         values, row_scale=None, col_scale=None) -> bytes:
    """Validate logical weights and return the packed blob (host bytes).

    mode: 'lut' / 'affine' / 'bitplane' or MODE_*.  Arrays: codes uint8
    [rows, cols]; table fp16 bits (uint16) [rows, 2^bits] (lut),
    [rows, cols/16] (affine scales) or [rows, cols/(32*2^bits), bits+1]
    (bit-plane coefficients C0..Ck); zeros uint16 [rows, cols/16] or None;
    row_ptr int32; col_idx int32; values uint16 fp16 bits.  row_scale /
    col_scale (fp16 bits [rows] / [cols]): two-axis scales (dsq_pack_two_axis)."""
    lib = library()
    m = {"lut": MODE_LUT_ROW, "affine": MODE_AFFINE_G16, "bitplane": MODE_BITPLANE}.get(mode, mode)
    nnz = int(np.asarray(row_ptr)[-1]) if row_ptr is not None and len(row_ptr) else 0
    d = Desc(int(rows), int(cols), int(bits), int(m), nnz)
    keep = [_arr(codes, np.uint8), _arr(table, np.uint16), _arr(zeros, np.uint16),
            _arr(row_ptr, np.int32), _arr(col_idx, np.int32), _arr(values, np.uint16)]
    two = row_scale is not None or col_scale is not None
    if two:
        keep += [_arr(row_scale, np.uint16), _arr(col_scale, np.uint16)]
    ptrs = [p for _, p in keep]
    fn, name = (lib.dsq_pack_two_axis, "dsq_pack_two_axis") if two else (lib.dsq_pack, "dsq_pack")
    size = ctypes.c_size_t(0)
    rc = fn(ctypes.byref(d), *ptrs, None, ctypes.byref(size))
    if rc != DSQ_ERR_BUFFER_TOO_SMALL:
        _check(rc, name)
    buf = ctypes.create_string_buffer(size.value)
    _check(fn(ctypes.byref(d), *ptrs, buf, ctypes.byref(size)), name)
    return buf.raw[:size.value]


def pack_intgrid(rows: int, cols: int, q, scales, row_ptr, col_idx, values) -> bytes:
    """Huffman-code an integer-grid matrix (dsq_pack_intgrid): q int16
    [rows, cols] (|q| <= 8191), scales fp16 bits [rows, cols/16], optional
    outliers as CSR."""
    lib = library()
    nnz = int(np.asarray(row_ptr)[-1]) if row_ptr is not None and len(row_ptr) else 0
    d = Desc(int(rows), int(cols), 14, MODE_INTGRID, nnz)
    keep = [_arr(q, np.int16), _arr(scales, np.uint16), _arr(row_ptr, np.int32),
            _arr(col_idx, np.int32), _arr(values, np.uint16)]
    ptrs = [p for _, p in keep]
    size = ctypes.c_size_t(0)
    rc = lib.dsq_pack_intgrid(ctypes.byref(d), *ptrs, None, ctypes.byref(size))
    if rc != DSQ_ERR_BUFFER_TOO_SMALL:
        _check(rc, "dsq_pack_intgrid")
    buf = ctypes.create_string_buffer(size.value)
    _check(lib.dsq_pack_intgrid(ctypes.byref(d), *ptrs, buf, ctypes.byref(size)), "dsq_pack_intgrid")
    return buf.raw[:size.value]


def pack_problem(p) -> bytes:
    """pack() from an object with rows, cols, bits, mode, codes, table, zeros,
    row_ptr, col_idx, values attributes."""
    if p.mode == "intgrid":
        return pack_intgrid(p.rows, p.cols, p.codes, p.table, p.row_ptr, p.col_idx, p.values)
    return pack(p.rows, p.cols, p.bits, p.mode, p.codes, p.table, p.zeros, p.row_ptr,
                p.col_idx, p.values, getattr(p, "row_scale", None), getattr(p, "col_scale", None))


def blob_desc(blob: bytes) -> Desc:
    d = Desc()
    _check(library().dsq_blob_desc(blob, len(blob), ctypes.byref(d)), "dsq_blob_desc")
    return d


def _stream_ptr(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


class Handle:
    """A packed matrix resident on one GPU."""

    def __init__(self, blob: bytes, device: int = 0):
        self._h = None
        h = ctypes.c_void_p()
        _check(library().dsq_create(blob, len(blob), int(device), ctypes.byref(h)), "dsq_create")
        self._h = h
        self.device = int(device)
        d = Desc()
        _check(library().dsq_handle_desc(h, ctypes.byref(d)), "dsq_handle_desc")
        self.rows, self.cols, self.bits, self.mode, self.nnz = d.rows, d.cols, d.bits, d.mode, d.nnz

    @property
    def device_bytes(self) -> int:
        return int(library().dsq_device_bytes(self._h))

    def gemv(self, x, y=None, stream=None):
        """y = x @ What^T.  x: cuda fp16 [batch, cols] (or [cols]); y optional
        cuda fp16 [batch, rows].  Asynchronous on ``stream`` (default: the
        current torch stream)."""
        import torch
        squeeze = x.dim() == 1
        if squeeze:
            x = x.unsqueeze(0)
        if x.dtype != torch.float16 or not x.is_cuda or not x.is_contiguous():
            raise ValueError("x must be a contiguous cuda float16 tensor")
        if x.shape[1] != self.cols:
            raise ValueError(f"x has {x.shape[1]} columns, the matrix {self.cols}")
        batch = x.shape[0]
        if y is None:
            y = torch.empty((batch, self.rows), dtype=torch.float16, device=x.device)
        elif (y.dtype != torch.float16 or not y.is_cuda or not y.is_contiguous()
              or tuple(y.shape) != (batch, self.rows)):
            raise ValueError("y must be a contiguous cuda float16 tensor [batch, rows]")
        _check(library().dsq_gemv(self._h, x.data_ptr(), y.data_ptr(), batch,
                                  _stream_ptr(stream)), "dsq_gemv")
        return y[0] if squeeze else y

    def launches_per_call(self, batch: int) -> int:
        """Kernel launches one gemv() of this batch makes."""
        n = library().dsq_gemv_launches(self._h, int(batch))
        if n < 0:
            raise DSQError(DSQ_ERR_INVALID_ARG, "dsq_gemv_launches")
        return n

    def gemv_host(self, x_host, y_host=None, x_dev=None, y_dev=None, stream=None):
        """End-to-end call from host memory: copy x (pinned cpu fp16
        [batch, cols]) to the device, run the product, copy y back into pinned
        cpu memory.  Asynchronous; synchronise the stream before reading y."""
        import torch
        if x_dev is None:
            x_dev = torch.empty(x_host.shape, dtype=torch.float16, device=f"cuda:{self.device}")
        if y_host is None:
            y_host = torch.empty((x_host.shape[0], self.rows), dtype=torch.float16).pin_memory()
        if y_dev is None:
            y_dev = torch.empty(y_host.shape, dtype=torch.float16, device=x_dev.device)
        s = torch.cuda.current_stream() if stream is None else stream
        with torch.cuda.stream(s):
            x_dev.copy_(x_host, non_blocking=True)
            self.gemv(x_dev, y_dev, stream=s)
            y_host.copy_(y_dev, non_blocking=True)
        return y_host

    def decode(self, out=None, stream=None):
        """W_dense as cuda fp16 [rows, cols] (outliers not added)."""
        import torch
        if out is None:
            out = torch.empty((self.rows, self.cols), dtype=torch.float16,
                              device=f"cuda:{self.device}")
        _check(library().dsq_decode(self._h, out.data_ptr(), _stream_ptr(stream)), "dsq_decode")
        return out

    def check(self):
        """Synchronise the device; raise if a kernel of this handle gave up a
        bounded wait since the last check."""
        _check(library().dsq_check(self._h), "dsq_check")

    def selftest_wait_timeout(self, stream=None):
        """Test hook: launch a kernel whose bounded wait runs out (about 2 s);
        the next check() raises DSQ_ERR_DEVICE."""
        _check(library().dsq_selftest_wait_timeout(self._h, _stream_ptr(stream)),
               "dsq_selftest_wait_timeout")

    def close(self):
        if self._h is not None:
            _check(library().dsq_destroy(self._h), "dsq_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


def gemv_noalloc(desc: Desc, packed_device, x, y, stream=None):
    """y = x @ What^T without a handle and without any device allocation in
    the library, for callers whose device memory all comes from a host
    program's own pool.  ``packed_device``: the dsq_pack blob already copied
    to the device by the caller (a cuda uint8 tensor, 256-byte aligned);
    ``x``: cuda fp16 [batch, cols]; ``y``: caller-allocated cuda fp16
    [batch, rows].  Calls that overlap on the GPU share one scratch array and
    race.  Asynchronous on ``stream`` (default: the current torch stream)."""
    import torch
    if packed_device.dtype != torch.uint8 or not packed_device.is_cuda or not packed_device.is_contiguous():
        raise ValueError("packed_device must be a contiguous cuda uint8 tensor")
    for name, t in (("x", x), ("y", y)):
        if t.dtype != torch.float16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 2:
            raise ValueError(f"{name} must be a contiguous 2-D cuda float16 tensor")
    batch = x.shape[0]
    if x.shape[1] != desc.cols or tuple(y.shape) != (batch, desc.rows):
        raise ValueError("x must be [batch, cols] and y [batch, rows]")
    _check(library().dsq_gemv_noalloc(ctypes.byref(desc), packed_device.data_ptr(), packed_device.numel(),
                                      x.data_ptr(), y.data_ptr(), batch, _stream_ptr(stream)),
           "dsq_gemv_noalloc")
    return y


def decompose(w, bits: int, mode: str, nnz: int, stream=None, workspace=None):
    """Outliers and quantized dense part of device fp32 weights w [rows, cols]
    (dsq_decompose): returns cuda tensors (codes, table, zeros or None,
    row_ptr, col_idx, values) -- the arrays pack() takes.  ``workspace``:
    an optional cuda uint8 tensor to reuse; one is allocated otherwise."""
    import torch
    if w.dtype != torch.float32 or not w.is_cuda or not w.is_contiguous() or w.dim() != 2:
        raise ValueError("w must be a contiguous 2-D cuda float32 tensor")
    rows, cols = w.shape
    m = {"lut": MODE_LUT_ROW, "affine": MODE_AFFINE_G16}[mode]
    d = Desc(rows, cols, int(bits), m, int(nnz))
    dev = w.device
    size = ctypes.c_size_t(0)
    rc = library().dsq_decompose(ctypes.byref(d), None, None, None, None, None, None, None, None,
                                 ctypes.byref(size), None)
    if rc != DSQ_ERR_BUFFER_TOO_SMALL:
        _check(rc, "dsq_decompose")
    if workspace is None or workspace.numel() < size.value:
        workspace = torch.empty(max(size.value, 1), dtype=torch.uint8, device=dev)
    codes = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
    if m == MODE_LUT_ROW:
        table = torch.empty((rows, 1 << bits), dtype=torch.float16, device=dev)
        zeros = None
    else:
        table = torch.empty((rows, cols // 16), dtype=torch.float16, device=dev)
        zeros = torch.empty((rows, cols // 16), dtype=torch.float16, device=dev)
    row_ptr = torch.empty(rows + 1, dtype=torch.int32, device=dev)
    col_idx = torch.empty(max(nnz, 1), dtype=torch.int32, device=dev)
    values = torch.empty(max(nnz, 1), dtype=torch.float16, device=dev)
    size = ctypes.c_size_t(workspace.numel())
    _check(library().dsq_decompose(ctypes.byref(d), w.data_ptr(), codes.data_ptr(), table.data_ptr(),
                                   None if zeros is None else zeros.data_ptr(), row_ptr.data_ptr(),
                                   col_idx.data_ptr(), values.data_ptr(), workspace.data_ptr(),
                                   ctypes.byref(size), _stream_ptr(stream)), "dsq_decompose")
    return codes, table, zeros, row_ptr, col_idx[:nnz], values[:nnz]


class KVCache:
    """The keys and values of one layer in 4-bit codes, in pages (dsq_kv_*).

    ``data``: cuda uint8 memory of KVCache.bytes_for(...) bytes to use (a
    stored cache, or a host program's own pool); allocated and zeroed
    otherwise.  A token's slot is page * page_tokens + offset.  Calls are
    asynchronous on ``stream`` (default: the current torch stream of the
    cache's device) and work on the cache's device, whichever is current; new
    tensors that they return are made on that stream.

        kv = KVCache(kv_heads=8, head_dim=128, pages=1024)
        kv.append(k, v, slots)                    # k, v: [tokens, kv_heads, head_dim]
        out = kv.attend(q, page_table, kv_lens)   # q: [batch, q_heads, head_dim]
        k, v = kv.read(slots)
    """

    def __init__(self, kv_heads: int, head_dim: int, pages: int, page_tokens: int = 64, device: int = 0,
                 data=None):
        import torch
        if data is not None:
            if data.dtype != torch.uint8 or not data.is_cuda or not data.is_contiguous():
                raise ValueError("data must be a contiguous cuda uint8 tensor")
            device = data.device.index
        self.desc = _kv_desc(device, kv_heads, head_dim, page_tokens, pages)
        size = self.bytes_for(kv_heads, head_dim, pages, page_tokens)
        if data is None:
            data = torch.zeros(size, dtype=torch.uint8, device=f"cuda:{int(device)}")
        elif data.numel() != size:
            raise ValueError(f"data has {data.numel()} bytes, the cache takes {size}")
        self.data = data
        self.device = data.device
        self.kv_heads, self.head_dim = int(kv_heads), int(head_dim)
        self.page_tokens, self.pages = int(page_tokens), int(pages)
        self._lib, self._torch, self._index = library(), torch, self.desc.device
        self._int32, self._int64 = torch.int32, torch.int64
        self._raw_stream = torch._C._cuda_getCurrentRawStream
        self._d, self._data = ctypes.byref(self.desc), data.data_ptr()
        self._dtypes = {torch.float16: DTYPE_F16, torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}

    @staticmethod
    def bytes_for(kv_heads: int, head_dim: int, pages: int, page_tokens: int = 64) -> int:
        """Bytes of a cache of that shape (dsq_kv_bytes)."""
        size = ctypes.c_size_t(0)
        d = _kv_desc(0, kv_heads, head_dim, page_tokens, pages)
        _check(library().dsq_kv_bytes(ctypes.byref(d), ctypes.byref(size)), "dsq_kv_bytes")
        return size.value

    def _stream(self, stream):
        # a decode step makes these calls by the dozen: the raw handle costs a
        # tenth of a torch.cuda.Stream object
        if stream is None:
            return self._raw_stream(self._index)
        return _stream_ptr(stream)

    def _new(self, stream, fill, shape, dtype):
        """A tensor made on ``stream``, so that what fills it and what may get
        its memory next is in order with the call."""
        if stream is None:
            return fill(shape, dtype=dtype, device=self.device)
        cuda = self._torch.cuda
        if not isinstance(stream, cuda.Stream):
            stream = cuda.ExternalStream(int(stream), device=self.device)
        with cuda.stream(stream):
            return fill(shape, dtype=dtype, device=self.device)

    def _rows(self, t, name, tokens, heads):
        if t.get_device() != self._index or t.shape != (tokens, heads, self.head_dim):
            raise ValueError(f"{name} must be [{tokens}, {heads}, {self.head_dim}] on {self.device}")
        strides = t.stride()
        if strides[2] != 1:
            raise ValueError(f"{name} must be contiguous in its last dimension")
        return strides

    def _kv_rows(self, k, v, slots):
        if (slots.dtype != self._int64 or slots.get_device() != self._index or slots.dim() != 1
                or not slots.is_contiguous()):
            raise ValueError(f"slots must be a contiguous 1-D int64 tensor on {self.device}")
        n = slots.shape[0]
        ks, vs = self._rows(k, "k", n, self.kv_heads), self._rows(v, "v", n, self.kv_heads)
        dtype = self._dtypes.get(k.dtype)
        if dtype is None or k.dtype != v.dtype:
            raise ValueError("k and v must have the same dtype: float16, bfloat16 or float32")
        return n, ctypes.byref(KVRows(k.data_ptr(), v.data_ptr(), ks[0], ks[1], vs[0], vs[1], dtype))

    def append(self, k, v, slots, stream=None):
        """Quantise k, v [tokens, kv_heads, head_dim] (float16 or bfloat16, any
        strides that are multiples of 8) into ``slots`` (int64 [tokens]; a
        negative slot passes its token over; no slot twice)."""
        n, rows = self._kv_rows(k, v, slots)
        rc = self._lib.dsq_kv_append(self._d, self._data, rows, slots.data_ptr(), n, self._stream(stream))
        if rc:
            _check(rc, "dsq_kv_append")

    def read(self, slots, dtype=None, k=None, v=None, stream=None):
        """(k, v): the values at ``slots``, [tokens, kv_heads, head_dim] in
        ``dtype`` (default float16) or in the given k and v, whose rows of
        negative slots stay as they are (new ones hold 0 there)."""
        if k is None or v is None:
            like = k if k is not None else v
            dtype = dtype or (like.dtype if like is not None else self._torch.float16)
            shape = (slots.shape[0], self.kv_heads, self.head_dim)
            k = self._new(stream, self._torch.zeros, shape, dtype) if k is None else k
            v = self._new(stream, self._torch.zeros, shape, dtype) if v is None else v
        if dtype is not None and k.dtype != dtype:
            raise ValueError("k and v must have the dtype asked for")
        n, rows = self._kv_rows(k, v, slots)
        rc = self._lib.dsq_kv_read(self._d, self._data, rows, slots.data_ptr(), n, self._stream(stream))
        if rc:
            _check(rc, "dsq_kv_read")
        return k, v

    def attend_workspace(self, q_tokens: int, q_heads: int, batch: int, stream=None):
        """Scratch for attend() calls of these sizes that follow one another;
        calls that may overlap need one each."""
        size = ctypes.c_size_t(0)
        (n,), (heads, batch) = _kv_numbers(64, q_tokens=q_tokens), _kv_numbers(32, q_heads=q_heads, batch=batch)
        # the size is asked for with a q_start, which a query of it does not read:
        # any number of rows may be any number of sequences'
        a = KVQueries(q_tokens=n, q_heads=heads, batch=batch, q_start=self._data or 256)
        rc = library().dsq_kv_attend(self._d, None, ctypes.byref(a), None, ctypes.byref(size), None)
        if rc != DSQ_ERR_BUFFER_TOO_SMALL:
            _check(rc, "dsq_kv_attend")
        return self._new(stream, self._torch.empty, max(size.value, 1), self._torch.uint8)

    def attend(self, q, page_table, kv_lens, q_start=None, scale=None, causal=True, window=0, out=None, lse=None,
               return_lse=False, workspace=None, stream=None):
        """softmax(scale * q K^T) V of queries over the cache (dsq_kv_attend).

        q: [q_tokens, q_heads, head_dim], float16 or bfloat16; page_table:
        int32 [batch, pages per sequence]; kv_lens: int32 [batch], the tokens
        of each sequence in the cache, those of its queries among them;
        q_start: int32 [batch + 1], the first row of each sequence (default:
        q_tokens / batch rows each); scale: default head_dim ** -0.5; window:
        see only the last that many tokens; out: not q's memory.  Returns out (like q), and with
        ``return_lse`` or ``lse`` also the fp32 log-sum-exp [q_tokens,
        q_heads].  Rows of no sequence stay as they are in a given out and
        lse, and hold 0 in new ones."""
        torch, device = self._torch, self.device
        if q.dim() != 3:
            raise ValueError(f"q must be [q_tokens, q_heads, {self.head_dim}]")
        n, heads = q.shape[0], q.shape[1]
        qs = self._rows(q, "q", n, heads)
        dtype = self._dtypes.get(q.dtype)
        if dtype is None:
            raise ValueError("q must be float16 or bfloat16")
        if page_table.dim() != 2 or kv_lens.dim() != 1 or kv_lens.shape[0] != page_table.shape[0]:
            raise ValueError("page_table must be [batch, pages] and kv_lens [batch]")
        batch, columns = page_table.shape
        for t in (page_table, kv_lens) if q_start is None else (page_table, kv_lens, q_start):
            if t.dtype != self._int32 or t.get_device() != self._index or not t.is_contiguous():
                raise ValueError(f"page_table, kv_lens and q_start must be contiguous int32 tensors on {device}")
        if q_start is not None and q_start.shape != (batch + 1,):
            raise ValueError("q_start must be [batch + 1]")
        if out is None:
            out = self._new(stream, torch.empty if q_start is None else torch.zeros, q.shape, q.dtype)
        elif out.dtype != q.dtype:
            raise ValueError("out must have q's dtype")
        os = self._rows(out, "out", n, heads)
        if lse is None:
            if return_lse:
                lse = self._new(stream, torch.zeros, (n, heads), torch.float32)
        elif (lse.dtype != torch.float32 or lse.get_device() != self._index or lse.shape != (n, heads)
              or not lse.is_contiguous()):
            raise ValueError(f"lse must be a contiguous float32 tensor [{n}, {heads}] on {device}")
        if workspace is None:
            workspace = self.attend_workspace(n, heads, batch, stream)
        elif workspace.get_device() != self._index or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {device}")
        a = KVQueries(q.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(), qs[0], qs[1], os[0], os[1],
                      n, dtype, heads, batch, columns, causal, _kv_window(window),
                      self.head_dim ** -0.5 if scale is None else scale, page_table.data_ptr(), kv_lens.data_ptr(),
                      None if q_start is None else q_start.data_ptr())
        size = ctypes.c_size_t(workspace.nbytes)
        rc = self._lib.dsq_kv_attend(self._d, self._data, ctypes.byref(a), workspace.data_ptr(), ctypes.byref(size),
                                     self._stream(stream))
        if rc:
            _check(rc, "dsq_kv_attend")
        return out if lse is None else (out, lse)

    def attend_kernel(self, q_tokens: int, q_heads: int, batch: int, table_pages: int, ragged=False, causal=True,
                      window=0) -> str:
        """The kernel that attend() calls of these sizes take, "few_rows" or
        "many_rows" (dsq_kv_attend_kernel).  ragged: with a q_start."""
        (n,), sizes = _kv_numbers(64, q_tokens=q_tokens), _kv_numbers(32, q_heads=q_heads, batch=batch, table_pages=table_pages)
        a = KVQueries(q_tokens=n, q_heads=sizes[0], batch=sizes[1], table_pages=sizes[2], causal=causal,
                      window=_kv_window(window), q_start=256 if ragged else None)
        which = self._lib.dsq_kv_attend_kernel(self._d, ctypes.byref(a))
        if which < 0:
            _check(which, "dsq_kv_attend_kernel")
        return ("few_rows", "many_rows")[which]

    def check(self):
        """Synchronise the device; raise if a kernel of an attend() on it, of any
        cache, gave up a bounded wait since the last check."""
        _check(self._lib.dsq_kv_check(self._d), "dsq_kv_check")

    def selftest_wait_timeout(self, stream=None):
        """Test hook: launch a kernel whose bounded wait runs out (about 2 s);
        the next check() raises DSQ_ERR_DEVICE."""
        _check(self._lib.dsq_kv_selftest_wait_timeout(self._d, self._stream(stream)), "dsq_kv_selftest_wait_timeout")
