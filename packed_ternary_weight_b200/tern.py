"""ctypes binding of libtern.so: argument marshalling only.

Every step of the computation runs in the library's CUDA kernels (or, for
packing, its host C++ code). Importing this module fails loudly if the shared
library has not been built; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtern.so")

OK, EINVAL, EFORMAT, EALIGN, ENOSPACE, EUNSUPPORTED, ECUDA, ETIMEOUT = range(8)
FMT = {"bitnet": 1, "tq": 2, "bt3": 3}
ACT_INT8, ACT_BF16, ACT_BF16_Q8 = 1, 2, 3
OUT_F32, OUT_BF16 = 1, 2
NORM_PLAIN, NORM_ADD, NORM_RELU2 = 1, 2, 3
F_PDL = 1


class TernError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {status_string(code)} ({code})")
        self.code = code


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"libtern.so not built ({_LIB_PATH}); run python -m packed_ternary_weight_b200.build")
    return ctypes.CDLL(_LIB_PATH)


lib = _load()


class Desc(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("n", ctypes.c_int32), ("k", ctypes.c_int32),
                ("planes", ctypes.c_int32), ("group", ctypes.c_int32), ("tensor_scale", ctypes.c_float),
                ("flags", ctypes.c_uint32)]


_vp, _sz = ctypes.c_void_p, ctypes.c_size_t
lib.tern_status_string.restype = ctypes.c_char_p
lib.tern_status_string.argtypes = [ctypes.c_int]
lib.tern_packed_size.argtypes = [ctypes.POINTER(Desc), ctypes.POINTER(_sz)]
lib.tern_pack.argtypes = [ctypes.POINTER(Desc), _vp, _vp, _vp, _vp, _vp, _sz, ctypes.POINTER(_sz)]
lib.tern_workspace_size.argtypes = [ctypes.POINTER(Desc), ctypes.c_int32, ctypes.POINTER(_sz)]
lib.tern_quantize_act.argtypes = [_vp, ctypes.c_int32, ctypes.c_int32, _vp, _vp, _vp]
lib.tern_gemv.argtypes = [ctypes.POINTER(Desc), _vp, ctypes.c_int, _vp, _vp, ctypes.c_int, _vp, _vp, _sz, _vp]
lib.tern_gemm_batched.argtypes = [ctypes.POINTER(Desc), _vp, ctypes.c_int32, ctypes.c_int, _vp, _vp, ctypes.c_int,
                                  _vp, _vp, _sz, _vp]
lib.tern_device_error.argtypes = [_vp]
lib.tern_gemv_noalloc.argtypes = [ctypes.POINTER(Desc), _vp, ctypes.c_int, _vp, _vp, ctypes.c_int, _vp, _vp]
lib.tern_stream_read.argtypes = [_vp, _sz, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                 ctypes.c_int32, _vp, _vp]
lib.tern_gemv_grouped.argtypes = [ctypes.c_int32, ctypes.POINTER(Desc), ctypes.POINTER(_vp), ctypes.c_int,
                                  ctypes.POINTER(_vp), ctypes.POINTER(_vp), ctypes.c_int, ctypes.POINTER(_vp), _vp]
lib.tern_selftest_wait.argtypes = [ctypes.c_uint64, _vp]
lib.tern_fit_tq.argtypes = [_vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _vp, _vp, _vp]
lib.tern_fit_bt.argtypes = [_vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _vp, _vp, _vp, _vp]


class DecodeModelC(ctypes.Structure):
    _fields_ = [("layers", ctypes.c_int32), ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("max_pos", ctypes.c_int32), ("eps", ctypes.c_float), ("packed", ctypes.POINTER(_vp)),
                ("d_gains", _vp), ("d_kcache", _vp), ("d_vcache", _vp), ("d_rope", _vp)]


lib.tern_decode_rope_table.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_double, _vp]
lib.tern_decode_workspace_size.argtypes = [ctypes.POINTER(DecodeModelC), ctypes.POINTER(_sz)]
lib.tern_decode_step.argtypes = [ctypes.POINTER(DecodeModelC), ctypes.c_int32, _vp, _vp, ctypes.c_int32,
                                 ctypes.c_int32, _vp, _vp, _vp, _sz, _vp]
for _f in (lib.tern_decode_rope_table, lib.tern_decode_workspace_size, lib.tern_decode_step):
    _f.restype = ctypes.c_int
for _f in (lib.tern_selftest_wait, lib.tern_fit_tq, lib.tern_fit_bt, lib.tern_packed_size, lib.tern_pack, lib.tern_workspace_size, lib.tern_quantize_act, lib.tern_gemv,
           lib.tern_gemm_batched, lib.tern_device_error, lib.tern_gemv_noalloc, lib.tern_gemv_grouped,
           lib.tern_stream_read):
    _f.restype = ctypes.c_int


class KV4CacheC(ctypes.Structure):
    _fields_ = [("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("d_pages", _vp)]


class KV4BatchC(ctypes.Structure):
    _fields_ = [("seqs", ctypes.c_int32), ("tokens", ctypes.c_int32), ("max_new", ctypes.c_int32),
                ("max_len", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("d_start", _vp), ("d_len", _vp),
                ("d_table", _vp)]


_i32, _i64, _cache_p, _batch_p = ctypes.c_int32, ctypes.c_int64, ctypes.POINTER(KV4CacheC), ctypes.POINTER(KV4BatchC)
lib.tern_norm_quantize.argtypes = [ctypes.c_int, _i32, _i32, ctypes.c_int, _vp, _i64, ctypes.c_int, _vp, _i64, _vp,
                                   ctypes.c_float, _vp, _i64, _vp, _i64, _vp, _vp]
lib.tern_kv4_cache_size.argtypes = [_cache_p, ctypes.POINTER(_sz)]
lib.tern_kv4_append.argtypes = [_cache_p, _batch_p, _i32, ctypes.c_int, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i32,
                                _vp, _vp]
lib.tern_kv4_read.argtypes = [_cache_p, _batch_p, ctypes.c_int, _vp, _i64, _vp, _i64, _vp]
lib.tern_kv4_attention_workspace_size.argtypes = [_cache_p, _i32, _i32, _i32, _i32, ctypes.POINTER(_sz)]
lib.tern_kv4_attention.argtypes = [_cache_p, _batch_p, _i32, ctypes.c_float, _vp, _vp, _vp, _sz, _vp]
lib.tern_gemm_i8.argtypes = [_i32, _i32, _i32, _vp, _i64, _vp, _vp, _i64, _vp, ctypes.c_int, _vp, _i64, _vp]
for _f in (lib.tern_norm_quantize, lib.tern_kv4_cache_size, lib.tern_kv4_append, lib.tern_kv4_read,
           lib.tern_kv4_attention_workspace_size, lib.tern_kv4_attention, lib.tern_gemm_i8):
    _f.restype = ctypes.c_int


def status_string(code: int) -> str:
    return lib.tern_status_string(code).decode()


def _check(code: int, what: str):
    if code != OK:
        raise TernError(code, what)


def make_desc(fmt: str, n: int, k: int, planes: int = 1, group: int = 0, tensor_scale: float = 0.0,
              flags: int = 0) -> Desc:
    return Desc(FMT[fmt], n, k, planes, group, tensor_scale, flags)


def desc_of(layer, flags: int = 0) -> Desc:
    """Descriptor of a synth.Layer (or anything with the same fields)."""
    return make_desc(layer.fmt, layer.n, layer.k, layer.planes, layer.group, layer.tensor_scale, flags)


def packed_size(desc: Desc) -> int:
    out = _sz()
    _check(lib.tern_packed_size(ctypes.byref(desc), ctypes.byref(out)), "tern_packed_size")
    return out.value


def _ptr(a):
    if a is None:
        return None
    if hasattr(a, "data_ptr"):
        return ctypes.c_void_p(a.data_ptr())
    return a.ctypes.data_as(ctypes.c_void_p)


def pack(desc: Desc, trits, scales_fp16=None, scale_idx=None, codebook=None) -> np.ndarray:
    """Pack logical weights (host numpy arrays) into a uint8 numpy buffer."""
    t = np.ascontiguousarray(trits, dtype=np.int8)
    s = None if scales_fp16 is None else np.ascontiguousarray(scales_fp16, dtype=np.float16).view(np.uint16)
    i = None if scale_idx is None else np.ascontiguousarray(scale_idx, dtype=np.uint8)
    c = None if codebook is None else np.ascontiguousarray(codebook, dtype=np.float32)
    size = packed_size(desc)
    out = np.empty(size, dtype=np.uint8)
    used = _sz()
    _check(lib.tern_pack(ctypes.byref(desc), _ptr(t), _ptr(s), _ptr(i), _ptr(c), _ptr(out), size,
                         ctypes.byref(used)), "tern_pack")
    return out


def pack_layer(layer, flags: int = 0):
    d = desc_of(layer, flags)
    return d, pack(d, layer.trits, layer.scales, layer.idx, layer.codebook)


def workspace_size(desc: Desc, m: int = 1) -> int:
    out = _sz()
    _check(lib.tern_workspace_size(ctypes.byref(desc), m, ctypes.byref(out)), "tern_workspace_size")
    return out.value


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def quantize_act(x_bf16, xq, xscale, stream=None):
    """x_bf16: device tensor [m][k] of bf16 (or int16/uint16 bits); xq int8 [m][k]; xscale float [m]."""
    m, k = x_bf16.shape
    _check(lib.tern_quantize_act(_ptr(x_bf16), m, k, _ptr(xq), _ptr(xscale), _stream(stream)), "tern_quantize_act")


def gemm_batched(desc: Desc, packed, m: int, act: int, x, xscale, out: int, y, ws=None, stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.tern_gemm_batched(ctypes.byref(desc), _ptr(packed), m, act, _ptr(x), _ptr(xscale), out, _ptr(y),
                                 _ptr(ws), ws_bytes, _stream(stream)), "tern_gemm_batched")


def gemv(desc: Desc, packed, act: int, x, xscale, out: int, y, ws=None, stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.tern_gemv(ctypes.byref(desc), _ptr(packed), act, _ptr(x), _ptr(xscale), out, _ptr(y), _ptr(ws),
                         ws_bytes, _stream(stream)), "tern_gemv")


class Grouped:
    """Marshalled arguments of tern_gemv_grouped, built once and launched many times."""

    def __init__(self, descs, packed, act: int, xs, xscales, out: int, ys):
        n = len(descs)
        self.count = n
        self.act, self.out = act, out
        self.descs = (Desc * n)(*descs)
        self.packed = (_vp * n)(*[p.data_ptr() for p in packed])
        self.xs = (_vp * n)(*[x.data_ptr() for x in xs])
        self.xscales = None if xscales is None else (_vp * n)(*[s.data_ptr() for s in xscales])
        self.ys = (_vp * n)(*[y.data_ptr() for y in ys])

    def launch(self, stream=None):
        _check(lib.tern_gemv_grouped(self.count, self.descs, self.packed, self.act, self.xs, self.xscales, self.out,
                                     self.ys, _stream(stream)), "tern_gemv_grouped")


def gemv_grouped(descs, packed, act: int, xs, xscales, out: int, ys, stream=None):
    Grouped(descs, packed, act, xs, xscales, out, ys).launch(stream)


def gemv_noalloc(desc: Desc, packed, act: int, x, xscale, out: int, y, stream=None):
    """tern_gemv with the library's fixed device scratch instead of a caller workspace."""
    _check(lib.tern_gemv_noalloc(ctypes.byref(desc), _ptr(packed), act, _ptr(x), _ptr(xscale), out, _ptr(y),
                                 _stream(stream)), "tern_gemv_noalloc")


def stream_read(src, mode: int, chunk: int, depth: int, ctas_per_sm: int, warps: int, sink, stream=None):
    """Read-ceiling kernel: stream all of `src` once with the given access shape."""
    _check(lib.tern_stream_read(_ptr(src), src.numel() * src.element_size(), mode, chunk, depth, ctas_per_sm, warps,
                                _ptr(sink), _stream(stream)), "tern_stream_read")


def device_error(stream=None) -> int:
    return lib.tern_device_error(_stream(stream))


def selftest_wait(limit_ns: int, stream=None):
    """Enqueue the failure-detection self-test: a bounded wait that expires after limit_ns."""
    _check(lib.tern_selftest_wait(limit_ns, _stream(stream)), "tern_selftest_wait")


def decode_rope_table(max_pos: int, head_dim: int = 128, theta: float = 500000.0) -> np.ndarray:
    """cos/sin table [max_pos][head_dim/2][2] (fp32) computed by the library."""
    out = np.empty((max_pos, head_dim // 2, 2), dtype=np.float32)
    _check(lib.tern_decode_rope_table(max_pos, head_dim, theta, _ptr(out)), "tern_decode_rope_table")
    return out


class DecodeModel:
    """Marshalled tern_decode_model: device buffers are caller-owned tensors; the host array of
    packed-buffer pointers lives as long as this object."""

    def __init__(self, packed, gains, kcache, vcache, rope, hidden: int, inter: int, heads: int, kv_heads: int,
                 max_pos: int, eps: float = 1e-5, head_dim: int = 128):
        n = len(packed)
        assert n % 7 == 0
        self._keep = (packed, gains, kcache, vcache, rope)
        self._ptrs = (_vp * n)(*[p.data_ptr() for p in packed])
        self.c = DecodeModelC(n // 7, hidden, inter, heads, kv_heads, head_dim, max_pos, eps,
                              ctypes.cast(self._ptrs, ctypes.POINTER(_vp)), gains.data_ptr(), kcache.data_ptr(),
                              vcache.data_ptr(), rope.data_ptr())

    def workspace_size(self) -> int:
        out = _sz()
        _check(lib.tern_decode_workspace_size(ctypes.byref(self.c), ctypes.byref(out)), "tern_decode_workspace_size")
        return out.value

    def step(self, pos: int, h_in, h_out, ws, first: int = 0, last: int | None = None, attn_in=None, trace=None,
             stream=None):
        last = 5 * self.c.layers - 1 if last is None else last
        _check(lib.tern_decode_step(ctypes.byref(self.c), pos, _ptr(h_in), _ptr(h_out), first, last, _ptr(attn_in),
                                    _ptr(trace), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
               "tern_decode_step")


def fit_tq(w, planes: int, group: int, trits, scales, stream=None):
    """Fit fp32 device weights [n][k] into TQ planes: trits int8 [planes][n][k], scales fp16 [planes][n][k/group]."""
    n, k = w.shape
    _check(lib.tern_fit_tq(_ptr(w), n, k, planes, group, _ptr(trits), _ptr(scales), _stream(stream)), "tern_fit_tq")


def fit_bt(w, depth: int, codebook, trits, idx, stream=None):
    """Fit fp32 device weights [n][k] into balanced ternary: trits int8 [depth][n][k], idx uint8 [n][k/16]."""
    n, k = w.shape
    _check(lib.tern_fit_bt(_ptr(w), n, k, depth, _ptr(codebook), _ptr(trits), _ptr(idx), _stream(stream)),
           "tern_fit_bt")


_torch = None
_OUT_TYPE: dict = {}


def _import_torch():
    """torch, imported on first use (packing needs none); its types as TERN_OUT_*."""
    global _torch, _current_stream, _current_device
    import torch
    _OUT_TYPE.update({torch.float32: OUT_F32, torch.bfloat16: OUT_BF16})
    _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda dev: torch.cuda.current_stream(dev).cuda_stream)  # the handle alone costs a tenth of the object
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _torch = torch
    return torch


def _bad(what: str):
    raise TernError(EINVAL, what)


def _type(t, what: str) -> int:
    """TERN_OUT_* of a float tensor."""
    o = _OUT_TYPE.get(t.dtype)
    return o if o is not None else _bad(f"{what}: {t.dtype} is neither float32 nor bfloat16")


def _rows(t, shape, what: str) -> int:
    """Row stride of a tensor of the shape (m, k) whose rows are contiguous."""
    if t.is_contiguous() and t.shape == shape:  # most calls
        return shape[1]
    if t.shape != shape:
        _bad(what)
    ld, one = t.stride()
    m, k = shape
    if one != 1 and k > 1:
        _bad(what)
    return ld if m > 1 else k


def _vector(t, n: int, dtype, what: str):
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        _bad(what)


def _launch(dev: int, stream, what: str, fn, *args):
    """Call an entry point on the device that the tensors are on (their get_device())."""
    if dev < 0:
        _bad(f"{what}: tensors are not on a CUDA device")
    if dev != _current_device():
        with _torch.cuda.device(dev):
            return _launch(dev, stream, what, fn, *args)
    code = fn(*args, _current_stream(dev) if stream is None else _stream(stream))
    if code != OK:
        raise TernError(code, what)


def norm_quantize(mode: int, x, r, gain, eps: float, sum, xq, xscale, stream=None):
    """RMSNorm of x (NORM_PLAIN), of x + r, which goes to `sum` (NORM_ADD), or of relu(x)^2 r (NORM_RELU2), quantised
    to int8 per row: x, r, sum [m][k] float32 or bfloat16 (sum of r's type, or r itself), gain float32 [k], xq int8
    [m][k], xscale float32 [m]."""
    what = "tern_norm_quantize"
    t = _torch or _import_torch()
    shape = x.shape
    m, k = shape
    dev = x.get_device()
    _vector(gain, k, t.float32, "tern_norm_quantize: gain")
    _vector(xscale, m, t.float32, "tern_norm_quantize: xscale")
    if xq.dtype is not t.int8:
        _bad(f"{what}: xq is int8")
    rt, rp, ldr, sp, lds = 0, None, 0, None, 0
    if mode != NORM_PLAIN:
        if r is None:
            _bad(f"{what}: r is missing")
        rt, rp, ldr = _type(r, what), r.data_ptr(), _rows(r, shape, "tern_norm_quantize: r")
        if r.get_device() != dev:
            _bad(f"{what}: tensors on several devices")
    if mode == NORM_ADD:
        if sum is None or sum.dtype is not r.dtype:
            _bad(f"{what}: sum has r's type")
        sp, lds = sum.data_ptr(), _rows(sum, shape, "tern_norm_quantize: sum")
        if sum.get_device() != dev:
            _bad(f"{what}: tensors on several devices")
    if gain.get_device() != dev or xq.get_device() != dev or xscale.get_device() != dev:
        _bad(f"{what}: tensors on several devices")
    _launch(dev, stream, what, lib.tern_norm_quantize, mode, m, k, _type(x, what), x.data_ptr(),
            _rows(x, shape, "tern_norm_quantize: x"), rt, rp, ldr, gain.data_ptr(), eps, sp, lds, xq.data_ptr(),
            _rows(xq, shape, "tern_norm_quantize: xq"), xscale.data_ptr())


def gemm_i8(x, xscale, w, wscale, y, stream=None):
    """y[m][n] = x[m][k] w[n][k]^T with a scale per row of x and of w: x, w int8 (row strides multiples of 16), xscale
    float32 [m], wscale float32 [n], y float32 or bfloat16."""
    what = "tern_gemm_i8"
    t = _torch or _import_torch()
    m, k = x.shape
    n = w.shape[0]
    if x.dtype is not t.int8 or w.dtype is not t.int8:
        _bad(f"{what}: x and w are int8")
    _vector(xscale, m, t.float32, "tern_gemm_i8: xscale")
    _vector(wscale, n, t.float32, "tern_gemm_i8: wscale")
    dev = x.get_device()
    if w.get_device() != dev or xscale.get_device() != dev or wscale.get_device() != dev or y.get_device() != dev:
        _bad(f"{what}: tensors on several devices")
    ldx, ldw = _rows(x, (m, k), "tern_gemm_i8: x"), _rows(w, (n, k), "tern_gemm_i8: w")
    if m <= 1:
        ldx = (ldx + 15) & ~15  # the stride of a single row is free
    if n <= 1:
        ldw = (ldw + 15) & ~15
    _launch(dev, stream, what, lib.tern_gemm_i8, m, n, k, x.data_ptr(), ldx, xscale.data_ptr(), w.data_ptr(), ldw,
            wscale.data_ptr(), _type(y, what), y.data_ptr(), _rows(y, (m, n), "tern_gemm_i8: y"))


class KV4Batch:
    """Marshalled tern_kv4_batch: start int32 [seqs + 1], len int32 [seqs] and table int32 [seqs][max_pages] on the
    device; tokens, max_new and max_len are host bounds that the launches are planned with."""

    def __init__(self, start, len, table, tokens: int, max_new: int, max_len: int):
        what = "tern_kv4_batch"
        i32 = (_torch or _import_torch()).int32
        seqs = start.numel() - 1
        _vector(start, seqs + 1, i32, "tern_kv4_batch: start")
        _vector(len, seqs, i32, "tern_kv4_batch: len")
        if table.dim() != 2 or table.shape[0] != seqs or table.dtype is not i32 or not table.is_contiguous():
            _bad(f"{what}: table")
        self.dev = start.get_device()
        if len.get_device() != self.dev or table.get_device() != self.dev:
            _bad(f"{what}: tensors on several devices")
        self._keep = (start, len, table)
        self.tokens = tokens
        self.c = KV4BatchC(seqs, tokens, max_new, max_len, table.shape[1], start.data_ptr(), len.data_ptr(),
                           table.data_ptr())
        self._ref = ctypes.byref(self.c)


class KV4Cache:
    """Marshalled tern_kv4_cache: `pages` is a contiguous uint8 tensor of whole pages, owned by the caller."""

    def __init__(self, pages, kv_heads: int, head_dim: int, page_size: int):
        what = "tern_kv4_cache"
        page_bytes = kv_heads * page_size * (head_dim + 8)
        if pages.dtype is not (_torch or _import_torch()).uint8 or not pages.is_contiguous():
            _bad(f"{what}: pages is contiguous uint8")
        if page_bytes <= 0 or pages.numel() % page_bytes:
            _bad(f"{what}: pages holds whole pages")
        self._keep, self.dev = pages, pages.get_device()
        self.kv_heads, self.head_dim = kv_heads, head_dim
        self.c = KV4CacheC(kv_heads, head_dim, page_size, pages.numel() // page_bytes, pages.data_ptr())
        self._ref = ctypes.byref(self.c)

    @staticmethod
    def size(kv_heads: int, head_dim: int, page_size: int, num_pages: int) -> int:
        """Bytes of a cache of num_pages pages."""
        out = _sz()
        c = KV4CacheC(kv_heads, head_dim, page_size, num_pages, None)
        _check(lib.tern_kv4_cache_size(ctypes.byref(c), ctypes.byref(out)), "tern_kv4_cache_size")
        return out.value

    def _width(self, t, tokens: int, heads: int, what: str) -> int:
        """Row stride of a token buffer [tokens][heads * head_dim] on the cache's device."""
        if t.get_device() != self.dev:
            _bad(f"{what}: tensors on several devices")
        return _rows(t, (tokens, heads * self.head_dim), what)

    def append(self, batch: KV4Batch, q, k, v, rope, q_out, stream=None):
        """Rotate q and k by position, store k and v. q [tokens][heads * head_dim] and q_out (bfloat16, contiguous)
        may both be None; q, k, v are float32 or bfloat16, rope is the float32 table of decode_rope_table."""
        what = "tern_kv4_append"
        n, d = batch.tokens, self.head_dim
        heads, ldq, qp, qo = 0, 0, None, None
        if q is not None:
            heads = q.shape[-1] // d
            ldq, qp = self._width(q, n, heads, "tern_kv4_append: q"), q.data_ptr()
            if q_out is None or q_out.get_device() != self.dev:
                _bad(f"{what}: q_out")
            _vector(q_out, n * heads * d, _torch.bfloat16, "tern_kv4_append: q_out")
            qo = q_out.data_ptr()
        ldk = self._width(k, n, self.kv_heads, "tern_kv4_append: k")
        ldv = self._width(v, n, self.kv_heads, "tern_kv4_append: v")
        if v.dtype is not k.dtype or (q is not None and q.dtype is not k.dtype):
            _bad(f"{what}: q, k and v have one type")
        max_pos = rope.shape[0]
        _vector(rope, max_pos * d, _torch.float32, "tern_kv4_append: rope")
        if rope.get_device() != self.dev or batch.dev != self.dev:
            _bad(f"{what}: tensors on several devices")
        _launch(self.dev, stream, what, lib.tern_kv4_append, self._ref, batch._ref, heads, _type(k, what), qp, ldq,
                k.data_ptr(), ldk, v.data_ptr(), ldv, rope.data_ptr(), max_pos, qo)

    def read(self, batch: KV4Batch, k, v, stream=None):
        """The cached keys and values of the batch's tokens into k and v [tokens][kv_heads * head_dim] (one may be
        None), float32 or bfloat16."""
        what = "tern_kv4_read"
        one = v if k is None else k
        if one is None:
            _bad(f"{what}: neither k nor v")
        ldk = 0 if k is None else self._width(k, batch.tokens, self.kv_heads, "tern_kv4_read: k")
        ldv = 0 if v is None else self._width(v, batch.tokens, self.kv_heads, "tern_kv4_read: v")
        if v is not None and v.dtype is not one.dtype:
            _bad(f"{what}: k and v have one type")
        if batch.dev != self.dev:
            _bad(f"{what}: tensors on several devices")
        _launch(self.dev, stream, what, lib.tern_kv4_read, self._ref, batch._ref, _type(one, what),
                None if k is None else k.data_ptr(), ldk, None if v is None else v.data_ptr(), ldv)

    def attention_workspace_size(self, seqs: int, max_new: int, max_len: int, heads: int) -> int:
        if 0 <= self.dev != _torch.cuda.current_device():  # planned for the multiprocessors of the cache's device
            with _torch.cuda.device(self.dev):
                return self.attention_workspace_size(seqs, max_new, max_len, heads)
        out = _sz()
        _check(lib.tern_kv4_attention_workspace_size(self._ref, seqs, max_new, max_len, heads, ctypes.byref(out)),
               "tern_kv4_attention_workspace_size")
        return out.value

    def attention(self, batch: KV4Batch, q, scale: float, out, ws=None, stream=None):
        """Causal attention of the batch's new tokens over the cache: q, out bfloat16 [tokens][heads * head_dim]
        contiguous (out may be q); ws uint8, contiguous, zero before its first use (attention_workspace_size)."""
        what = "tern_kv4_attention"
        width, dev = q.shape[-1], self.dev
        heads = width // self.head_dim
        bf16 = _torch.bfloat16
        _vector(q, batch.tokens * heads * self.head_dim, bf16, "tern_kv4_attention: q")
        _vector(out, batch.tokens * width, bf16, "tern_kv4_attention: out")
        if ws is not None and not ws.is_contiguous():
            _bad(f"{what}: the workspace is not contiguous")
        if batch.dev != dev or q.get_device() != dev or out.get_device() != dev or (ws is not None and ws.get_device() != dev):
            _bad(f"{what}: tensors on several devices")
        _launch(dev, stream, what, lib.tern_kv4_attention, self._ref, batch._ref, heads, scale, q.data_ptr(),
                out.data_ptr(), None if ws is None else ws.data_ptr(), 0 if ws is None else ws.nbytes)
