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


def _type(t, what: str) -> int:
    """TERN_OUT_* of a float tensor."""
    name = str(t.dtype)
    if name == "torch.float32":
        return OUT_F32
    if name == "torch.bfloat16":
        return OUT_BF16
    raise TernError(EINVAL, f"{what}: {name} is neither float32 nor bfloat16")


def _want(ok: bool, what: str):
    if not ok:
        raise TernError(EINVAL, what)


def _rows(t, m: int, k: int, what: str) -> int:
    """Row stride of a tensor [m][k] whose rows are contiguous."""
    _want(t.dim() == 2 and t.shape[0] == m and t.shape[1] == k and (k == 1 or t.stride(1) == 1), what)
    return t.stride(0) if m > 1 else max(k, t.stride(0))


def _vector(t, n: int, name: str, what: str):
    _want(str(t.dtype) == name and t.numel() == n and t.is_contiguous(), what)


def _launch(dev, stream, what: str, fn, *args):
    """Call an entry point on the device that the tensors are on."""
    import torch
    _want(dev.type == "cuda", f"{what}: tensors are not on a CUDA device")
    if dev.index == torch.cuda.current_device():
        return _check(fn(*args, _stream(stream)), what)
    with torch.cuda.device(dev):
        _check(fn(*args, _stream(stream)), what)


def norm_quantize(mode: int, x, r, gain, eps: float, sum, xq, xscale, stream=None):
    """RMSNorm of x (NORM_PLAIN), of x + r, which goes to `sum` (NORM_ADD), or of relu(x)^2 r (NORM_RELU2), quantised
    to int8 per row: x, r, sum [m][k] float32 or bfloat16 (sum of r's type, or r itself), gain float32 [k], xq int8
    [m][k], xscale float32 [m]."""
    what = "tern_norm_quantize"
    m, k = x.shape
    two, add = mode != NORM_PLAIN, mode == NORM_ADD
    _want(not two or r is not None, f"{what}: r is missing")
    _want(not add or (sum is not None and sum.dtype == r.dtype), f"{what}: sum has r's type")
    _vector(gain, k, "torch.float32", f"{what}: gain")
    _vector(xscale, m, "torch.float32", f"{what}: xscale")
    _want(str(xq.dtype) == "torch.int8", f"{what}: xq is int8")
    dev = x.device
    _want(gain.device == dev and xq.device == dev and xscale.device == dev and (not two or r.device == dev) and
          (not add or sum.device == dev), f"{what}: tensors on several devices")
    _launch(dev, stream, what, lib.tern_norm_quantize, mode, m, k, _type(x, what), x.data_ptr(),
            _rows(x, m, k, f"{what}: x"), _type(r, what) if two else 0, r.data_ptr() if two else None,
            _rows(r, m, k, f"{what}: r") if two else 0, gain.data_ptr(), eps, sum.data_ptr() if add else None,
            _rows(sum, m, k, f"{what}: sum") if add else 0, xq.data_ptr(), _rows(xq, m, k, f"{what}: xq"),
            xscale.data_ptr())


def gemm_i8(x, xscale, w, wscale, y, stream=None):
    """y[m][n] = x[m][k] w[n][k]^T with a scale per row of x and of w: x, w int8 (row strides multiples of 16), xscale
    float32 [m], wscale float32 [n], y float32 or bfloat16."""
    what = "tern_gemm_i8"
    m, k = x.shape
    n = w.shape[0]
    _want(str(x.dtype) == "torch.int8" and str(w.dtype) == "torch.int8", f"{what}: x and w are int8")
    _vector(xscale, m, "torch.float32", f"{what}: xscale")
    _vector(wscale, n, "torch.float32", f"{what}: wscale")
    dev = x.device
    _want(w.device == dev and xscale.device == dev and wscale.device == dev and y.device == dev,
          f"{what}: tensors on several devices")
    ldx, ldw = _rows(x, m, k, f"{what}: x"), _rows(w, n, k, f"{what}: w")
    if m <= 1:
        ldx = (ldx + 15) & ~15  # the stride of a single row is free
    if n <= 1:
        ldw = (ldw + 15) & ~15
    _launch(dev, stream, what, lib.tern_gemm_i8, m, n, k, x.data_ptr(), ldx, xscale.data_ptr(), w.data_ptr(), ldw,
            wscale.data_ptr(), _type(y, what), y.data_ptr(), _rows(y, m, n, f"{what}: y"))


class KV4Batch:
    """Marshalled tern_kv4_batch: start int32 [seqs + 1], len int32 [seqs] and table int32 [seqs][max_pages] on the
    device; tokens, max_new and max_len are host bounds that the launches are planned with."""

    def __init__(self, start, len, table, tokens: int, max_new: int, max_len: int):
        what = "tern_kv4_batch"
        seqs = start.numel() - 1
        _vector(start, seqs + 1, "torch.int32", f"{what}: start")
        _vector(len, seqs, "torch.int32", f"{what}: len")
        _want(table.dim() == 2 and table.shape[0] == seqs, f"{what}: table")
        _vector(table, table.numel(), "torch.int32", f"{what}: table")
        _want(len.device == start.device and table.device == start.device, f"{what}: tensors on several devices")
        self._keep = (start, len, table)
        self.device, self.tokens = start.device, tokens
        self.c = KV4BatchC(seqs, tokens, max_new, max_len, table.shape[1], start.data_ptr(), len.data_ptr(),
                           table.data_ptr())


class KV4Cache:
    """Marshalled tern_kv4_cache: `pages` is a contiguous uint8 tensor of whole pages, owned by the caller."""

    def __init__(self, pages, kv_heads: int, head_dim: int, page_size: int):
        what = "tern_kv4_cache"
        _want(str(pages.dtype) == "torch.uint8" and pages.is_contiguous(), f"{what}: pages is contiguous uint8")
        page_bytes = kv_heads * page_size * (head_dim + 8)
        _want(page_bytes > 0 and pages.numel() % page_bytes == 0, f"{what}: pages holds whole pages")
        self._keep, self.device = pages, pages.device
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

    def _heads(self, t, tokens: int, what: str):
        """Heads and row stride of a token buffer [tokens][heads * head_dim]."""
        _want(t.device == self.device, f"{what}: tensors on several devices")
        _want(t.dim() == 2 and t.shape[1] % self.head_dim == 0, what)
        return t.shape[1] // self.head_dim, _rows(t, tokens, t.shape[1], what)

    def append(self, batch: KV4Batch, q, k, v, rope, q_out, stream=None):
        """Rotate q and k by position, store k and v. q [tokens][heads * head_dim] and q_out (bfloat16, contiguous)
        may both be None; q, k, v are float32 or bfloat16, rope is the float32 table of decode_rope_table."""
        what = "tern_kv4_append"
        n = batch.tokens
        heads, ldq = (0, 0) if q is None else self._heads(q, n, f"{what}: q")
        hk, ldk = self._heads(k, n, f"{what}: k")
        hv, ldv = self._heads(v, n, f"{what}: v")
        _want(hk == self.kv_heads and hv == hk, f"{what}: k and v have the cache's heads")
        _want(v.dtype == k.dtype and (q is None or q.dtype == k.dtype), f"{what}: q, k and v have one type")
        if q is not None:
            _want(q_out is not None and q_out.device == self.device, f"{what}: q_out")
            _vector(q_out, n * heads * self.head_dim, "torch.bfloat16", f"{what}: q_out")
        _want(rope.dim() == 3 and rope.shape[1] * 2 == self.head_dim and rope.shape[2] == 2 and
              rope.device == self.device and batch.device == self.device, f"{what}: rope")
        _vector(rope, rope.numel(), "torch.float32", f"{what}: rope")
        _launch(self.device, stream, what, lib.tern_kv4_append, self._ref, ctypes.byref(batch.c), heads,
                _type(k, what), None if q is None else q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv,
                rope.data_ptr(), rope.shape[0], None if q is None else q_out.data_ptr())

    def read(self, batch: KV4Batch, k, v, stream=None):
        """The cached keys and values of the batch's tokens into k and v [tokens][kv_heads * head_dim] (one may be
        None), float32 or bfloat16."""
        what = "tern_kv4_read"
        _want(k is not None or v is not None, f"{what}: neither k nor v")
        hk, ldk = (self.kv_heads, 0) if k is None else self._heads(k, batch.tokens, f"{what}: k")
        hv, ldv = (self.kv_heads, 0) if v is None else self._heads(v, batch.tokens, f"{what}: v")
        _want(hk == self.kv_heads and hv == hk, f"{what}: k and v have the cache's heads")
        _want(k is None or v is None or k.dtype == v.dtype, f"{what}: k and v have one type")
        _want(batch.device == self.device, f"{what}: tensors on several devices")
        _launch(self.device, stream, what, lib.tern_kv4_read, self._ref, ctypes.byref(batch.c),
                _type(v if k is None else k, what), None if k is None else k.data_ptr(), ldk,
                None if v is None else v.data_ptr(), ldv)

    def attention_workspace_size(self, seqs: int, max_new: int, max_len: int, heads: int) -> int:
        out = _sz()
        _check(lib.tern_kv4_attention_workspace_size(self._ref, seqs, max_new, max_len, heads, ctypes.byref(out)),
               "tern_kv4_attention_workspace_size")
        return out.value

    def attention(self, batch: KV4Batch, q, scale: float, out, ws=None, stream=None):
        """Causal attention of the batch's new tokens over the cache: q, out bfloat16 [tokens][heads * head_dim]
        contiguous (out may be q); ws uint8, zero before its first use (attention_workspace_size)."""
        what = "tern_kv4_attention"
        _want(q.dim() == 2 and q.shape[1] % self.head_dim == 0 and batch.device == self.device and
              q.device == self.device and out.device == self.device and (ws is None or ws.device == self.device),
              f"{what}: q")
        heads = q.shape[1] // self.head_dim
        _vector(q, batch.tokens * q.shape[1], "torch.bfloat16", f"{what}: q")
        _vector(out, q.numel(), "torch.bfloat16", f"{what}: out")
        _launch(self.device, stream, what, lib.tern_kv4_attention, self._ref, ctypes.byref(batch.c), heads, scale,
                q.data_ptr(), out.data_ptr(), None if ws is None else ws.data_ptr(),
                0 if ws is None else ws.numel() * ws.element_size())
