"""Host-side checks of the operators of a step of many tokens: refusals of every entry point (no device call is
reached), sizes, and pins of the oracle."""
import ctypes
import math

import numpy as np
import pytest

from oracle import decode, prompt
from packed_ternary_weight_b200 import tern

P = 0x10000  # an aligned address that no refused call may reach
NULL = None


def cache(kvh=5, d=128, page=64, pages=8, ptr=P):
    return tern.KV4CacheC(kvh, d, page, pages, ptr)


def batch(seqs=2, tokens=4, max_new=2, max_len=100, max_pages=2, start=P, length=P, table=P):
    return tern.KV4BatchC(seqs, tokens, max_new, max_len, max_pages, start, length, table)


def norm(mode=2, m=3, k=64, xt=1, x=P, ldx=64, rt=1, r=P, ldr=64, gain=P, eps=1e-5, s=P, lds=64, xq=P, ldq=64, xs=P):
    return tern.lib.tern_norm_quantize(mode, m, k, xt, x, ldx, rt, r, ldr, gain, eps, s, lds, xq, ldq, xs, NULL)


@pytest.mark.parametrize("bad", [dict(mode=0), dict(mode=4), dict(xt=3), dict(rt=0), dict(m=-1), dict(k=0), dict(ldx=63),
                                 dict(ldr=63), dict(lds=63), dict(ldq=63), dict(eps=0.0), dict(eps=float("nan")), dict(x=NULL),
                                 dict(r=NULL), dict(gain=NULL), dict(s=NULL), dict(xq=NULL), dict(xs=NULL),
                                 dict(r=P, s=P, lds=96)])
def test_norm_refuses(bad):
    assert norm(**bad) == tern.EINVAL


def test_norm_alignment_and_nothing_to_do():
    for bad in (dict(x=P + 2), dict(r=P + 2), dict(gain=P + 1), dict(xs=P + 2), dict(s=P + 2), dict(x=P + 1, xt=2)):
        assert norm(**bad) == tern.EALIGN
    assert norm(m=0, x=NULL, r=NULL, s=NULL, xq=NULL, xs=NULL) == tern.OK


def gemm(m=3, n=5, k=40, x=P, ldx=48, sx=P, w=P, ldw=48, sw=P, out=1, y=P, ldy=5):
    return tern.lib.tern_gemm_i8(m, n, k, x, ldx, sx, w, ldw, sw, out, y, ldy, NULL)


@pytest.mark.parametrize("bad", [dict(m=-1), dict(n=0), dict(k=0), dict(k=131072, ldx=131072, ldw=131072), dict(ldx=40), dict(ldw=56),
                                 dict(ldx=32), dict(ldw=32), dict(ldy=4), dict(out=0), dict(x=NULL), dict(w=NULL), dict(sx=NULL),
                                 dict(sw=NULL), dict(y=NULL)])
def test_gemm_refuses(bad):
    assert gemm(**bad) == tern.EINVAL


def test_gemm_alignment_and_nothing_to_do():
    for bad in (dict(x=P + 8), dict(w=P + 4), dict(sx=P + 2), dict(sw=P + 1), dict(y=P + 2), dict(y=P + 1, out=2)):
        assert gemm(**bad) == tern.EALIGN
    assert gemm(m=0, x=NULL, y=NULL, sx=NULL) == tern.OK


def test_sizes_beyond_the_indices():
    big = (1 << 30) + 1
    for bad in (dict(m=big), dict(k=big, ldx=big, ldr=big, lds=big, ldq=big)):
        assert norm(**bad) == tern.EINVAL
    for bad in (dict(m=big), dict(n=big, ldy=big), dict(m=(1 << 31) - 1), dict(m=1 << 24, n=1 << 20, ldy=1 << 20)):
        assert gemm(**bad) == tern.EINVAL


def append(c=None, b=None, heads=20, type=1, q=P, ldq=2560, k=P, ldk=640, v=P, ldv=640, rope=P, max_pos=100, qo=P):
    c, b = c or cache(), b or batch()
    return tern.lib.tern_kv4_append(ctypes.byref(c), ctypes.byref(b), heads, type, q, ldq, k, ldk, v, ldv, rope, max_pos, qo, NULL)


def read(c=None, b=None, type=1, k=P, ldk=640, v=P, ldv=640):
    c, b = c or cache(), b or batch()
    return tern.lib.tern_kv4_read(ctypes.byref(c), ctypes.byref(b), type, k, ldk, v, ldv, NULL)


def attend(c=None, b=None, heads=20, scale=0.1, q=P, out=P, ws=P, n=1 << 40):
    c, b = c or cache(), b or batch()
    return tern.lib.tern_kv4_attention(ctypes.byref(c), ctypes.byref(b), heads, scale, q, out, ws, n, NULL)


@pytest.mark.parametrize("call", [append, read, attend])
def test_cache_and_batch_refusals(call):
    for c in (cache(kvh=0), cache(kvh=1025), cache(pages=0), cache(ptr=NULL)):
        assert call(c=c) == tern.EINVAL
    for c in (cache(d=96), cache(d=256), cache(page=8), cache(page=48), cache(page=512)):
        assert call(c=c) == tern.EUNSUPPORTED
    assert call(c=cache(ptr=P + 8)) == tern.EALIGN
    for b in (batch(seqs=-1), batch(seqs=65536), batch(tokens=-1), batch(max_new=-1), batch(max_len=-1), batch(max_pages=-1),
              batch(start=NULL), batch(length=NULL), batch(table=NULL)):
        assert call(b=b) == tern.EINVAL
    for b in (batch(start=P + 2), batch(length=P + 1), batch(table=P + 2)):
        assert call(b=b) == tern.EALIGN
    for b in (batch(seqs=0, start=NULL), batch(tokens=0, table=NULL), batch(max_new=0)):
        assert call(b=b) == tern.OK


@pytest.mark.parametrize("bad", [dict(type=0), dict(heads=-1), dict(ldq=2552), dict(ldq=2564), dict(ldk=632), dict(ldv=641), dict(max_pos=0),
                                 dict(q=NULL), dict(k=NULL), dict(v=NULL), dict(rope=NULL), dict(qo=NULL)])
def test_append_refuses(bad):
    assert append(**bad) == tern.EINVAL


def test_alignment_of_token_buffers():
    for bad in (dict(q=P + 8), dict(k=P + 4), dict(v=P + 2), dict(rope=P + 8), dict(qo=P + 4)):
        assert append(**bad) == tern.EALIGN
    for bad in (dict(k=P + 4), dict(v=P + 2)):
        assert read(**bad) == tern.EALIGN
    for bad in (dict(q=P + 8), dict(out=P + 2)):
        assert attend(**bad) == tern.EALIGN


def test_read_and_attention_refuse():
    for bad in (dict(type=3), dict(ldk=632), dict(ldv=644)):
        assert read(**bad) == tern.EINVAL
    assert read(k=NULL, v=NULL) == tern.OK
    for bad in (dict(heads=0), dict(heads=21), dict(scale=float("inf")), dict(scale=float("nan")), dict(q=NULL), dict(out=NULL)):
        assert attend(**bad) == tern.EINVAL


def test_attention_workspace():
    size = ctypes.c_size_t()
    c = cache()

    def need(seqs, new, length, heads=20):
        assert tern.lib.tern_kv4_attention_workspace_size(ctypes.byref(c), seqs, new, length, heads, ctypes.byref(size)) == tern.OK
        return size.value

    assert need(0, 1, 100) == 0
    assert need(1, 1, 100) == 0                       # one chunk: nothing to join
    assert need(1, 1, 8192) > 0
    b = batch(seqs=1, tokens=1, max_new=1, max_len=8192, max_pages=128)
    assert attend(b=b, ws=NULL, n=0) == tern.ENOSPACE
    assert attend(b=b, n=255) == tern.ENOSPACE
    assert attend(b=b, ws=P + 128) == tern.EALIGN
    f = tern.lib.tern_kv4_attention_workspace_size
    assert f(ctypes.byref(c), 1, 1, 100, 21, ctypes.byref(size)) == tern.EINVAL
    assert f(ctypes.byref(c), -1, 1, 100, 20, ctypes.byref(size)) == tern.EINVAL
    assert f(ctypes.byref(c), 1, 1, 100, 20, None) == tern.EINVAL


def test_workspace_covers_smaller_batches():
    # a workspace sized for a bound serves every batch within it
    c = cache(kvh=4)
    size = ctypes.c_size_t()

    def need(seqs, new, length):
        assert tern.lib.tern_kv4_attention_workspace_size(ctypes.byref(c), seqs, new, length, 16, ctypes.byref(size)) == tern.OK
        return size.value

    for bound in ((8, 4, 5000), (64, 1, 8192), (3, 40, 20000), (2, 1000, 3000)):
        top = need(*bound)
        for s in {1, bound[0] // 2, bound[0]}:
            for n in {1, 2, 3, bound[1] // 2, bound[1]}:
                for ln in {16, 256, 257, 1000, bound[2] // 3, bound[2]}:
                    if s and n and n <= bound[1] and ln <= bound[2]:
                        assert need(s, n, ln) <= top, (bound, s, n, ln)


@pytest.mark.parametrize("page,d", [(16, 64), (64, 128), (256, 128)])
def test_cache_size(page, d):
    assert tern.KV4Cache.size(5, d, page, 7) == 7 * 5 * page * (d + 8)


# ------------------------------------------------------------ oracle pins
def test_oracle_four_bit_codes_by_hand():
    x = np.zeros((1, 64), np.float32)
    x[0, :16] = np.arange(16) * 0.5 - 2.0              # min -2, max 5.5, scale 0.5: codes 0..15, exact
    x[0, 16:] = -2.0
    c, s, m = prompt.quantize4(x)
    assert s[0] == np.float16(0.5) and m[0] == np.float16(-2)
    assert np.array_equal(c[0, :16], np.arange(16)) and not c[0, 16:].any()
    c, s, m = prompt.quantize4(np.full((1, 64), 3.25, np.float32))
    assert s[0] == 0 and m[0] == np.float16(3.25) and not c.any()
    # a code is off by at most half a step, and the step and the minimum by an fp16 rounding (2^-11)
    g = np.random.default_rng(1)
    x = g.standard_normal((50, 128)).astype(np.float32)
    c, s, m = prompt.quantize4(x)
    back = m.astype(np.float64)[:, None] + s.astype(np.float64)[:, None] * c
    s64 = s.astype(np.float64)[:, None]
    assert (np.abs(back - x) <= 0.5 * s64 * 1.0001 + 15 * s64 * 2.0 ** -11 + 2.0 ** -11 * np.abs(m.astype(np.float64))[:, None]).all()


def test_oracle_norm_agrees_with_the_decode_oracle():
    g = np.random.default_rng(2)
    x, r, gain = (g.standard_normal((3, 200)).astype(np.float32) for _ in range(3))
    v, q, s = prompt.norm_quantize("add", x, r, gain[0], 1e-5)
    for i in range(3):
        y = decode.rmsnorm((x[i] + r[i]).astype(np.float32), gain[0])
        q1, s1 = decode.quantize_f32(y)
        assert np.array_equal(q[i], q1[0]) and s[i] == s1[0]


def test_oracle_rotation_agrees_with_the_decode_oracle():
    g = np.random.default_rng(3)
    x = g.standard_normal((2, 3, 128)).astype(np.float32)
    cs = [decode.rope_cos_sin(p) for p in (0, 17)]
    y = prompt.rotate(x, np.stack([c for c, _ in cs]), np.stack([s for _, s in cs]))
    for i in range(2):
        for h in range(3):
            assert np.array_equal(y[i, h], decode.rope(x[i, h], *cs[i]))


def test_oracle_attention_by_hand():
    # two positions, one head; the first token sees only the first position
    d, page = 64, 16
    raw = np.zeros((1, 1, prompt.block_bytes(page, d)), np.uint8)
    c = prompt.Cache(raw, 1, d, page)
    ones, seven = np.full(d, 1, np.uint8), np.full(d, 7, np.uint8)
    c.put(0, 0, 0, 0, ones, 0.5, 0.0)
    c.put(0, 1, 0, 0, seven, 0.25, -1.0)
    c.put(0, 0, 0, 1, seven, 1.0, 0.0)
    c.put(0, 1, 0, 1, ones, 2.0, 1.0)
    assert c.raw[0, 0, 0] == 0x11 and c.raw[0, 0, d // 2] == 0x77 and c.raw[0, 0, page * d // 2] == 0x77
    q = np.full((2, 1, d), 1 / 16, np.float32)
    out, tol = prompt.attention(c, np.array([[0]]), np.array([0, 2]), np.array([2]), 1, 0.5, q)
    a, b = 0.5 * 64 / 16 * 0.5, 0.5 * 64 / 16 * 0.75
    w = 1 / (1 + math.exp(b - a))
    assert np.allclose(out[0], 7.0) and np.allclose(out[1], w * 7 + (1 - w) * 3, rtol=1e-12)
    assert (tol > 0).all()
