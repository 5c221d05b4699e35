"""Attention over the 4-bit cache: queries over the whole range of bf16, the rounding of the weights, which kernel takes
a sequence, and cut prompts, each against a bound of its own."""
import math

import numpy as np
import pytest

from oracle import prompt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tern():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from packed_ternary_weight_b200 import tern as t
    t.device_error()
    return t


def util():
    from tests import prompt_util
    return prompt_util


def attend(tern, b, heads, scale, q, max_new=None):
    """The kernel's output [tokens][heads][d] as fp64."""
    cache, batch = b.device(max_new)
    q = util().bf16_dev(q.reshape(b.rows, heads * b.d))
    out = torch.full_like(q, 9.0)
    cache.attention(batch, q, scale, out, util().workspace(cache, heads, len(b.new), max_new or int(b.new.max()), int(b.len.max())))
    torch.cuda.synchronize()
    assert tern.device_error() == tern.OK
    return q.float().cpu().numpy().reshape(b.rows, heads, b.d), out.double().cpu().numpy().reshape(b.rows, heads, b.d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,heads", [(1, 4), (5, 4), (60, 2)])
@pytest.mark.parametrize("kind", ["normal", "one sign", "one row"])
def test_queries_at_the_top_of_the_range(tern, d, new, heads, kind):
    # q near 2^121 and a scale that keeps the scores ordinary: neither a row's factor nor its sum may leave fp32
    b = util().Batch([new], [300], 1, d, 16, seed=41)
    b.fill_values()
    q = b.g.standard_normal((new, heads, d))
    if kind == "one sign":
        q = np.abs(q) + 0.5                                # the sum of a row is beyond fp32
    if kind == "one row":
        q[:, 1:] *= 2.0 ** -121
    scale = 2.0 ** -121 / math.sqrt(d)
    q, got = attend(tern, b, heads, scale, q * 2.0 ** 121)
    ref, tol = prompt.attention(b.oracle_cache(), b.table, b.start, b.len, heads, scale, q)
    assert (np.abs(got - ref) <= tol).all(), float(np.nanmax(np.abs(got - ref) / tol))


@pytest.mark.parametrize("new", [1, 3])
@pytest.mark.parametrize("d,length", [(64, 500), (128, 900)])
def test_roundings_of_the_weights_cancel_in_the_offset(tern, new, d, length):
    # Values of codes 7 and 8 about zero, and weights that are all alike but for one position in 32, so that all of them
    # are rounded the same way: the offset 7.5 scale, fifteen times the values, must not bring that rounding in.
    b = util().Batch([new], [length], 1, d, 16, seed=42)
    c, heads = b.oracle_cache(), 8
    for j in range(length):
        at = (int(b.table[0, j // 16]), j % 16, 0)
        c.put(*at, 0, np.zeros(d, np.uint8), np.float16(0), np.float16(j % 32 == 0))
        c.put(*at, 1, b.g.integers(7, 9, d).astype(np.uint8), np.float16(0.75), np.float16(-5.625))
    q = np.zeros((new, heads, d))
    q += np.linspace(0.07, 0.95, new * heads).reshape(new, heads, 1) / d   # the others' weight is 2^-(that)
    q, got = attend(tern, b, heads, math.log(2.0), q)
    ref, tol = prompt.attention(b.oracle_cache(), b.table, b.start, b.len, heads, math.log(2.0), q)
    assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,group", [(17, 1), (8, 4), (11, 3), (12, 4), (2, 8), (1, 5)])
@pytest.mark.parametrize("offset", [0.0, 6.0])
def test_one_sequence_of_few_rows(tern, d, new, group, offset):
    # up to 48 query rows of a single sequence multiply by the codes, and are held to that kernel's bound
    b = util().Batch([new], [300 + new], 2, d, 32, seed=43 + new)
    c = b.oracle_cache()
    for j in range(int(b.len[0])):
        for h in range(2):
            for w in range(2):
                codes, s, m = prompt.quantize4((b.g.standard_normal((1, d)) + w * offset).astype(np.float32))
                c.put(int(b.table[0, j // 32]), j % 32, h, w, codes[0], s[0], m[0])
    heads = 2 * group
    q, got = attend(tern, b, heads, d ** -0.5, b.g.standard_normal((new, heads, d)))
    ref, tol = prompt.attention(b.oracle_cache(), b.table, b.start, b.len, heads, d ** -0.5, q)
    assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())


@pytest.mark.parametrize("new,bound", [(1, 400), (3, 4000)])
def test_a_generous_bound_does_not_choose_the_kernel(tern, new, bound):
    # the buffers have few rows: the result is that of the exact bound
    b = util().Batch([new], [900], 2, 64, 16, seed=44)
    b.fill_values()
    q = b.g.standard_normal((new, 8, 64))
    want, got = attend(tern, b, 8, 0.125, q)[1], attend(tern, b, 8, 0.125, q, max_new=bound)[1]
    assert np.array_equal(got, want)


@pytest.mark.parametrize("new,length", [([16], [3500]), ([13, 20], [3000, 2500])])
def test_cut_prompts_of_wide_heads(tern, new, length):
    # few rows and long histories at D = 128: one tile's blocks go to several CTAs, whose parts are joined
    b = util().Batch(new, length, 1, 128, 64, seed=45)
    b.fill_values()
    q, got = attend(tern, b, 4, 128 ** -0.5, b.g.standard_normal((b.rows, 4, 128)))
    ref, tol = prompt.attention(b.oracle_cache(), b.table, b.start, b.len, 4, 128 ** -0.5, q)
    assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())


@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d,n", [(64, 5), (128, 900)])        # one head per group of lanes; several
def test_appended_values_that_are_not_finite_show(tern, bad, dt, d, n):
    # a key head or value head with a value that the cache cannot hold reads as not finite; all others are as without it
    u, kvh, heads = util(), 2, 6
    b = u.Batch([n], [n], kvh, d, 16, seed=46)
    k, v, q = (torch.from_numpy(b.g.standard_normal((n, h * d)).astype(np.float32)).to(dt).cuda() for h in (kvh, kvh, heads))
    rope = torch.from_numpy(tern.decode_rope_table(n, d)).cuda()
    cache, batch = b.device()
    qo = torch.empty((n, heads * d), dtype=torch.bfloat16, device="cuda")
    res = []
    for _ in range(2):
        cache.append(batch, q, k, v, rope, qo)
        ko, vo = torch.empty((n, kvh * d), device="cuda"), torch.empty((n, kvh * d), device="cuda")
        cache.read(batch, ko, vo)
        res.append((ko.view(n, kvh, d), vo.view(n, kvh, d)))
        k[1, 7], v[3, d + 9] = float(bad), float(bad)        # token 1's first key head, token 3's second value head
    (k0, v0), (k1, v1) = res
    assert not k1[1, 0].isfinite().any() and not v1[3, 1].isfinite().any()
    k1[1, 0], v1[3, 1] = k0[1, 0], v0[3, 1]
    assert torch.equal(k0, k1) and torch.equal(v0, v1)
    out = torch.empty_like(qo)
    cache.attention(batch, qo, d ** -0.5, out, u.workspace(cache, heads, 1, n, n))
    o = out.view(n, kvh, 3, d)
    assert o[:3, 1].isfinite().all() and not o[3:, 1].isfinite().any()     # values of the second head, from token 3 on
    assert o[:1, 0].isfinite().all()
    if bad == "nan":
        assert not o[1:, 0].isfinite().any()                               # keys of the first, from token 1 on
    assert tern.device_error() == tern.OK


def test_a_query_that_is_not_a_number_in_a_prompt(tern):
    b = util().Batch([60], [300], 1, 64, 16, seed=47)
    b.fill_values()
    q = b.g.standard_normal((60, 2, 64))
    want = attend(tern, b, 2, 0.125, q)[1]
    q[7, 1, 5], q[9, 0, 3] = float("nan"), float("inf")
    got = attend(tern, b, 2, 0.125, q)[1]
    assert not np.isfinite(got[7, 1]).any() and not np.isfinite(got[9, 0]).any()
    got[7, 1], got[9, 0] = want[7, 1], want[9, 0]
    assert np.array_equal(got, want)
