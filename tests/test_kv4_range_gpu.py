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
