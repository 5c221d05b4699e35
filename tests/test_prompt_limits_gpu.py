"""Operators of a step of many tokens at the ends of what their documentation allows: values at the border of the
cache's range, and calls of every kind under way at once on several streams."""
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


def test_values_at_the_border_of_the_range(tern):
    from tests import prompt_util as u
    d, heads = 64, 4
    b = u.Batch([1, 20], [40, 30], 1, d, 16, seed=31)          # the kernel for few rows and the prompt kernel
    c = b.oracle_cache()
    for s in range(2):
        for j in range(int(b.len[s])):
            for w in range(2):
                x = b.g.uniform(-65000, 65000, d).astype(np.float32)
                x[:2] = 65000, -65000                              # min + 15 scale at its largest
                codes, sc, m = prompt.quantize4(x[None])
                c.put(int(b.table[s, j // 16]), j % 16, 0, w, codes[0], sc[0], m[0])
    q = u.bf16_dev(b.g.standard_normal((b.rows, heads * d)) * 1e-4)
    cache, batch = b.device()
    out = torch.empty_like(q)
    cache.attention(batch, q, 0.1, out, u.workspace(cache, heads, 2, 20, 40))
    ref, tol = prompt.attention(c, b.table, b.start, b.len, heads, 0.1, q.float().cpu().numpy().reshape(-1, heads, d))
    err = np.abs(out.float().cpu().numpy().reshape(ref.shape) - ref)
    assert (err <= tol).all(), float(np.nanmax(err / tol))
    assert tern.device_error() == tern.OK


def test_calls_of_every_kind_at_once(tern):
    # each stream repeats one operator on buffers of its own; the results are those of the same calls one by one
    from tests import prompt_util as u
    g = torch.Generator().manual_seed(7)

    def attention(new, length, kvh, heads, seed):
        b = u.Batch(new, length, kvh, 128, 64, seed=seed)
        b.raw[:] = b.g.integers(0, 256, b.raw.size)
        c = b.oracle_cache()
        for page in range(b.raw.size // (kvh * prompt.block_bytes(64, 128))):
            for h in range(kvh):
                for w in range(2):
                    for slot in range(64):
                        c.put(page, slot, h, w, b.g.integers(0, 16, 128), np.float16(0.1), np.float16(-0.7))
        cache, batch = b.device()
        q = u.bf16_dev(b.g.standard_normal((b.rows, heads * 128)))
        ws = u.workspace(cache, heads, len(new), max(new), max(length))
        return lambda out: cache.attention(batch, q, 0.1, out, ws), torch.empty_like(q)

    def gemm(m, n, k):
        x = torch.randint(-127, 128, (m, k), dtype=torch.int8, generator=g).cuda()
        w = torch.randint(-127, 128, (n, k), dtype=torch.int8, generator=g).cuda()
        sx, sw = torch.rand(m, generator=g).cuda(), torch.rand(n, generator=g).cuda()
        return lambda out: tern.gemm_i8(x, sx, w, sw, out), torch.empty((m, n), device="cuda")

    def norm(m, k):
        x, r = torch.randn(m, k, generator=g).cuda(), torch.randn(m, k, generator=g).cuda()
        gain, s, sx = torch.rand(k, generator=g).cuda(), torch.empty(m, k, device="cuda"), torch.empty(m, device="cuda")
        return lambda out: tern.norm_quantize(tern.NORM_ADD, x, r, gain, 1e-5, s, out, sx), \
            torch.empty((m, k), dtype=torch.int8, device="cuda")

    calls = [attention([300, 200], [700, 200], 2, 8, 1), attention([1] * 9, [900] * 9, 2, 8, 2),
             gemm(500, 20000, 512), gemm(3, 1280, 2560), gemm(90, 2560, 1280), norm(700, 2560)]
    want = []
    for call, out in calls:
        call(out)
        torch.cuda.synchronize()
        want.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(12):
        for (call, out), stream in zip(calls, streams):
            with torch.cuda.stream(stream):
                call(out)
    torch.cuda.synchronize()
    for (_, out), w in zip(calls, want):
        assert torch.equal(out, w)
    assert tern.device_error() == tern.OK


@pytest.mark.parametrize("group", [1, 4, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_at_the_border_of_the_kernels(tern, group, d):
    # 48 query rows per kv head and one token more, beside single tokens; in place as well
    from tests import prompt_util as u
    n = 48 // group
    b = u.Batch([n, n + 1, 1, n], [600, 300, 520, n], 2, d, 32, seed=group)
    b.fill_values()
    heads, scale = 2 * group, d ** -0.5
    q = u.bf16_dev(b.g.standard_normal((b.rows, heads * d)))
    cache, batch = b.device()
    out, ws = torch.empty_like(q), u.workspace(cache, heads, 4, n + 1, 600)
    cache.attention(batch, q, scale, out, ws)
    ref, tol = prompt.attention(b.oracle_cache(), b.table, b.start, b.len, heads, scale, q.float().cpu().numpy().reshape(-1, heads, d))
    assert (np.abs(out.float().cpu().numpy().reshape(ref.shape) - ref) <= tol).all()
    cache.attention(batch, q, scale, q, ws)
    assert torch.equal(q, out) and tern.device_error() == tern.OK


def test_prompts_among_many_sequences(tern):
    # more sequences than a CTA has threads: the search for a share goes over them in turns
    from tests import prompt_util as u
    new = [1] * 800
    length = [1 + s % 5 for s in range(800)]
    for s, n in ((3, 60), (400, 130), (671, 49), (672, 70), (799, 50)):
        new[s], length[s] = n, n + 7 * (s % 4)
    new[10] = new[700] = length[10] = 0
    b = u.Batch(new, length, 1, 64, 16, seed=8)
    b.fill_values()
    q = u.bf16_dev(b.g.standard_normal((b.rows, 64)))
    cache, batch = b.device()
    out = torch.empty_like(q)
    cache.attention(batch, q, 0.125, out, u.workspace(cache, 1, 800, 130, max(length)))
    ref, tol = prompt.attention(b.oracle_cache(), b.table, b.start, b.len, 1, 0.125, q.float().cpu().numpy().reshape(-1, 1, 64))
    assert (np.abs(out.float().cpu().numpy().reshape(ref.shape) - ref) <= tol).all()
    assert tern.device_error() == tern.OK
