"""tern_gemm_i8 against the exact integer product: the definition rounds three times in a stated order, so the outputs
must be equal bit for bit."""
import numpy as np
import pytest

from oracle import prompt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tern():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from packed_ternary_weight_b200 import tern as t
    return t


def codes(g, rows, k, ld):
    a = torch.randint(-128, 128, (rows, ld), generator=g, dtype=torch.int32).to(torch.int8)
    return a.cuda()[:, :k]


def check(tern, m, n, k, out=torch.float32, pad=0, ypad=0, seed=0, x=None, w=None):
    g = torch.Generator().manual_seed(seed)
    ld = (k + 15) // 16 * 16 + 16 * pad
    x = codes(g, m, k, ld) if x is None else x
    w = codes(g, n, k, ld) if w is None else w
    sx, sw = (torch.rand(m, generator=g) * 0.01 + 1e-4).cuda(), (torch.rand(n, generator=g) * 0.01 + 1e-4).cuda()
    y = torch.full((m + 1, n + ypad), 5.0, dtype=out, device="cuda")
    tern.gemm_i8(x, sx, w, sw, y[:m, :n])
    torch.cuda.synchronize()
    ref = prompt.gemm_i8(x.cpu().numpy(), sx.cpu().numpy(), w.cpu().numpy(), sw.cpu().numpy())
    if out == torch.bfloat16:
        ref = prompt.bf16_value(ref)
    assert np.array_equal(y[:m, :n].float().cpu().numpy(), ref)
    assert (y[m:] == 5).all() and (y[:, n:] == 5).all()   # nothing beyond the output is written


@pytest.mark.parametrize("m", [1, 2, 3, 7, 8, 9, 15, 16, 17, 31, 32, 33, 48, 64, 65, 100, 128, 129, 200, 255, 256, 257, 300, 513])
def test_tokens(tern, m):
    check(tern, m, 200, 272, seed=m)
    check(tern, m, 200, 272, torch.bfloat16, seed=m)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 63, 127, 128, 129, 255, 256, 257, 1000, 20000])
@pytest.mark.parametrize("m", [1, 5, 20, 140])
def test_channels(tern, m, n):
    check(tern, m, n, 160, seed=n)


@pytest.mark.parametrize("k", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 100, 127, 128, 129, 255, 257, 511, 513, 1000, 2560, 6912, 14336])
@pytest.mark.parametrize("m", [1, 6, 24, 150])
def test_depths(tern, m, k):
    check(tern, m, 70, k, seed=k)


@pytest.mark.parametrize("m", [1, 9, 40, 260])
def test_strides(tern, m):
    check(tern, m, 130, 200, pad=1, ypad=3)
    check(tern, m, 130, 200, torch.bfloat16, pad=2, ypad=1)


@pytest.mark.parametrize("m", [1, 8, 30, 300])
def test_largest_sums(tern, m):
    k = 131071                                            # 128 * 128 * k is the last below 2^31
    ld = 131072
    x = torch.full((m, ld), -128, dtype=torch.int8, device="cuda")[:, :k]
    w = torch.full((9, ld), -128, dtype=torch.int8, device="cuda")[:, :k]
    w[1] = 127
    check(tern, m, 9, k, x=x, w=w)


@pytest.mark.parametrize("m,n,k", [(700, 1000, 2560), (61, 2560, 6912), (1, 40000, 512), (1500, 300, 640)])
def test_larger(tern, m, n, k):
    check(tern, m, n, k, torch.bfloat16, seed=m)


@pytest.mark.parametrize("m,n,k", [(65, 19000, 64), (96, 18945, 1), (257, 9600, 272), (300, 9473, 100), (512, 9500, 129), (513, 6400, 640),
                                   (1023, 5000, 500), (4096, 1300, 333)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_many_tiles(tern, m, n, k, out):
    # more tiles than multiprocessors: several per CTA, odd ends on every side
    check(tern, m, n, k, out, pad=1, ypad=2, seed=m)


def test_weights_quantised_per_channel(tern):
    # tern_quantize_act gives the weights and their scales
    g = torch.Generator().manual_seed(3)
    w = (torch.randn((300, 256), generator=g) * 0.05).bfloat16().cuda()
    wq, sw = torch.empty((300, 256), dtype=torch.int8, device="cuda"), torch.empty(300, device="cuda")
    tern.quantize_act(w, wq, sw)
    x = torch.randint(-127, 128, (4, 256), generator=g, dtype=torch.int32).to(torch.int8).cuda()
    sx = torch.full((4,), 0.02, device="cuda")
    y = torch.empty((4, 300), device="cuda")
    tern.gemm_i8(x, sx, wq, sw, y)
    ref = (x.double() * 0.02) @ w.double().t()
    # each weight is off by at most half its channel's step
    bound = 0.5001 * sw.double()[None] * (x.double().abs().sum(1) * 0.02)[:, None] + 1e-6
    assert ((y.double() - ref).abs() <= bound).all()


def test_streams_and_replay(tern):
    g = torch.Generator().manual_seed(4)
    for m in (1, 30, 400):
        x, w = codes(g, m, 512, 512), codes(g, 384, 512, 512)
        sx, sw = torch.rand(m, generator=g).cuda(), torch.rand(384, generator=g).cuda()
        y, y2 = torch.empty((m, 384), device="cuda"), torch.empty((m, 384), device="cuda")
        tern.gemm_i8(x, sx, w, sw, y)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            tern.gemm_i8(x, sx, w, sw, y2)
        torch.cuda.synchronize()
        assert torch.equal(y, y2)
        with torch.cuda.graph(graph):
            tern.gemm_i8(x, sx, w, sw, y2)
        x.copy_(codes(g, m, 512, 512))
        graph.replay()
        tern.gemm_i8(x, sx, w, sw, y)
        torch.cuda.synchronize()
        assert torch.equal(y, y2)


def test_binding_refuses(tern):
    x, w = torch.zeros((2, 32), dtype=torch.int8, device="cuda"), torch.zeros((5, 32), dtype=torch.int8, device="cuda")
    sx, sw, y = torch.zeros(2, device="cuda"), torch.zeros(5, device="cuda"), torch.zeros((2, 5), device="cuda")
    for bad in (dict(x=x.float()), dict(w=w[:, :16]), dict(xscale=sw), dict(wscale=sx), dict(y=y.half()), dict(y=y[:, :4]),
                dict(x=x.t().contiguous().t()), dict(w=w.cpu()), dict(x=torch.zeros((2, 40), dtype=torch.int8, device="cuda")[:, 8:])):
        with pytest.raises(tern.TernError):
            tern.gemm_i8(**(dict(x=x, xscale=sx, w=w, wscale=sw, y=y) | bad))
