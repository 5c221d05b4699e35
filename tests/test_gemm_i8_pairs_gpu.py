"""tern_gemm_i8 on pairs of CTAs whose odd one has little or nothing to store, many calls in a row on two streams: the
odd CTA ends as early as it may, and what the even one still sends to it must have come by then."""
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


@pytest.mark.parametrize("m,n,k", [(256, 256 * 80 + 64, 64), (256, 256 * 76 + 128, 1040), (500, 256 * 40 + 1, 144), (255, 256 * 75 - 130, 4096)])
def test_odd_halves_without_channels(tern, m, n, k):
    g = torch.Generator().manual_seed(m + k)
    x = torch.randint(-128, 128, (m, k), generator=g, dtype=torch.int32).to(torch.int8).cuda()
    w = torch.randint(-128, 128, (n, k), generator=g, dtype=torch.int32).to(torch.int8).cuda()
    sx, sw = (torch.rand(m, generator=g) * 0.01 + 1e-4).cuda(), (torch.rand(n, generator=g) * 0.01 + 1e-4).cuda()
    want = torch.from_numpy(prompt.gemm_i8(x.cpu().numpy(), sx.cpu().numpy(), w.cpu().numpy(), sw.cpu().numpy())).cuda()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ys = [torch.zeros((m, n), device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for _ in range(25):
        for y, s in zip(ys, streams):
            with torch.cuda.stream(s):
                tern.gemm_i8(x, sx, w, sw, y)
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in ys)
    assert tern.device_error() == tern.OK
