"""tern_norm_quantize on rows with values that are not finite: the row's scale says so, whichever kernel takes it, and
the other rows are as without it."""
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


@pytest.mark.parametrize("k", [641, 640, 6912, 16384, 20000])   # rows read three times; in registers; too long for them
@pytest.mark.parametrize("mode", ["plain", "add", "relu2"])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_a_row_that_is_not_finite_shows_in_its_scale(tern, k, mode, dt):
    m = 6
    g = torch.Generator().manual_seed(k)
    x, r = torch.randn((m, k), generator=g).to(dt), torch.randn((m, k), generator=g).to(dt)
    bad = {1: float("nan"), 3: float("inf")}
    for row, v in bad.items():
        (x if mode == "plain" or row == 1 else r)[row, k // 2] = v
    gain = 1 + 0.1 * torch.randn(k, generator=g)
    xq, xs = torch.full((m, k), 77, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    s = torch.empty((m, k), dtype=dt, device="cuda") if mode == "add" else None
    code = {"plain": tern.NORM_PLAIN, "add": tern.NORM_ADD, "relu2": tern.NORM_RELU2}[mode]
    tern.norm_quantize(code, x.cuda(), r.cuda(), gain.cuda(), 1e-5, s, xq, xs)
    torch.cuda.synchronize()
    ok = [0, 2, 4, 5]
    _, q, sc = prompt.norm_quantize(mode, x.float().numpy()[ok], r.float().numpy()[ok], gain.numpy(), 1e-5, dt == torch.bfloat16)
    assert np.array_equal(xq.cpu().numpy()[ok], q) and np.array_equal(xs.cpu().numpy()[ok], sc)
    for row in bad:
        assert not np.isfinite(float(xs[row])) and (xq[row] == 0).all()


@pytest.mark.parametrize("k", [65, 64, 20000])
def test_a_gain_that_overflows(tern, k):
    x = torch.ones((2, k), device="cuda")
    x[1] = 0
    gain = torch.ones(k, device="cuda")
    gain[3] = 3e38
    x[0, 3] = 4                                           # 4 / rms times 3e38 is beyond fp32
    xq, xs = torch.full((2, k), 77, dtype=torch.int8, device="cuda"), torch.empty(2, device="cuda")
    tern.norm_quantize(tern.NORM_PLAIN, x, None, gain, 1e-5, None, xq, xs)
    assert not np.isfinite(float(xs[0])) and (xq[0] == 0).all()
    assert float(xs[1]) == 0 and (xq[1] == 0).all()
