"""tern_norm_quantize against the oracle. The definition rounds every step to fp32 and the sum of squares is formed in
fp64, where its error (about k 2^-53) is far below the half step of the one rounding to fp32, so all outputs must be
equal bit for bit."""
import numpy as np
import pytest

from oracle import prompt
from packed_ternary_weight_b200 import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tern():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from packed_ternary_weight_b200 import tern as t
    return t


DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def host(t):
    return t.float().cpu().numpy()


def check(tern, mode, m, k, xt="f32", rt="f32", pad=0, seed=0, shape=None, in_place=False, offset=0):
    g = torch.Generator().manual_seed(seed)

    def rows(dt, fill=None):
        a = torch.randn((m, k + pad + offset), generator=g)
        if fill is not None:
            fill(a)
        return a.to(dt).cuda()[:, offset:k + offset]

    x, r = rows(DT[xt], shape), rows(DT[rt])
    gain = (1 + 0.1 * torch.randn(k, generator=g)).cuda()
    hx, hr = host(x), host(r)
    total = r if in_place else torch.full((m, k + pad + offset), 7.0, dtype=DT[rt], device="cuda")[:, offset:k + offset]
    xq = torch.full((m, k + pad), 77, dtype=torch.int8, device="cuda")
    xs = torch.empty(m, device="cuda")
    code = {"plain": tern.NORM_PLAIN, "add": tern.NORM_ADD, "relu2": tern.NORM_RELU2}[mode]
    tern.norm_quantize(code, x, None if mode == "plain" else r, gain, 1e-5, total if mode == "add" else None, xq[:, :k], xs)
    torch.cuda.synchronize()
    v, q, s = prompt.norm_quantize(mode, hx, hr, gain.cpu().numpy(), 1e-5, rt == "bf16")
    if mode == "add":
        assert np.array_equal(host(total), v)
    assert np.array_equal(xq[:, :k].cpu().numpy(), q)
    assert np.array_equal(xs.cpu().numpy(), s)
    assert (xq[:, k:] == 77).all()                       # what lies between the rows is left alone


@pytest.mark.parametrize("mode", ["plain", "add", "relu2"])
@pytest.mark.parametrize("xt,rt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
def test_types(tern, mode, xt, rt):
    check(tern, mode, 5, 2560, xt, rt)


@pytest.mark.parametrize("mode", ["plain", "add", "relu2"])
@pytest.mark.parametrize("k", [1, 2, 3, 4, 31, 100, 255, 1023, 1024, 4096, 6912, 14336, 16384, 16388, 20000])
def test_widths(tern, mode, k):
    check(tern, mode, 3, k, "bf16", "f32", seed=k)


@pytest.mark.parametrize("m", [1, 2, 147, 149, 1000, 5000])
def test_row_counts(tern, m):
    check(tern, "add", m, 512, "bf16", "f32", seed=m)


@pytest.mark.parametrize("seed", range(6))
def test_borders_of_the_rounding(tern, seed):
    # enough values that some stand at a half after the product's own rounding, where a fused product and sum would
    # round the other way (one in about 2^17 values)
    check(tern, "plain", 300, 4096, "bf16", "f32", seed=seed)
    check(tern, "relu2", 40, 6912, "f32", "f32", seed=seed)


@pytest.mark.parametrize("pad", [1, 4, 8])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_strides(tern, pad, xt):
    check(tern, "add", 7, 640, xt, xt, pad=pad)
    check(tern, "relu2", 7, 641, xt, xt, pad=pad)


@pytest.mark.parametrize("k", [640, 20000])
def test_unaligned_rows_and_in_place(tern, k):
    check(tern, "add", 4, k, offset=1)
    check(tern, "add", 4, k, "bf16", "bf16", offset=2)
    check(tern, "add", 4, k, "bf16", "f32", in_place=True)


def test_extreme_rows(tern):
    def fill(a):
        a[0] = 0                                         # an empty row: zeros and scale 0
        a[1] = 1e-30                                     # eps dominates
        a[2] = 0
        a[2, 5] = 3e38                                   # squares beyond fp32
        a[3] *= 1e18
        a[4] = -0.0
    check(tern, "plain", 6, 256, shape=fill)
    check(tern, "relu2", 6, 256, shape=lambda a: a[0].fill_(-1.0))   # the gate closes a whole row


def test_feeds_the_ternary_product(tern):
    lay = synth.bitnet_layer(320, 640, seed=5)
    d, buf = tern.pack_layer(lay)
    m = 20
    x = torch.randn((m, 640), generator=torch.Generator().manual_seed(1)).cuda()
    gain = torch.ones(640, device="cuda")
    xq, xs = torch.empty((m, 640), dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    y = torch.empty((m, 320), device="cuda")
    ws = torch.zeros(tern.workspace_size(d, m), dtype=torch.uint8, device="cuda")
    tern.norm_quantize(tern.NORM_PLAIN, x, None, gain, 1e-5, None, xq, xs)
    tern.gemm_batched(d, torch.from_numpy(buf).cuda(), m, tern.ACT_INT8, xq, xs, tern.OUT_F32, y, ws)
    torch.cuda.synchronize()
    import oracle
    _, q, s = prompt.norm_quantize("plain", host(x), None, gain.cpu().numpy(), 1e-5)
    assert np.array_equal(y.cpu().numpy(), oracle.gemv_bitnet_int8(lay.trits, q, s, lay.tensor_scale))


def test_binding_refuses(tern):
    x = torch.zeros((2, 8), device="cuda")
    q, s, g = torch.zeros((2, 8), dtype=torch.int8, device="cuda"), torch.zeros(2, device="cuda"), torch.zeros(8, device="cuda")
    for bad in (dict(x=x.double()), dict(gain=g[:4]), dict(xq=x), dict(xscale=s.double()), dict(x=x.t().contiguous().t()),
                dict(r=None), dict(sum=None), dict(sum=x.bfloat16()), dict(r=torch.zeros((3, 8), device="cuda")), dict(gain=g.cpu())):
        a = dict(x=x, r=x, gain=g, eps=1e-5, sum=x, xq=q, xscale=s) | bad
        with pytest.raises(tern.TernError):
            tern.norm_quantize(tern.NORM_ADD, **a)
