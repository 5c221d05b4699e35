"""Checks of the binding that need no device: they come before anything is launched."""
import pytest

torch = pytest.importorskip("torch")

from packed_ternary_weight_b200 import tern  # noqa: E402


def attention(ws):
    i32 = dict(dtype=torch.int32)
    cache = tern.KV4Cache(torch.zeros(2 * 16 * 72, dtype=torch.uint8), 1, 64, 16)
    batch = tern.KV4Batch(torch.tensor([0, 1], **i32), torch.tensor([20], **i32), torch.tensor([[0, 1]], **i32), 1, 1, 20)
    q = torch.zeros((1, 64), dtype=torch.bfloat16)
    cache.attention(batch, q, 0.1, torch.zeros_like(q), ws)


@pytest.mark.parametrize("ws", [torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(64, dtype=torch.uint8)[::2],
                                torch.zeros((8, 8), dtype=torch.uint8).t()])
def test_a_workspace_has_the_bytes_it_says(ws):
    # a view that repeats or skips bytes counts more of them than stand behind its address
    with pytest.raises(tern.TernError, match="workspace"):
        attention(ws)


def test_tensors_off_the_device():
    for ws in (None, torch.zeros(64, dtype=torch.uint8)):
        with pytest.raises(tern.TernError, match="not on a CUDA device"):
            attention(ws)
