"""Rotary positions, cache and attention without a GPU: refusals at the edges of what is accepted."""
import pytest

from tests.test_attn_cpu import UNSUPPORTED, _kv, _kv_create
from vector_quantized_weight_b200 import eva_vq


def test_caps_beyond_the_accurate_range_are_refused():
    assert _kv_create(_kv(softcap=2e30)) == UNSUPPORTED


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_devices_that_are_not_cuda_are_refused(device):
    with pytest.raises(ValueError):
        eva_vq.HeadRope(2, 2, 64, device=device)
    with pytest.raises(ValueError):
        eva_vq.KVCache(2, 2, 64, num_pages=1, max_seqs=1, max_pages=1, device=device)


def test_buffers_that_are_not_cuda_are_refused():
    import torch
    k = torch.zeros((1, 2, 64, 64), dtype=torch.int8)
    with pytest.raises(ValueError):
        eva_vq.KVCache(2, 2, 64, num_pages=1, max_seqs=1, max_pages=1, k=k)


def test_cuda_without_a_number_is_the_current_device(monkeypatch):
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    for device, number in ((None, 3), ("cuda", 3), (torch.device("cuda"), 3), ("cuda:1", 1), (torch.device("cuda", 0), 0)):
        assert eva_vq._cuda_device(device) == torch.device("cuda", number)
