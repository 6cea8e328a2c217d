"""The KV-cache binding on the GPU: the memory of handles and of temporaries."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_handle_gives_its_memory_back(gpu):
    """Caches made, used and dropped one after the other take no more memory than one."""
    pages = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    lens = torch.tensor([20, 5], dtype=torch.int32, device="cuda")
    K, Q = (torch.randn(2, h, 64, device="cuda").bfloat16() for h in (2, 8))
    before = torch.cuda.memory_allocated()
    for _ in range(3):
        cache = gpu.make_qcache(64, 256, 2, 64, 8)
        assert torch.cuda.memory_allocated() >= before + 2 * 64 * 256 * 2 * 64
        gpu.qcache_write(cache, K, K, pages, lens)
        out = gpu.qcache_attend(cache, Q, pages, lens)
        torch.cuda.synchronize()
        del cache, out
        assert torch.cuda.memory_allocated() == before
