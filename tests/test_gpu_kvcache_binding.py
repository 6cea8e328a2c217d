"""The KV-cache binding on the GPU: the memory of handles and of temporaries."""
import numpy as np
import pytest
import torch

from kv_util import Batch, bf16, dev_bf16

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


def test_temporaries_of_another_stream(gpu):
    """Memory that was just given back on the current stream, where work on it is still queued, is not what a call on
    another stream works in."""
    rng = np.random.default_rng(1)
    b = Batch(rng, [3000, 60], [1, 1], 64, 2, 128, 8, starts=False).device(gpu)     # with partial results in ws
    Q = dev_bf16(bf16(rng.standard_normal((2, 16, 128)))[1])
    want = gpu.qcache_attend(b.cache, Q, b.d_pages, b.d_lens)
    kv = gpu.qcache_read(b.cache, b.d_pages, b.d_lens)
    nbytes = gpu.qcache_attend_ws(b.cache, 2, 2, b.pages.shape[1], 16)
    s = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        junk = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (Q.numel() * 2, 4 * 2 * 128 * 2, nbytes)]
        big = torch.empty(1 << 28, device="cuda")
        for _ in range(8):
            big.fill_(1.0)                           # about a millisecond of work queued on the current stream
        for t in junk:
            t.fill_(255)
        del junk, t
        out = gpu.qcache_attend(b.cache, Q, b.d_pages, b.d_lens, stream=s)
        K, V = gpu.qcache_read(b.cache, b.d_pages, b.d_lens, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(K, kv[0]) and torch.equal(V, kv[1])


def test_captured_on_an_explicit_stream(gpu):
    """The capturing stream named explicitly, outputs and workspaces from the graph's own memory, replayed beside eager
    work on the current stream."""
    rng = np.random.default_rng(2)
    b = Batch(rng, [3000, 60], [1, 1], 64, 2, 128, 8, starts=False, prefix=100).device(gpu)
    Q = dev_bf16(bf16(rng.standard_normal((2, 16, 128)))[1])
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()

    def calls(stream):
        return [gpu.qcache_attend(b.cache, Q, b.d_pages, b.d_lens, stream=stream),
                gpu.qcache_attend_shared(b.cache, Q, b.d_prefix, 100, b.d_pages, b.d_lens, stream=stream),
                *gpu.qcache_read(b.cache, b.d_pages, b.d_lens, stream=stream)]

    calls(None)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        outs = calls(s)
    for i in range(3):
        Q.normal_()
        b.d_lens -= 7
        want = calls(None)
        torch.cuda.synchronize()
        g.replay()
        torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want)), f"replay {i}"
