"""The KV-cache binding on the CPU: what a handle keeps alive and where a
call's temporaries come from."""
import gc
import weakref

import pytest
import torch

import compressed_gemv_amd as cg


@pytest.fixture
def lib():
    import os
    if not os.path.exists(cg.lib_path()):
        import __graft_entry__
        __graft_entry__.build()
    return cg.load()


def _buffers():
    codes, meta = cg.qcache_sizes(4, 16, 2, 64, 8)
    return [torch.zeros(n, dtype=d) for n, d in ((codes, torch.uint8), (meta // 4, torch.int32)) * 2]


def test_a_handle_lets_its_buffers_go(lib, monkeypatch):
    """The buffers live as long as the handle and no longer, without the cycle collector's help."""
    monkeypatch.setattr(cg, "_need_cuda", lambda *t: None)
    bufs = _buffers()
    cache = cg.make_qcache(4, 16, 2, 64, 8, *bufs)
    refs = [weakref.ref(t) for t in bufs]
    gc.disable()
    try:
        del bufs
        assert all(r() is not None for r in refs)
        del cache
        assert all(r() is None for r in refs)
    finally:
        gc.enable()
