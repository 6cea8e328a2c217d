"""The KV-cache binding on the CPU: what a handle keeps alive and where a
call's temporaries come from."""
import gc
import weakref

import numpy as np
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


class _Stream:
    device, cuda_stream = torch.device("cpu"), 7


class _Lib:
    """The library with its launches noted instead of made."""

    def __init__(self, real, calls):
        self._real, self._calls = real, calls

    def __getattr__(self, name):
        if name in ("qcache_read", "qcache_attend", "qcache_attend_shared"):
            return lambda *a: self._calls.append((name, a[-1])) or cg.Q_OK
        return getattr(self._real, name)


def test_temporaries_come_from_the_streams_own_pool(lib, monkeypatch):
    """With an explicit stream every tensor the binding allocates is allocated on that stream, and what the caller
    gets back is recorded on the current one as well."""
    inside, made, recorded, calls = [], [], [], []

    class on:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            inside.append(self.stream)

        def __exit__(self, *e):
            inside.pop()

    real_empty = torch.empty

    def empty(*a, **kw):
        t = real_empty(*a, **kw)
        made.append((t.data_ptr(), inside[-1] if inside else None))
        return t

    stream, current = _Stream(), object()
    cache = cg.qcache(4, 16, 2, 64, 8, *(0x10000,) * 4)
    cache._tensors, cache._device, cache._index = (), torch.device("cpu"), -1
    bf = dict(dtype=torch.bfloat16)
    Q, pages, lens = torch.zeros(3, 8, 64, **bf), torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    with monkeypatch.context() as m:
        m.setattr(cg, "load", lambda: _Lib(lib, calls))
        m.setattr(torch, "empty", empty)
        m.setattr(torch.cuda, "stream", on)
        m.setattr(torch.cuda, "device", lambda d: on(None))
        m.setattr(torch.cuda, "current_stream", lambda d=None: current)
        m.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s)))
        outs = [cg.qcache_attend(cache, Q, pages, lens, stream=stream),
                cg.qcache_attend_shared(cache, Q, pages[0], 20, pages, lens, stream=stream),
                cg.qcache_read(cache, pages, lens, stream=stream)[0]]
    assert calls == [("qcache_attend", 7), ("qcache_attend_shared", 7), ("qcache_read", 7)]
    assert len(made) == 5                                  # two outputs with a workspace each, K and V together
    assert all(s is stream for _, s in made)
    assert recorded == [(o.data_ptr(), current) for o in outs]


def test_a_stream_of_another_device_is_refused(lib):
    cache = cg.qcache(4, 16, 2, 64, 8, *(0x10000,) * 4)
    cache._tensors, cache._device, cache._index = (), torch.device("cpu"), -1
    bf = dict(dtype=torch.bfloat16)
    K, Q = torch.zeros(3, 2, 64, **bf), torch.zeros(3, 8, 64, **bf)
    pages, lens = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)

    class other:
        device, cuda_stream = torch.device("cuda", 1), 7

    for call in (lambda: cg.qcache_write(cache, K, K, pages, lens, stream=other),
                 lambda: cg.qcache_read(cache, pages, lens, stream=other),
                 lambda: cg.qcache_read(cache, pages, lens, K=K, V=K, stream=other),
                 lambda: cg.qcache_attend(cache, Q, pages, lens, stream=other),
                 lambda: cg.qcache_attend_shared(cache, Q, pages[0], 20, pages, lens, stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()


def test_a_scale_beyond_the_kernels_constants_is_refused(lib):
    """scale * log2(e) * 2^69 * s is held in fp32: finite up to a scale of 2^45 for the largest s there is."""
    largest = 2 * 65504 / 15
    with np.errstate(over="ignore"):
        product = [np.float32(2.0 ** p * np.log2(np.e)) * np.float32(2.0 ** 69) * np.float32(largest) for p in (45, 46)]
    assert np.isfinite(product[0]) and np.isinf(product[1])
    c, s = cg.qcache(4, 16, 2, 64, 8, *(0x10000,) * 4), cg.qseqs(3, 7, 2, *(0x10000,) * 3)
    for scale, status in ((2.0 ** 45, cg.Q_EWORKSPACE), (-2.0 ** 45, cg.Q_EWORKSPACE), (2.0 ** 45 * 1.001, cg.Q_EUNSUPPORTED),
                          (-2.0 ** 59, cg.Q_EUNSUPPORTED), (3e38, cg.Q_EUNSUPPORTED)):
        # a good scale gets as far as the workspace, which is missing
        assert lib.qcache_attend(c, s, 0x10000, 512, 8, scale, 0x10000, 512, cg.Q_BF16, None, 0, None) == status, scale
        assert lib.qcache_attend_shared(c, s, 0x10000, 5, 0x10000, 512, 8, scale, 0x10000, 512, cg.Q_BF16, None, 0,
                                        None) == status, scale
