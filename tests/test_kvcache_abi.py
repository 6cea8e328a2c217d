"""The KV-cache entry points (include/qcache.h) on the CPU: every declared
symbol is exported, sizes, refusals before any HIP call, and the binding's
checks of tensors."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import compressed_gemv_amd as cg
import oracle

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qcache.h")
P = ctypes.c_void_p
GOOD, ODD = 0x10000, 0x10008


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(cg.lib_path()):
        import __graft_entry__
        __graft_entry__.build()
    return cg.load()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*int\s+([a-z_]+)\s*\(", text, flags=re.M)))
    assert names == ["qcache_attend", "qcache_attend_shared", "qcache_attend_ws", "qcache_read", "qcache_sizes",
                     "qcache_write"]
    for n in names:
        assert hasattr(lib, n), n


def test_sizes(lib):
    assert cg.qcache_sizes(10, 16, 8, 128, 8) == (10 * 16 * 8 * 128, 10 * 16 * 8 * 4)
    assert cg.qcache_sizes(1, 256, 1, 64, 4) == (256 * 32, 256 * 4)
    # a cache beyond 32-bit offsets
    assert cg.qcache_sizes(1 << 20, 256, 8, 128, 8) == (1 << 38, 1 << 33)


@pytest.mark.parametrize("args,status", [
    ((0, 16, 8, 128, 8), cg.Q_EINVAL), ((1, 16, 0, 128, 8), cg.Q_EINVAL), ((1, 8, 8, 128, 8), cg.Q_EINVAL),
    ((1, 48, 8, 128, 8), cg.Q_EINVAL), ((1, 512, 8, 128, 8), cg.Q_EINVAL), ((1, 16, 8, 128, 6), cg.Q_EINVAL),
    ((1, 16, 8, 0, 8), cg.Q_EINVAL), ((1, 16, 8, 96, 8), cg.Q_EUNSUPPORTED), ((1, 16, 8, 256, 8), cg.Q_EUNSUPPORTED),
    ((1, 16, 2000, 128, 8), cg.Q_EUNSUPPORTED), ((1 << 31, 16, 8, 128, 8), cg.Q_EUNSUPPORTED),
])
def test_sizes_refused(lib, args, status):
    assert lib.qcache_sizes(*args, None, None) == status


def _cache(**kw):
    d = dict(n_pages=4, page_size=16, heads=2, head_dim=64, bits=8, k_codes=GOOD, k_meta=GOOD, v_codes=GOOD, v_meta=GOOD)
    d.update(kw)
    return cg.qcache(*(d[n] for n, _ in cg.qcache._fields_))


def _seqs(**kw):
    d = dict(B=3, T=7, max_pages=2, pages=GOOD, lens=GOOD, starts=GOOD)
    d.update(kw)
    return cg.qseqs(*(d[n] for n, _ in cg.qseqs._fields_))


BAD_CACHES = [(dict(bits=5), cg.Q_EINVAL), (dict(page_size=24), cg.Q_EINVAL), (dict(k_codes=None), cg.Q_EINVAL),
              (dict(v_meta=None), cg.Q_EINVAL), (dict(k_meta=ODD), cg.Q_EALIGN), (dict(v_codes=ODD), cg.Q_EALIGN),
              (dict(head_dim=32), cg.Q_EUNSUPPORTED)]
BAD_SEQS = [(dict(B=0), cg.Q_EINVAL), (dict(B=65537), cg.Q_EINVAL), (dict(T=0), cg.Q_EINVAL),
            (dict(max_pages=0), cg.Q_EINVAL), (dict(pages=None), cg.Q_EINVAL), (dict(lens=None), cg.Q_EINVAL),
            (dict(starts=None), cg.Q_EINVAL), (dict(pages=GOOD + 2), cg.Q_EALIGN), (dict(lens=GOOD + 1), cg.Q_EALIGN),
            (dict(starts=GOOD + 2), cg.Q_EALIGN), (dict(T=1 << 29), cg.Q_EUNSUPPORTED),
            (dict(max_pages=1 << 27), cg.Q_EUNSUPPORTED)]


@pytest.mark.parametrize("fn", ["qcache_write", "qcache_read"])
def test_write_and_read_refuse(lib, fn):
    f = getattr(lib, fn)

    def call(c, s, K=GOOD, ks=128, V=GOOD, vs=128, dt=cg.Q_BF16):
        return f(None if c is None else ctypes.byref(c), None if s is None else ctypes.byref(s), K, ks, V, vs, dt, None)

    assert call(None, _seqs()) == cg.Q_EINVAL and call(_cache(), None) == cg.Q_EINVAL
    for kw, st in BAD_CACHES:
        assert call(_cache(**kw), _seqs()) == st, kw
    for kw, st in BAD_SEQS:
        assert call(_cache(), _seqs(**kw)) == st, kw
    for kw, st in [(dict(K=None), cg.Q_EINVAL), (dict(V=None), cg.Q_EINVAL), (dict(dt=cg.Q_F16 if hasattr(cg, "Q_F16") else 2), cg.Q_EINVAL),
                   (dict(ks=120), cg.Q_EINVAL), (dict(vs=-128), cg.Q_EINVAL), (dict(K=ODD), cg.Q_EALIGN),
                   (dict(vs=132), cg.Q_EALIGN), (dict(ks=130, dt=cg.Q_F32), cg.Q_EALIGN),
                   (dict(ks=1 << 31), cg.Q_EUNSUPPORTED)]:
        assert call(_cache(), _seqs(), **kw) == st, kw


def test_attend_refuses(lib):
    def call(c=None, s=None, Q=GOOD, qs=512, heads=8, scale=0.1, out=GOOD, os_=512, dt=cg.Q_BF16, ws=GOOD, nws=1 << 40,
             shared=False, prefix=GOOD, n=5):
        c, s = ctypes.byref(c or _cache()), ctypes.byref(s or _seqs())
        if shared:
            return lib.qcache_attend_shared(c, s, prefix, n, Q, qs, heads, scale, out, os_, dt, ws, nws, None)
        return lib.qcache_attend(c, s, Q, qs, heads, scale, out, os_, dt, ws, nws, None)

    for shared in (False, True):
        for kw, st in BAD_CACHES:
            assert call(c=_cache(**kw), shared=shared) == st, kw
        for kw, st in BAD_SEQS:
            assert call(s=_seqs(**kw), shared=shared) == st, kw
        for kw, st in [(dict(Q=None), cg.Q_EINVAL), (dict(out=None), cg.Q_EINVAL), (dict(heads=0), cg.Q_EINVAL),
                       (dict(heads=7), cg.Q_EINVAL), (dict(heads=2 * 65, qs=130 * 64, os_=130 * 64), cg.Q_EUNSUPPORTED),
                       (dict(scale=float("nan")), cg.Q_EINVAL), (dict(scale=float("inf")), cg.Q_EINVAL),
                       (dict(dt=2), cg.Q_EINVAL), (dict(qs=500), cg.Q_EINVAL), (dict(os_=511), cg.Q_EINVAL),
                       (dict(qs=516), cg.Q_EALIGN), (dict(os_=514, dt=cg.Q_F32), cg.Q_EALIGN), (dict(Q=ODD), cg.Q_EALIGN),
                       (dict(out=ODD), cg.Q_EALIGN), (dict(ws=None), cg.Q_EWORKSPACE), (dict(nws=0), cg.Q_EWORKSPACE),
                       (dict(ws=ODD), cg.Q_EALIGN)]:
            assert call(shared=shared, **kw) == st, kw
    for kw, st in [(dict(prefix=None), cg.Q_EINVAL), (dict(n=0), cg.Q_EINVAL), (dict(n=-3), cg.Q_EINVAL),
                   (dict(prefix=GOOD + 2), cg.Q_EALIGN), (dict(n=1 << 31), cg.Q_EUNSUPPORTED)]:
        assert call(shared=True, **kw) == st, kw


def test_workspace_query(lib):
    n = ctypes.c_size_t()
    q = lambda c, s, h, p: lib.qcache_attend_ws(ctypes.byref(c), ctypes.byref(s), h, p, ctypes.byref(n))   # noqa: E731
    bare = _seqs(pages=None, lens=None, starts=None)      # the query reads sizes only
    assert q(_cache(k_codes=None), bare, 8, 0) == cg.Q_OK and n.value > 0
    assert q(_cache(), bare, 3, 0) == cg.Q_EINVAL
    assert q(_cache(), bare, 8, -1) == cg.Q_EINVAL
    assert q(_cache(), _seqs(B=0), 8, 0) == cg.Q_EINVAL
    assert q(_cache(), _seqs(T=1 << 28), 128, 0) == cg.Q_EUNSUPPORTED
    assert lib.qcache_attend_ws(ctypes.byref(_cache()), ctypes.byref(bare), 8, 0, None) == cg.Q_EINVAL


# ---------------------------------------------------------------- binding
def _bare():
    c = _cache()
    c._tensors, c._device, c._index = (), torch.device("cuda", 0), 0
    return c


def test_binding_checks(lib):
    c = _bare()
    bf = dict(dtype=torch.bfloat16)
    K, pages, lens = torch.zeros(3, 2, 64, **bf), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    starts = torch.zeros(4, dtype=torch.int32)
    Q = torch.zeros(3, 8, 64, **bf)

    def refuses(match, fn, *a, **kw):
        with pytest.raises(ValueError, match=match):
            fn(*a, **kw)

    for fn, first in ((cg.qcache_write, (c, K, K)), (cg.qcache_attend, (c, Q))):
        refuses("pages", fn, *first, pages.long(), lens)
        refuses("pages", fn, *first, pages[0], lens)
        refuses("lens", fn, *first, pages, lens[:2])
        refuses("lens", fn, *first, pages, lens.long())
        refuses("starts", fn, *first, pages, lens, starts[:3])
        refuses("starts", fn, *first, pages[:2], lens[:2])          # three rows, two sequences
        refuses("CUDA", fn, *first, pages, lens)
    refuses("K", cg.qcache_write, c, K[:, :1], K, pages, lens)
    refuses("V", cg.qcache_write, c, K, K.float(), pages, lens)
    refuses("V", cg.qcache_write, c, K, K[:2], pages, lens)
    refuses("contiguous", cg.qcache_write, c, K.transpose(1, 2).contiguous().transpose(1, 2), K, pages, lens)
    refuses("dtype", cg.qcache_write, c, K.half(), K.half(), pages, lens)
    refuses("rows", cg.qcache_read, c, pages, lens, starts)
    refuses("both", cg.qcache_read, c, pages, lens, K=K)
    refuses("dtype", cg.qcache_attend, c, Q.float(), pages, lens)
    refuses("Q", cg.qcache_attend, c, Q[:, :7], pages, lens)
    refuses("Q", cg.qcache_attend, c, Q[:, :, :32], pages, lens)
    refuses("out", cg.qcache_attend, c, Q, pages, lens, out=Q[:2])
    refuses("out", cg.qcache_attend, c, Q, pages, lens, out=Q.half())
    refuses("prefix_pages", cg.qcache_attend_shared, c, Q, pages[0].long(), 5, pages, lens)
    refuses("prefix_pages", cg.qcache_attend_shared, c, Q, pages[0], 33, pages, lens)
    refuses("prefix_len", cg.qcache_attend_shared, c, Q, pages[0], 0, pages, lens)
    codes, meta = (torch.zeros(n, dtype=torch.uint8) for n in cg.qcache_sizes(4, 16, 2, 64, 8))
    refuses("k_meta", cg.make_qcache, 4, 16, 2, 64, 8, codes, meta[:-4], codes, meta)
    refuses("v_codes", cg.make_qcache, 4, 16, 2, 64, 8, codes, meta, None, meta)
    refuses("CUDA", cg.make_qcache, 4, 16, 2, 64, 8, codes, meta, codes, meta)


# ----------------------------------------------------------------- oracle
@pytest.mark.parametrize("head_dim", [32, 64])
def test_oracle_rows_are_the_group_packers(head_dim):
    """At 4 bits and a row of 32 or 64 values the cache's encoder is the group encoder."""
    W = np.random.default_rng(0).standard_normal((50, head_dim)).astype(np.float32)
    q, s, o = oracle.rtn.quantize(W, 4, head_dim)
    q2, s2, o2 = oracle.kvcache.quantize_rows(W, 4)
    assert np.array_equal(q, q2) and np.array_equal(s[:, 0], s2) and np.array_equal(o[:, 0], o2)


@pytest.mark.parametrize("bits", [4, 8])
def test_oracle_rows_bounds(bits):
    rng = np.random.default_rng(bits)
    x = rng.standard_normal((200, 128)) * 10.0 ** rng.uniform(-3, 4, (200, 1))
    q, s, o = oracle.kvcache.quantize_rows(x, bits)
    err = np.abs(oracle.kvcache.row_values(q, s, o) - np.clip(x, -65280, 65280))
    assert np.all(err <= s.astype(np.float64)[:, None] / 2 * (1 + 1e-12))
    assert np.abs(oracle.kvcache.row_values(q, s, o)).max() <= 65504
    # the largest rows there are: no level leaves fp16
    big = np.where(np.arange(64) % 2, 65280.0, -65280.0)[None] * np.linspace(0.9, 1.2, 40)[:, None]
    assert np.abs(oracle.kvcache.row_values(*oracle.kvcache.quantize_rows(big, bits))).max() <= 65504
    codes = oracle.kvcache.pack_codes(q, bits)
    assert np.array_equal(oracle.kvcache.unpack_codes(codes, bits), q)


def test_oracle_attention_by_hand():
    """One head, three tokens, by the softmax written out; rows past the end and an empty row."""
    c = oracle.kvcache.Cache(2, 16, 1, 64, 8)
    rng = np.random.default_rng(1)
    x, y = rng.standard_normal((2, 3, 1, 64))
    pages, lens, starts = np.array([[1], [0]], np.int32), np.array([3, 0], np.int32), np.array([0, 3, 4], np.int32)
    c.write(x, y, pages, lens, np.array([0, 3, 3]))
    k, v, owned = c.read(3, pages, lens, np.array([0, 3, 3]))
    assert owned.all() and np.abs(k - x).max() < 0.02 and np.abs(v - y).max() < 0.02
    Q = rng.standard_normal((5, 1, 64))
    out, _, owned = c.attend(Q, pages, lens, starts)
    assert owned.tolist() == [True] * 4 + [False]
    assert np.array_equal(out[0, 0], v[0, 0]) and np.all(out[3] == 0)
    w = np.exp(Q[2, 0] @ k[:, 0].T / 8)
    assert np.allclose(out[2, 0], (w / w.sum()) @ v[:, 0])
    # the first two tokens as a prefix
    pre, _, _ = c.attend(Q[2:3], np.array([[0]], np.int32), np.array([0], np.int32), None, None, np.array([1]), 2)
    w = w[:2]
    assert np.allclose(pre[0, 0], (w / w.sum()) @ v[:2, 0])
