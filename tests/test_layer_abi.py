"""The entry points of include/qlayer.h on the CPU: every declared symbol is
exported, sizes, and refusals before any HIP call."""
import ctypes
import os
import re

import pytest

import compressed_gemv_amd as cg

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qlayer.h")
GOOD, ODD = 0x10000, 0x10008
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(cg.lib_path()):
        import __graft_entry__
        __graft_entry__.build()
    return cg.load()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*int\s+([a-z_]+)\s*\(", text, flags=re.M)))
    assert names == ["qadapt", "qadapt_ws", "qnorm_rope", "qprompt_attend"]
    for n in names:
        assert hasattr(lib, n), n


# ------------------------------------------------------------------ adapters
def adapters(**kw):
    d = dict(n=3, K=64, N=40, rank=16, A=GOOD, B=GOOD, scales=GOOD, ranks=None)
    d.update(kw)
    return cg.qadapters(*(d[n] for n, _ in cg.qadapters._fields_))


BAD_SETS = [(dict(n=0), cg.Q_EINVAL), (dict(K=0), cg.Q_EINVAL), (dict(N=0), cg.Q_EINVAL), (dict(rank=0), cg.Q_EINVAL),
            (dict(K=60), cg.Q_EINVAL), (dict(rank=12), cg.Q_EINVAL), (dict(rank=136), cg.Q_EUNSUPPORTED),
            (dict(n=(1 << 20) + 1), cg.Q_EUNSUPPORTED), (dict(K=1 << 23), cg.Q_EUNSUPPORTED),
            (dict(N=1 << 25), cg.Q_EUNSUPPORTED)]
BAD_BUFFERS = [(dict(A=None), cg.Q_EINVAL), (dict(B=None), cg.Q_EINVAL), (dict(scales=None), cg.Q_EINVAL),
               (dict(A=ODD), cg.Q_EALIGN), (dict(B=ODD), cg.Q_EALIGN), (dict(scales=GOOD + 2), cg.Q_EALIGN),
               (dict(ranks=GOOD + 1), cg.Q_EALIGN)]


def call_adapt(lib, a, **kw):
    d = dict(B=2, T=9, ids=GOOD, starts=GOOD, x=GOOD, xs=64, y=GOOD, ys=40, out=GOOD * 2, os=40, dt=cg.Q_F32, ws=GOOD, n=BIG)
    d.update(kw)
    return lib.qadapt(a, d["B"], d["T"], d["ids"], d["starts"], d["x"], d["xs"], d["y"], d["ys"], d["out"], d["os"], d["dt"],
                      d["ws"], d["n"], None)


@pytest.mark.parametrize("kw,status", BAD_SETS + BAD_BUFFERS)
def test_adapter_sets_refused(lib, kw, status):
    assert call_adapt(lib, adapters(**kw)) == status
    n = ctypes.c_size_t()
    assert lib.qadapt_ws(adapters(**kw), 2, 9, ctypes.byref(n)) == (status if (kw, status) in BAD_SETS else cg.Q_OK)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), cg.Q_EINVAL), (dict(T=0), cg.Q_EINVAL), (dict(T=(1 << 27) + 1), cg.Q_EUNSUPPORTED),
    (dict(B=65537, T=1 << 20), cg.Q_EINVAL), (dict(B=70000), cg.Q_EINVAL), (dict(starts=None), cg.Q_EINVAL),
    (dict(ids=None), cg.Q_EINVAL), (dict(x=None), cg.Q_EINVAL), (dict(y=None), cg.Q_EINVAL), (dict(out=None), cg.Q_EINVAL),
    (dict(dt=cg.Q_F16), cg.Q_EINVAL), (dict(xs=56), cg.Q_EINVAL), (dict(ys=39), cg.Q_EINVAL), (dict(os=39), cg.Q_EINVAL),
    (dict(out=GOOD, os=48), cg.Q_EINVAL), (dict(ids=GOOD + 2), cg.Q_EALIGN), (dict(starts=GOOD + 2), cg.Q_EALIGN),
    (dict(x=ODD), cg.Q_EALIGN), (dict(xs=68), cg.Q_EALIGN), (dict(y=GOOD + 2), cg.Q_EALIGN), (dict(out=GOOD + 2), cg.Q_EALIGN),
    (dict(y=GOOD + 1, dt=cg.Q_BF16), cg.Q_EALIGN), (dict(xs=1 << 24), cg.Q_EUNSUPPORTED), (dict(ys=1 << 31), cg.Q_EUNSUPPORTED),
    (dict(ws=None), cg.Q_EWORKSPACE), (dict(n=100), cg.Q_EWORKSPACE), (dict(ws=ODD), cg.Q_EALIGN)])
def test_adapt_refuses(lib, kw, status):
    assert call_adapt(lib, adapters(), **kw) == status


def test_adapt_without_a_set(lib):
    n = ctypes.c_size_t()
    assert call_adapt(lib, None) == cg.Q_EINVAL
    assert lib.qadapt_ws(None, 1, 1, ctypes.byref(n)) == cg.Q_EINVAL
    assert lib.qadapt_ws(adapters(), 1, 1, None) == cg.Q_EINVAL


def test_adapt_workspace_covers_both_kinds_of_rows(lib):
    """Partial sums of A_a x: fp32 [splits][T][rank padded to 16]."""
    n = ctypes.c_size_t()
    for T, B in ((1, 1), (64, 64), (5000, 3), (1, 65536)):
        assert lib.qadapt_ws(adapters(K=8192, rank=24), B, T, ctypes.byref(n)) == cg.Q_OK
        assert n.value % (T * 32 * 4) == 0 and 1 <= n.value // (T * 32 * 4) <= 32


# --------------------------------------------------------------------- norms
def rope(**kw):
    d = dict(head_dim=64, q_heads=4, kv_heads=2, rot=64, pairs=0, freqs=GOOD, q_weight=GOOD, k_weight=GOOD,
             w_dtype=cg.Q_BF16, eps=1e-6, offset=0)
    d.update(kw)
    return cg.qrope(*(d[n] for n, _ in cg.qrope._fields_))


def call_rope(lib, p, **kw):
    d = dict(B=2, T=9, lens=GOOD, starts=GOOD, Q=GOOD, qs=256, K=GOOD, ks=128, i=cg.Q_BF16, Qo=GOOD * 2, qos=256, Ko=GOOD * 3,
             kos=128, o=cg.Q_BF16)
    d.update(kw)
    return lib.qnorm_rope(p, d["B"], d["T"], d["lens"], d["starts"], d["Q"], d["qs"], d["K"], d["ks"], d["i"], d["Qo"], d["qos"],
                          d["Ko"], d["kos"], d["o"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=0), cg.Q_EINVAL), (dict(head_dim=96), cg.Q_EUNSUPPORTED), (dict(q_heads=-1), cg.Q_EINVAL),
    (dict(q_heads=0, kv_heads=0), cg.Q_EINVAL), (dict(q_heads=65536), cg.Q_EUNSUPPORTED), (dict(rot=80), cg.Q_EINVAL),
    (dict(rot=-16), cg.Q_EINVAL), (dict(rot=7), cg.Q_EINVAL), (dict(rot=24), cg.Q_EUNSUPPORTED), (dict(freqs=None), cg.Q_EINVAL),
    (dict(freqs=GOOD + 4), cg.Q_EALIGN), (dict(q_weight=ODD), cg.Q_EALIGN), (dict(k_weight=ODD), cg.Q_EALIGN),
    (dict(w_dtype=cg.Q_F16), cg.Q_EINVAL), (dict(eps=0.0), cg.Q_EINVAL), (dict(eps=float("nan")), cg.Q_EINVAL),
    (dict(eps=float("inf")), cg.Q_EINVAL), (dict(eps=-1.0), cg.Q_EINVAL), (dict(offset=1 << 31), cg.Q_EUNSUPPORTED),
    (dict(offset=-(1 << 31)), cg.Q_EUNSUPPORTED)])
def test_rope_descriptions_refused(lib, kw, status):
    assert call_rope(lib, rope(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), cg.Q_EINVAL), (dict(T=0), cg.Q_EINVAL), (dict(T=(1 << 27) + 1), cg.Q_EUNSUPPORTED), (dict(B=65537), cg.Q_EINVAL),
    (dict(lens=None), cg.Q_EINVAL), (dict(starts=None), cg.Q_EINVAL), (dict(lens=GOOD + 2), cg.Q_EALIGN),
    (dict(starts=GOOD + 1), cg.Q_EALIGN), (dict(Q=None), cg.Q_EINVAL), (dict(Ko=None), cg.Q_EINVAL), (dict(Q=ODD), cg.Q_EALIGN),
    (dict(qs=248), cg.Q_EINVAL), (dict(qs=260), cg.Q_EALIGN), (dict(kos=1 << 31), cg.Q_EUNSUPPORTED), (dict(i=cg.Q_F16), cg.Q_EINVAL),
    (dict(o=7), cg.Q_EINVAL), (dict(Qo=GOOD, qos=512), cg.Q_EINVAL), (dict(Qo=GOOD, o=cg.Q_F32), cg.Q_EINVAL)])
def test_rope_refuses(lib, kw, status):
    assert call_rope(lib, rope(), **kw) == status


def test_rope_without_a_description(lib):
    assert call_rope(lib, None) == cg.Q_EINVAL


# ------------------------------------------------------------------- prompts
def call_prompt(lib, **kw):
    d = dict(D=64, hq=4, h=2, B=2, T=9, starts=GOOD, Q=GOOD, qs=256, K=GOOD, ks=128, V=GOOD, vs=128, scale=0.1, out=GOOD * 2,
             os=256, o=cg.Q_BF16)
    d.update(kw)
    return lib.qprompt_attend(d["D"], d["hq"], d["h"], d["B"], d["T"], d["starts"], d["Q"], d["qs"], d["K"], d["ks"], d["V"], d["vs"],
                              d["scale"], d["out"], d["os"], d["o"], None)


SIZES = [(dict(D=0), cg.Q_EINVAL), (dict(D=96), cg.Q_EUNSUPPORTED), (dict(hq=5), cg.Q_EINVAL), (dict(hq=0), cg.Q_EINVAL),
         (dict(h=0), cg.Q_EINVAL), (dict(hq=130), cg.Q_EUNSUPPORTED), (dict(hq=2048, h=2048), cg.Q_EUNSUPPORTED),
         (dict(B=0), cg.Q_EINVAL), (dict(B=65537), cg.Q_EINVAL), (dict(T=0), cg.Q_EINVAL), (dict(T=(1 << 27) + 1), cg.Q_EUNSUPPORTED),
         (dict(hq=64, T=1 << 26), cg.Q_EUNSUPPORTED)]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(starts=None), cg.Q_EINVAL), (dict(starts=GOOD + 2), cg.Q_EALIGN), (dict(Q=None), cg.Q_EINVAL), (dict(K=None), cg.Q_EINVAL),
    (dict(V=None), cg.Q_EINVAL), (dict(out=None), cg.Q_EINVAL), (dict(Q=ODD), cg.Q_EALIGN), (dict(vs=132), cg.Q_EALIGN),
    (dict(ks=120), cg.Q_EINVAL), (dict(qs=1 << 31), cg.Q_EUNSUPPORTED), (dict(scale=float("nan")), cg.Q_EINVAL),
    (dict(scale=float("inf")), cg.Q_EINVAL), (dict(scale=1e14), cg.Q_EUNSUPPORTED), (dict(o=cg.Q_F16), cg.Q_EINVAL)])
def test_prompt_refuses(lib, kw, status):
    assert call_prompt(lib, **kw) == status
